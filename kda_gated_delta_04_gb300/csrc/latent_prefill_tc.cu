// latent_prefill_tc.cu -- expanded latent attention over packed sequences on the tensor cores
// (bf16 I/O).
//
//   s_ij = scale q_i . [k_nope_j, k_pe_j]  (192 channels),  o_i = sum_j softmax_j(s_i) v_j  (128)
//
// A sequence of lq queries and lk keys is aligned at its end: query i sees keys j <= i + lk - lq
// (causal) or all.  Bound by the tensor cores: 640 FLOP per (query, key, head) against a few bytes.
//
// A pair of CTAs (a cluster of two, one CTA per SM) holds 512 queries of one head as two tiles of 256
// and passes over the keys in tiles of 128.  A matrix instruction spans the pair (M = 256): each CTA
// holds its 128 queries of a tile, half of K's rows and half of V's columns, so that a key tile takes
// 40 KB a CTA instead of 80, and an instruction reads 6 KB of shared memory in its 64 cycles instead
// of 8 (the limit).  One CTA alone left 4,600 cycles for what the tensor cores do in 2,560: its ring
// held 1.6 key tiles, and the copies' writes competed with operand reads at the limit.
//
//   S [256 x 128] = Q [256 x 192] K^T          12 steps of K = 16, operands in shared memory
//   O [256 x 128] += P [256 x 128] V            8 steps, P (bf16) in tensor memory over its S
//
// Tensor memory is full: two O, two S of 128 columns (a tile that is alone has both S).  The two query
// tiles take turns: while one tile's softmax runs (a warpgroup each, a thread per query, so that maximum
// and sum need no other thread), the tensor cores run the other tile's products, O += P V of key tile j
// and S of j + 1.
// Where there are few jobs and many keys, two or four pairs (one cluster) share the keys of a job and join
// their parts through distributed shared memory.
// Warps 0 to 7: softmax; 8: copies (TMA); 9: matrix instructions (in the leading CTA); 10: the jobs;
// 11: a check of the offsets (first CTA).
//
// 4,096 tokens, 32 heads, causal: 131 us, 1.31 PFLOP/s; 1,024 tokens behind 13,047 keys 207 us, 1.37 (other inputs
// on every call).  The comparisons at the constants below repeat one call on the same inputs, in bursts of 2 ms after a
// pause; the 4,096 tokens take 124 us so.  Cycles by that, over 4 to 32 key tiles and 1 to 6 jobs a pair, within 2 %:
// 13,600 a call, 6,900 a job and 3,290 a key tile of a pair, for which the products need 2,560.
#include <math.h>

#include "latent.cuh"
#include "latent_ptx.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

using namespace ptx;
using tc::kdesc;

constexpr int kT = 384, kM = 128, kN = 128;   // threads; queries of a tile in one CTA; keys per tile
constexpr int kPairM = 4 * kM;                // queries of a pair of CTAs
constexpr uint32_t kPanelQ = 128 * 128;       // bytes: 128 queries x 64 channels
constexpr uint32_t kPanelK = 64 * 128;        // half of a tile's keys x 64 channels
constexpr uint32_t kTileK = 3 * kPanelK, kTileV = 128 * 128;  // a CTA's part of a K and a V tile
constexpr int kStages = 3;                    // key tiles in shared memory
constexpr int kJobs = 4;                      // records of jobs
// Key tiles of a job during whose copies the next one is asked for already: what hides the 2,000 cycles that
// asking for and finding it take.  A job taken sooner is one that a pair that comes free cannot have: with 4
// for shared key tiles a prompt of 4,096 tokens takes 130 us instead of 124 (its last jobs have 4), while 64
// prompts of 150 to 250 tokens, side by side, take 79 us with 2 and 74 with 4 or 8 (16 heads).
constexpr int kShort = 2, kShortApart = 8;
constexpr int kAhead = 2;                     // key tiles brought into L2 before their copy
constexpr uint32_t kOffQ = 0;                 // two tiles of three panels
constexpr uint32_t kOffK = kOffQ + 6 * kPanelQ;
constexpr uint32_t kOffV = kOffK + kStages * kTileK;
constexpr uint32_t kOffMisc = kOffV + kStages * kTileV;
constexpr uint64_t kWait = tc::kWaitNs;
constexpr float kSlack = 8.f;  // log2: how far scores may pass the held maximum before it is moved
constexpr uint32_t kColO = 0, kColS = 256;    // + 128 x query tile

// A query tile: queries [q0, q0 + rows) of a head (256 at most, 128 for each CTA) against the keys of their
// sequence, klen from k0; the first query sees the keys up to `off` when causal; n key tiles.
struct alignas(16) Part {
    int q0, k0, rows, klen, off, h, n;
    int tail;  // where the last key tile reaches past the sequence's keys: its V buffer + 4 x parity there
    __device__ __forceinline__ bool has_tail() const { return n > 0 && n * kN > klen; }
};

// What a pair of CTAs works on: two query tiles of one sequence and head that share every key tile (the
// second sees all that the first does), or, of sequences with no more than 256 queries left, one each of
// two, whose key tiles come in turn.
enum : int { kDone = 0, kShared = 1, kApart = 2 };
struct Job {
    Part part[2];
    int kind;
    int base[2];  // + j: key tile j of all jobs, where the query tile is alone (see alone_from)
    int unused;
};

// Place of key tile j of query tile i among the job's key tiles.
__device__ __forceinline__ int place(bool apart, int n0, int n1, int i, int j)
{
    return !apart ? j : (i ? j + min(j + 1, n0) : j + min(j, n1));
}

// Where a query tile's key tiles outnumber the other's, S goes to the other's buffer and the own one in turn
// from this key tile on, a key tile ahead, so that it is computed while the softmax before it runs: by then the
// other's last product has been issued, and what a tile alone would wait for is half of its time.  256 queries
// behind 15,000 keys: 40 heads 118 us, with one buffer 180; 8 heads (their keys shared by four pairs) 39 and 55; 4
// times 200 behind 3,000, 8 heads, 31.5 and 43.  What it costs: prompts of one key tile, which have nothing to
// compute ahead, 300 of 10 to 30 tokens, 16 heads, 193 us and 182; 64 of 150 to 250 tokens 74 and 72.
__device__ __forceinline__ int alone_from(int i, int n0, int n1) { return i ? n0 + 1 : n1 + 2; }
__device__ __forceinline__ bool in_other(int alone, int j) { return j >= alone && !((j - alone) & 1); }

// Barriers of the leading CTA only: q_full, k_full, v_full (bytes that both CTAs copy), p_full,
// o_empty and next_empty (a warp's arrival each, both CTAs).  The others each CTA has for itself; what the matrix
// instructions signal arrives in both.
struct Misc {
    uint64_t q_full[2], q_empty[2], k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[2], s_other[2], p_full[2][4], o_full[2], o_empty[2], v_tail[kStages], drained;
    uint64_t next_full, next_empty;  // the number asked for: each CTA; both CTAs have read it, in the leading one
    uint64_t job_full[kJobs], job_empty[kJobs], copied[2];  // copied: all of a job's tiles
    alignas(16) uint4 next;
    alignas(16) Job job[kJobs];      // for this CTA's other warps
    uint32_t tmem;
    int abort;
};
constexpr int kSmem = kOffMisc + (int)sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory");

// Waits for a phase; gives up after kWait ns or as soon as another role of the CTA has.  The same
// answer on every lane of the (converged) warp.
template <bool CLUSTER>
__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    auto test = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    bool ok = test();
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            for (int i = 0; i < 32 && !ok; ++i) ok = test();
            if (ok || *abort) break;
            if (globaltimer_ns() - t0 > kWait) {
                *abort = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32])
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
          "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]),
          "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]),
          "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
}

// 32 bytes to global memory: whole sectors (16-byte aligned; in one instruction where 32-byte aligned).
__device__ __forceinline__ void store32(__nv_bfloat16 *p, const uint32_t (&w)[8])
{
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Query tiles of cluster `pair` of the grid: heads innermost, the tiles with the most keys first.  A whole
// warp; part[0].rows is 0 where the number has no tile.
__device__ __forceinline__ void make_parts(const LatentPrefill &p, const LatentLane &mine, int count, uint32_t inverse,
                                           int pair, int lane, Part (&part)[2])
{
    // pair / heads from floor((2^32 - 1) / heads), which is short by two at most
    int order = (int)__umulhi((uint32_t)pair, inverse), h = pair - order * p.heads;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (h >= p.heads) {
            h -= p.heads;
            ++order;
        }
    const LatentTile at = latent_tile(p, mine, order, count, kPairM, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        Part &x = part[i];
        x.q0 = at.q0 + 2 * kM * i;
        x.k0 = at.k0;
        x.rows = max(0, min(2 * kM, at.rows - 2 * kM * i));
        x.klen = at.klen;
        x.off = at.off + 2 * kM * i;
        x.h = h;
        const int keys = p.causal ? max(0, min(x.klen, x.off + x.rows)) : x.klen;
        x.n = x.rows > 0 ? (keys + kN - 1) / kN : 0;
        x.tail = 0;
    }
}

// The jobs of this pair as the other warps of a CTA read them.  Every warp of a role takes them in step.
struct Jobs {
    Misc &mi;
    int count;
    __device__ __forceinline__ Jobs(Misc &m) : mi(m), count(0) {}
    // The next job, to be read before done(); null: there is none, or a wait gave up
    __device__ __forceinline__ const Job *take()
    {
        const Job *job = &mi.job[count % kJobs];
        if (!all_wait<false>(&mi.job_full[count % kJobs], (count / kJobs) & 1, &mi.abort)) return nullptr;
        return job->kind == kDone ? nullptr : job;
    }
    __device__ __forceinline__ void done(int lane)
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.job_empty[count % kJobs]);
        ++count;
    }
};

// One warp of each CTA: finds the jobs, its own cluster's, then those of clusters that were still waiting
// to be launched.  The next one is asked for when the last copy of the present one has been issued: early
// enough for the answer to be there, and no sooner, so that the last jobs go to the pairs that are done
// first; a short job's successor is asked for when the copies of the one before are done.
// A job of one query tile takes another such beside it (`beside`: the grid has more clusters than can run
// at once), since alone it leaves the tensor cores to wait for its softmax and the other way round: 64
// prompts of 150 to 250 tokens, 16 heads, 74 us instead of 97; 300 of 10 to 30 tokens 193 instead of 307.
// Both CTAs of the pair come to the same jobs.
template <int SPLIT>
__device__ __forceinline__ void job_role(Misc &mi, const LatentPrefill &p, bool beside, int rank, int team, int lane)
{
    volatile int *abort = &mi.abort;
    const bool lead = lane == 0, leader = rank == 0;
    int t = 0, asked = 0;       // key tiles of the jobs before, numbers asked for so far
    int at = blockIdx.x / (2 * SPLIT);  // the number at hand; -1: there is none left
    bool used = false;          // it is in a job already
    uint32_t tails = 0;         // parity of the tails so far in each V buffer
    const LatentLane mine = latent_lane(p, kPairM, lane);
    const int tiles = (int)(gridDim.x / (2 * SPLIT)) / p.heads;
    const uint32_t inverse = 0xffffffffu / (uint32_t)p.heads;
    for (int count = 0;; ++count) {
        Job &job = mi.job[count % kJobs];
        if (count >= kJobs && !all_wait<false>(&mi.job_empty[count % kJobs], (count / kJobs - 1) & 1, abort)) return;
        int kind = kDone, n0 = 0, n1 = 0;
        bool tail0 = false, tail1 = false;
        for (;;) {
            if (SPLIT > 1 && used) at = -1;
            if (SPLIT == 1 && used && at >= 0) {
                if (lead) mbar_arrive_expect_tx(&mi.next_full, 16);
                if (leader) {
                    if (asked > 0 && !all_wait<true>(&mi.next_empty, (asked - 1) & 1, abort)) return;
                    if (lead) cluster_take(&mi.next, &mi.next_full);
                }
                __syncwarp();
                if (!all_wait<false>(&mi.next_full, asked & 1, abort)) return;
                at = cluster_taken(&mi.next) >> 1;  // (-1 stays -1)
                fence_proxy_async_smem();           // read before it is written again
                __syncwarp();
                if (lead) mbar_arrive_cluster(map_to_rank(&mi.next_empty, 0));
                ++asked;
                used = false;
            }
            if (at < 0) break;
            Part part[2];
            make_parts(p, mine, tiles, inverse, at, lane, part);
            if constexpr (SPLIT > 1) {  // this pair's key tiles
                const int n = max(part[0].n, part[1].n), from = n * team / SPLIT, to = n * (team + 1) / SPLIT;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Part &x = part[i];
                    x.n = max(0, min(to, x.n) - from);
                    x.k0 += from * kN;
                    x.klen -= from * kN;
                    x.off -= from * kN;
                }
            }
            const bool lone = beside && part[1].rows == 0;
            if (part[0].rows == 0) {
                used = true;
            } else if (kind == kDone) {
                used = true;
                if (lead) {
                    job.part[0] = part[0];
                    job.part[1] = part[1];
                }
                kind = kShared;
                n0 = part[0].n, n1 = part[1].n;
                tail0 = part[0].has_tail(), tail1 = part[1].has_tail();
                if (!lone) break;
            } else {  // a second one beside the first, or the next job
                if (lone) {
                    used = true;
                    if (lead) job.part[1] = part[0];
                    kind = kApart;
                    n1 = part[0].n;
                    tail1 = part[0].has_tail();
                }
                break;
            }
        }
        const bool apart = kind == kApart;
        const int all = apart ? n0 + n1 : max(n0, n1);
        if (tail0 || tail1) {
            // buffers and parities of the tails; of two, the one copied first counts first
            const int e0 = place(apart, n0, n1, 0, n0 - 1), e1 = place(apart, n0, n1, 1, n1 - 1);
            const bool swap = apart && e1 < e0;
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                const bool one = (k == 1) != swap;
                if (!(one ? tail1 : tail0)) continue;
                const int slot = (t + (one ? e1 : e0)) % kStages;
                if (lead) job.part[one].tail = slot | (int)((tails >> slot) & 1) << 2;
                // (where both share it, it is the second's)
                if (apart || one || n1 == 0) tails ^= 1u << slot;
            }
        }
        if (lead) {
            job.kind = kind;
            job.base[0] = t + (apart ? n1 : 0);
            job.base[1] = t + (apart ? n0 : 0);
            mbar_arrive(&mi.job_full[count % kJobs]);
        }
        t += all;
        __syncwarp();
        if (kind == kDone) return;
        if (count > 0 && !all_wait<false>(&mi.copied[(count - 1) & 1], ((count - 1) >> 1) & 1, abort)) return;
        if (all > (apart ? kShortApart : kShort) && !all_wait<false>(&mi.copied[count & 1], (count >> 1) & 1, abort)) return;
    }
}

// One warp of each CTA: copies the tiles of the jobs.
__device__ __forceinline__ void copy_role(unsigned char *sm, Misc &mi, const CUtensorMap &tq, const CUtensorMap &tk,
                                          const CUtensorMap &tp, const CUtensorMap &tv, int q_step, int k_step,
                                          int v_step, int rank, int home, int lane)
{
    volatile int *abort = &mi.abort;
    const bool lead = lane == 0, leader = rank == 0;
    int t = 0, nq0 = 0, nq1 = 0;  // key tiles and queries copied so far
    Jobs jobs(mi);
    while (const Job *next = jobs.take()) {
        const Job &job = *next;
        const bool apart = job.kind == kApart;
        const int n0 = job.part[0].n, n1 = job.part[1].n, all = apart ? n0 + n1 : max(n0, n1);
        bool ok = true;
        auto ahead = [&](const Part &x, int j) {  // this CTA's part of a key tile into L2
            if (!lead || j >= x.n) return;
            const int k = x.k0 + kN * j, kh = x.h * k_step;
            tma_prefetch_3d(&tk, 0, kh, k + 64 * rank);
            tma_prefetch_3d(&tk, 64, kh, k + 64 * rank);
            tma_prefetch_3d(&tp, 0, 0, k + 64 * rank);
            tma_prefetch_3d(&tv, 64 * rank, x.h * v_step, k);
        };
        auto queries = [&](int i, int &nq) -> bool {
            const Part x = job.part[i];
            if (x.n == 0) return true;
            if (nq > 0 && !all_wait<false>(&mi.q_empty[i], (nq - 1) & 1, abort)) return false;
            if (lead) {
                if (leader) mbar_arrive_expect_tx(&mi.q_full[i], 2 * 3 * kPanelQ);
                const uint32_t bar = map_to_rank(&mi.q_full[i], home);
#pragma unroll
                for (int c = 0; c < 3; ++c)
                    tma_load_3d_pair(sm + kOffQ + (3 * i + c) * kPanelQ, &tq, bar, 64 * c, x.h * q_step, x.q0 + kM * rank);
            }
            ++nq;
            return true;
        };
        if (lead) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const Part x = job.part[i];
                if (x.n > 0)
#pragma unroll
                    for (int c = 0; c < 3; ++c) tma_prefetch_3d(&tq, 64 * c, x.h * q_step, x.q0 + kM * rank);
            }
        }
        const int only = n1 > 0;  // shared key tiles: the second sees them all
#pragma unroll 1
        for (int u = 0; u < kAhead; ++u) {
            const Part x = job.part[apart ? u & 1 : only];
            ahead(x, apart ? u >> 1 : u);
        }
        int j0 = 0, j1 = 0;  // key tiles copied of each
#pragma unroll 1
        for (int u = 0; u < all; ++u, ++t) {
            const int i = apart ? (j1 < n1 && (j0 > j1 || j0 == n0)) : only;
            const int j = i ? j1++ : j0++;
            const Part x = job.part[i];
            ahead(x, j + (apart ? kAhead / 2 : kAhead));
            const int slot = t % kStages, k = x.k0 + kN * j, kh = x.h * k_step;
            if (t >= kStages && !(ok = all_wait<false>(&mi.k_empty[slot], (t / kStages - 1) & 1, abort))) break;
            if (lead) {
                if (leader) mbar_arrive_expect_tx(&mi.k_full[slot], 2 * kTileK);
                const uint32_t bar = map_to_rank(&mi.k_full[slot], home);
                unsigned char *dst = sm + kOffK + slot * kTileK;
                tma_load_3d_pair(dst, &tk, bar, 0, kh, k + 64 * rank);
                tma_load_3d_pair(dst + kPanelK, &tk, bar, 64, kh, k + 64 * rank);
                tma_load_3d_pair(dst + 2 * kPanelK, &tp, bar, 0, 0, k + 64 * rank);
            }
            if (u == 0 && !(ok = queries(0, nq0) && queries(1, nq1))) break;
            if (t >= kStages && !(ok = all_wait<false>(&mi.v_empty[slot], (t / kStages - 1) & 1, abort))) break;
            if (lead) {
                unsigned char *dst = sm + kOffV + slot * kTileV;
                if (j + 1 == x.n && x.has_tail()) {
                    // each CTA's softmax waits for this part itself (it clears the rows past the end) and
                    // answers for it with its weights
                    if (leader) mbar_arrive(&mi.v_full[slot]);
                    mbar_arrive_expect_tx(&mi.v_tail[slot], kTileV);
                    tma_load_3d(dst, &tv, &mi.v_tail[slot], 64 * rank, x.h * v_step, k);
                } else {
                    if (leader) mbar_arrive_expect_tx(&mi.v_full[slot], 2 * kTileV);
                    tma_load_3d_pair(dst, &tv, map_to_rank(&mi.v_full[slot], home), 64 * rank, x.h * v_step, k);
                }
            }
        }
        if (!ok) break;
        if (lead) mbar_arrive(&mi.copied[jobs.count & 1]);
        jobs.done(lane);
    }
    if (*abort && lead) {  // the copies in flight land before the pair goes (the other CTA stays for this one)
        if (leader) {
            if (nq0) mbar_wait_ns(&mi.q_full[0], (nq0 - 1) & 1, kWait);
            if (nq1) mbar_wait_ns(&mi.q_full[1], (nq1 - 1) & 1, kWait);
            for (int k = max(0, t - kStages); k < t; ++k) {
                mbar_wait_ns(&mi.k_full[k % kStages], (k / kStages) & 1, kWait);
                mbar_wait_ns(&mi.v_full[k % kStages], (k / kStages) & 1, kWait);
            }
        }
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000) {}  // the tail's copies and an answer on its way: 1 ms
    }
}

// One warp of the leading CTA, in step: for each key tile and query tile in turn O += P V, then S of the
// next key tile.  (A warp for each query tile: 6% slower; both tiles' softmax then run at the same time and
// share the exponential units.)
__device__ __forceinline__ bool mma_role(uint32_t sb, Misc &mi, uint32_t tmem, uint32_t pair, int lane)
{
    constexpr uint32_t id_s = idesc_bf16(2 * kM, kN, false, false), id_o = idesc_bf16(2 * kM, 128, false, true);
    volatile int *abort = &mi.abort;
    const uint32_t lead = elect_lead();
    int t0 = 0;                  // key tiles of the jobs before
    int np0 = 0, np1 = 0;        // products O += P V of each query tile so far, P in its own buffer
    int nother0 = 0, nother1 = 0;  // and in the other's
    int nj0 = 0, nj1 = 0;        // jobs of each query tile so far
    Jobs jobs(mi);
    while (const Job *job = jobs.take()) {
        const int n0 = job->part[0].n, n1 = job->part[1].n;
        const bool apart = job->kind == kApart;
        jobs.done(lane);
        const bool back0 = apart || n1 == 0;  // a key tile is given back by the last query tile that reads it
        auto k_ready = [&](int i, int j) {
            const int t = t0 + place(apart, n0, n1, i, j);
            return all_wait<true>(&mi.k_full[t % kStages], (t / kStages) & 1, abort);
        };
        auto scores = [&](int i, int j) {  // S_i of key tile j
            const int slot = (t0 + place(apart, n0, n1, i, j)) % kStages;
            const bool other = in_other(alone_from(i, n0, n1), j);
            const uint32_t d = tmem + kColS + 128 * (i ^ (int)other), a = sb + kOffQ + 3 * i * kPanelQ;
            const uint32_t b = sb + kOffK + slot * kTileK;
#pragma unroll
            for (int c = 0; c < 3; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16_pair(lead, d, kdesc(a + c * kPanelQ + k * 32), kdesc(b + c * kPanelK + k * 32), id_s,
                                  c > 0 || k > 0);
            mma_commit_pair(lead, other ? &mi.s_other[i] : &mi.s_full[i], pair);
            if (i == 1 || back0) mma_commit_pair(lead, &mi.k_empty[slot], pair);
            if (j + 1 == (i ? n1 : n0)) mma_commit_pair(lead, &mi.q_empty[i], pair);
        };
        auto step = [&](int i, int j, int &np, int &nother, int nj, int &next) -> bool {
            // O_i += P_i V of key tile j, S_i of the next (alone: the next two)
            const int t = t0 + place(apart, n0, n1, i, j), slot = t % kStages, alone = alone_from(i, n0, n1);
            const int n = i ? n1 : n0;
            const bool other = in_other(alone, j);
            const uint32_t parity = (other ? nother++ : np++) & 1;
            if (j == 0 && nj > 0 && !all_wait<true>(&mi.o_empty[i], (nj - 1) & 1, abort)) return false;
            const uint32_t d = tmem + kColO + 128 * i, a = tmem + kColS + 128 * (i ^ (int)other);
            const uint32_t b = sb + kOffV + slot * kTileV;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k == 0 && !all_wait<true>(&mi.v_full[slot], (t / kStages) & 1, abort)) return false;
                if ((k & 3) == 0) {  // a half of the keys
                    if (!all_wait<true>(&mi.p_full[i][2 * (int)other + (k >> 2)], parity, abort)) return false;
                    tc_fence_after_sync();
                }
                mma_tmem_a_pair(lead, d, a + 8 * k, sdesc(b + k * 2048, kTileV, 1024, kSw128B), id_o, j > 0 || k > 0);
            }
            if (i == 1 || back0) mma_commit_pair(lead, &mi.v_empty[slot], pair);
            if (j + 1 == n) mma_commit_pair(lead, &mi.o_full[i], pair);
            const int to = min(n, j + 2 >= alone ? j + 3 : j + 2);
#pragma unroll 1
            for (; next < to; ++next) {
                if (!k_ready(i, next)) return false;
                tc_fence_after_sync();
                scores(i, next);
            }
            return true;
        };
        if (n0 > 0) {
            if (!all_wait<true>(&mi.q_full[0], nj0 & 1, abort) || !k_ready(0, 0)) return false;
            tc_fence_after_sync();
            scores(0, 0);
        }
        if (n1 > 0) {
            if (!all_wait<true>(&mi.q_full[1], nj1 & 1, abort) || !k_ready(1, 0)) return false;
            tc_fence_after_sync();
            scores(1, 0);
        }
        int next0 = 1, next1 = 1;  // scores issued so far
#pragma unroll 1
        for (int j = 0; j < max(n0, n1); ++j) {
            if (j < n0 && !step(0, j, np0, nother0, nj0, next0)) return false;
            if (j < n1 && !step(1, j, np1, nother1, nj1, next1)) return false;
        }
        t0 += apart ? n0 + n1 : max(n0, n1);
        nj0 += n0 > 0;
        nj1 += n1 > 0;
    }
    return !*abort;
}

// What a thread has of its query's softmax at the end; any: there were keys.
struct Held {
    float m, l;
    bool any;
};

// A warpgroup of each CTA per query tile, a thread per query.
template <int SPLIT>
__device__ __forceinline__ void softmax_role(unsigned char *sm, Misc &mi, const LatentPrefill &p, uint32_t tmem, int i,
                                             int rank, int home, Held &held)
{
    volatile int *abort = &mi.abort;
    const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t quarter = (uint32_t)((row >> 5) * 32) << 16;
    const uint32_t to = tmem + kColO + 128 * i + quarter;
    const uint32_t p_full = map_to_rank(&mi.p_full[i][0], home), o_empty = map_to_rank(&mi.o_empty[i], home);
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    int ns = 0, nother = 0, nj = 0;  // score tiles in its own and in the other's buffer, jobs of this query tile
    Jobs jobs(mi);
    while (const Job *job = jobs.take()) {
        const Part at = job->part[i];
        const int alone = alone_from(i, job->part[0].n, job->part[1].n), base = job->base[i];
        jobs.done(lane);
        const int klen = at.klen, n = at.n, mine = kM * rank + row;
        // last key this query sees
        const int last = p.causal ? min(at.off + mine, klen - 1) : klen - 1;
        // this query's row of the output, or none
        const int64_t out = mine < at.rows ? (int64_t)(at.q0 + mine) * p.heads + at.h : -1;
        float m = -INFINITY, l = 0.f;  // held maximum (log2 units) and the sum of the weights
        for (int j = 0; j < n; ++j) {
            const bool other = in_other(alone, j);
            const uint32_t ts = tmem + kColS + 128 * (i ^ (int)other) + quarter;
            if (!all_wait<false>(other ? &mi.s_other[i] : &mi.s_full[i], (other ? nother++ : ns++) & 1, abort)) return;
            tc_fence_after_sync();
            float s[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, *reinterpret_cast<float(*)[32]>(&s[32 * c]));
            const int seen = max(-1, min(kN, last - j * kN));  // columns 0 .. seen
            const bool special = __any_sync(0xffffffffu, seen < kN - 1) || p.scale_log2 <= 0.f;
            tmem_ld_wait();
            // one branch for all that is rare: the rest is straight code that the scheduler can interleave
            if (special) {
                const float sign = p.scale_log2 > 0.f ? 1.f : (p.scale_log2 < 0.f ? -1.f : 0.f);
#pragma unroll
                for (int c = 0; c < 128; ++c) s[c] = c <= seen ? s[c] * sign : -INFINITY;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 128; c += 2) top[(c >> 1) & 3] = max3(top[(c >> 1) & 3], s[c], s[c + 1]);
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
            // the maximum is moved only where a score passes it by kSlack: weights are below 2^kSlack, and
            // the precision of fp32 and bf16 does not depend on that
            const bool rise = mx > m + kSlack;
            const int left = klen - j * kN;
            if (__any_sync(0xffffffffu, rise) || left < kN) {
                float f = 1.f;
                if (rise) {
                    f = tc::exp2_approx(m - mx);
                    m = mx;
                    l *= f;
                }
                // what O holds follows (its last product finished before this S did, but for a tile that is alone:
                // there the product's end gives its V buffer back)
                if (j > 0 && __any_sync(0xffffffffu, rise)) {
                    const int t = base + j - 1;
                    if (j >= alone && !all_wait<false>(&mi.v_empty[t % kStages], (t / kStages) & 1, abort)) return;
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 128; c += 16) {
                        float x[16];
                        tmem_ld16(to + c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] *= f;
                        tmem_st16(to + c, x);
                    }
                }
                // keys past the sequence's end are other sequences' rows: their weight is 0, so their values
                // must be finite
                if (left < kN) {
                    const int slot = at.tail & 3;
                    if (!all_wait<false>(&mi.v_tail[slot], at.tail >> 2, abort)) return;
                    for (int e = row; e < (kN - left) * 8; e += 128)
                        *reinterpret_cast<uint4 *>(sm + kOffV + slot * kTileV + (left + (e >> 3)) * 128 + (e & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    fence_cluster();
                }
            }
            const float base = m == -INFINITY ? 0.f : -m;
            const float2 scale2 = make_float2(scale, scale), base2 = make_float2(base, base);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 &x = *reinterpret_cast<float2 *>(&s[32 * c + 2 * k]);
                    x = fma2(x, scale2, base2);
                    x.x = tc::exp2_approx(x.x);
                    x.y = tc::exp2_approx(x.y);
                    // bf16: the product's operands share one type, and V is bf16
                    w[k] = __uint_as_float(tc::pack_bf16x2(x.x, x.y));
                }
                tmem_st16(ts + 16 * c, w);
                if (c & 1) {  // the product starts on the first half of the keys
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(p_full + 8 * (2 * (int)other + (c >> 1)));
                }
            }
            float2 sum[4] = {};
#pragma unroll
            for (int k = 0; k < 64; ++k) sum[k & 3] = add2(sum[k & 3], *reinterpret_cast<float2 *>(&s[2 * k]));
            const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
            l += all.x + all.y;
        }
        if constexpr (SPLIT > 1) {  // the only job: what it leaves is joined by all
            held = Held{m, l, n > 0};
            if (n > 0) all_wait<false>(&mi.o_full[i], 0, abort);
            return;
        }
        if (out >= 0 && p.lse) p.lse[out] = m * kLn2 + logf(l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + out * kLatN;
        if (n == 0) {
            const uint32_t zero[8] = {};
            if (out >= 0)
#pragma unroll
                for (int k = 0; k < 128; k += 16) store32(o + k, zero);
            continue;
        }
        if (!all_wait<false>(&mi.o_full[i], nj & 1, abort)) return;
        tc_fence_after_sync();
        ++nj;
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(to + 32 * c, *reinterpret_cast<float(*)[32]>(&x[32 * c]));
        tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(o_empty);  // the next job's products may start
        if (out < 0) continue;
#pragma unroll
        for (int k = 0; k < 128; k += 16) {
            uint32_t w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = tc::pack_bf16x2(x[k + 2 * u] * inv, x[k + 2 * u + 1] * inv);
            store32(o + k, w);
        }
    }
}

// The pairs of a cluster that had a share of the keys each: their unnormalised outputs (fp32) and sums, over
// the tiles' buffers (256 rows of 512 bytes, the 16-byte pieces of a row in an order that spreads a column's
// over the banks; then maximum and sum of each row), and their join.  The warps of the softmax.
__device__ __forceinline__ void put_part(unsigned char *sm, uint32_t tmem, int i, int row, const Held &held)
{
    const uint32_t to = tmem + kColO + 128 * i + ((uint32_t)((row >> 5) * 32) << 16);
    unsigned char *o = sm + (128 * i + row) * 512;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        float x[32] = {};
        if (held.any) {
            tmem_ld32(to + 32 * c, x);
            tmem_ld_wait();
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4 *>(o + (((8 * c + k) ^ (row & 31)) << 4)) =
                make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
    }
    *reinterpret_cast<float2 *>(sm + 256 * 512 + (128 * i + row) * 8) = make_float2(held.m, held.l);
}
template <int SPLIT>
__device__ __forceinline__ void join_parts(const unsigned char *sm, const Misc &mi, const LatentPrefill &p, int rank,
                                           int team, int warp, int lane)
{
    if (mi.job[0].kind == kDone) return;
    constexpr int kShare = 256 / SPLIT;  // rows that this CTA writes
#pragma unroll 1
    for (int r = team * kShare + warp; r < (team + 1) * kShare; r += 8) {
        const Part &x = mi.job[0].part[r >> 7];
        const int mine = kM * rank + (r & 127);
        if (mine >= x.rows) continue;
        const float *stats = reinterpret_cast<const float *>(sm + 256 * 512 + r * 8);
        const float *o = reinterpret_cast<const float *>(sm + r * 512 + ((lane ^ (r & 31)) << 4));
        float m[SPLIT], top = -INFINITY, l = 0.f;
        float4 part[SPLIT], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < SPLIT; ++u) {
            m[u] = peer_load(stats, 2 * u + rank);
            part[u] = peer_load4(o, 2 * u + rank);
            top = fmaxf(top, m[u]);
        }
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int u = 0; u < SPLIT; ++u) {
            const float f = exp2f(m[u] - base);
            l += f * peer_load(stats + 1, 2 * u + rank);
            sum.x += f * part[u].x; sum.y += f * part[u].y; sum.z += f * part[u].z; sum.w += f * part[u].w;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t out = (int64_t)(x.q0 + mine) * p.heads + x.h;
        uint2 w;
        w.x = tc::pack_bf16x2(sum.x * inv, sum.y * inv);
        w.y = tc::pack_bf16x2(sum.z * inv, sum.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + out * kLatN + 4 * lane) = w;
        if (p.lse && lane == 0) p.lse[out] = top * kLn2 + logf(l);
    }
}

// SPLIT: pairs (in a cluster) that share a job's keys.
template <int SPLIT>
__global__ void __launch_bounds__(kT, 1)
latent_prefill_tc_kernel(const LatentPrefill p, const __grid_constant__ CUtensorMap tq,
                         const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tp,
                         const __grid_constant__ CUtensorMap tv, int q_step, int k_step, int v_step, bool beside)
{
    extern __shared__ __align__(1024) unsigned char sm[];
    Misc &mi = *reinterpret_cast<Misc *>(sm + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int place = (int)cluster_rank(), rank = place & 1;
    const int team = place >> 1, home = SPLIT > 1 ? place & ~1 : 0;  // which pair; its leading CTA
    if (smem_u32(sm) & 1023u) {    // the swizzled panels need it; never seen
        if (tid == 0 && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&mi.q_full[i], 1);
            mbar_init(&mi.q_empty[i], 1);
            mbar_init(&mi.s_full[i], 1);
            mbar_init(&mi.s_other[i], 1);
            for (int k = 0; k < 4; ++k) mbar_init(&mi.p_full[i][k], 8);
            mbar_init(&mi.copied[i], 1);
            mbar_init(&mi.o_full[i], 1);
            mbar_init(&mi.o_empty[i], 8);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&mi.k_full[i], 1);
            mbar_init(&mi.k_empty[i], 1);
            mbar_init(&mi.v_full[i], 1);
            mbar_init(&mi.v_empty[i], 1);
            mbar_init(&mi.v_tail[i], 1);
        }
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&mi.job_full[i], 1);
            mbar_init(&mi.job_empty[i], rank == 0 ? 10 : 9);  // warps: softmax, copies, matrix instructions
        }
        mbar_init(&mi.drained, 1);
        mbar_init(&mi.next_full, 1);
        mbar_init(&mi.next_empty, 2);
        fence_mbar_init();
        mi.abort = 0;
    }
    if (warp == 9) tmem_alloc_pair(&mi.tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are ready
    pdl_wait();
    tc_fence_after_sync();
    const uint32_t tmem = mi.tmem;
    // registers: 384 x 168 = 64,512 at launch; 256 x 200 + 128 x 56 = 58,368 now
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        Held held;
        softmax_role<SPLIT>(sm, mi, p, tmem, warp >> 2, rank, home, held);
        if constexpr (SPLIT > 1) {
            __syncwarp();
            __syncthreads();  // both query tiles' products are done
            tc_fence_after_sync();
            const bool whole = mi.job[0].kind != kDone && !mi.abort;
            if (whole) put_part(sm, tmem, warp >> 2, tid & 127, held);
            __syncwarp();
            cluster_sync();
            if (whole) join_parts<SPLIT>(sm, mi, p, rank, team, warp, lane);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 8) {
            copy_role(sm, mi, tq, tk, tp, tv, q_step, k_step, v_step, rank, home, lane);
        } else if (warp == 9 && rank == 0) {
            // (the reduction's result is uniform to the compiler, the loaded word is not)
            if (!mma_role(smem_u32(sm), mi, __reduce_or_sync(0xffffffffu, tmem), 3u << home, lane)) {
                // nothing in flight when tensor memory is given back
                mma_commit_pair(lane == 0, &mi.drained, 3u << home);
                if (lane == 0) mbar_wait_ns(&mi.drained, 0, kWait);
            }
        } else if (warp == 10) {
            job_role<SPLIT>(mi, p, beside, rank, team, lane);
        } else if (warp == 11 && blockIdx.x == 0) {
            latent_check_cu(p.cu_q, p.num_seqs, p.q_tokens, p.errors);
            latent_check_cu(p.cu_k, p.num_seqs, p.k_tokens, p.errors);
        }
        if constexpr (SPLIT > 1) {
            __syncwarp();
            __syncthreads();
            cluster_sync();
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA goes while the other's instructions use its memory
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, 512);
    }
    if (tid == 0 && mi.abort && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
}

// [tokens][heads][channels] with any strides as a tensor of boxes of `box_rows` tokens x 64 channels of
// one head; `step` is the head coordinate's step: 0 where the heads share their rows.
bool make_map(CUtensorMap *m, const void *ptr, int channels, int64_t heads, int64_t hs, int64_t tokens, int64_t ts,
              int box_rows, int *step)
{
    tc::EncodeTiledFn enc = tc::encode_fn();
    if (!enc) return false;
    *step = hs == 0 ? 0 : 1;
    if (hs == 0) {  // one head, or one for all
        heads = 1;
        hs = channels;
    }
    if (ts == 0) ts = channels;  // one token
    const cuuint64_t dims[3] = {(cuuint64_t)channels, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ts * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs that share a job's keys: as many as leave every cluster an SM for each of its CTAs at once (15
// clusters of eight CTAs or 36 of four do), where the share saves more than the larger cluster and the join
// cost, 4 us.  512 queries behind 7,500 keys, us with one, two, four pairs: 15 heads 115, 70, 42; 16 heads 115,
// 69, 79; 36 heads 117, 74, 121; 37 heads 117, 136, 122.  Few keys, 8 heads: 512 queries and keys (4 tiles)
// 14.8, 17.5, 13.7; 64 queries and keys 9.2, 13.0, 13.4.  16 heads: 512 queries behind 1,000 keys 29.7, 25.3, 35,
// behind 512 21.7, 20.8, 30; 200 behind 1,000 18.4, 19.9, 32.  The key tiles are an average and the jobs include
// numbers without a tile, since the lengths are on the device: one long history beside several short prompts is not
// shared.
int key_split(const LatentPrefill &p, int64_t jobs)
{
    const int64_t tiles = p.k_tokens / p.num_seqs / kN;  // key tiles of a sequence, on average
    return jobs <= 15 && tiles >= 4 ? 4 : jobs <= 36 && tiles >= 10 ? 2 : 1;
}

}  // namespace

cudaError_t launch_latent_prefill_tc(const LatentPrefill &p)
{
    // one sequence: its tiles; more: as latent_tile numbers them (numbers without a tile are passed over)
    const int64_t tiles = p.num_seqs == 1 ? (p.q_tokens + kPairM - 1) / kPairM : p.q_tokens / kPairM + p.num_seqs;
    const int64_t blocks = 2 * tiles * p.heads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    CUtensorMap tq, tk, tp, tv;
    int q_step = 0, k_step = 0, v_step = 0, one = 0;
    // without keys no copy of keys runs; the maps still need an address
    const bool keys = p.k_tokens > 0;
    const void *kn = keys ? p.k_nope : p.q, *kp = keys ? p.k_pe : p.q, *v = keys ? p.v : p.q;
    const int64_t tokens = keys ? p.k_tokens : 1;
    if (!make_map(&tq, p.q, kLatQK, p.heads, p.q_hs, p.q_tokens, p.q_ts, kM, &q_step) ||
        !make_map(&tk, kn, kLatN, p.heads, p.kn_hs, tokens, p.kn_ts, 64, &k_step) ||
        !make_map(&tp, kp, kLatP, 1, 0, tokens, p.kp_ts, 64, &one) ||
        !make_map(&tv, v, kLatN, p.heads, p.v_hs, tokens, p.v_ts, kN, &v_step))
        return cudaErrorInvalidValue;
    auto launch = [&](auto kernel, int split, int *configured) -> cudaError_t {
        const cudaError_t err = tc::allow_smem(kernel, kSmem, configured);
        if (err != cudaSuccess) return err;
        return latent_launch(kernel, dim3((unsigned)(blocks * split)), kT, kSmem, p.stream, 2 * split, p, tq, tk, tp, tv,
                             q_step, k_step, v_step, blocks > 152 /* CTAs at once */);
    };
    static int set1 = -1, set2 = -1, set4 = -1;
    const int split = key_split(p, tiles * p.heads);
    return split == 4   ? launch(latent_prefill_tc_kernel<4>, 4, &set4)
           : split == 2 ? launch(latent_prefill_tc_kernel<2>, 2, &set2)
                        : launch(latent_prefill_tc_kernel<1>, 1, &set1);
}

}  // namespace kda
