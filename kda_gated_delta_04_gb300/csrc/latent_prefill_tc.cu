// latent_prefill_tc.cu -- expanded latent attention over packed sequences on the tensor cores
// (bf16 I/O).
//
//   s_ij = scale q_i . [k_nope_j, k_pe_j]  (192 channels),  o_i = sum_j softmax_j(s_i) v_j  (128)
//
// A sequence of lq queries and lk keys is aligned at its end: query i sees keys j <= i + lk - lq
// (causal) or all.  Bound by the tensor cores: 640 FLOP per (query, key, head) against a few bytes.
//
// One CTA per SM holds 256 queries of one head as two tiles of 128 and passes over the keys in
// tiles of 128.  Both products have M = 128 queries in the 128 lanes of tensor memory:
//
//   S [128 x 128] = Q [128 x 192] K^T          12 steps of K = 16, operands in shared memory
//   O [128 x 128] += P [128 x 128] V            8 steps, P (bf16) in tensor memory over its S
//
// Tensor memory is full: two O, two S of 128 columns.  The two query tiles take turns: while one
// tile's softmax runs (a warpgroup each, a thread per query, so that maximum and sum need no other
// thread), the tensor cores run the other tile's products, O += P V of key tile j and S of j + 1.
// K arrives in a ring of four 64-channel panels, each given back as soon as the second query tile
// has read it, V in two buffers.  Warps 0 to 7: softmax; 8: copies (TMA); 9: matrix instructions;
// 10 and 11 only make up the warpgroup whose registers the softmax takes over.
#include <math.h>

#include "latent.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

using namespace ptx;
using tc::kdesc;

constexpr int kT = 384, kM = 128, kN = 128;   // threads; queries and keys per tile
constexpr uint32_t kPanel = 128 * 128;        // bytes: 128 rows x 64 channels
constexpr int kNK = 4, kNV = 2;               // K panel slots, V buffers
constexpr int kAhead = 4;                     // key tiles brought into L2 before their copy
constexpr uint32_t kOffQ = 0;                 // two tiles of three panels
constexpr uint32_t kOffK = kOffQ + 6 * kPanel;
constexpr uint32_t kOffV = kOffK + kNK * kPanel;
constexpr uint32_t kOffMisc = kOffV + kNV * 2 * kPanel;
constexpr uint64_t kWait = tc::kWaitNs;
constexpr float kSlack = 8.f;  // log2: how far scores may pass the held maximum before it is moved
constexpr uint32_t kColO = 0, kColS = 256;    // + 128 x query tile

struct Misc {
    uint64_t q_full[2], k_full[kNK], k_empty[kNK], v_full[kNV], v_empty[kNV], s_full[2], p_full[2][2], o_full[2], drained;
    uint32_t tmem;
    int abort;
};
constexpr int kSmem = kOffMisc + (int)sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory");

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWait) {
            *abort = 1;
            return false;
        }
    }
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

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
          "l"(reinterpret_cast<unsigned long long &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// What one CTA works on, and how many key tiles each of its query tiles sees.
struct Job {
    LatentTile at;   // of all 256 queries
    int64_t lk;      // the sequence's keys
    int n0, n1, nmax;
    __device__ __forceinline__ int n(int i) const { return i ? n1 : n0; }
    __device__ __forceinline__ int rows(int i) const { return max(0, min(kM, at.rows - kM * i)); }
    __device__ __forceinline__ int64_t off(int i) const { return at.off + kM * i; }
};

__device__ __forceinline__ Job make_job(const LatentPrefill &p, int tile)
{
    Job j;
    j.at = latent_tile(p, tile, 2 * kM);
    j.lk = j.at.klen;
    auto tiles = [&](int i) {
        int64_t keys = j.lk;
        if (p.causal) keys = max((int64_t)0, min(keys, j.off(i) + j.rows(i)));
        return j.rows(i) > 0 ? (int)((keys + kN - 1) / kN) : 0;
    };
    j.n0 = tiles(0);
    j.n1 = tiles(1);
    j.nmax = max(j.n0, j.n1);
    return j;
}

__device__ __forceinline__ void copy_role(unsigned char *sm, Misc &mi, const Job &job, const CUtensorMap &tq,
                                          const CUtensorMap &tk, const CUtensorMap &tp, const CUtensorMap &tv, int h,
                                          int kh, int vh)
{
    volatile int *abort = &mi.abort;
    int nk = 0, nv = 0;
    const int k0 = (int)job.at.k0, q0 = (int)job.at.q0;
    auto queries = [&](int i) {
        if (job.n(i) == 0) return;
        mbar_arrive_expect_tx(&mi.q_full[i], 3 * kPanel);
#pragma unroll
        for (int c = 0; c < 3; ++c)
            tma_load_3d(sm + kOffQ + (3 * i + c) * kPanel, &tq, &mi.q_full[i], 64 * c, h, q0 + kM * i);
    };
    auto ahead = [&](int j) {  // key tile j into L2
        if (j >= job.nmax) return;
        const int k = k0 + kN * j;
        tma_prefetch_3d(&tk, 0, kh, k);
        tma_prefetch_3d(&tk, 64, kh, k);
        tma_prefetch_3d(&tp, 0, 0, k);
        tma_prefetch_3d(&tv, 0, vh, k);
        tma_prefetch_3d(&tv, 64, vh, k);
    };
    queries(0);
    bool ok = true;
    for (int j = 1; j < kAhead; ++j) ahead(j);
    for (int j = 0; j < job.nmax && ok; ++j) {
        ahead(j + kAhead);
        for (int c = 0; c < 3 && ok; ++c) {
            const int slot = nk % kNK;
            if (nk >= kNK) ok = wait(&mi.k_empty[slot], (nk / kNK - 1) & 1, abort);
            if (!ok) break;
            mbar_arrive_expect_tx(&mi.k_full[slot], kPanel);
            unsigned char *dst = sm + kOffK + slot * kPanel;
            if (c < 2) tma_load_3d(dst, &tk, &mi.k_full[slot], 64 * c, kh, k0 + kN * j);
            else tma_load_3d(dst, &tp, &mi.k_full[slot], 0, 0, k0 + kN * j);
            ++nk;
        }
        if (j == 0) queries(1);
        if (!ok) break;
        const int slot = nv % kNV;
        if (nv >= kNV) ok = wait(&mi.v_empty[slot], (nv / kNV - 1) & 1, abort);
        if (!ok) break;
        mbar_arrive_expect_tx(&mi.v_full[slot], 2 * kPanel);
#pragma unroll
        for (int c = 0; c < 2; ++c)
            tma_load_3d(sm + kOffV + (2 * slot + c) * kPanel, &tv, &mi.v_full[slot], 64 * c, vh, k0 + kN * j);
        ++nv;
    }
    if (!ok) {  // the copies in flight land before the CTA goes
        for (int i = 0; i < 2; ++i)
            if (job.n(i)) mbar_wait_ns(&mi.q_full[i], 0, kWait);
        for (int k = max(0, nk - kNK); k < nk; ++k) mbar_wait_ns(&mi.k_full[k % kNK], (k / kNK) & 1, kWait);
        for (int k = max(0, nv - kNV); k < nv; ++k) mbar_wait_ns(&mi.v_full[k % kNV], (k / kNV) & 1, kWait);
    }
}

// A whole warp's wait: the same answer on every lane.
__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

// Executed by one whole warp in step.
__device__ __forceinline__ void mma_role(uint32_t sb, Misc &mi, const Job &job, uint32_t tmem)
{
    constexpr uint32_t id_s = idesc_bf16(kM, kN, false, false), id_o = idesc_bf16(kM, 128, false, true);
    volatile int *abort = &mi.abort;
    const uint32_t lead = elect_lead();
    // the second query tile, where there is one, sees every key tile that the first sees
    const bool two = job.n(1) > 0;
    auto scores = [&](int i, int j) -> bool {  // S_i of key tile j
        const uint32_t d = tmem + kColS + 128 * i;
#pragma unroll 1
        for (int c = 0; c < 3; ++c) {
            const int nk = 3 * j + c, slot = nk % kNK;
            if (!all_wait(&mi.k_full[slot], (nk / kNK) & 1, abort)) return false;
            if (c == 0) tc_fence_after_sync();
            const uint32_t a = sb + kOffQ + (3 * i + c) * kPanel, b = sb + kOffK + slot * kPanel;
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16_lead(lead, d, kdesc(a + k * 32), kdesc(b + k * 32), id_s, c > 0 || k > 0);
            if (i == (two ? 1 : 0)) mma_commit_lead(lead, &mi.k_empty[slot]);
        }
        mma_commit_lead(lead, &mi.s_full[i]);
        return true;
    };
    auto values = [&](int i, int j) -> bool {  // O_i += P_i V of key tile j
        const int slot = j % kNV;
        if (!all_wait(&mi.v_full[slot], (j / kNV) & 1, abort)) return false;
        const uint32_t d = tmem + kColO + 128 * i, a = tmem + kColS + 128 * i, b = sb + kOffV + 2 * slot * kPanel;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if ((k & 3) == 0) {
                if (!all_wait(&mi.p_full[i][k >> 2], j & 1, abort)) return false;
                tc_fence_after_sync();
            }
            mma_tmem_a_lead(lead, d, a + 8 * k, sdesc(b + k * 2048, kPanel, 1024, kSw128B), id_o, j > 0 || k > 0);
        }
        if (i == (two ? 1 : 0)) mma_commit_lead(lead, &mi.v_empty[slot]);
        if (j + 1 == job.n(i)) mma_commit_lead(lead, &mi.o_full[i]);
        return true;
    };
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        if (job.n(i) == 0) continue;
        if (!all_wait(&mi.q_full[i], 0, abort)) return;
        if (!scores(i, 0)) return;
    }
#pragma unroll 1
    for (int j = 0; j < job.nmax; ++j)
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (j >= job.n(i)) continue;
            if (!values(i, j)) return;
            if (j + 1 < job.n(i) && !scores(i, j + 1)) return;
        }
}

__device__ __forceinline__ void softmax_role(unsigned char *sm, Misc &mi, const LatentPrefill &p, const Job &job,
                                             uint32_t tmem, int i, int h)
{
    volatile int *abort = &mi.abort;
    const int row = threadIdx.x & 127;
    const uint32_t quarter = (uint32_t)((row >> 5) * 32) << 16;
    const uint32_t ts = tmem + kColS + 128 * i + quarter, to = tmem + kColO + 128 * i + quarter;
    const int64_t last = p.causal ? min(job.off(i) + row, job.lk - 1) : job.lk - 1;  // last key this query sees
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    float m = -INFINITY, l = 0.f;  // held maximum (log2 units) and the sum of the weights
    for (int j = 0; j < job.n(i); ++j) {
        if (!__all_sync(0xffffffffu, wait(&mi.s_full[i], j & 1, abort))) return;
        tc_fence_after_sync();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, *reinterpret_cast<float(*)[32]>(&s[32 * c]));
        const int seen = (int)max((int64_t)-1, min((int64_t)kN, last - (int64_t)j * kN));  // columns 0 .. seen
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
        const int64_t left = job.lk - (int64_t)j * kN;
        if (__any_sync(0xffffffffu, rise) || left < kN) {
            float f = 1.f;
            if (rise) {
                f = tc::exp2_approx(m - mx);
                m = mx;
                l *= f;
            }
            // what O holds follows (its last product finished before this S did)
            if (j > 0 && __any_sync(0xffffffffu, rise)) {
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
                const int slot = j % kNV;
                if (!__all_sync(0xffffffffu, wait(&mi.v_full[slot], (j / kNV) & 1, abort))) return;
                for (int e = row; e < (kN - (int)left) * 16; e += 128) {
                    const int r = (int)left + (e >> 4), c = e & 15;
                    *reinterpret_cast<uint4 *>(sm + kOffV + (2 * slot + (c >> 3)) * kPanel + r * 128 + (c & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
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
                mbar_arrive(&mi.p_full[i][c >> 1]);
            }
        }
        float2 sum[4] = {};
#pragma unroll
        for (int k = 0; k < 64; ++k) sum[k & 3] = add2(sum[k & 3], *reinterpret_cast<float2 *>(&s[2 * k]));
        const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += all.x + all.y;
    }
    // O's rows out, through this warp's part of the query tile's memory so that a row is stored whole
    const int lane = row & 31, warp0 = row & ~31;
    const int64_t q = job.at.q0 + kM * i;
    if (p.lse && row < job.rows(i)) p.lse[(q + row) * p.heads + h] = m * kLn2 + logf(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    unsigned char *stage = sm + kOffQ + 3 * i * kPanel + warp0 * 256;
    if (job.n(i) > 0) {
        if (!__all_sync(0xffffffffu, wait(&mi.o_full[i], 0, abort))) return;
        tc_fence_after_sync();
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float x[16];
        if (job.n(i) > 0) {
            tmem_ld16(to + 16 * c, x);
            tmem_ld_wait();
        }
        float y[2][8];
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k >> 3][k & 7] = job.n(i) > 0 ? x[k] * inv : 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4 *>(stage + lane * 256 + (((2 * c + k) ^ (lane & 15)) << 4)) = tc::pack_bf16x8(y[k]);
    }
    __syncwarp();
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + (q * p.heads + h) * kLatN;
#pragma unroll 4
    for (int r = lane >> 4; r < 32; r += 2) {
        const int c = lane & 15;
        const uint4 x = *reinterpret_cast<const uint4 *>(stage + r * 256 + ((c ^ (r & 15)) << 4));
        if (warp0 + r < job.rows(i))
            *reinterpret_cast<uint4 *>(o + (int64_t)(warp0 + r) * p.heads * kLatN + 8 * c) = x;
    }
}

__global__ void __launch_bounds__(kT, 1)
latent_prefill_tc_kernel(const LatentPrefill p, const __grid_constant__ CUtensorMap tq,
                         const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tp,
                         const __grid_constant__ CUtensorMap tv, int q_step, int k_step, int v_step)
{
    extern __shared__ __align__(1024) unsigned char sm[];
    Misc &mi = *reinterpret_cast<Misc *>(sm + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // heads innermost, the tiles with the most keys first
    const int h = blockIdx.x % p.heads, tile = (int)(gridDim.x / p.heads - 1 - blockIdx.x / p.heads);
    const Job job = make_job(p, tile);
    if (blockIdx.x == 0) {
        latent_check_cu(p.cu_q, p.num_seqs, p.q_tokens, p.errors);
        latent_check_cu(p.cu_k, p.num_seqs, p.k_tokens, p.errors);
    }
    if (job.at.rows <= 0) return;
    if (smem_u32(sm) & 1023u) {  // the swizzled panels need it; never seen
        if (tid == 0 && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&mi.q_full[i], 1);
            mbar_init(&mi.s_full[i], 1);
            mbar_init(&mi.p_full[i][0], 128);
            mbar_init(&mi.p_full[i][1], 128);
            mbar_init(&mi.o_full[i], 1);
        }
        for (int i = 0; i < kNK; ++i) {
            mbar_init(&mi.k_full[i], 1);
            mbar_init(&mi.k_empty[i], 1);
        }
        for (int i = 0; i < kNV; ++i) {
            mbar_init(&mi.v_full[i], 1);
            mbar_init(&mi.v_empty[i], 1);
        }
        mbar_init(&mi.drained, 1);
        fence_mbar_init();
        mi.abort = 0;
    }
    if (warp == 9) {
        tmem_alloc(&mi.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = mi.tmem;
    // registers: 384 x 168 at launch; 256 x 216 + 128 x 64 now
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int i = warp >> 2;
        if (job.rows(i) > 0) softmax_role(sm, mi, p, job, tmem, i, h);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 8) {
            if (lane == 0) copy_role(sm, mi, job, tq, tk, tp, tv, h * q_step, h * k_step, h * v_step);
        } else if (warp == 9) {
            // (the reduction's result is uniform to the compiler, the loaded word is not)
            mma_role(smem_u32(sm), mi, job, __reduce_or_sync(0xffffffffu, tmem));
            __syncwarp();
            if (lane == 0 && *(volatile int *)&mi.abort) {  // nothing in flight when tensor memory is given back
                mma_commit(&mi.drained);
                mbar_wait_ns(&mi.drained, 0, kWait);
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && mi.abort && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
}

// [tokens][heads][channels] with any strides as a tensor of boxes of 128 tokens x 64 channels of one
// head; `step` is the head coordinate's step: 0 where the heads share their rows.
bool make_map(CUtensorMap *m, const void *ptr, int channels, int64_t heads, int64_t hs, int64_t tokens, int64_t ts,
              int *step)
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
    const cuuint32_t box[3] = {64, 1, 128}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_latent_prefill_tc(const LatentPrefill &p)
{
    const int64_t blocks = (p.q_tokens / (2 * kM) + p.num_seqs) * p.heads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    CUtensorMap tq, tk, tp, tv;
    int q_step = 0, k_step = 0, v_step = 0, one = 0;
    // without keys no copy of keys runs; the maps still need an address
    const bool keys = p.k_tokens > 0;
    const void *kn = keys ? p.k_nope : p.q, *kp = keys ? p.k_pe : p.q, *v = keys ? p.v : p.q;
    const int64_t tokens = keys ? p.k_tokens : 1;
    if (!make_map(&tq, p.q, kLatQK, p.heads, p.q_hs, p.q_tokens, p.q_ts, &q_step) ||
        !make_map(&tk, kn, kLatN, p.heads, p.kn_hs, tokens, p.kn_ts, &k_step) ||
        !make_map(&tp, kp, kLatP, 1, 0, tokens, p.kp_ts, &one) ||
        !make_map(&tv, v, kLatN, p.heads, p.v_hs, tokens, p.v_ts, &v_step))
        return cudaErrorInvalidValue;
    static int configured = -1;
    const cudaError_t err = tc::allow_smem(latent_prefill_tc_kernel, kSmem, &configured);
    if (err != cudaSuccess) return err;
    latent_prefill_tc_kernel<<<(unsigned)blocks, kT, kSmem, p.stream>>>(p, tq, tk, tp, tv, q_step, k_step, v_step);
    return cudaGetLastError();
}

}  // namespace kda
