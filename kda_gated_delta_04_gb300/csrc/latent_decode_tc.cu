// latent_decode_tc.cu -- absorbed latent attention for one token per sequence on the tensor cores
// (bf16 I/O).
//
//   s_hj = scale q_h . c_j  (576 channels),  o_h = sum_j softmax_j(s_h) c_j[:512],  j < len
//
// All heads read the same cache rows, so a row is worth one read: 1,152 bytes against
// 2 x 1,088 x H operations.  Up to about 128 heads the cache's bytes are the bound.  Both products
// are computed transposed, cache rows (or channels) as the M dimension and heads as N:
//
//   S^T [64 rows x H]   = C [64 x 576] Q^T            (M = 64, N = H, 36 steps of K = 16)
//   O^T [512 x H]      += C[:, :512]^T P^T [64 x H]   (4 x M = 128, N = H, 4 steps of K = 16)
//
// so that no part of a matrix instruction is spent on padding a few heads to a tile of 128: a
// tile's cost is reading it from shared memory twice, below the time HBM takes to deliver it.  O^T
// stays in tensor memory for the whole of a sequence (4 H columns), the two S^T buffers beside it.
//
// One CTA per SM, 384 threads: warp 0 copies cache rows (TMA), warps 1 and 2 issue the two products,
// warp 3 copies a sequence's queries, warps 4 to 11 do the softmax (a
// warpgroup for each half of the heads).  The cache rows arrive as 64-row
// panels of 64 channels in rings of pieces: the position channels (read by S^T only, freed early)
// in one, pairs of latent panels (read by both products) in the other.  S^T of tile t + 1 is issued
// before O^T of tile t, so the softmax of one tile runs beside the products of its neighbours, and
// the rings hold 2 to 2.7 tiles: while one is worked on, the others are in flight (100 KB and more a
// SM; 45 KB cover HBM's latency at its full rate).  256 sequences of 1 to 8,192 rows, 32 heads: 217 to 222 us, 5.8 to
// 5.9 TB/s.  That is with pages of 64 rows and more: a copy never leaves a page, and a tile of 9 copies of 8 KB takes
// 36 of 2 KB with pages of 16 rows or 48 (215 us become 263) and 72 of 1 KB with 8 (380); pages of 32 are as good
// as whole tiles (218).
#include <math.h>

#include "latent.cuh"
#include "latent_ptx.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

using namespace ptx;
using tc::kdesc;

constexpr int kT = 384;
constexpr int kSoft = 256;                // threads of the softmax: two warpgroups, half of the heads each
constexpr int kRows = 64;                 // cache rows per tile
constexpr uint32_t kPanel = kRows * 128;  // bytes of a panel: 64 rows x 64 channels
constexpr uint32_t kPair = 2 * kPanel;
constexpr int kSmemMax = 232448;          // 227 KB, the most a CTA can have
constexpr uint64_t kWait = tc::kWaitNs;
constexpr float kSlack = 8.f;  // log2: how far scores may pass the held maximum before it is moved

template <int NH>
struct Cfg {
    static constexpr int NP = NH == 64 ? 1 : 2;  // P buffers (one where a second would cost a piece of the ring)
    static constexpr int NB = NH == 64 ? 2 : (NH == 32 ? 2 : 3);    // position-panel slots
    static constexpr int NA = NH == 64 ? 8 : (NH == 32 ? 10 : 11);  // latent-pair slots (4 a tile)
    static constexpr uint32_t Q = 0;
    static constexpr uint32_t P = Q + 9 * NH * 128;
    static constexpr uint32_t A = P + NP * NH * 128;
    static constexpr uint32_t B = A + NA * kPair;
    static constexpr uint32_t MISC = B + NB * kPanel;
    static constexpr uint32_t COLS = NH == 64 ? 512 : (NH == 32 ? 256 : 128);  // 6 NH columns, a power of two
    static constexpr uint32_t SCOL = 4 * NH;                                   // S^T buffers after O^T
};

template <int NH>
struct Misc {
    uint64_t full_a[Cfg<NH>::NA], empty_a[Cfg<NH>::NA], full_b[Cfg<NH>::NB], empty_b[Cfg<NH>::NB];
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], q_full, q_empty, o_full, o_empty, drained;
    uint32_t tmem;
    int abort;
    alignas(16) float red[2][4][NH];  // (read as float4) per warp: a tile's column maxima (by tile parity), at the end the sums
    float fac[NH];        // rescaling factors, at the end 1 / sum
    int scan[kT / 32 + 2];
};

// Waits for a phase; gives up after kWait ns or as soon as another role has.
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

// A whole warp's wait: the same answer on every lane.
__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

// The units of this CTA, in order, as each role walks them.
struct Units {
    const LatentDecode &p;
    LatentWalk w;
    int64_t capacity;
    int len, n, tile0, tiles;  // current unit: rows, tiles, this CTA's part
    bool first;
    __device__ __forceinline__ Units(const LatentDecode &p_, const LatentWalk &w_)
        : p(p_), w(w_), capacity((int64_t)p_.table_width * p_.page_size), len(0), n(0), tile0(0), tiles(0), first(true)
    {
    }
    __device__ __forceinline__ bool next()
    {
        if (tiles > 0) {
            first = false;
            advance();
        }
        while (w.g < w.g_end) {
            bool ignore = false;
            len = latent_len(p.lens, w.b, capacity, ignore);
            n = (len + kRows - 1) / kRows;
            if (n > 0) {
                tile0 = w.tile;
                tiles = (int)min((int64_t)(n - tile0), w.g_end - w.g);
                w.g += tiles;
                return true;
            }
            advance();
        }
        return false;
    }
    __device__ __forceinline__ void advance()
    {
        w.tile = 0;
        if (++w.b == p.batch) {
            w.b = 0;
            ++w.hg;
        }
    }
};

// Reduces r[0..n) over 16 lanes (a half warp), splitting the values among them: afterwards r[0..)
// of a lane holds the results of the columns starting at the returned index, `per` of them.
template <int N, bool MAX>
__device__ __forceinline__ int half_warp_reduce(float (&r)[N], int lane)
{
    int at = 0, cnt = N;
#pragma unroll
    for (int m = 8; m; m >>= 1) {
        if (cnt > 1) {
            const int half = cnt / 2;
            const bool up = lane & m;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i >= half) break;
                const float send = up ? r[i] : r[i + half], keep = up ? r[i + half] : r[i];
                const float got = __shfl_xor_sync(0xffffffffu, send, m);
                r[i] = MAX ? fmaxf(keep, got) : keep + got;
            }
            at += up ? half : 0;
            cnt = half;
        } else {
            const float got = __shfl_xor_sync(0xffffffffu, r[0], m);
            r[0] = MAX ? fmaxf(r[0], got) : r[0] + got;
        }
    }
    return at;
}

// This thread's half of a row of S^T: N columns (16 lanes a warp hold rows, two threads each).
template <int N>
__device__ __forceinline__ void load_scores(uint32_t t, float (&s)[N])
{
    if constexpr (N == 4) tmem_ld16x2_x4<4>(t, s);
    else if constexpr (N == 8) tmem_ld16x2_x8<8>(t, s);
    else tmem_ld16x2_x16<16>(t, s);
}

// 8 or 16 consecutive columns of a lane.
__device__ __forceinline__ void load_cols(uint32_t t, float (&x)[8]) { tmem_ld8(t, x); }
__device__ __forceinline__ void load_cols(uint32_t t, float (&x)[16]) { tmem_ld16(t, x); }
__device__ __forceinline__ void store_cols(uint32_t t, const float (&x)[8])
{
    tmem_st8(t, *reinterpret_cast<const uint32_t(*)[8]>(&x));
}
__device__ __forceinline__ void store_cols(uint32_t t, const float (&x)[16]) { tmem_st16(t, x); }

template <int NH>
__device__ __forceinline__ void copy_role(unsigned char *sm, Misc<NH> &mi, const LatentDecode &p, Units u,
                                          const CUtensorMap &tm, int piece_rows, int lane)
{
    using C = Cfg<NH>;
    const int pieces = kRows / piece_rows;  // copies per panel: 1, 2, 4 or 8
    const int batch = 32 / pieces;          // tiles whose pages the warp looks up at once
    const int64_t outside = max(p.num_pages * (int64_t)p.page_size, (int64_t)1);  // past the cache: copied as zeros
    int ts = 0, na = 0, nb = 0;
    volatile int *abort = &mi.abort;
    while (u.next()) {
        // row of the cache at which piece (lane % pieces) of tile (t + lane / pieces) starts
        auto entry = [&](int t, int &j) -> int {  // its page; -1: it is past the end
            j = (u.tile0 + t + lane / pieces) * kRows + (lane % pieces) * piece_rows;
            return t + lane / pieces < u.tiles && j < u.len ? p.table[u.w.b * p.table_stride + j / p.page_size] : -1;
        };
        auto row_of = [&](int page, int j, bool asked) -> int {
            if (page >= 0 && page < p.num_pages) return page * p.page_size + j % p.page_size;
            if (asked && p.errors) atomicOr(p.errors, DEV_ERR_PAGE);
            return (int)outside;
        };
        auto asked = [&](int t, int j) { return t + lane / pieces < u.tiles && j < u.len; };
        int j0, j1;
        const int page0 = entry(0, j0), page1 = entry(batch, j1);  // (both loads on their way)
        int rows = row_of(page0, j0, asked(0, j0)), later = row_of(page1, j1, asked(batch, j1));
        for (int t = 0; t < u.tiles; ++t, ++ts) {
            const int in = t % batch;
            if (in == 0 && t > 0) {
                rows = later;
                const int page = entry(t + batch, j1);
                later = row_of(page, j1, asked(t + batch, j1));
            }
            const int row = __shfl_sync(0xffffffffu, rows, in * pieces + (lane & (pieces - 1)));
            bool ok = true;
            if (nb >= C::NB) ok = wait(&mi.empty_b[nb % C::NB], (nb / C::NB - 1) & 1, abort);
            if (!__all_sync(0xffffffffu, ok)) goto gave_up;
            uint64_t *bar = &mi.full_b[nb % C::NB];
            unsigned char *dst = sm + C::B + (nb % C::NB) * kPanel;
            if (lane == 0) mbar_arrive_expect_tx(bar, kPanel);
            __syncwarp();
            if (lane < pieces) tma_load_3d(dst + lane * piece_rows * 128, &tm, bar, 0, row, 8);
            ++nb;
            for (int i = 0; i < 4; ++i, ++na) {
                const int slot = na % C::NA;
                if (na >= C::NA) ok = wait(&mi.empty_a[slot], (na / C::NA - 1) & 1, abort);
                if (!__all_sync(0xffffffffu, ok)) goto gave_up;
                bar = &mi.full_a[slot];
                dst = sm + C::A + slot * kPair;
                if (lane == 0) mbar_arrive_expect_tx(bar, kPair);
                __syncwarp();
                if (lane < pieces) {
                    tma_load_3d(dst + lane * piece_rows * 128, &tm, bar, 0, row, 2 * i);
                    tma_load_3d(dst + kPanel + lane * piece_rows * 128, &tm, bar, 0, row, 2 * i + 1);
                }
            }
        }
    }
    return;
gave_up:  // the copies in flight land before the CTA goes
    if (lane == 0) {
        for (int k = max(0, nb - C::NB); k < nb; ++k) mbar_wait_ns(&mi.full_b[k % C::NB], (k / C::NB) & 1, kWait);
        for (int k = max(0, na - C::NA); k < na; ++k) mbar_wait_ns(&mi.full_a[k % C::NA], (k / C::NA) & 1, kWait);
    }
}

// S^T of every tile; one warp, in step.
template <int NH>
__device__ __forceinline__ bool score_role(uint32_t sb, Misc<NH> &mi, Units u, uint32_t tmem)
{
    using C = Cfg<NH>;
    constexpr uint32_t id = idesc_bf16(64, NH, false, false);
    volatile int *abort = &mi.abort;
    const uint32_t lead = elect_lead();
    int ts = 0, units = 0;
    while (u.next()) {
        if (!all_wait(&mi.q_full, units & 1, abort)) return false;
        ++units;
        for (int t = 0; t < u.tiles; ++t, ++ts) {
            if (ts >= 2 && !all_wait(&mi.s_empty[ts & 1], (ts / 2 - 1) & 1, abort)) return false;
            if (!all_wait(&mi.full_b[ts % C::NB], (ts / C::NB) & 1, abort)) return false;
            tc_fence_after_sync();
            const uint32_t d = tmem + C::SCOL + (ts & 1) * NH;
            const uint32_t b = sb + C::B + (ts % C::NB) * kPanel;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16_lead(lead, d, kdesc(b + k * 32), kdesc(sb + C::Q + 8 * NH * 128 + k * 32), id, k > 0);
            mma_commit_lead(lead, &mi.empty_b[ts % C::NB]);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int na = 4 * ts + i, slot = na % C::NA;
                if (!all_wait(&mi.full_a[slot], (na / C::NA) & 1, abort)) return false;
                const uint32_t a = sb + C::A + slot * kPair;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_bf16_lead(lead, d, kdesc(a + (k >> 2) * kPanel + (k & 3) * 32),
                                  kdesc(sb + C::Q + (2 * i + (k >> 2)) * NH * 128 + (k & 3) * 32), id, 1);
            }
            mma_commit_lead(lead, &mi.s_full[ts & 1]);
            if (t + 1 == u.tiles) mma_commit_lead(lead, &mi.q_empty);
        }
    }
    return true;
}

// O^T += C^T P^T of every tile; one warp, in step.  Its own warp, so that the waits of one product
// (about 100 cycles each, ready or not) pass while the other's instructions run.
template <int NH>
__device__ __forceinline__ bool value_role(uint32_t sb, Misc<NH> &mi, Units u, uint32_t tmem)
{
    using C = Cfg<NH>;
    constexpr uint32_t id = idesc_bf16(128, NH, true, false);
    volatile int *abort = &mi.abort;
    const uint32_t lead = elect_lead();
    int ts = 0, units = 0;
    while (u.next()) {
        if (units > 0 && !all_wait(&mi.o_empty, (units - 1) & 1, abort)) return false;
        ++units;
        for (int t = 0; t < u.tiles; ++t, ++ts) {
            if (!all_wait(&mi.p_full[ts % C::NP], (ts / C::NP) & 1, abort)) return false;
            tc_fence_after_sync();
            const uint32_t pb = sb + C::P + (ts % C::NP) * (NH * 128);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int slot = (4 * ts + i) % C::NA;
                const uint32_t a = sb + C::A + slot * kPair;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16_lead(lead, tmem + i * NH, sdesc(a + k * 2048, kPanel, 1024, kSw128B), kdesc(pb + k * 32), id,
                                  t > 0 || k > 0);
                mma_commit_lead(lead, &mi.empty_a[slot]);
            }
            mma_commit_lead(lead, &mi.p_empty[ts % C::NP]);
            if (t + 1 == u.tiles) mma_commit_lead(lead, &mi.o_full);
        }
    }
    return true;
}

// The queries of each unit (TMA); one warp, so that the cache rows' copies never wait for it.
template <int NH>
__device__ __forceinline__ void query_role(unsigned char *sm, Misc<NH> &mi, const LatentDecode &p, Units u,
                                           const CUtensorMap &tq, int b_step, int h_step, int lane)
{
    using C = Cfg<NH>;
    volatile int *abort = &mi.abort;
    int units = 0;
    bool ok = true;
    while (ok && u.next()) {
        if (units > 0 && !(ok = all_wait(&mi.q_empty, (units - 1) & 1, abort))) break;
        if (lane == 0) {
            mbar_arrive_expect_tx(&mi.q_full, 9 * NH * 128);
#pragma unroll
            for (int c = 0; c < 9; ++c)
                tma_load_3d(sm + C::Q + c * NH * 128, &tq, &mi.q_full, 64 * c, u.w.hg * NH * h_step, u.w.b * b_step);
        }
        ++units;
    }
    if (!ok && units > 0 && lane == 0) mbar_wait_ns(&mi.q_full, (units - 1) & 1, kWait);
}

// Softmax of half of the heads (`part`): one warpgroup.  A thread has one cache row of the tile and N
// heads of it; a head's maximum is taken over 16 lanes and then four warps.
template <int NH>
__device__ __forceinline__ void softmax_role(unsigned char *sm, Misc<NH> &mi, const LatentDecode &p, Units u,
                                             uint32_t tmem, int part, int tid)
{
    using C = Cfg<NH>;
    constexpr int N = NH / 4, HALF = NH / 2, CH = HALF < 16 ? HALF : 16;
    volatile int *abort = &mi.abort;
    const int warp = tid >> 5, lane = tid & 31, side = lane >> 4, row = 16 * warp + (lane & 15);
    const int head0 = part * HALF, mine = head0 + side * N;  // first head of the warpgroup, of this thread
    const uint32_t quarter = (uint32_t)(warp * 32) << 16, bar = 1 + part;
    int ts = 0, units = 0;
    bool bad = false;  // a wait gave up: the next barrier takes all four warps out together
    // every head column of O^T that this warpgroup has: 4 M tiles x HALF columns, CH at a time
    auto columns = [&](auto &&f) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < HALF; c += CH) f(i, head0 + c);
    };
    while (u.next()) {
        if (part == 0 && tid == 0) latent_record_join(p, u.w, u.w.g - u.tiles, u.tile0, u.n, u.tiles, u.first, NH);
        float m[N], l[N];  // of heads mine + i: the held maximum (log2 units), this row's share of the sum
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
        for (int t = 0; t < u.tiles; ++t, ++ts) {
            float s[N], r[N];
            bad |= !wait(&mi.s_full[ts & 1], (ts / 2) & 1, abort);
            __syncwarp();
            tc_fence_after_sync();
            load_scores<N>(tmem + C::SCOL + (ts & 1) * NH + head0 + quarter, s);
            tmem_ld_wait();
            tc_fence_before_sync();
            mbar_arrive(&mi.s_empty[ts & 1]);
            const int left = u.len - (u.tile0 + t) * kRows;  // rows of the tile that count
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = s[i] = row < left ? s[i] * p.scale_log2 : -INFINITY;
            const int at = mine + half_warp_reduce<N, true>(r, lane);
            mi.red[ts & 1][warp][at] = r[0];
            if (bar_sync_or(bar, 128, bad)) return;
            bool rise = false;
            float top[N];
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                float4 a = *reinterpret_cast<const float4 *>(&mi.red[ts & 1][0][mine + i]);
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                    const float4 b = *reinterpret_cast<const float4 *>(&mi.red[ts & 1][w][mine + i]);
                    a = make_float4(fmaxf(a.x, b.x), fmaxf(a.y, b.y), fmaxf(a.z, b.z), fmaxf(a.w, b.w));
                }
                top[i] = a.x; top[i + 1] = a.y; top[i + 2] = a.z; top[i + 3] = a.w;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) rise |= top[i] > m[i] + kSlack;
            // the same in the four warps (each has both sides): all see the same maxima
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float mn = fmaxf(m[i], top[i]);
                    const float f = mn == m[i] ? 1.f : tc::exp2_approx(m[i] - mn);
                    m[i] = mn;
                    l[i] *= f;
                    if (warp == 0 && (lane & 15) == 0) mi.fac[mine + i] = f;
                }
                if (t > 0) {  // what O^T holds follows
                    bad |= !wait(&mi.p_empty[(ts - 1) % C::NP], ((ts - 1) / C::NP) & 1, abort);
                    if (bar_sync_or(bar, 128, bad)) return;
                    tc_fence_after_sync();
                    columns([&](int i, int h) {
                        float x[CH];
                        load_cols(tmem + quarter + i * NH + h, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < CH; ++k) x[k] *= mi.fac[h + k];
                        store_cols(tmem + quarter + i * NH + h, x);
                    });
                    tmem_st_wait();
                    tc_fence_before_sync();
                    if (bar_sync_or(bar, 128, bad)) return;  // the factors are read before the next rise
                }
            }
            if (ts >= C::NP) bad |= !wait(&mi.p_empty[ts % C::NP], (ts / C::NP - 1) & 1, abort);
            unsigned char *pb = sm + C::P + (ts % C::NP) * (NH * 128);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float e = tc::exp2_approx(s[i] - (m[i] == -INFINITY ? 0.f : m[i]));
                l[i] += e;
                // bf16: the product's operands share one type, and V is bf16
                tc::store_bf16(pb + tc::km16(mine + i, row, NH), e);
            }
            if (left < kRows) {  // rows past the end may hold anything: their weight is 0, so their values must be finite
                for (int e = part * 128 + tid; e < (kRows - left) * 64; e += kSoft) {
                    const int rr = left + (e >> 6), c = e & 63;  // 16-byte piece c of the row's 8 panels
                    const int slot = (4 * ts + (c >> 4)) % C::NA;
                    *reinterpret_cast<uint4 *>(sm + C::A + slot * kPair + ((c >> 3) & 1) * kPanel + rr * 128 +
                                               (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&mi.p_full[ts % C::NP]);
        }
        // the unit's end: sums over the rows, then O^T out
        float r[N];
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = l[i];
        const int at = mine + half_warp_reduce<N, false>(r, lane);
        bad |= !wait(&mi.o_full, units & 1, abort);
        ++units;
        if (bar_sync_or(bar, 128, bad)) return;  // every read of the last maxima is done
        mi.red[0][warp][at] = r[0];
        if (warp == 0 && (lane & 15) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) mi.red[1][0][mine + i] = m[i];
        if (bar_sync_or(bar, 128, bad)) return;
        const int h0 = u.w.hg * NH, hs = min(NH, p.heads - h0);
        const bool whole = u.tiles == u.n;
        const int slot = u.first ? 2 * u.w.cta : 2 * u.w.cta + 1;
        if (tid < HALF) {
            const int h = head0 + tid;
            const float sum = (mi.red[0][0][h] + mi.red[0][1][h]) + (mi.red[0][2][h] + mi.red[0][3][h]);
            const float mx = mi.red[1][0][h];
            mi.fac[h] = sum == 0.f ? 0.f : 1.f / sum;
            if (whole) {
                if (p.lse && h < hs) p.lse[(int64_t)u.w.b * p.heads + h0 + h] = mx * kLn2 + logf(sum);
            } else {
                float *ml = latent_ml(p.workspace) + ((size_t)slot * NH + h) * 2;
                ml[0] = mx;
                ml[1] = sum;
            }
        }
        if (bar_sync_or(bar, 128, bad)) return;
        tc_fence_after_sync();
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + ((int64_t)u.w.b * p.heads + h0) * kLatR + tid;
        float *out = latent_part(p.workspace, NH) + (size_t)slot * NH * kLatR + tid;
        columns([&](int i, int h) {  // channels 128 i + tid of heads h ...
            float x[CH];
            load_cols(tmem + quarter + i * NH + h, x);
            tmem_ld_wait();
            if (whole) {
#pragma unroll
                for (int k = 0; k < CH; ++k)
                    if (h + k < hs) store_io(o + (size_t)(h + k) * kLatR + 128 * i, x[k] * mi.fac[h + k]);
            } else {
#pragma unroll
                for (int k = 0; k < CH; ++k)
                    if (h + k < hs) out[(size_t)(h + k) * kLatR + 128 * i] = x[k];
            }
        });
        tc_fence_before_sync();
        mbar_arrive(&mi.o_empty);
        if (bar_sync_or(bar, 128, bad)) return;  // fac and red are free again
    }
}

template <int NH>
__global__ void __launch_bounds__(kT, 1)
latent_decode_tc_kernel(const LatentDecode p, const __grid_constant__ CUtensorMap tm,
                        const __grid_constant__ CUtensorMap tq, int piece_rows, int b_step, int h_step)
{
    using C = Cfg<NH>;
    static_assert(C::MISC + sizeof(Misc<NH>) <= kSmemMax, "shared memory");
    extern __shared__ __align__(1024) unsigned char sm[];
    Misc<NH> &mi = *reinterpret_cast<Misc<NH> *>(sm + C::MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(sm) & 1023u) {  // the swizzled panels need it; never seen
        if (tid == 0 && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        prefetch_tmap(&tm);
        prefetch_tmap(&tq);
        for (int i = 0; i < C::NA; ++i) {
            mbar_init(&mi.full_a[i], 1);
            mbar_init(&mi.empty_a[i], 1);
        }
        for (int i = 0; i < C::NB; ++i) {
            mbar_init(&mi.full_b[i], 1);
            mbar_init(&mi.empty_b[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&mi.s_full[i], 1);
            mbar_init(&mi.s_empty[i], kSoft);
            mbar_init(&mi.p_full[i], kSoft);
            mbar_init(&mi.p_empty[i], 1);
        }
        mbar_init(&mi.q_full, 1);
        mbar_init(&mi.q_empty, 1);
        mbar_init(&mi.o_full, 1);
        mbar_init(&mi.o_empty, kSoft);
        mbar_init(&mi.drained, 2);
        fence_mbar_init();
        mi.abort = 0;
    }
    if (warp == 1) {
        tmem_alloc(&mi.tmem, C::COLS);
        tmem_relinquish();
    }
    pdl_wait();
    const LatentWalk w = latent_walk<kT, __nv_bfloat16>(p, kRows, NH, mi.scan);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = mi.tmem;
    pdl_launch_dependents();
    if (w.cta < w.ctas) {
        const Units u(p, w);
        if (warp == 0) copy_role<NH>(sm, mi, p, u, tm, piece_rows, lane);
        else if (warp < 3) {
            // (the reduction's result is uniform to the compiler, the loaded word is not)
            const uint32_t t = __reduce_or_sync(0xffffffffu, tmem);
            if (!(warp == 1 ? score_role<NH>(smem_u32(sm), mi, u, t) : value_role<NH>(smem_u32(sm), mi, u, t))) {
                // nothing in flight when tensor memory is given back
                mma_commit_lead(lane == 0, &mi.drained);
                if (lane == 0) mbar_wait_ns(&mi.drained, 0, kWait);
            }
        } else if (warp == 3) query_role<NH>(sm, mi, p, u, tq, b_step, h_step, lane);
        else softmax_role<NH>(sm, mi, p, u, tmem, (warp - 4) >> 2, (tid - 128) & 127);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::COLS);
    }
    if (tid == 0 && mi.abort && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
}

template <int NH>
cudaError_t launch(const LatentDecode &p, int grid)
{
    tc::EncodeTiledFn enc = tc::encode_fn();
    if (!enc) return cudaErrorNotSupported;
    static int configured = -1;
    cudaError_t err = tc::allow_smem(latent_decode_tc_kernel<NH>, kSmemMax, &configured);
    if (err != cudaSuccess) return err;
    // the cache as [channel panel][row][64 channels]; a copy is one panel of the rows that tile and
    // page have in common
    int piece = 64;
    while (p.page_size % piece) piece /= 2;
    const int64_t rows = p.num_pages * p.page_size;
    CUtensorMap tm;
    const cuuint64_t dims[3] = {64, (cuuint64_t)(rows > 0 ? rows : 1), 9};
    const cuuint64_t strides[2] = {kLatC * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)piece, 1}, es[3] = {1, 1, 1};
    // (without pages every copy starts past the one row that is declared)
    void *base = rows > 0 ? const_cast<void *>(p.cache) : static_cast<void *>(p.workspace);
    if (enc(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    // the queries as [batch][heads][channels]; a step of 0 where heads or sequences share their rows
    const int h_step = p.q_hs ? 1 : 0, b_step = p.q_bs ? 1 : 0;
    CUtensorMap tq;
    const cuuint64_t qdims[3] = {kLatC, (cuuint64_t)(h_step ? p.heads : 1), (cuuint64_t)(b_step ? p.batch : 1)};
    const cuuint64_t qstrides[2] = {(cuuint64_t)(h_step ? p.q_hs : kLatC) * 2, (cuuint64_t)(b_step ? p.q_bs : kLatC) * 2};
    const cuuint32_t qbox[3] = {64, NH, 1};
    if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p.q), qdims, qstrides, qbox, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    err = latent_launch(latent_decode_tc_kernel<NH>, dim3((unsigned)grid), kT, kSmemMax, p.stream, 1, p, tm, tq, piece,
                        b_step, h_step);
    return err != cudaSuccess ? err : launch_latent_join(p, NH, grid);
}

// Heads of a tile: the least of 16, 32 and 64 that holds them all (else tiles of 64), since a smaller tile leaves
// more shared memory to the ring and costs the tensor cores less, and each further tile reads the cache rows once
// more (from L2).
// 256 sequences of up to 8,192 rows: 16 heads 210 us in a tile of 16, 216 of 32, 243 of 64; 32 heads 217 in a
// tile of 32, 249 of 64.  48 of up to 8,192 rows, 128 heads: 117 us in tiles of 64, 175 of 32.  The tile of 64
// has a ring of two cache tiles, too short to hide a copy's latency: the tensor pipe is 42 % busy.
int head_tile(int heads) { return heads <= 16 ? 16 : (heads <= 32 ? 32 : 64); }

}  // namespace

size_t latent_decode_tc_ws_bytes(int heads) { return latent_ws_bytes(head_tile(heads), 152); }

cudaError_t launch_latent_decode_tc(const LatentDecode &p)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    const int nh = head_tile(p.heads);
    // no more CTAs than there can be tiles
    const int64_t per_seq = ((int64_t)p.table_width * p.page_size + kRows - 1) / kRows;
    const int64_t most = per_seq * p.batch * ((p.heads + nh - 1) / nh);
    int grid = sms < 152 ? sms : 152;
    if (most < grid) grid = most > 0 ? (int)most : 1;
    return nh == 16 ? launch<16>(p, grid) : nh == 32 ? launch<32>(p, grid) : launch<64>(p, grid);
}

}  // namespace kda
