// linear_tc.cu -- projections on the tensor cores (bf16 rows on 16 bytes).
//
//   y [rows x n] = act(x [rows x k] w^T [k x n] + b) + r
//
// A tile of y is 128 rows by `width` columns of one CTA, or 256 rows by `width` of a pair (a cluster of two):
// there each CTA holds its 128 rows of x and half of w's rows, and an instruction spans both (M = 256).  The
// accumulators, fp32 in tensor memory, are doubled, so that a tile's epilogue runs while the next one's
// products do.
// Warp 0: copies (TMA); 1: matrix instructions (of a pair: in the leading CTA); 2: tensor memory; 4 to 7: the
// epilogue, a thread a row.
#include "latent_ptx.cuh"
#include "layer.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

using namespace ptx;
using tc::kdesc;

constexpr int kThreads = 256, kM = 128;
constexpr int kMaxStages = 8, kMaxWidth = 256, kDepth = 64;  // kDepth: channels of a panel, a swizzled row of 128 bytes
constexpr int kSmem = 232448;
constexpr uint64_t kWait = tc::kWaitNs;

struct Misc {
    uint64_t full[kMaxStages], empty[kMaxStages];  // full: of a pair, the leading CTA's
    uint64_t done[2], drained, freed[2];           // done: in both CTAs; freed: the leading one's
    uint32_t tmem;
    int abort;
};
// rows that an instruction reads behind those that a short last panel holds
constexpr int kSlack = kM * 128;
constexpr int kStageBytes = (kSmem - (int)sizeof(Misc) - kSlack) / 1024 * 1024;

// What the host decides for a call.
struct Plan {
    int width;        // columns of a tile
    int box;          // rows of x that a copy brings
    int panels;       // panels of a stage
    int stages;
    int tiles_m, tiles_n, group;  // tiles_m in groups that are worked on together
    uint32_t columns; // of tensor memory
    bool vec;         // rows of y start on 16 bytes
    bool vec_r, vec_b;  // those of the residual; the bias
};

// Waits for a phase; gives up after kWait ns or as soon as another role of the CTA has.  The same answer on every lane
// of the (converged) warp.
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

__device__ __forceinline__ void tile_at(const Plan &pl, int tile, int &m, int &n)
{
    const int per = pl.group * pl.tiles_n, g = tile / per, first = g * pl.group;
    const int tall = min(pl.group, pl.tiles_m - first), in = tile - g * per;
    n = in / tall;
    m = first + in - n * tall;
}

template <typename OUT>
__device__ __forceinline__ void activate16(float (&v)[16], int act)
{
    switch (act) {
    case KDA_ACT_SILU:
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activate<OUT>(v[i], KDA_ACT_SILU);
        break;
    case KDA_ACT_GELU:
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activate<OUT>(v[i], KDA_ACT_GELU);
        break;
    case KDA_ACT_SIGMOID:
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activate<OUT>(v[i], KDA_ACT_SIGMOID);
        break;
    case KDA_ACT_SOFTPLUS:
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activate<OUT>(v[i], KDA_ACT_SOFTPLUS);
        break;
    default: break;
    }
}

// 32 bytes to global memory, a whole sector (16-byte aligned; in one instruction where 32-byte aligned).
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8])
{
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// 16 consecutive elements of a row.
template <typename OUT>
struct Raw16 {
    uint32_t w[4 * sizeof(OUT)];
    __device__ __forceinline__ void load(const OUT *p)
    {
#pragma unroll
        for (size_t i = 0; i < sizeof(OUT); ++i) {
            const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(OUT) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[16])
    {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (sizeof(OUT) == 4) w[i] = __float_as_uint(v[i]);
            else if (i & 1) w[i >> 1] = tc::pack_bf16x2(v[i - 1], v[i]);
        }
    }
    __device__ __forceinline__ void store(OUT *p) const
    {
#pragma unroll
        for (size_t i = 0; i < sizeof(OUT) / 2; ++i)
            store32(reinterpret_cast<uint32_t *>(p) + 8 * i, *reinterpret_cast<const uint32_t(*)[8]>(&w[8 * i]));
    }
};

template <typename OUT, bool PAIR>
__device__ __forceinline__ void epilogue_role(Misc &mi, const Linear &p, const Plan &pl, uint32_t tmem, int rank, int first,
                                              int step)
{
    volatile int *abort = &mi.abort;
    const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t quarter = (uint32_t)((row >> 5) * 32) << 16;
    const __nv_bfloat16 *bias = static_cast<const __nv_bfloat16 *>(p.bias);
    int count = 0;
    for (int tile = first; tile < pl.tiles_m * pl.tiles_n; tile += step, ++count) {
        int m, n;
        tile_at(pl, tile, m, n);
        const int buf = count & 1, c0 = n * pl.width, left = min(pl.width, p.n - c0);
        const int64_t at = (int64_t)m * (PAIR ? 2 * kM : kM) + rank * kM + row;
        const bool mine = at < p.rows;
        const OUT *r = static_cast<const OUT *>(p.residual) + at * p.rs + c0;
        OUT *y = static_cast<OUT *>(p.y) + at * p.ys + c0;
        // the residual's next 16 columns are on their way while these are worked on
        const bool whole_r = p.residual && mine && pl.vec_r;
        Raw16<OUT> next;
        if (whole_r && left >= 16) next.load(r);
        if (!all_wait<false>(&mi.done[buf], (count >> 1) & 1, abort)) return;
        tc_fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < left; c += 16) {
            float v[16];
            tmem_ld16(tmem + buf * kMaxWidth + c + quarter, v);
            const Raw16<OUT> now = next;
            if (whole_r && left - c >= 32) next.load(r + c + 16);
            tmem_ld_wait();
            if (c + 16 >= left) {  // the accumulators may be written again
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_cluster(map_to_rank(&mi.freed[buf], 0));
                    else mbar_arrive(&mi.freed[buf]);
                }
            }
            if (bias) {
                Raw16<__nv_bfloat16> b;
                if (pl.vec_b && left - c >= 16) {
                    b.load(bias + c0 + c);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += b.get(i);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < left) v[i] += load_io(bias + c0 + c + i);
                }
            }
            activate16<OUT>(v, p.act);
            if (!mine) continue;
            if (left - c >= 16 && pl.vec && (!p.residual || pl.vec_r)) {
                if (p.residual)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += now.get(i);
                Raw16<OUT> out;
                out.set(v);
                out.store(y + c);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < left) {
                        if (p.residual) v[i] += load_io(r + c + i);
                        store_io(y + c + i, v[i]);
                    }
            }
        }
    }
}

template <typename OUT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
linear_tc_kernel(const Linear p, const Plan pl, const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw)
{
    extern __shared__ __align__(1024) unsigned char sm[];
    Misc &mi = *reinterpret_cast<Misc *>(sm + kStageBytes + kSlack);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    if (smem_u32(sm) & 1023u) {  // the swizzled panels need it; never seen
        if (tid == 0 && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&mi.full[i], 1);
            mbar_init(&mi.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&mi.done[i], 1);
            mbar_init(&mi.freed[i], PAIR ? 8 : 4);
        }
        mbar_init(&mi.drained, 1);
        fence_mbar_init();
        mi.abort = 0;
    }
    if (warp == 2) {
        if (PAIR) {
            tmem_alloc_pair(&mi.tmem, pl.columns);
        } else {
            tmem_alloc(&mi.tmem, pl.columns);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (PAIR) cluster_sync();
    tc_fence_after_sync();
    // only now: a CTA of the next kernel must not take the tensor memory that one of this kernel is waiting for
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t tmem = mi.tmem;
    const int first = PAIR ? blockIdx.x / 2 : blockIdx.x, step = PAIR ? gridDim.x / 2 : gridDim.x;
    const int tiles = pl.tiles_m * pl.tiles_n, all_panels = (p.k + kDepth - 1) / kDepth;
    const int steps = (all_panels + pl.panels - 1) / pl.panels;
    const int half = PAIR ? pl.width / 2 : pl.width;  // rows of w that this CTA holds
    const uint32_t panel_x = pl.box * 128, panel_w = half * 128, stage_bytes = pl.panels * (panel_x + panel_w);
    volatile int *abort = &mi.abort;

    if (warp == 0) {
        const bool lead = elect_lead();
        int t = 0;  // stages so far
        for (int tile = first; tile < tiles; tile += step) {
            int m, n;
            tile_at(pl, tile, m, n);
            const int row_x = m * (PAIR ? 2 * kM : kM) + rank * kM, row_w = n * pl.width + rank * half;
            bool ok = true;
            for (int s = 0; s < steps; ++s, ++t) {
                const int slot = t % pl.stages, count = min(pl.panels, all_panels - s * pl.panels);
                if (t >= pl.stages && !(ok = all_wait<PAIR>(&mi.empty[slot], (t / pl.stages - 1) & 1, abort))) break;
                if (lead) {
                    unsigned char *dst = sm + slot * stage_bytes;
                    if (rank == 0) mbar_arrive_expect_tx(&mi.full[slot], (PAIR ? 2 : 1) * count * (panel_x + panel_w));
                    const uint32_t bar = PAIR ? map_to_rank(&mi.full[slot], 0) : 0;
                    for (int i = 0; i < count; ++i) {
                        const int k = (s * pl.panels + i) * kDepth;
                        unsigned char *dx = dst + i * panel_x, *dw = dst + pl.panels * panel_x + i * panel_w;
                        if (PAIR) {
                            tma_load_3d_pair(dx, &tx, bar, k, 0, row_x);
                            tma_load_3d_pair(dw, &tw, bar, k, 0, row_w);
                        } else {
                            tma_load_3d(dx, &tx, &mi.full[slot], k, 0, row_x);
                            tma_load_3d(dw, &tw, &mi.full[slot], k, 0, row_w);
                        }
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        // no copy in flight when the CTAs go, whatever became of the products
        if (lead && rank == 0)
            for (int k = max(0, t - pl.stages); k < t; ++k)
                mbar_wait_ns(&mi.full[k % pl.stages], (k / pl.stages) & 1, kWait);
    } else if (warp == 1 && rank == 0) {
        const uint32_t lead = elect_lead(), base = __reduce_or_sync(0xffffffffu, tmem), sb = smem_u32(sm);
        const uint32_t id = idesc_bf16(PAIR ? 2 * kM : kM, pl.width, false, false);
        int t = 0, count = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step, ++count) {
            const int buf = count & 1;
            if (count >= 2 && !(ok = all_wait<PAIR>(&mi.freed[buf], ((count >> 1) - 1) & 1, abort))) break;
            tc_fence_after_sync();
            const uint32_t d = base + buf * kMaxWidth;
            for (int s = 0; s < steps; ++s, ++t) {
                const int slot = t % pl.stages, held = min(pl.panels, all_panels - s * pl.panels);
                if (!(ok = all_wait<PAIR>(&mi.full[slot], (t / pl.stages) & 1, abort))) break;
                tc_fence_after_sync();
                const uint32_t a = sb + slot * stage_bytes, b = a + pl.panels * panel_x;
                for (int i = 0; i < held; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t da = kdesc(a + i * panel_x + k * 32), db = kdesc(b + i * panel_w + k * 32);
                        if (PAIR) mma_bf16_pair(lead, d, da, db, id, s > 0 || i > 0 || k > 0);
                        else mma_bf16_lead(lead, d, da, db, id, s > 0 || i > 0 || k > 0);
                    }
                if (PAIR) mma_commit_pair(lead, &mi.empty[slot]);
                else mma_commit_lead(lead, &mi.empty[slot]);
            }
            if (!ok) break;
            if (PAIR) mma_commit_pair(lead, &mi.done[buf]);
            else mma_commit_lead(lead, &mi.done[buf]);
        }
        // nothing in flight when tensor memory is given back, whatever became of the epilogue
        if (PAIR) mma_commit_pair(lead, &mi.drained);
        else mma_commit_lead(lead, &mi.drained);
        if (lane == 0) mbar_wait_ns(&mi.drained, 0, kWait);
    } else if (warp >= 4) {
        epilogue_role<OUT, PAIR>(mi, p, pl, tmem, rank, first, step);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA goes while the other's instructions use its memory
    if (warp == 2) {
        tc_fence_after_sync();
        if (PAIR) tmem_dealloc_pair(tmem, pl.columns);
        else tmem_dealloc(tmem, pl.columns);
    }
    if (tid == 0 && mi.abort && p.errors) atomicOr(p.errors, DEV_ERR_TIMEOUT);
}

bool make_map(CUtensorMap *m, const void *ptr, int k, int64_t rows, int64_t stride, int box_rows)
{
    tc::EncodeTiledFn enc = tc::encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)k, 1, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {kDepth, 1, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rows_on(const void *p, int64_t stride, int64_t rows, size_t es)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || (size_t)stride * es % 16 == 0);
}

// The width of a tile: as few rounds of `at_once` tiles as possible, each as narrow as possible (`extra`: what a
// round costs beside its columns, in columns).
int tile_width(int n, int64_t tiles_m, int at_once, int extra)
{
    int best = 0;
    int64_t least = 0;
    for (int w = 16; w <= kMaxWidth; w += 16) {
        const int64_t tiles = tiles_m * ((n + w - 1) / w), cost = (tiles + at_once - 1) / at_once * (w + extra);
        if (best == 0 || cost < least) {
            best = w;
            least = cost;
        }
        if (w >= n) break;
    }
    return best;
}

}  // namespace

bool linear_tc_takes(const Linear &p)
{
    auto fits = [&](const void *q, int64_t stride, int64_t rows) {
        return rows_on(q, stride, rows, 2) && (rows <= 1 || stride >= p.k);
    };
    return p.dtype == KDA_DTYPE_BF16 && p.k % 8 == 0 && fits(p.x, p.xs, p.rows) && fits(p.w, p.ws, p.n);
}

cudaError_t launch_linear_tc(const Linear &p)
{
    constexpr int kSms = 152;
    const bool pair = p.rows > kM && p.n > 64;
    Plan pl;
    const int tall = pair ? 2 * kM : kM;
    const int64_t tiles_m = (p.rows + tall - 1) / tall;
    pl.width = tile_width(p.n, tiles_m, pair ? kSms / 2 : kSms, 32);
    const int64_t tiles_n = (p.n + pl.width - 1) / pl.width;
    if (tiles_m * tiles_n > INT32_MAX) return cudaErrorInvalidValue;
    pl.tiles_m = (int)tiles_m; pl.tiles_n = (int)tiles_n;
    pl.group = 8;
    pl.box = (int)(p.rows < kM ? (p.rows + 7) / 8 * 8 : kM);
    const int half = pair ? pl.width / 2 : pl.width, panel = (pl.box + half) * 128;
    pl.panels = panel <= 8192 ? 4 : panel <= 16384 ? 2 : 1;
    pl.stages = kStageBytes / (panel * pl.panels);
    if (pl.stages > kMaxStages) pl.stages = kMaxStages;
    pl.columns = 512;
    const size_t eo = p.out_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    pl.vec = rows_on(p.y, p.ys, p.rows, eo);
    pl.vec_r = rows_on(p.residual, p.rs, p.rows, eo);
    pl.vec_b = rows_on(p.bias, 0, 1, 2);
    CUtensorMap tx, tw;
    if (!make_map(&tx, p.x, p.k, p.rows, p.rows > 1 ? p.xs : p.k, pl.box) ||
        !make_map(&tw, p.w, p.k, p.n, p.n > 1 ? p.ws : p.k, half))
        return cudaErrorInvalidValue;
    const int64_t at_once = pair ? kSms / 2 : kSms, tiles = tiles_m * tiles_n;
    const unsigned blocks = (unsigned)((tiles < at_once ? tiles : at_once) * (pair ? 2 : 1));
    auto launch = [&](auto kernel, int *configured) -> cudaError_t {
        const cudaError_t err = tc::allow_smem(kernel, kSmem, configured);
        if (err != cudaSuccess) return err;
        return latent_launch(kernel, dim3(blocks), kThreads, kSmem, p.stream, pair ? 2 : 1, p, pl, tx, tw);
    };
    static int set[4] = {-1, -1, -1, -1};
    const bool f32 = p.out_dtype == KDA_DTYPE_F32;
    return pair ? f32 ? launch(linear_tc_kernel<float, true>, &set[0]) : launch(linear_tc_kernel<__nv_bfloat16, true>, &set[1])
                : f32 ? launch(linear_tc_kernel<float, false>, &set[2]) : launch(linear_tc_kernel<__nv_bfloat16, false>, &set[3]);
}

}  // namespace kda
