// latent_decode_simt.cu -- absorbed latent attention for one token per sequence on the CUDA cores
// (fp32 I/O, exact fp32 products), and the kernel that joins the parts of a split sequence for
// this form and the tensor-core one.
//
//   s_hj = scale q_h . c_j  (576 channels),  o_h = sum_j softmax_j(s_h) c_j[:512],  j < len
//
// One pass over the cache rows with a running maximum m and sum l per head (base 2): a tile's rows
// enter with p = 2^(s - m), and what is held is scaled by 2^(m_old - m) when m rises.  Bound by the chain of
// a tile (copy, products, softmax, products) and not by the fp32 rate or HBM: 16 sequences of 1 to 2,048
// rows, 8 heads, 24.6 us, of which HBM needs 5 and the products 3.6.
#include <math.h>

#include "latent.cuh"
#include "latent_ptx.cuh"

namespace kda {
namespace {

using namespace ptx;

constexpr int kT = 256;        // threads
constexpr int kRows = 32;      // cache rows per tile, one per lane
constexpr int kHeads = 8;      // heads per tile
constexpr int kLdK = kLatC + 4;  // row stride (floats) of the tile: 16-byte reads of 8 rows cover all banks
constexpr int kSpan = kLatC / 8;  // channels of one warp in the score product

struct Smem {
    float q[kHeads][kLatC];
    float k[kRows][kLdK];
    const float *row[2][kRows];  // where the tile's rows lie (null: zeros), by tile parity
    float red[8][kHeads][kRows];
    float p[kRows][kHeads];
    float alpha[kHeads];
    float ml[kHeads][2];
    int scan[kT / 32 + 2];
};

// Two CTAs on an SM overlap one's loads with the other's products.  Scores: warp w multiplies
// channels [72 w, 72 w + 72) for the tile's 32 rows (a lane each) and 8 heads, then the eight
// partial products are summed.  Output: a thread owns two of the 512 channels for 8 heads.
__global__ void __launch_bounds__(kT, 2) latent_decode_simt_kernel(const LatentDecode p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t capacity = (int64_t)p.table_width * p.page_size;
    pdl_wait();
    LatentWalk w = latent_walk<kT, float>(p, kRows, kHeads, sm.scan);
    pdl_launch_dependents();
    if (w.cta >= w.ctas) return;
    const float *cache = static_cast<const float *>(p.cache);
    bool first_unit = true;
    while (w.g < w.g_end) {
        bool ignore = false;
        const int len = latent_len(p.lens, w.b, capacity, ignore);
        const int n = (len + kRows - 1) / kRows;
        if (n == 0) {
            if (++w.b == p.batch) { w.b = 0; ++w.hg; }
            continue;
        }
        const int tile0 = w.tile, tiles = (int)min((int64_t)(n - tile0), w.g_end - w.g);
        if (tid == 0) latent_record_join(p, w, w.g, tile0, n, tiles, first_unit, kHeads);
        const int h0 = w.hg * kHeads, hs = min(kHeads, p.heads - h0);
        // the row pointers of tile t: one warp looks the pages up
        auto look_up = [&](int t) {
            const int j = t * kRows + lane;
            const float *at = nullptr;  // rows past the end count nothing, whatever they hold
            if (j < len) {
                const int page = j / p.page_size;
                const int64_t x = p.table[w.b * p.table_stride + page];
                if (x >= 0 && x < p.num_pages) at = cache + (x * p.page_size + (j - page * p.page_size)) * kLatC;
                else if (p.errors) atomicOr(p.errors, DEV_ERR_PAGE);
            }
            sm.row[t & 1][lane] = at;
        };
        __syncthreads();  // the previous unit's reads of q, k and the row pointers
        if (warp == 0) look_up(tile0);
        for (int e = tid; e < kHeads * (kLatC / 4); e += kT) {
            const int h = e / (kLatC / 4), c = 4 * (e - h * (kLatC / 4));
            cp_async16(&sm.q[h][c],
                       static_cast<const float *>(p.q) + w.b * p.q_bs + (h0 + (h < hs ? h : 0)) * p.q_hs + c, h < hs);
        }
        float m = -INFINITY, l = 0.f;  // of head `warp`, the same on every lane (l: this lane's rows)
        float acc[kHeads][2];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) acc[h][0] = acc[h][1] = 0.f;
        for (int t = tile0; t < tile0 + tiles; ++t) {
            const int j0 = t * kRows, rows = min(kRows, len - j0);
            __syncthreads();  // the previous tile's reads of k and p; this one's row pointers are there
            // a warp has four rows: 576 channels are 4.5 copies of 16 bytes a lane
#pragma unroll
            for (int r = 4 * warp; r < 4 * warp + 4; ++r) {
                const float *at = sm.row[t & 1][r];
#pragma unroll
                for (int u = 0; u < 5; ++u) {
                    const int c = 4 * (lane + 32 * u);
                    if (c < kLatC) cp_async16(&sm.k[r][c], at ? at + c : cache, at != nullptr);
                }
            }
            cp_async_commit();
            if (warp == 0 && t + 1 < tile0 + tiles) look_up(t + 1);
            cp_async_wait<0>();
            __syncthreads();
            float s[kHeads];
#pragma unroll
            for (int h = 0; h < kHeads; ++h) s[h] = 0.f;
#pragma unroll 6
            for (int c = warp * kSpan; c < (warp + 1) * kSpan; c += 4) {
                const float4 k = *reinterpret_cast<const float4 *>(&sm.k[lane][c]);
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    const float4 q = *reinterpret_cast<const float4 *>(&sm.q[h][c]);
                    s[h] += q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
                }
            }
#pragma unroll
            for (int h = 0; h < kHeads; ++h) sm.red[warp][h][lane] = s[h];
            __syncthreads();
            // head `warp`, row `lane`
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x += sm.red[i][warp][lane];
            x = lane < rows ? x * p.scale_log2 : -INFINITY;
            float mx = x;
#pragma unroll
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
            const float a = exp2f(m - base), e = exp2f(x - base);
            l = l * a + e;
            m = mn;
            sm.p[lane][warp] = e;
            if (lane == 0) sm.alpha[warp] = a;
            __syncthreads();
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                const float f = sm.alpha[h];
                acc[h][0] *= f;
                acc[h][1] *= f;
            }
#pragma unroll 8
            for (int r = 0; r < kRows; ++r) {
                const float2 v = *reinterpret_cast<const float2 *>(&sm.k[r][2 * tid]);
                const float4 pa = *reinterpret_cast<const float4 *>(&sm.p[r][0]);
                const float4 pb = *reinterpret_cast<const float4 *>(&sm.p[r][4]);
                const float ph[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    acc[h][0] += ph[h] * v.x;
                    acc[h][1] += ph[h] * v.y;
                }
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0) {
            sm.ml[warp][0] = m;
            sm.ml[warp][1] = l;
        }
        __syncthreads();
        if (tiles == n) {  // the whole unit
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                if (h >= hs) break;
                const float inv = sm.ml[h][1] == 0.f ? 0.f : 1.f / sm.ml[h][1];
                float *o = static_cast<float *>(p.o) + ((int64_t)w.b * p.heads + h0 + h) * kLatR + 2 * tid;
                *reinterpret_cast<float2 *>(o) = make_float2(acc[h][0] * inv, acc[h][1] * inv);
            }
            if (p.lse && tid < hs)
                p.lse[(int64_t)w.b * p.heads + h0 + tid] = sm.ml[tid][0] * kLn2 + logf(sm.ml[tid][1]);
        } else {
            const int slot = first_unit ? 2 * w.cta : 2 * w.cta + 1;
            float *part = latent_part(p.workspace, kHeads) + (size_t)slot * kHeads * kLatR + 2 * tid;
#pragma unroll
            for (int h = 0; h < kHeads; ++h)
                *reinterpret_cast<float2 *>(part + h * kLatR) = make_float2(acc[h][0], acc[h][1]);
            if (tid < kHeads) {
                float *ml = latent_ml(p.workspace) + ((size_t)slot * kHeads + tid) * 2;
                ml[0] = sm.ml[tid][0];
                ml[1] = sm.ml[tid][1];
            }
        }
        first_unit = false;
        w.g += tiles;
        w.tile = 0;
        if (++w.b == p.batch) { w.b = 0; ++w.hg; }
    }
}

// Joins one split unit's parts for one head: o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.  One
// CTA per (record, head), 128 threads with a float4 of the output each for every one of GROUPS groups
// of parts (i mod GROUPS; a fixed order, so the same bits on every call).  Bound by the latency of its
// loads: the first parts are asked for beside the maxima.  One group where there are many records (most
// say at once that there is nothing to join, the others have few parts), four where there are few
// (long sequences, dozens of parts): two sequences of 131k rows, 32 heads, 76 parts each: 15 us with
// one group, 5 with four.
template <typename IO, int GROUPS>
__global__ void __launch_bounds__(128 * GROUPS)
latent_join_kernel(const char *ws, int head_tile, int heads, IO *o, float *lse)
{
    constexpr int kAsk = 4;  // parts asked for at a time
    __shared__ float s_w[kLatMaxGrid];
    __shared__ float s_red[4 * GROUPS];
    __shared__ float4 s_o[GROUPS > 1 ? GROUPS - 1 : 1][128];
    pdl_wait();  // launched early behind the kernel that wrote the parts
    pdl_launch_dependents();
    const LatentJoin j = reinterpret_cast<const LatentJoin *>(ws)[blockIdx.x];
    const int hl = blockIdx.y, h = j.h0 + hl, tid = threadIdx.x, quad = tid & 127, group = tid >> 7;
    if (j.b < 0 || h >= heads) return;
    const int parts = j.c_last - j.c_first + 1;
    auto slot = [&](int i) { return i == 0 ? j.first_slot : 2 * (j.c_first + i); };
    const float *ml = latent_ml(const_cast<char *>(ws));
    const float *part = latent_part(const_cast<char *>(ws), head_tile) + (size_t)hl * kLatR + 4 * quad;
    auto load = [&](int i) {
        return i < parts ? *reinterpret_cast<const float4 *>(part + (size_t)slot(i) * head_tile * kLatR)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 x[kAsk];
#pragma unroll
    for (int u = 0; u < kAsk; ++u) x[u] = load(group + u * GROUPS);
    float mx = -INFINITY;
    for (int i = tid; i < parts; i += 128 * GROUPS) mx = fmaxf(mx, ml[((size_t)slot(i) * head_tile + hl) * 2]);
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4 * GROUPS; ++w) mx = fmaxf(mx, s_red[w]);
    const float base = mx == -INFINITY ? 0.f : mx;
    __syncthreads();
    float l = 0.f;
    for (int i = tid; i < parts; i += 128 * GROUPS) {
        const float2 y = *reinterpret_cast<const float2 *>(ml + ((size_t)slot(i) * head_tile + hl) * 2);
        const float f = exp2f(y.x - base);
        s_w[i] = f;
        l += f * y.y;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if ((tid & 31) == 0) s_red[tid >> 5] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < 4 * GROUPS; ++w) l += s_red[w];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = group; i < parts; i += kAsk * GROUPS) {
        float4 y[kAsk];
#pragma unroll
        for (int u = 0; u < kAsk; ++u) y[u] = load(i + (kAsk + u) * GROUPS);
#pragma unroll
        for (int u = 0; u < kAsk; ++u) {
            const float f = i + u * GROUPS < parts ? s_w[i + u * GROUPS] : 0.f;
            acc.x += f * x[u].x; acc.y += f * x[u].y; acc.z += f * x[u].z; acc.w += f * x[u].w;
            x[u] = y[u];
        }
    }
    if (GROUPS > 1) {
        if (group > 0) s_o[group - 1][quad] = acc;
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 0; g < GROUPS - 1; ++g) {
            const float4 y = s_o[g][quad];
            acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float out[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    store_io4(o + ((int64_t)j.b * heads + h) * kLatR + 4 * quad, out);
    if (lse && tid == 0) lse[(int64_t)j.b * heads + h] = mx * kLn2 + logf(l);
}

template <typename IO>
cudaError_t launch_join(const LatentDecode &p, int head_tile, int grid)
{
    const int records = latent_join_by_unit(p.batch, p.heads, head_tile, grid)
                            ? p.batch * ((p.heads + head_tile - 1) / head_tile) : grid;
    const int heads = p.heads < head_tile ? p.heads : head_tile;
    const bool few = records * heads <= 4 * 152;  // one wave of 512 threads a CTA
    return latent_launch(few ? latent_join_kernel<IO, 4> : latent_join_kernel<IO, 1>,
                         dim3((unsigned)records, (unsigned)heads), few ? 512 : 128, 0, p.stream, 1,
                         (const char *)p.workspace, head_tile, p.heads, static_cast<IO *>(p.o), p.lse);
}

int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

}  // namespace

cudaError_t launch_latent_join(const LatentDecode &p, int head_tile, int grid)
{
    return p.dtype == KDA_DTYPE_BF16 ? launch_join<__nv_bfloat16>(p, head_tile, grid)
                                     : launch_join<float>(p, head_tile, grid);
}

size_t latent_decode_simt_ws_bytes() { return latent_ws_bytes(kHeads, kLatMaxGrid); }

cudaError_t launch_latent_decode_simt(const LatentDecode &p)
{
    const cudaError_t err = cudaFuncSetAttribute(latent_decode_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)sizeof(Smem));
    if (err != cudaSuccess) return err;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t per_seq = ((int64_t)p.table_width * p.page_size + kRows - 1) / kRows;
    const int64_t most = per_seq * p.batch * ((p.heads + kHeads - 1) / kHeads);  // no more CTAs than there can be tiles
    int grid = 2 * sms < kLatMaxGrid ? 2 * sms : kLatMaxGrid;
    if (most < grid) grid = most > 0 ? (int)most : 1;
    const cudaError_t launched =
        latent_launch(latent_decode_simt_kernel, dim3((unsigned)grid), kT, sizeof(Smem), p.stream, 1, p);
    return launched != cudaSuccess ? launched : launch_latent_join(p, kHeads, grid);
}

}  // namespace kda
