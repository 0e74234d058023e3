// linear_simt.cu -- projections on the CUDA cores: fp32, and bf16 rows that the tensor cores' copies
// cannot take (odd strides or addresses).
//
//   y_mn = act(sum_k x_mk w_nk + b_n) + r_mn        exact products, fp32 sums in the order of k
#include "latent_ptx.cuh"
#include "layer.cuh"

namespace kda {
namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;

template <typename IO, typename OUT>
__global__ void __launch_bounds__(kThreads)
linear_simt_kernel(const Linear p, int tiles_n)
{
    __shared__ float sx[kDepth][kTile + 4], sw[kDepth][kTile + 4];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kTile;
    const int n0 = (int)(blockIdx.x % tiles_n) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const IO *x = static_cast<const IO *>(p.x), *w = static_cast<const IO *>(p.w);
    float acc[4][4] = {};
    for (int k0 = 0; k0 < p.k; k0 += kDepth) {
#pragma unroll
        for (int e = threadIdx.x; e < kTile * kDepth; e += kThreads) {
            const int r = e / kDepth, k = e % kDepth;
            const bool in = k0 + k < p.k;
            sx[k][r] = in && m0 + r < p.rows ? load_io(x + (m0 + r) * p.xs + k0 + k) : 0.f;
            sw[k][r] = in && n0 + r < p.n ? load_io(w + (int64_t)(n0 + r) * p.ws + k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            const float4 a = *reinterpret_cast<const float4 *>(&sx[k][4 * ty]), b = *reinterpret_cast<const float4 *>(&sw[k][4 * tx]);
            const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 4 * ty + i;
        if (m >= p.rows) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + 4 * tx + j;
            if (n >= p.n) break;
            float v = acc[i][j];
            if (p.bias) v += load_io(static_cast<const IO *>(p.bias) + n);
            v = activate<OUT>(v, p.act);
            if (p.residual) v += load_io(static_cast<const OUT *>(p.residual) + m * p.rs + n);
            store_io(static_cast<OUT *>(p.y) + m * p.ys + n, v);
        }
    }
}

}  // namespace

cudaError_t launch_linear_simt(const Linear &p)
{
    const int tiles_n = (p.n + kTile - 1) / kTile;
    const dim3 grid((unsigned)((p.rows + kTile - 1) / kTile * tiles_n));
    auto *kernel = p.dtype == KDA_DTYPE_F32       ? linear_simt_kernel<float, float>
                   : p.out_dtype == KDA_DTYPE_F32 ? linear_simt_kernel<__nv_bfloat16, float>
                                                  : linear_simt_kernel<__nv_bfloat16, __nv_bfloat16>;
    return latent_launch(kernel, grid, kThreads, 0, p.stream, 1, p, tiles_n);
}

}  // namespace kda
