// scan_step.cu -- the selective scan of one token of every sequence.
//
//   h_cn <- exp(d_c A_cn) h_cn + d_c B_n x_c;   y_c = (sum_n C_n h_cn + D_c x_c) silu(z_c)
//
// Bound by memory: the states, fp32, are read and written once.  A thread has four states of a channel, so that
// a warp's states are 512 bytes in a row, and kSeqs sequences, whose states are asked for at once; A is
// read once for them.
#include "latent_ptx.cuh"
#include "layer.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128, kSeqs = 4;

template <typename IO, int N>
__global__ void __launch_bounds__(kThreads)
scan_step_kernel(const Scan p, int channel_blocks)
{
    constexpr int L = N / 4, CH = kThreads / L;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int n0 = (int)(blockIdx.x / channel_blocks) * kSeqs, lane = threadIdx.x % L;
    const int ch = (blockIdx.x % channel_blocks) * CH + threadIdx.x / L, c = min(ch, p.channels - 1);
    const bool mine = ch < p.channels;
    const int group = c / (p.channels / p.groups);
    const int64_t at = (int64_t)c * N + 4 * lane, all = (int64_t)p.channels * N;
    int64_t init[kSeqs], fin[kSeqs];
    float4 h[kSeqs];
    float x[kSeqs], dt[kSeqs], z[kSeqs], b[kSeqs][4], cc[kSeqs][4];
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int n = n0 + i;
        init[i] = fin[i] = -1;
        if (n < p.seq.num_seqs && !packed_entries(p.seq, n, init[i], fin[i]) && blockIdx.x % channel_blocks == 0 &&
            threadIdx.x == 0 && p.seq.errors)
            atomicOr(p.seq.errors, DEV_ERR_SLOT);
    }
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int64_t n = min(n0 + i, p.seq.num_seqs - 1);
        h[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (init[i] >= 0) h[i] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.seq.init) + init[i] * all + at);
        x[i] = load_io(static_cast<const IO *>(p.x) + n * p.xs + c);
        dt[i] = load_io(static_cast<const IO *>(p.dt) + n * p.dts + c);
        z[i] = p.z ? load_io(static_cast<const IO *>(p.z) + n * p.zs + c) : 0.f;
        load_io4(static_cast<const IO *>(p.b) + n * p.bs + group * N + 4 * lane, b[i]);
        load_io4(static_cast<const IO *>(p.c) + n * p.cs + group * N + 4 * lane, cc[i]);
    }
    float4 a = *reinterpret_cast<const float4 *>(p.a + at);
    a.x *= tc::kLog2e; a.y *= tc::kLog2e; a.z *= tc::kLog2e; a.w *= tc::kLog2e;
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.d ? p.d[c] : 0.f;
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        float d = dt[i] + bias;
        if (p.softplus) d = softplus(d);
        const float dx = d * x[i];
        h[i].x = fmaf(tc::exp2_approx(d * a.x), h[i].x, dx * b[i][0]);
        h[i].y = fmaf(tc::exp2_approx(d * a.y), h[i].y, dx * b[i][1]);
        h[i].z = fmaf(tc::exp2_approx(d * a.z), h[i].z, dx * b[i][2]);
        h[i].w = fmaf(tc::exp2_approx(d * a.w), h[i].w, dx * b[i][3]);
        float y = fmaf(h[i].x, cc[i][0], h[i].y * cc[i][1]) + fmaf(h[i].z, cc[i][2], h[i].w * cc[i][3]);
#pragma unroll
        for (int m = L / 2; m; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (!mine || n0 + i >= p.seq.num_seqs) continue;
        if (fin[i] >= 0) *reinterpret_cast<float4 *>(static_cast<float *>(p.seq.fin) + fin[i] * all + at) = h[i];
        if (lane == 0) {
            y = fmaf(skip, x[i], y);
            if (p.z) y *= silu_io<IO>(z[i]);
            store_io(static_cast<IO *>(p.y) + (int64_t)(n0 + i) * p.ys + c, y);
        }
    }
}

template <typename IO, int N>
cudaError_t launch(const Scan &p)
{
    constexpr int CH = kThreads / (N / 4);
    const int channel_blocks = (p.channels + CH - 1) / CH;
    const int64_t blocks = (int64_t)channel_blocks * ((p.seq.num_seqs + kSeqs - 1) / kSeqs);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return latent_launch(scan_step_kernel<IO, N>, dim3((unsigned)blocks), kThreads, 0, p.stream, 1, p, channel_blocks);
}

}  // namespace

cudaError_t launch_scan_step(const Scan &p)
{
    const bool half = p.dtype == KDA_DTYPE_BF16;
    switch (p.states) {
    case 8: return half ? launch<__nv_bfloat16, 8>(p) : launch<float, 8>(p);
    case 16: return half ? launch<__nv_bfloat16, 16>(p) : launch<float, 16>(p);
    case 32: return half ? launch<__nv_bfloat16, 32>(p) : launch<float, 32>(p);
    default: return half ? launch<__nv_bfloat16, 64>(p) : launch<float, 64>(p);
    }
}

}  // namespace kda
