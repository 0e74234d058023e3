// scan.cu -- the selective scan over packed sequences.
//
//   d = softplus(dt + dt_bias);  h_cn <- exp(d_c A_cn) h_cn + d_c B_n x_c;
//   y_c = (sum_n C_n h_cn + D_c x_c) silu(z_c)
//
// Per token and channel d_state exponentials and 5 d_state other operations against 8 bytes of bf16: bound by
// the exponential units (16 a cycle and SM).  Only h's product and sum are in order of the tokens, 4 cycles each,
// so that the scan stays in order and the channels fill the GPU: 32 channels of 16 states a CTA, four states a
// thread.
//
// Warps 0 to 3 scan; warps 4 to 7 bring the tokens in and out, kChunk at a time, a chunk ahead and one behind:
// d and d x, which all states of a channel share, are computed once and handed over in shared memory, as are
// the sums, to which D x and the gate are applied where they are stored.
#include "latent_ptx.cuh"
#include "layer.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

constexpr int kScanThreads = 128, kThreads = 256;
constexpr int kChunk = 32;  // tokens handed over at a time

template <typename IO> struct Raw8 { uint4 q[sizeof(IO) / 2]; };

template <typename IO>
__device__ __forceinline__ Raw8<IO> load8(const IO *p)
{
    Raw8<IO> r;
#pragma unroll
    for (size_t i = 0; i < sizeof(IO) / 2; ++i) r.q[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}
template <typename IO>
__device__ __forceinline__ void store8(IO *p, const Raw8<IO> &r)
{
#pragma unroll
    for (size_t i = 0; i < sizeof(IO) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = r.q[i];
}
template <typename IO>
__device__ __forceinline__ void widen(const Raw8<IO> &r, float (&x)[8])
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(IO) == 2)
            x[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        else
            x[i] = __uint_as_float(w[i]);
    }
}
template <typename IO>
__device__ __forceinline__ Raw8<IO> narrow(const float (&x)[8])
{
    Raw8<IO> r;
    uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(IO) == 2) {
            if (i & 1) w[i >> 1] = tc::pack_bf16x2(x[i - 1], x[i]);
        } else {
            w[i] = __float_as_uint(x[i]);
        }
    }
    return r;
}

// Channels of a CTA and the buffers of its chunks.
template <typename IO, int N>
struct Shape {
    static constexpr int kLanes = N / 4;                    // lanes of a channel, four states each
    static constexpr int kCh = kScanThreads / kLanes;       // channels
    static constexpr int kRowY = kCh + 8;                   // (lanes of a channel store rows that follow one another)
    static constexpr int kItems = (kChunk * kCh / 8 + 127) / 128;     // pieces of 8 channels a thread brings in
    static constexpr int kItemsBC = (kChunk * 2 * N / 8 + 127) / 128;
    float2 dd[2][kChunk][kCh];                              // d, d x
    float bc[2][kChunk][2 * N];
    float y[2][kChunk][kRowY];
    alignas(16) IO x[3][kChunk][kCh], z[3][kChunk][kCh];
};

// Sums over the kLanes lanes of a channel of v[u], u < kLanes, to lane u.
template <int L>
__device__ __forceinline__ float spread_sums(float (&v)[L], int lane)
{
#pragma unroll
    for (int m = L / 2; m; m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int u = 0; u < m; ++u) {
            const float give = up ? v[u] : v[u + m], keep = up ? v[u + m] : v[u];
            v[u] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
    return v[0];
}

template <typename IO, int N>
__global__ void __launch_bounds__(kThreads)
scan_kernel(const Scan p, int group_blocks)
{
    using S = Shape<IO, N>;
    constexpr int L = S::kLanes, CH = S::kCh;
    extern __shared__ __align__(16) unsigned char raw_smem[];
    S &sm = *reinterpret_cast<S *>(raw_smem);
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int blocks = p.groups * group_blocks, n = blockIdx.x / blocks, block = blockIdx.x % blocks;
    const int group = block / group_blocks, per_group = p.channels / p.groups;
    const int c0 = group * per_group + (block % group_blocks) * CH;   // first channel
    const int held = min(CH, (group + 1) * per_group - c0);            // channels: a multiple of 8
    int first, end;
    packed_range(p.seq, n, first, end);
    const int len = end - first, chunks = (len + kChunk - 1) / kChunk;

    if (threadIdx.x < kScanThreads) {
        const int lane = threadIdx.x % L, ch = threadIdx.x / L;
        const bool mine = ch < held;
        int64_t init, fin;
        const bool good = packed_entries(p.seq, n, init, fin);
        if (threadIdx.x == 0 && block == 0) {
            packed_check(p.seq, n);
            if (n == 0) packed_check(p.seq, p.seq.num_seqs);
            if (!good && p.seq.errors) atomicOr(p.seq.errors, DEV_ERR_SLOT);
        }
        const int64_t at = (int64_t)(c0 + ch) * N + 4 * lane, all = (int64_t)p.channels * N;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), h = a;
        if (mine) {
            a = *reinterpret_cast<const float4 *>(p.a + at);
            if (init >= 0) h = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.seq.init) + init * all + at);
        }
        a.x *= tc::kLog2e; a.y *= tc::kLog2e; a.z *= tc::kLog2e; a.w *= tc::kLog2e;
        __syncthreads();
        for (int k = 0; k < chunks; ++k) {
            const int buf = k & 1, count = min(kChunk, len - k * kChunk);
            auto step = [&](int t) {
                const float2 dd = sm.dd[buf][t][ch];
                const float4 b = *reinterpret_cast<const float4 *>(&sm.bc[buf][t][4 * lane]);
                const float4 c = *reinterpret_cast<const float4 *>(&sm.bc[buf][t][N + 4 * lane]);
                h.x = fmaf(tc::exp2_approx(dd.x * a.x), h.x, dd.y * b.x);
                h.y = fmaf(tc::exp2_approx(dd.x * a.y), h.y, dd.y * b.y);
                h.z = fmaf(tc::exp2_approx(dd.x * a.z), h.z, dd.y * b.z);
                h.w = fmaf(tc::exp2_approx(dd.x * a.w), h.w, dd.y * b.w);
                return fmaf(h.x, c.x, h.y * c.y) + fmaf(h.z, c.z, h.w * c.w);
            };
#pragma unroll 2
            for (int t = 0; t < count; t += L) {
                float v[L];
                if (t + L <= count) {
#pragma unroll
                    for (int u = 0; u < L; ++u) v[u] = step(t + u);
                } else {
#pragma unroll
                    for (int u = 0; u < L; ++u) v[u] = t + u < count ? step(t + u) : 0.f;
                }
                sm.y[buf][t + lane][ch] = spread_sums<L>(v, lane);
            }
            __syncthreads();
        }
        if (fin >= 0 && mine) *reinterpret_cast<float4 *>(static_cast<float *>(p.seq.fin) + fin * all + at) = h;
        return;
    }

    // tokens in and out
    const int tid = threadIdx.x - kScanThreads;
    Raw8<IO> rx[S::kItems], rdt[S::kItems], rz[S::kItems], rbc[S::kItemsBC];
    auto ask = [&](int k) {  // a chunk's rows
#pragma unroll
        for (int i = 0; i < S::kItems; ++i) {
            const int e = i * 128 + tid, t = k * kChunk + e / (CH / 8), c = e % (CH / 8) * 8;
            if (e < kChunk * CH / 8 && t < len && c < held) {
                const int64_t row = first + t;
                rx[i] = load8(static_cast<const IO *>(p.x) + row * p.xs + c0 + c);
                rdt[i] = load8(static_cast<const IO *>(p.dt) + row * p.dts + c0 + c);
                if (p.z) rz[i] = load8(static_cast<const IO *>(p.z) + row * p.zs + c0 + c);
            }
        }
#pragma unroll
        for (int i = 0; i < S::kItemsBC; ++i) {
            const int e = i * 128 + tid, t = k * kChunk + e / (N / 4), s = e % (N / 4) * 8;
            if (e < kChunk * N / 4 && t < len) {
                const int64_t row = first + t;
                rbc[i] = s < N ? load8(static_cast<const IO *>(p.b) + row * p.bs + group * N + s)
                               : load8(static_cast<const IO *>(p.c) + row * p.cs + group * N + s - N);
            }
        }
    };
    auto put = [&](int k) {
        const int buf = k & 1;
#pragma unroll
        for (int i = 0; i < S::kItems; ++i) {
            const int e = i * 128 + tid, t = e / (CH / 8), c = e % (CH / 8) * 8;
            if (e < kChunk * CH / 8 && k * kChunk + t < len && c < held) {
                float x[8], d[8], bias[8] = {};
                widen(rx[i], x);
                widen(rdt[i], d);
                if (p.dt_bias) widen(load8(p.dt_bias + c0 + c), bias);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    d[u] += bias[u];
                    if (p.softplus) d[u] = softplus(d[u]);
                    sm.dd[buf][t][c + u] = make_float2(d[u], d[u] * x[u]);
                }
                store8(&sm.x[k % 3][t][c], rx[i]);
                if (p.z) store8(&sm.z[k % 3][t][c], rz[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < S::kItemsBC; ++i) {
            const int e = i * 128 + tid, t = e / (N / 4), s = e % (N / 4) * 8;
            if (e < kChunk * N / 4 && k * kChunk + t < len) {
                float v[8];
                widen(rbc[i], v);
#pragma unroll
                for (int u = 0; u < 8; u += 4)
                    *reinterpret_cast<float4 *>(&sm.bc[buf][t][s + u]) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
            }
        }
    };
    auto out = [&](int k) {
        const int buf = k & 1;
#pragma unroll
        for (int i = 0; i < S::kItems; ++i) {
            const int e = i * 128 + tid, t = e / (CH / 8), c = e % (CH / 8) * 8;
            if (e < kChunk * CH / 8 && k * kChunk + t < len && c < held) {
                float x[8], z[8], skip[8] = {}, y[8];
                widen(load8(&sm.x[k % 3][t][c]), x);
                if (p.d) widen(load8(p.d + c0 + c), skip);
                if (p.z) widen(load8(&sm.z[k % 3][t][c]), z);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    y[u] = fmaf(skip[u], x[u], sm.y[buf][t][c + u]);
                    if (p.z) y[u] *= silu_io<IO>(z[u]);
                }
                store8(static_cast<IO *>(p.y) + (int64_t)(first + k * kChunk + t) * p.ys + c0 + c, narrow<IO>(y));
            }
        }
    };
    if (chunks > 0) {
        ask(0);
        put(0);
        if (chunks > 1) ask(1);
    }
    __syncthreads();
    for (int k = 0; k < chunks; ++k) {  // while chunk k is scanned
        if (k + 1 < chunks) put(k + 1);
        if (k + 2 < chunks) ask(k + 2);
        if (k > 0) out(k - 1);
        __syncthreads();
    }
    if (chunks > 0) out(chunks - 1);
}

template <typename IO, int N>
cudaError_t launch(const Scan &p)
{
    using S = Shape<IO, N>;
    static int configured = -1;
    const cudaError_t err = tc::allow_smem(scan_kernel<IO, N>, (int)sizeof(S), &configured);
    if (err != cudaSuccess) return err;
    const int group_blocks = (p.channels / p.groups + S::kCh - 1) / S::kCh;
    const int64_t blocks = (int64_t)group_blocks * p.groups * p.seq.num_seqs;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return latent_launch(scan_kernel<IO, N>, dim3((unsigned)blocks), kThreads, sizeof(S), p.stream, 1, p, group_blocks);
}

}  // namespace

cudaError_t launch_scan(const Scan &p)
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
