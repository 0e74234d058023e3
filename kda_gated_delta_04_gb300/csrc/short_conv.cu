// short_conv.cu -- the short causal convolution over packed sequences, with its states.
//
//   y_tc = act(b_c + sum_{j < W} w_cj x_{t - W + 1 + j, c}),   state: the last W - 1 rows of [state; x]
//
// Bound by memory: an element is read once and written once, W products between.  A thread has 16 bytes of
// channels and walks along the tokens, the last W - 1 rows in registers.  The work is of two kinds, in one
// launch:
//  - runs of kRun tokens, whatever sequences they fall in: a token is computed here where all W rows of it
//    are its sequence's;
//  - heads, one for each sequence: its first W - 1 tokens, whose rows come from the state in part, and
//    the new state.  A head reads and writes all that a sequence's state takes part in, thread by thread, so
//    that the new state may replace the old one.  A batch of single tokens is heads only.
#include "latent_ptx.cuh"
#include "layer.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 16;   // tokens of a run
constexpr int kBatch = 8;  // rows asked for at once

template <typename IO> constexpr int kVec = 16 / (int)sizeof(IO);

template <typename IO>
__device__ __forceinline__ void widen(const uint4 &r, float (&x)[kVec<IO>])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if constexpr (sizeof(IO) == 2) {
            x[2 * u] = __uint_as_float(w[u] << 16);
            x[2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
        } else {
            x[u] = __uint_as_float(w[u]);
        }
    }
}
template <typename IO>
__device__ __forceinline__ uint4 narrow(const float (&x)[kVec<IO>])
{
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if constexpr (sizeof(IO) == 2) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * u], x[2 * u + 1]);
            w[u] = *reinterpret_cast<const uint32_t *>(&v);
        } else {
            w[u] = __float_as_uint(x[u]);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's channels: their taps and bias, and where their rows are.
template <typename IO, int W>
struct Channels {
    static constexpr int V = kVec<IO>;
    float tap[V * W], bias[V];
    const IO *x;
    IO *y;
    __device__ __forceinline__ Channels(const ShortConv &p, int c)
    {
        const uint4 *w = reinterpret_cast<const uint4 *>(static_cast<const IO *>(p.weight) + (int64_t)c * W);
#pragma unroll
        for (int j = 0; j < W; ++j) widen<IO>(__ldg(w + j), *reinterpret_cast<float(*)[V]>(&tap[V * j]));
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = 0.f;
        if (p.bias) widen<IO>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const IO *>(p.bias) + c)), bias);
        x = static_cast<const IO *>(p.x) + c;
        const int part = c / p.part;
        y = static_cast<IO *>(p.y) + part * p.part_stride + (c - part * p.part);
    }
    // row[0 .. W - 1]: the rows of a token, the oldest first
    __device__ __forceinline__ uint4 token(const float (&row)[W][V], bool silu) const
    {
        float a[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a[v] = bias[v];
#pragma unroll
            for (int j = 0; j < W; ++j) a[v] = fmaf(tap[v * W + j], row[j][v], a[v]);
            if (silu) a[v] = silu_io<IO>(a[v]);
        }
        return narrow<IO>(a);
    }
};

template <typename IO, int W>
__device__ __forceinline__ void head(const ShortConv &p, int n, int c)
{
    constexpr int V = kVec<IO>;
    int first, end;
    int64_t init, fin;
    packed_range(p.seq, n, first, end);
    if (!packed_entries(p.seq, n, init, fin) && c == 0 && p.seq.errors) atomicOr(p.seq.errors, DEV_ERR_SLOT);
    const int len = end - first, mine = min(len, W - 1);
    const IO *x = static_cast<const IO *>(p.x) + c;
    // the W - 1 rows of the state, and the sequence's first ones
    uint4 raw[2 * W - 2], last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (init >= 0)
            raw[j] = *reinterpret_cast<const uint4 *>(static_cast<const IO *>(p.seq.init) +
                                                      (init * (W - 1) + j) * p.channels + c);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        if (j < mine) raw[W - 1 + j] = *reinterpret_cast<const uint4 *>(x + (int64_t)(first + j) * p.xs);
    // the last W - 1 rows of both
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        if (len >= W - 1) last[j] = *reinterpret_cast<const uint4 *>(x + (int64_t)(end - (W - 1) + j) * p.xs);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        if (len == k)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) last[j] = raw[k + j];
    if (fin >= 0)
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<uint4 *>(static_cast<IO *>(p.seq.fin) + (fin * (W - 1) + j) * p.channels + c) = last[j];
    if (mine == 0) return;
    const Channels<IO, W> ch(p, c);
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t >= mine) break;
        float row[W][V];
#pragma unroll
        for (int j = 0; j < W; ++j) widen<IO>(raw[t + j], row[j]);
        *reinterpret_cast<uint4 *>(ch.y + (int64_t)(first + t) * p.ys) = ch.token(row, p.silu);
    }
}

// The last sequence that starts at or before token t (of malformed offsets, some sequence).
__device__ __forceinline__ int sequence_of(const Packed &s, int t)
{
    int lo = 0, hi = s.num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Bit i: all W rows of token t0 + i are its sequence's.  A whole warp.
template <int W>
__device__ __forceinline__ uint32_t whole_tokens(const Packed &s, int t0, int lane)
{
    const int t = t0 + lane;
    bool whole = false;
    if (lane < kRun && t < s.tokens) {
        int first, end;
        packed_range(s, s.cu ? sequence_of(s, t) : t / s.each, first, end);
        whole = t - first >= W - 1 && t < end;
    }
    return __ballot_sync(0xffffffffu, whole);
}

template <typename IO, int W>
__device__ __forceinline__ void run(const ShortConv &p, int t0, int c)
{
    constexpr int V = kVec<IO>;
    const Channels<IO, W> ch(p, c);
    const int total = (int)p.seq.tokens;
    uint4 raw[kBatch];
    float row[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int t = max(t0 - (W - 1) + j, 0);
        widen<IO>(*reinterpret_cast<const uint4 *>(ch.x + (int64_t)t * p.xs), row[j]);
    }
    uint32_t whole = 0;
#pragma unroll
    for (int b = 0; b < kRun; b += kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int t = min(t0 + b + i, total - 1);
            raw[i] = *reinterpret_cast<const uint4 *>(ch.x + (int64_t)t * p.xs);
        }
        if (b == 0) whole = whole_tokens<W>(p.seq, t0, threadIdx.x & 31);  // (after the rows are on their way)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            widen<IO>(raw[i], row[W - 1]);
            if (whole >> (b + i) & 1)
                *reinterpret_cast<uint4 *>(ch.y + (int64_t)(t0 + b + i) * p.ys) = ch.token(row, p.silu);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) row[j][v] = row[j + 1][v];
        }
    }
}

// Blocks: the heads of each sequence, then the runs; channels innermost.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads)
short_conv_kernel(const ShortConv p, int channel_blocks, int64_t head_blocks)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int64_t unit = blockIdx.x / channel_blocks;
    const int c = ((blockIdx.x % channel_blocks) * kThreads + threadIdx.x) * kVec<IO>;
    const bool mine = c < p.channels;
    if (unit < head_blocks) {
        if (blockIdx.x % channel_blocks == 0 && threadIdx.x == 0) {
            packed_check(p.seq, (int)unit);
            if (unit == 0) packed_check(p.seq, p.seq.num_seqs);
        }
        if (mine) head<IO, W>(p, (int)unit, c);
    } else {
        // (threads without channels keep the warp whole: the last channels, computed and stored again, the same)
        run<IO, W>(p, (int)(unit - head_blocks) * kRun, mine ? c : p.channels - kVec<IO>);
    }
}

template <typename IO, int W>
cudaError_t launch(const ShortConv &p)
{
    const int channel_blocks = (p.channels / kVec<IO> + kThreads - 1) / kThreads;
    const int64_t heads = p.seq.num_seqs;
    // sequences of equal, few tokens have no others than their first W - 1
    const int64_t runs = !p.seq.cu && p.seq.each < W ? 0 : (p.seq.tokens + kRun - 1) / kRun;
    const int64_t blocks = (heads + runs) * channel_blocks;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return latent_launch(short_conv_kernel<IO, W>, dim3((unsigned)blocks), kThreads, 0, p.stream, 1, p, channel_blocks, heads);
}

}  // namespace

cudaError_t launch_short_conv(const ShortConv &p)
{
    const bool half = p.dtype == KDA_DTYPE_BF16;
    switch (p.width) {
    case 2: return half ? launch<__nv_bfloat16, 2>(p) : launch<float, 2>(p);
    case 3: return half ? launch<__nv_bfloat16, 3>(p) : launch<float, 3>(p);
    default: return half ? launch<__nv_bfloat16, 4>(p) : launch<float, 4>(p);
    }
}

}  // namespace kda
