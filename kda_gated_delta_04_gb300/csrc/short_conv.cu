// short_conv.cu -- the short causal convolution over packed sequences, with its states.
//
//   y_tc = act(b_c + sum_{j < W} w_cj x_{t - W + 1 + j, c}),   state: the last W - 1 rows of [state; x]
//
// Bound by memory: an element is read once and written once, W products between.  A thread has four channels
// (16 bytes of bf16 took 126 registers and 40 us where this takes 38) and walks along the tokens, the last W - 1 rows
// in registers: 4,096 tokens of 12,288 channels in bf16 37.9 us, 5.3 TB/s.  The work is of two kinds, in one launch:
//  - runs of tokens, whatever sequences they fall in: a token is computed here where all W rows of it
//    are its sequence's;
//  - heads, one for each sequence: its first W - 1 tokens, whose rows come from the state in part, and
//    the new state.  A head reads and writes all that a sequence's state takes part in, thread by thread, so
//    that the new state may replace the old one.  A batch of single tokens is heads only.
#include "latent_ptx.cuh"
#include "layer.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
// Tokens of a run.  4,096 tokens of 12,288 channels in bf16, us with 8, 16, 32: 41.4, 37.9, 40.6; 7,800 tokens of
// 2,048 channels in fp32 28.1, 30.9, 34.7.
template <typename IO> constexpr int kRun = sizeof(IO) == 2 ? 16 : 8;
constexpr int kBatch = 8;  // rows asked for at once
constexpr int kSeqs = 4;   // sequences of a thread that takes single tokens (256 of 12,288 channels 10.0 us; 1: 11.7)

// A thread's four channels of a row, as they lie in memory.
constexpr int V = 4;
template <typename IO> struct Raw;
template <> struct Raw<__nv_bfloat16> { using Type = uint2; };
template <> struct Raw<float> { using Type = uint4; };
template <typename IO> using Raw4 = typename Raw<IO>::Type;

template <typename IO>
__device__ __forceinline__ Raw4<IO> load_raw(const IO *p) { return *reinterpret_cast<const Raw4<IO> *>(p); }
template <typename IO>
__device__ __forceinline__ void store_raw(IO *p, const Raw4<IO> &r) { *reinterpret_cast<Raw4<IO> *>(p) = r; }
__device__ __forceinline__ void widen(const uint2 &r, float (&x)[V])
{
    x[0] = __uint_as_float(r.x << 16); x[1] = __uint_as_float(r.x & 0xffff0000u);
    x[2] = __uint_as_float(r.y << 16); x[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void widen(const uint4 &r, float (&x)[V])
{
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y); x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
}

// A thread's channels: their taps and bias, and where their rows are.
template <typename IO, int W>
struct Channels {
    float tap[V * W], bias[V];
    const IO *x;
    IO *y;
    __device__ __forceinline__ Channels(const ShortConv &p, int c)
    {
        const IO *w = static_cast<const IO *>(p.weight) + (int64_t)c * W;
#pragma unroll
        for (int j = 0; j < W; ++j) widen(load_raw(w + V * j), *reinterpret_cast<float(*)[V]>(&tap[V * j]));
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = 0.f;
        if (p.bias) widen(load_raw(static_cast<const IO *>(p.bias) + c), bias);
        x = static_cast<const IO *>(p.x) + c;
        const int part = c / p.part;
        y = static_cast<IO *>(p.y) + part * p.part_stride + (c - part * p.part);
    }
    // Token t from its rows row[0 .. W - 1], the oldest first.
    __device__ __forceinline__ void token(const ShortConv &p, const float (&row)[W][V], int64_t t) const
    {
        float a[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a[v] = bias[v];
#pragma unroll
            for (int j = 0; j < W; ++j) a[v] = fmaf(tap[v * W + j], row[j][v], a[v]);
            if (p.silu) a[v] = silu_io<IO>(a[v]);
        }
        store_io4(y + t * p.ys, a);
    }
};

template <typename IO, int W>
__device__ __forceinline__ void head(const ShortConv &p, int n, int c)
{
    int first, end;
    int64_t init, fin;
    packed_range(p.seq, n, first, end);
    if (!packed_entries(p.seq, n, init, fin) && c == 0 && p.seq.errors) atomicOr(p.seq.errors, DEV_ERR_SLOT);
    const int len = end - first, mine = min(len, W - 1);
    const IO *x = static_cast<const IO *>(p.x) + c;
    // the W - 1 rows of the state, and the sequence's first ones
    Raw4<IO> raw[2 * W - 2], last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        raw[j] = Raw4<IO>{};
        if (init >= 0) raw[j] = load_raw(static_cast<const IO *>(p.seq.init) + (init * (W - 1) + j) * p.channels + c);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        if (j < mine) raw[W - 1 + j] = load_raw(x + (int64_t)(first + j) * p.xs);
    // the last W - 1 rows of both
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        if (len >= W - 1) last[j] = load_raw(x + (int64_t)(end - (W - 1) + j) * p.xs);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        if (len == k)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) last[j] = raw[k + j];
    if (fin >= 0)
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_raw(static_cast<IO *>(p.seq.fin) + (fin * (W - 1) + j) * p.channels + c, last[j]);
    if (mine == 0) return;
    const Channels<IO, W> ch(p, c);
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t >= mine) break;
        float row[W][V];
#pragma unroll
        for (int j = 0; j < W; ++j) widen(raw[t + j], row[j]);
        ch.token(p, row, first + t);
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
template <int W, int RUN>
__device__ __forceinline__ uint32_t whole_tokens(const Packed &s, int t0, int lane)
{
    const int t = t0 + lane;
    bool whole = false;
    if (lane < RUN && t < s.tokens) {
        int first, end;
        packed_range(s, s.cu ? sequence_of(s, t) : t / s.each, first, end);
        whole = t - first >= W - 1 && t < end;
    }
    return __ballot_sync(0xffffffffu, whole);
}

template <typename IO, int W>
__device__ __forceinline__ void run(const ShortConv &p, int t0, int c)
{
    const Channels<IO, W> ch(p, c);
    const int total = (int)p.seq.tokens;
    constexpr int B = kBatch;
    Raw4<IO> raw[B], before[W - 1];
    float row[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) before[j] = load_raw(ch.x + (int64_t)max(t0 - (W - 1) + j, 0) * p.xs);
    uint32_t whole = 0;
#pragma unroll
    for (int b = 0; b < kRun<IO>; b += B) {
#pragma unroll
        for (int i = 0; i < B; ++i) raw[i] = load_raw(ch.x + (int64_t)min(t0 + b + i, total - 1) * p.xs);
        if (b == 0) {
            whole = whole_tokens<W, kRun<IO>>(p.seq, t0, threadIdx.x & 31);  // (after the rows are on their way)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) widen(before[j], row[j]);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
            widen(raw[i], row[W - 1]);
            if (whole >> (b + i) & 1) ch.token(p, row, t0 + b + i);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) row[j][v] = row[j + 1][v];
        }
    }
}

// One token of each of kSeqs sequences: what head does where all sequences are one token, with everything of them
// asked for at once.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads, sizeof(IO) == 2 ? 6 : 4)
short_conv_step_kernel(const ShortConv p, int channel_blocks)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int n0 = (int)(blockIdx.x / channel_blocks) * kSeqs;
    const int own = ((blockIdx.x % channel_blocks) * kThreads + threadIdx.x) * V, c = min(own, p.channels - V);
    const bool mine = own < p.channels;
    // lane i of a warp reads sequence i's entries
    const int lane = threadIdx.x & 31;
    int64_t own_init = -1, own_fin = -1;
    if (lane < kSeqs && n0 + lane < p.seq.num_seqs &&
        !packed_entries(p.seq, n0 + lane, own_init, own_fin) && blockIdx.x % channel_blocks == 0 && threadIdx.x < 32 && p.seq.errors)
        atomicOr(p.seq.errors, DEV_ERR_SLOT);
    int fin[kSeqs];
    Raw4<IO> raw[kSeqs][W];
    const IO *x = static_cast<const IO *>(p.x) + n0 * p.xs + c;
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        raw[i][W - 1] = load_raw(x);
        if (n0 + i + 1 < p.seq.num_seqs) x += p.xs;
    }
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int init = __shfl_sync(0xffffffffu, (int)own_init, i);
        fin[i] = __shfl_sync(0xffffffffu, (int)own_fin, i);
        const IO *from = static_cast<const IO *>(p.seq.init) + (int64_t)init * (W - 1) * p.channels + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            raw[i][j] = Raw4<IO>{};
            if (init >= 0) raw[i][j] = load_raw(from + (int64_t)j * p.channels);
        }
    }
    if (!mine) return;
    const Channels<IO, W> ch(p, c);
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        if (n0 + i >= p.seq.num_seqs) break;
        if (fin[i] >= 0) {
            IO *to = static_cast<IO *>(p.seq.fin) + (int64_t)fin[i] * (W - 1) * p.channels + c;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) store_raw(to + (int64_t)j * p.channels, raw[i][j + 1]);
        }
        float row[W][V];
#pragma unroll
        for (int j = 0; j < W; ++j) widen(raw[i][j], row[j]);
        ch.token(p, row, n0 + i);
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
    const int c = ((blockIdx.x % channel_blocks) * kThreads + threadIdx.x) * V;
    const bool mine = c < p.channels;
    if (unit < head_blocks) {
        if (blockIdx.x % channel_blocks == 0 && threadIdx.x == 0) {
            packed_check(p.seq, (int)unit);
            if (unit == 0) packed_check(p.seq, p.seq.num_seqs);
        }
        if (mine) head<IO, W>(p, (int)unit, c);
    } else {
        // (threads without channels keep the warp whole: the last channels, computed and stored again, the same)
        run<IO, W>(p, (int)(unit - head_blocks) * kRun<IO>, mine ? c : p.channels - V);
    }
}

template <typename IO, int W>
cudaError_t launch(const ShortConv &p)
{
    const int channel_blocks = (p.channels / V + kThreads - 1) / kThreads;
    const int64_t heads = p.seq.num_seqs;
    if (!p.seq.cu && p.seq.each == 1) {
        const int64_t blocks = (heads + kSeqs - 1) / kSeqs * channel_blocks;
        if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
        return latent_launch(short_conv_step_kernel<IO, W>, dim3((unsigned)blocks), kThreads, 0, p.stream, 1, p, channel_blocks);
    }
    // sequences of equal, few tokens have no others than their first W - 1
    const int64_t runs = !p.seq.cu && p.seq.each < W ? 0 : (p.seq.tokens + kRun<IO> - 1) / kRun<IO>;
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
