// latent_append.cu -- one token's row into the latent cache: the latent vector normalised
// (RMSNorm), its position key rotated, both written to the token's cache slot, and in the same
// launch the rotation of the token's queries.
//
//   y = w x / sqrt(mean(x^2) + eps)            (512 channels; no weight: y = x)
//   (a, b)_i -> (a cos_i - b sin_i, b cos_i + a sin_i), i < 32   (position channels)
//
// The pair i is (i, i + 32) or, interleaved, (2i, 2i + 1).  Sums and products are fp32, rounded
// once when stored.  Bound by memory (T large) or by the latency of one dependent chain,
// position -> table row -> store (T small).  A warp's unit of work is either a token's latent row and
// position key, or the position channels of 16 of its query heads (32 lanes = 8 heads x 4 quarters of the
// pairs, two heads and 2 x 8 pairs a lane), so that small batches spread over 1 + H / 16 warps a token.  In
// large ones each of the 16 warps that an SM holds walks on through the units, the numbers (position, slot)
// two units ahead and the rows one: 32,768 tokens of 32 heads 69 us (386 MB, 5.6 TB/s), 64 tokens 3.2.  A
// warp a unit and CTA took 72 and was bound by the launching of CTAs, 0.6 ns each.
#include "latent.cuh"
#include "latent_ptx.cuh"

namespace kda {
namespace {

constexpr int kWarps = 2, kMaxBlocks = 152 * 8;  // 16 warps a SM: what 128 registers a thread leave room for

// Eight consecutive elements as they lie in memory (16-byte aligned): what is neither normalised
// nor rotated is stored again bit for bit.
template <typename IO> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 a; };
template <> struct Raw8<float> { float4 a, b; };

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, Raw8<__nv_bfloat16> &r)
{
    r.a = *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void load8(const float *p, Raw8<float> &r)
{
    r.a = *reinterpret_cast<const float4 *>(p);
    r.b = *reinterpret_cast<const float4 *>(p + 4);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Raw8<__nv_bfloat16> &r)
{
    *reinterpret_cast<uint4 *>(p) = r.a;
}
__device__ __forceinline__ void store8(float *p, const Raw8<float> &r)
{
    *reinterpret_cast<float4 *>(p) = r.a;
    *reinterpret_cast<float4 *>(p + 4) = r.b;
}
__device__ __forceinline__ void widen(const Raw8<__nv_bfloat16> &r, float (&x)[8])
{
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        x[2 * u] = __uint_as_float(w[u] << 16);
        x[2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen(const Raw8<float> &r, float (&x)[8])
{
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void narrow(const float (&x)[8], Raw8<__nv_bfloat16> &r)
{
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * u], x[2 * u + 1]);
        w[u] = *reinterpret_cast<const uint32_t *>(&v);
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void narrow(const float (&x)[8], Raw8<float> &r)
{
    r.a = make_float4(x[0], x[1], x[2], x[3]);
    r.b = make_float4(x[4], x[5], x[6], x[7]);
}

// Quarter j (8 pairs) of a 64-channel row: elements [lo, lo + 8) and [hi, hi + 8) of it.
__device__ __forceinline__ void quarter_at(int j, bool interleaved, int &lo, int &hi)
{
    lo = interleaved ? 16 * j : 8 * j;
    hi = interleaved ? 16 * j + 8 : 32 + 8 * j;
}

// Rotates the 8 pairs held as row[lo..] and row[hi..] (see quarter_at).
template <typename IO>
__device__ __forceinline__ void rotate8(Raw8<IO> &rx, Raw8<IO> &ry, const Raw8<float> &rc, const Raw8<float> &rs,
                                        bool interleaved)
{
    float x[8], y[8], c[8], s[8];
    widen(rx, x);
    widen(ry, y);
    widen(rc, c);
    widen(rs, s);
    if (interleaved) {  // pair i: elements 2i, 2i + 1 of x ++ y
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1], d = y[2 * i], e = y[2 * i + 1];
            x[2 * i] = a * c[i] - b * s[i];
            x[2 * i + 1] = b * c[i] + a * s[i];
            y[2 * i] = d * c[4 + i] - e * s[4 + i];
            y[2 * i + 1] = e * c[4 + i] + d * s[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i], b = y[i];
            x[i] = a * c[i] - b * s[i];
            y[i] = b * c[i] + a * s[i];
        }
    }
    narrow(x, rx);
    narrow(y, ry);
}

constexpr int kUnitHeads = 16;  // heads of a query unit, two a lane

// A unit as its warp has it in flight: of a token's latent row and position key, r[0], r[1] the latent's
// channels 8 lane and 256 + 8 lane, r[2], r[3] a quarter of the key (lanes 0 to 3); of its queries two
// heads' quarters.
template <typename IO>
struct Item {
    int t, unit, pos, slot;
    Raw8<IO> r[4];
    Raw8<float> c, s;
};

// The numbers of a unit: loaded two units ahead, as everything else hangs on the position.
template <typename IO>
__device__ __forceinline__ void ask_numbers(const LatentAppend &p, int64_t work, int64_t total, int units, Item<IO> &it)
{
    it.t = -1;
    if (work >= total) return;
    it.t = (int)(work / units);
    it.unit = (int)(work - (int64_t)it.t * units);
    it.pos = p.cos_sin ? p.positions[it.t] : 0;
    it.slot = it.unit == 0 ? p.slots[it.t] : -1;
}

// Its rows and its row of the table: loaded one unit ahead.
template <typename IO>
__device__ __forceinline__ void ask_rows(const LatentAppend &p, Item<IO> &it, int lane, int lo, int hi)
{
    if (it.t < 0) return;
    if (it.unit == 0) {
        const IO *row = static_cast<const IO *>(p.latent) + it.t * p.latent_stride;
        load8(row + 8 * lane, it.r[0]);
        load8(row + 256 + 8 * lane, it.r[1]);
        if (lane < 4) {
            const IO *kr = static_cast<const IO *>(p.k_pe) + it.t * p.k_pe_stride;
            load8(kr + lo, it.r[2]);
            load8(kr + hi, it.r[3]);
        }
    } else {
        const int head = (it.unit - 1) * kUnitHeads + (lane >> 2);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (head + 8 * u < p.heads) {
                const IO *qr = static_cast<const IO *>(p.q_pe) + it.t * p.q_ts + (head + 8 * u) * p.q_hs;
                load8(qr + lo, it.r[2 * u]);
                load8(qr + hi, it.r[2 * u + 1]);
            }
    }
    if (p.cos_sin && it.pos >= 0 && it.pos < p.num_positions) {
        const float *cs = p.cos_sin + (size_t)it.pos * kLatP + 8 * (lane & 3);
        load8(cs, it.c);
        load8(cs + kLatP / 2, it.s);
    }
}

template <typename IO>
__device__ __forceinline__ void finish(const LatentAppend &p, Item<IO> &it, int lane, int lo, int hi)
{
    if (p.cos_sin && (it.pos < 0 || it.pos >= p.num_positions)) {  // the token is left out
        if (it.unit == 0 && lane == 0 && p.errors) atomicOr(p.errors, DEV_ERR_POSITION);
        return;
    }
    if (it.unit > 0) {
        const int head = (it.unit - 1) * kUnitHeads + (lane >> 2);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (head + 8 * u < p.heads) {
                if (p.cos_sin) rotate8(it.r[2 * u], it.r[2 * u + 1], it.c, it.s, p.interleaved);
                IO *qo = static_cast<IO *>(p.q_pe_out) + it.t * p.qo_ts + (head + 8 * u) * p.qo_hs;
                store8(qo + lo, it.r[2 * u]);
                store8(qo + hi, it.r[2 * u + 1]);
            }
        return;
    }
    if (p.cos_sin && lane < 4) rotate8(it.r[2], it.r[3], it.c, it.s, p.interleaved);
    if (p.norm_weight) {
        const IO *w = static_cast<const IO *>(p.norm_weight);
        Raw8<IO> r0, r1;
        load8(w + 8 * lane, r0);
        load8(w + 256 + 8 * lane, r1);
        float a[8], b[8], w0[8], w1[8];
        widen(it.r[0], a);
        widen(it.r[1], b);
        widen(r0, w0);
        widen(r1, w1);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
        for (int m = 16; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float rn = 1.f / sqrtf(ss * (1.f / kLatR) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] *= rn * w0[i];
            b[i] *= rn * w1[i];
        }
        narrow(a, it.r[0]);
        narrow(b, it.r[1]);
    }
    if (p.latent_out) {
        IO *out = static_cast<IO *>(p.latent_out) + it.t * p.lo_stride;
        store8(out + 8 * lane, it.r[0]);
        store8(out + 256 + 8 * lane, it.r[1]);
    }
    if (p.k_pe_out && lane < 4) {
        IO *out = static_cast<IO *>(p.k_pe_out) + it.t * p.ko_stride;
        store8(out + lo, it.r[2]);
        store8(out + hi, it.r[3]);
    }
    if (it.slot < 0 || it.slot >= p.num_slots) {  // -1: not cached
        if (it.slot != -1 && lane == 0 && p.errors) atomicOr(p.errors, DEV_ERR_SLOT);
        return;
    }
    IO *c = static_cast<IO *>(p.cache) + (int64_t)it.slot * kLatC;
    store8(c + 8 * lane, it.r[0]);
    store8(c + 256 + 8 * lane, it.r[1]);
    if (lane < 4) {
        store8(c + kLatR + lo, it.r[2]);
        store8(c + kLatR + hi, it.r[3]);
    }
}

// q_pe / q_pe_out, latent / latent_out and k_pe / k_pe_out may be the same rows: a unit is read and written
// by the same lanes, and no other unit touches its rows.
template <typename IO>
__global__ void __launch_bounds__(32 * kWarps)
latent_append_kernel(const LatentAppend p)
{
    const int lane = threadIdx.x & 31;
    const int units = 1 + (p.q_pe_out ? (p.heads + kUnitHeads - 1) / kUnitHeads : 0);
    const int64_t total = (int64_t)p.tokens * units, step = (int64_t)gridDim.x * kWarps;
    int64_t work = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    int lo, hi;
    quarter_at(lane & 3, p.interleaved, lo, hi);
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    Item<IO> it, next, after;
    ask_numbers(p, work, total, units, it);
    ask_numbers(p, work + step, total, units, next);
    ask_rows(p, it, lane, lo, hi);
    while (it.t >= 0) {
        work += step;
        ask_numbers(p, work + step, total, units, after);
        ask_rows(p, next, lane, lo, hi);
        finish(p, it, lane, lo, hi);
        it = next;
        next = after;
    }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppend &p)
{
    const int64_t units = 1 + (p.q_pe_out ? (p.heads + kUnitHeads - 1) / kUnitHeads : 0);
    const int64_t needed = (p.tokens * units + kWarps - 1) / kWarps;
    if (needed == 0) return cudaSuccess;
    const int blocks = (int)(needed < kMaxBlocks ? needed : kMaxBlocks);
    return latent_launch(p.dtype == KDA_DTYPE_BF16 ? latent_append_kernel<__nv_bfloat16> : latent_append_kernel<float>,
                         dim3((unsigned)blocks), 32 * kWarps, 0, p.stream, 1, p);
}

}  // namespace kda
