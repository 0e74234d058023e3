// latent_append.cu -- one token's row into the latent cache: the latent vector normalised
// (RMSNorm), its position key rotated, both written to the token's cache slot, and in the same
// launch the rotation of the token's queries.
//
//   y = w x / sqrt(mean(x^2) + eps)            (512 channels; no weight: y = x)
//   (a, b)_i -> (a cos_i - b sin_i, b cos_i + a sin_i), i < 32   (position channels)
//
// The pair i is (i, i + 32) or, interleaved, (2i, 2i + 1).  Sums and products are fp32, rounded
// once when stored.  Bound by memory (T large) or by the latency of one dependent chain,
// position -> table row -> store (T small).  A warp is one unit of work and one CTA: either a token's
// latent row and position key, or the position channels of 16 of its query heads (32 lanes = 8 heads x 4
// quarters of the pairs, two heads and 2 x 8 pairs a lane).  Small batches so spread over 1 + H / 16 CTAs a
// token, and large ones keep up to 2 KB a warp in flight while warps come and go singly: 32,768 tokens of 32
// heads 72 us (386 MB, 5.4 TB/s); CTAs of four warps 76, one head a lane 79, one warp and one head 88.
#include "latent.cuh"

namespace kda {
namespace {

constexpr int kWarps = 1;

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
__device__ __forceinline__ void rotate8(Raw8<IO> &rx, Raw8<IO> &ry, const float (&c)[8], const float (&s)[8],
                                        bool interleaved)
{
    float x[8], y[8];
    widen(rx, x);
    widen(ry, y);
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

constexpr int kRounds = 2;  // heads of a lane in a query unit
constexpr int kUnitHeads = 8 * kRounds;

// q_pe / q_pe_out, latent / latent_out and k_pe / k_pe_out may be the same rows: a lane reads
// what it overwrites before it does.
template <typename IO>
__global__ void __launch_bounds__(32 * kWarps)
latent_append_kernel(const LatentAppend p)
{
    const int lane = threadIdx.x & 31;
    const int units = 1 + (p.q_pe_out ? (p.heads + kUnitHeads - 1) / kUnitHeads : 0);
    const int64_t work = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (work >= (int64_t)p.tokens * units) return;
    const int t = (int)(work / units), unit = (int)(work - (int64_t)t * units);
    const int j = lane & 3;
    int lo, hi;
    quarter_at(j, p.interleaved, lo, hi);
    const int pos = p.cos_sin ? p.positions[t] : 0;

    // the loads that depend on nothing, beside the chain position -> table row
    Raw8<IO> x[kRounds], y[kRounds], x0, x1;
    const int head = (unit - 1) * kUnitHeads + (lane >> 2);
    int64_t slot = -1;
    if (unit == 0) {
        slot = p.slots[t];
        const IO *row = static_cast<const IO *>(p.latent) + t * p.latent_stride;
        load8(row + 8 * lane, x0);
        load8(row + 256 + 8 * lane, x1);
        if (lane < 4) {
            const IO *kr = static_cast<const IO *>(p.k_pe) + t * p.k_pe_stride;
            load8(kr + lo, x[0]);
            load8(kr + hi, y[0]);
        }
    } else {
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (head + 8 * r < p.heads) {
                const IO *qr = static_cast<const IO *>(p.q_pe) + t * p.q_ts + (head + 8 * r) * p.q_hs;
                load8(qr + lo, x[r]);
                load8(qr + hi, y[r]);
            }
    }
    if (p.cos_sin && (pos < 0 || pos >= p.num_positions)) {  // the token is left out
        if (unit == 0 && lane == 0 && p.errors) atomicOr(p.errors, DEV_ERR_POSITION);
        return;
    }
    if (p.cos_sin && (unit > 0 || lane < 4)) {
        const float *cs = p.cos_sin + (size_t)pos * kLatP + 8 * j;
        Raw8<float> rc, rs;
        load8(cs, rc);
        load8(cs + kLatP / 2, rs);
        float c[8], s[8];
        widen(rc, c);
        widen(rs, s);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (unit == 0 ? r == 0 : head + 8 * r < p.heads) rotate8(x[r], y[r], c, s, p.interleaved);
    }
    if (unit > 0) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (head + 8 * r < p.heads) {
                IO *qo = static_cast<IO *>(p.q_pe_out) + t * p.qo_ts + (head + 8 * r) * p.qo_hs;
                store8(qo + lo, x[r]);
                store8(qo + hi, y[r]);
            }
        return;
    }
    if (p.norm_weight) {
        const IO *w = static_cast<const IO *>(p.norm_weight);
        Raw8<IO> r0, r1;
        load8(w + 8 * lane, r0);
        load8(w + 256 + 8 * lane, r1);
        float a[8], b[8], w0[8], w1[8];
        widen(x0, a);
        widen(x1, b);
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
        narrow(a, x0);
        narrow(b, x1);
    }
    if (p.latent_out) {
        IO *out = static_cast<IO *>(p.latent_out) + t * p.lo_stride;
        store8(out + 8 * lane, x0);
        store8(out + 256 + 8 * lane, x1);
    }
    if (p.k_pe_out && lane < 4) {
        IO *out = static_cast<IO *>(p.k_pe_out) + t * p.ko_stride;
        store8(out + lo, x[0]);
        store8(out + hi, y[0]);
    }
    if (slot < 0 || slot >= p.num_slots) {  // -1: not cached
        if (slot != -1 && lane == 0 && p.errors) atomicOr(p.errors, DEV_ERR_SLOT);
        return;
    }
    IO *c = static_cast<IO *>(p.cache) + slot * kLatC;
    store8(c + 8 * lane, x0);
    store8(c + 256 + 8 * lane, x1);
    if (lane < 4) {
        store8(c + kLatR + lo, x[0]);
        store8(c + kLatR + hi, y[0]);
    }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppend &p)
{
    const int64_t units = 1 + (p.q_pe_out ? (p.heads + kUnitHeads - 1) / kUnitHeads : 0);
    const int64_t blocks = (p.tokens * units + kWarps - 1) / kWarps;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (p.dtype == KDA_DTYPE_BF16)
        latent_append_kernel<__nv_bfloat16><<<(unsigned)blocks, 32 * kWarps, 0, p.stream>>>(p);
    else
        latent_append_kernel<float><<<(unsigned)blocks, 32 * kWarps, 0, p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
