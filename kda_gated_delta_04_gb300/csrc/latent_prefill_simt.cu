// latent_prefill_simt.cu -- expanded latent attention over packed sequences on the CUDA cores
// (fp32 I/O, exact fp32 products).
//
//   s_ij = scale q_i . [k_nope_j, k_pe_j],  o_i = sum_j softmax_j(s_i) v_j
//
// A sequence of lq queries and lk keys is aligned at its end: query i sees keys j <= i + lk - lq
// (causal) or all.  64 queries of one head pass over the keys in tiles of 64 with a running maximum and
// sum per query (base 2).  Bound by the fp32 rate: 128 products a cycle and SM, 10,240 cycles a tile.
// K and V have one buffer each: K of the next tile is copied (cp.async) while the softmax and the value
// product run, V while the scores do.
//
// With fewer query tiles than SMs a cluster of two or four CTAs shares a query tile, each taking every
// second or fourth key tile, and the results are joined through distributed shared memory (1,027 tokens, 4
// heads, 68 tiles: 60 us with four, 91 with two, 164 with one).  4,096 tokens, 8 heads: 1.1 ms, 39 TFLOP/s:
// the products take half of the cycles, the reads of their operands from shared memory the rest.
#include <math.h>

#include "latent.cuh"
#include "latent_ptx.cuh"

namespace kda {
namespace {

using namespace ptx;

constexpr int kT = 256, kM = 64, kN = 64;  // threads, queries and keys per tile
constexpr int kLdQ = kLatQK + 4, kLdV = kLatN, kLdS = kN + 4;  // row strides (floats)

struct Smem {
    float q[kM][kLdQ];
    float k[kN][kLdQ];
    union {
        struct {
            float v[kN][kLdV];
            float p[kM][kLdS];
        };
        float o[kM][kLatN];  // a CTA's unnormalised output, for the join
    };
    float m[kM], l[kM];
};

// Threads are 16 x 16: thread (ty, tx) has queries 4 ty .. 4 ty + 3, and keys tx + 16 j or output
// channels 4 tx + 64 j.  The 16 threads of a query row are half a warp.  CS: CTAs per query tile.
template <int CS>
__global__ void __launch_bounds__(kT, 1) latent_prefill_simt_kernel(const LatentPrefill p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int rank = CS > 1 ? (int)cluster_rank() : 0, unit = blockIdx.x / CS;
    const int h = unit % p.heads;
    pdl_wait();
    const LatentLane mine = latent_lane(p, kM, tid & 31);
    const LatentTile at = latent_tile(p, mine, unit / p.heads, (int)(gridDim.x / CS / p.heads), kM, tid & 31);
    if (blockIdx.x == 0 && tid < 32) {
        latent_check_cu(p.cu_q, p.num_seqs, p.q_tokens, p.errors);
        latent_check_cu(p.cu_k, p.num_seqs, p.k_tokens, p.errors);
    }
    if (at.rows <= 0) return;  // every CTA of the cluster
    const float *q = static_cast<const float *>(p.q) + h * p.q_hs, *kn = static_cast<const float *>(p.k_nope) + h * p.kn_hs;
    const float *kp = static_cast<const float *>(p.k_pe), *v = static_cast<const float *>(p.v) + h * p.v_hs;
    auto copy_k = [&](int j0) {
        for (int e = tid; e < kN * (kLatQK / 4); e += kT) {
            const int r = e / (kLatQK / 4), c = 4 * (e - r * (kLatQK / 4));
            const bool ok = j0 + r < at.keys;
            const int64_t j = ok ? at.k0 + j0 + r : 0;
            cp_async16(&sm.k[r][c], c < kLatN ? kn + j * p.kn_ts + c : kp + j * p.kp_ts + (c - kLatN), ok);
        }
        cp_async_commit();
    };
    auto copy_v = [&](int j0) {
        for (int e = tid; e < kN * (kLatN / 4); e += kT) {
            const int r = e / (kLatN / 4), c = 4 * (e - r * (kLatN / 4));
            const bool ok = j0 + r < at.keys;
            cp_async16(&sm.v[r][c], v + (ok ? at.k0 + j0 + r : 0) * (int64_t)p.v_ts + c, ok);
        }
        cp_async_commit();
    };
    const int first = rank * kN, step = CS * kN;
    for (int e = tid; e < kM * (kLatQK / 4); e += kT) {
        const int r = e / (kLatQK / 4), c = 4 * (e - r * (kLatQK / 4));
        const bool ok = r < at.rows;
        cp_async16(&sm.q[r][c], q + (at.q0 + (ok ? r : 0)) * (int64_t)p.q_ts + c, ok);
    }
    copy_k(first);
    copy_v(first);
    float m[4], l[4];
    alignas(8) float acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = first; j0 < at.keys; j0 += step) {
        cp_async_wait<1>();  // K (V may still be on its way)
        __syncthreads();
        float s[4][4];
        float2 s2[4][4] = {};  // channels two by two, added at the end
#pragma unroll 4
        for (int c = 0; c < kLatQK; c += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(&sm.q[4 * ty + i][c]);
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][c]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s2[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s2[i][j]);
                    s2[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s2[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
        __syncthreads();  // K is read
        copy_k(j0 + step);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = p.causal ? at.off + 4 * ty + i : at.keys - 1;  // last key this query sees
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + tx + 16 * j;
                s[i][j] = key <= last && key < at.keys ? s[i][j] * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int d = 8; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - base);
            m[i] = mn;
            l[i] *= f;
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[i][c] *= f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2f(s[i][j] - base);
                l[i] += e;
                sm.p[4 * ty + i][tx + 16 * j] = e;
            }
        }
        cp_async_wait<1>();  // V (the next K may still be on its way)
        __syncthreads();
#pragma unroll 4
        for (int r = 0; r < kN; r += 4) {
            float4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(&sm.p[4 * ty + i][r]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 va = *reinterpret_cast<const float4 *>(&sm.v[r + u][4 * tx]);
                const float4 vb = *reinterpret_cast<const float4 *>(&sm.v[r + u][64 + 4 * tx]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = u == 0 ? w[i].x : u == 1 ? w[i].y : u == 2 ? w[i].z : w[i].w;
                    const float2 xx = make_float2(x, x);
                    float2 *o = reinterpret_cast<float2 *>(acc[i]);
                    o[0] = fma2(xx, make_float2(va.x, va.y), o[0]);
                    o[1] = fma2(xx, make_float2(va.z, va.w), o[1]);
                    o[2] = fma2(xx, make_float2(vb.x, vb.y), o[2]);
                    o[3] = fma2(xx, make_float2(vb.z, vb.w), o[3]);
                }
            }
        }
        __syncthreads();  // V is read
        copy_v(j0 + step);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 8; d; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    }
    cp_async_wait<0>();
    if constexpr (CS > 1) {
        // every CTA's part where the others can read it, then each writes a share of the rows
        __syncthreads();  // o lies over v and p
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            *reinterpret_cast<float4 *>(&sm.o[r][4 * tx]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            *reinterpret_cast<float4 *>(&sm.o[r][64 + 4 * tx]) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            if (tx == 0) {
                sm.m[r] = m[i];
                sm.l[r] = l[i];
            }
        }
        cluster_sync();
        constexpr int kShare = kM / CS;
        for (int e = tid; e < kShare * (kLatN / 4); e += kT) {
            const int r = rank * kShare + e / (kLatN / 4), c = 4 * (e % (kLatN / 4));
            float pm[CS], top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int u = 0; u < CS; ++u) {
                pm[u] = peer_load(&sm.m[r], u);
                top = fmaxf(top, pm[u]);
            }
            const float base = top == -INFINITY ? 0.f : top;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < CS; ++u) {
                const float f = exp2f(pm[u] - base);
                const float4 y = peer_load4(&sm.o[r][c], u);
                sum += f * peer_load(&sm.l[r], u);
                x.x += f * y.x; x.y += f * y.y; x.z += f * y.z; x.w += f * y.w;
            }
            if (r >= at.rows) continue;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int64_t row = (int64_t)(at.q0 + r) * p.heads + h;
            store4_io(static_cast<float *>(p.o) + row * kLatN + c, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
            if (p.lse && c == 0) p.lse[row] = top * kLn2 + logf(sum);
        }
        cluster_sync();  // no CTA goes while another reads its part
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= at.rows) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const float lo[4] = {acc[i][0] * inv, acc[i][1] * inv, acc[i][2] * inv, acc[i][3] * inv};
        const float hi[4] = {acc[i][4] * inv, acc[i][5] * inv, acc[i][6] * inv, acc[i][7] * inv};
        const int64_t row = (int64_t)(at.q0 + r) * p.heads + h;
        float *o = static_cast<float *>(p.o) + row * kLatN + 4 * tx;
        store_io4(o, lo);
        store_io4(o + 64, hi);
        if (p.lse && tx == 0) p.lse[row] = m[i] * kLn2 + logf(l[i]);
    }
}

template <int CS>
cudaError_t launch(const LatentPrefill &p, int64_t units)
{
    cudaError_t err = cudaFuncSetAttribute(latent_prefill_simt_kernel<CS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)sizeof(Smem));
    if (err != cudaSuccess) return err;
    return latent_launch(latent_prefill_simt_kernel<CS>, dim3((unsigned)(units * CS)), kT, sizeof(Smem), p.stream, CS, p);
}

}  // namespace

cudaError_t launch_latent_prefill_simt(const LatentPrefill &p)
{
    const int64_t tiles = p.num_seqs == 1 ? (p.q_tokens + kM - 1) / kM : p.q_tokens / kM + p.num_seqs;
    const int64_t units = tiles * p.heads;
    if (4 * units > 0x7fffffff) return cudaErrorInvalidValue;
    // Four CTAs a tile up to half a tile an SM, two up to one: each CTA costs some 13 us beside its key tiles
    // (9 us each), one runs on an SM, and with more tiles than SMs they share the time out without it.  136
    // tiles of 1,027 tokens 98 us with two CTAs, 119 with four, 165 with one; 272 of them 165 with one, 193
    // with two; 112 tiles of sequences of 1 to 600 tokens 54 with two, 66 with four, 99 with one.
    return units <= 152 / 2 ? launch<4>(p, units) : units <= 152 ? launch<2>(p, units) : launch<1>(p, units);
}

}  // namespace kda
