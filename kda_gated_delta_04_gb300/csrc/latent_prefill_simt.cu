// latent_prefill_simt.cu -- expanded latent attention over packed sequences on the CUDA cores
// (fp32 I/O, exact fp32 products).
//
//   s_ij = scale q_i . [k_nope_j, k_pe_j],  o_i = sum_j softmax_j(s_i) v_j
//
// A sequence of lq queries and lk keys is aligned at its end: query i sees keys j <= i + lk - lq
// (causal) or all.  One CTA holds 64 queries of one head and passes over the keys in tiles of 64
// with a running maximum and sum per query (base 2).
#include <math.h>

#include "latent.cuh"

namespace kda {
namespace {

constexpr int kT = 256, kM = 64, kN = 64;  // threads, queries and keys per tile
constexpr int kLdQ = kLatQK + 4, kLdV = kLatN, kLdS = kN + 4;  // row strides (floats)

struct Smem {
    float q[kM][kLdQ];
    float k[kN][kLdQ];
    float v[kN][kLdV];
    float p[kM][kLdS];
};

// Threads are 16 x 16: thread (ty, tx) has queries 4 ty .. 4 ty + 3, and keys tx + 16 j or output
// channels 4 tx + 64 j.  The 16 threads of a query row are half a warp.
template <typename IO>
__global__ void __launch_bounds__(kT, 1) latent_prefill_simt_kernel(const LatentPrefill p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int h = blockIdx.y;
    // Query tiles are numbered so that sequence n's start at cu_q[n] / 64 + n: increasing in n,
    // with room for every tile, found by bisection.  Late tiles (most keys) run first.
    const int tile = (int)(gridDim.x - 1 - blockIdx.x);
    const LatentTile at = latent_tile(p, tile, kM);
    if (tile == 0 && h == 0 && tid < 32) {
        latent_check_cu(p.cu_q, p.num_seqs, p.q_tokens, p.errors);
        latent_check_cu(p.cu_k, p.num_seqs, p.k_tokens, p.errors);
    }
    if (at.rows <= 0) return;
    for (int e = tid; e < kM * (kLatQK / 4); e += kT) {
        const int r = e / (kLatQK / 4), c = 4 * (e - r * (kLatQK / 4));
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < at.rows) x = load4_io(static_cast<const IO *>(p.q) + (int64_t)(at.q0 + r) * p.q_ts + h * p.q_hs + c);
        *reinterpret_cast<float4 *>(&sm.q[r][c]) = x;
    }
    float m[4], l[4], acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = 0; j0 < at.keys; j0 += kN) {
        __syncthreads();
        for (int e = tid; e < kN * (kLatQK / 4); e += kT) {
            const int r = e / (kLatQK / 4), c = 4 * (e - r * (kLatQK / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + r < at.keys) {
                const int64_t j = at.k0 + j0 + r;
                x = c < kLatN ? load4_io(static_cast<const IO *>(p.k_nope) + j * p.kn_ts + h * p.kn_hs + c)
                              : load4_io(static_cast<const IO *>(p.k_pe) + j * p.kp_ts + (c - kLatN));
            }
            *reinterpret_cast<float4 *>(&sm.k[r][c]) = x;
        }
        for (int e = tid; e < kN * (kLatN / 4); e += kT) {
            const int r = e / (kLatN / 4), c = 4 * (e - r * (kLatN / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + r < at.keys)
                x = load4_io(static_cast<const IO *>(p.v) + (int64_t)(at.k0 + j0 + r) * p.v_ts + h * p.v_hs + c);
            *reinterpret_cast<float4 *>(&sm.v[r][c]) = x;
        }
        __syncthreads();
        float s[4][4] = {};
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
                for (int j = 0; j < 4; ++j)
                    s[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
        }
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
        __syncwarp();  // a query row's weights are written and read by the same half warp
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
                    acc[i][0] += x * va.x; acc[i][1] += x * va.y; acc[i][2] += x * va.z; acc[i][3] += x * va.w;
                    acc[i][4] += x * vb.x; acc[i][5] += x * vb.y; acc[i][6] += x * vb.z; acc[i][7] += x * vb.w;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 8; d; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        const int r = 4 * ty + i;
        if (r >= at.rows) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const float lo[4] = {acc[i][0] * inv, acc[i][1] * inv, acc[i][2] * inv, acc[i][3] * inv};
        const float hi[4] = {acc[i][4] * inv, acc[i][5] * inv, acc[i][6] * inv, acc[i][7] * inv};
        IO *o = static_cast<IO *>(p.o) + ((int64_t)(at.q0 + r) * p.heads + h) * kLatN + 4 * tx;
        store_io4(o, lo);
        store_io4(o + 64, hi);
        if (p.lse && tx == 0) p.lse[(int64_t)(at.q0 + r) * p.heads + h] = m[i] * kLn2 + logf(l[i]);
    }
}

template <typename IO>
cudaError_t launch_simt(const LatentPrefill &p)
{
    const cudaError_t err = cudaFuncSetAttribute(latent_prefill_simt_kernel<IO>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (err != cudaSuccess) return err;
    const dim3 grid((unsigned)(p.q_tokens / kM + p.num_seqs), (unsigned)p.heads);
    latent_prefill_simt_kernel<IO><<<grid, kT, sizeof(Smem), p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_prefill_simt(const LatentPrefill &p)
{
    return launch_simt<float>(p);
}

}  // namespace kda
