// linear_simt.cu -- projections on the CUDA cores: fp32, and bf16 rows that the tensor cores' copies
// cannot take (odd strides or addresses).
//
//   y_mn = act(sum_k x_mk w_nk + b_n) + r_mn        exact products, fp32 sums
//
// Many outputs: tiles of 64 x 128, in four groups of 64 threads that take every fourth step of eight inputs, 16 x 8
// outputs a thread, so that the 24 operands of a step, which shared memory gives to registers at 128 bytes a cycle,
// keep the 128 products' units busy for longer; products come two an instruction.  The next steps' inputs are on their
// way meanwhile, element by element, as rows may start anywhere: fp32 to shared memory, bf16 through registers.  1,027
// rows, 1,025 inputs, 1,003 outputs, fp32: 72 us, 29 TFLOP/s (of 75); through registers 81; two groups with 8 x 8 a
// thread 90; tiles of 64 x 64 with 4 x 4 a thread 105.  Without the copies the products and their operands take 56.
// Few outputs: a CTA has four outputs of eight rows and its threads share the inputs.
#include "latent_ptx.cuh"
#include "layer.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

constexpr int kInputs = 16;  // that lie in a row and are asked for by neighbouring threads (us with 8, 16, 32: 72.1, 71.7, 76.4)
constexpr int kTileM = 64, kTileN = 128, kDepth = 8, kGroup = 64, kGroups = 4, kThreads = kGroups * kGroup;

template <typename OUT>
__device__ __forceinline__ void finish(const Linear &p, int64_t m, int n, float v, float bias)
{
    v = activate<OUT>(v + bias, p.act);
    if (p.residual) v += load_io(static_cast<const OUT *>(p.residual) + m * p.rs + n);
    store_io(static_cast<OUT *>(p.y) + m * p.ys + n, v);
}

// (a row's pitch: 16-byte pieces, and the rows of a warp's stores in banks of their own)
struct Stage {
    float x[kDepth][kTileM + 4], w[kDepth][kTileN + 4];
};
// Steps in shared memory: fp32 comes by asynchronous copies of an element, two steps ahead; bf16 through registers.
template <typename IO> constexpr int kStages = sizeof(IO) == 4 ? 3 : 2;
template <typename IO> constexpr int kTileSmem = kStages<IO> * kGroups * (int)sizeof(Stage);

// 4 bytes to shared memory; zero where there are none (`from` is a valid address all the same).
__device__ __forceinline__ void cp_async4(float *to, const float *from, bool some)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(to)), "l"(from), "r"(some ? 4 : 0) : "memory");
}

template <typename IO, typename OUT>
__global__ void __launch_bounds__(kThreads)
linear_tile_kernel(const Linear p, int tiles_n)
{
    extern __shared__ __align__(16) unsigned char raw_smem[];
    Stage(*stage)[kGroups] = reinterpret_cast<Stage(*)[kGroups]>(raw_smem);
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kTileM;
    const int n0 = (int)(blockIdx.x % tiles_n) * kTileN;
    const int group = threadIdx.x / kGroup, tid = threadIdx.x % kGroup;
    // a thread's outputs: rows 4 ty + 16 i + .. (i < 4), columns 4 tx + 64 j + .. (j < 2)
    const int tx = tid & 15, ty = tid >> 4;
    // what it brings in, of all groups' inputs: lk, lk + kInputs, .. of rows lr, lr + kStep, ..
    constexpr int kAll = kGroups * kDepth, kStep = kThreads / kInputs, kTimes = kAll / kInputs, R = kStages<IO>;
    constexpr int kX = kTileM / kStep, kW = kTileN / kStep;
    const int lk = threadIdx.x % kInputs, lr = threadIdx.x / kInputs;
    // (rows past the last: the last again, whose outputs are not stored)
    const int64_t mr = min(m0 + lr, p.rows - 1);
    const int nr = min(n0 + lr, p.n - 1), nx = (int)min((p.rows - 1 - mr) / kStep, (int64_t)kX), nw = (p.n - 1 - nr) / kStep;
    const IO *x = static_cast<const IO *>(p.x) + mr * p.xs, *w = static_cast<const IO *>(p.w) + nr * p.ws;
    const int64_t step_x = kStep * p.xs, step_w = kStep * p.ws;
    auto each = [&](int k0, auto take_x, auto take_w) {  // of a step's inputs what this thread brings in
#pragma unroll
        for (int h = 0; h < kTimes; ++h) {
            const int k = k0 + h * kInputs + lk;
            const bool in = k < p.k;
            const IO *at = x + (in ? k : 0);
#pragma unroll
            for (int i = 0; i < kX; ++i) {
                take_x(h, i, at, in);
                if (i < nx) at += step_x;
            }
            at = w + (in ? k : 0);
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                take_w(h, i, at, in);
                if (i < nw) at += step_w;
            }
        }
    };
    auto to_x = [&](Stage *to, int h, int i) { return &to[(h * kInputs + lk) / kDepth].x[lk % kDepth][lr + i * kStep]; };
    auto to_w = [&](Stage *to, int h, int i) { return &to[(h * kInputs + lk) / kDepth].w[lk % kDepth][lr + i * kStep]; };
    float2 acc[16][4] = {};
    auto products = [&](const Stage &at) {
#pragma unroll 2
        for (int k = 0; k < kDepth; ++k) {
            const float4 b0 = *reinterpret_cast<const float4 *>(&at.w[k][4 * tx]);
            const float4 b1 = *reinterpret_cast<const float4 *>(&at.w[k][4 * tx + 64]);
            const float2 b[4] = {{b0.x, b0.y}, {b0.z, b0.w}, {b1.x, b1.y}, {b1.z, b1.w}};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 a4 = *reinterpret_cast<const float4 *>(&at.x[k][4 * ty + 16 * i]);
                const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[4 * i + u][j] = ptx::fma2(make_float2(a[u], a[u]), b[j], acc[4 * i + u][j]);
            }
        }
    };
    if constexpr (sizeof(IO) == 4) {
        auto ask = [&](int k0, Stage *to) {
            if (k0 < p.k)
                each(k0, [&](int h, int i, const IO *at, bool in) { cp_async4(to_x(to, h, i), at, in); },
                     [&](int h, int i, const IO *at, bool in) { cp_async4(to_w(to, h, i), at, in); });
            ptx::cp_async_commit();  // (a group for every step, empty past the last)
        };
#pragma unroll
        for (int i = 0; i < R - 1; ++i) ask(i * kAll, stage[i]);
        int now = 0, next = R - 1;
#pragma unroll 1
        for (int k0 = 0; k0 < p.k; k0 += kAll) {
            ptx::cp_async_wait<R - 2>();
            __syncthreads();  // this step has come, and the one before has been used
            ask(k0 + (R - 1) * kAll, stage[next]);
            products(stage[now][group]);
            now = now + 1 == R ? 0 : now + 1;
            next = next + 1 == R ? 0 : next + 1;
        }
        ptx::cp_async_wait<0>();
        __syncthreads();
    } else {
        float rx[kTimes][kX], rw[kTimes][kW];
        auto ask = [&](int k0) {
            each(k0, [&](int h, int i, const IO *at, bool in) { rx[h][i] = in ? load_io(at) : 0.f; },
                 [&](int h, int i, const IO *at, bool in) { rw[h][i] = in ? load_io(at) : 0.f; });
        };
        auto put = [&](Stage *to) {
#pragma unroll
            for (int h = 0; h < kTimes; ++h) {
#pragma unroll
                for (int i = 0; i < kX; ++i) *to_x(to, h, i) = rx[h][i];
#pragma unroll
                for (int i = 0; i < kW; ++i) *to_w(to, h, i) = rw[h][i];
            }
        };
        ask(0);
        put(stage[0]);
        __syncthreads();
        int buf = 0;
#pragma unroll 1
        for (int k0 = 0; k0 < p.k; k0 += kAll, buf ^= 1) {
            const bool more = k0 + kAll < p.k;
            if (more) ask(k0 + kAll);
            products(stage[buf][group]);
            if (more) put(stage[buf ^ 1]);
            __syncthreads();
        }
    }
    // The groups' sums, four rows of each thread at a time: group g makes the outputs of the rows of i = g.
    float4 *part = reinterpret_cast<float4 *>(raw_smem);
    static_assert(kTileSmem<IO> >= (kGroups - 1) * 8 * kGroup * (int)sizeof(float4));
    float2 mine[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows of i: the other groups give theirs to group i
        if (group != i) {
            const int from = group < i ? group : group - 1;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    part[((from * 4 + u) * 2 + j) * kGroup + tid] = make_float4(
                        acc[4 * i + u][2 * j].x, acc[4 * i + u][2 * j].y, acc[4 * i + u][2 * j + 1].x, acc[4 * i + u][2 * j + 1].y);
        }
        __syncthreads();
        if (group == i)
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float4 v = make_float4(acc[4 * i + u][2 * j].x, acc[4 * i + u][2 * j].y, acc[4 * i + u][2 * j + 1].x,
                                           acc[4 * i + u][2 * j + 1].y);
#pragma unroll
                    for (int g = 0; g < kGroups - 1; ++g) {
                        const float4 q = part[((g * 4 + u) * 2 + j) * kGroup + tid];
                        v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
                    }
                    mine[u][2 * j] = make_float2(v.x, v.y);
                    mine[u][2 * j + 1] = make_float2(v.z, v.w);
                }
        __syncthreads();
    }
    float bias[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int n = n0 + 4 * tx + (j & 3) + (j >> 2) * 64;
        bias[j] = p.bias && n < p.n ? load_io(static_cast<const IO *>(p.bias) + n) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t m = m0 + 4 * ty + 16 * group + u;
        if (m >= p.rows) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = n0 + 4 * tx + (j & 3) + (j >> 2) * 64;
            if (n < p.n) finish<OUT>(p, m, n, j & 1 ? mine[u][j >> 1].y : mine[u][j >> 1].x, bias[j]);
        }
    }
}

constexpr int kFewThreads = 256, kFewM = 8, kFewN = 4;

template <typename IO, typename OUT>
__global__ void __launch_bounds__(kFewThreads)
linear_few_simt_kernel(const Linear p, int tiles_n)
{
    __shared__ float part[kFewThreads / 32][kFewM * kFewN];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kFewM;
    const int n0 = (int)(blockIdx.x % tiles_n) * kFewN;
    const IO *x = static_cast<const IO *>(p.x) + m0 * p.xs, *w = static_cast<const IO *>(p.w) + (int64_t)n0 * p.ws;
    float acc[kFewM * kFewN] = {};
    for (int k = threadIdx.x; k < p.k; k += kFewThreads) {
        float b[kFewN], a[kFewM];
#pragma unroll
        for (int j = 0; j < kFewN; ++j) b[j] = n0 + j < p.n ? load_io(w + j * p.ws + k) : 0.f;
#pragma unroll
        for (int i = 0; i < kFewM; ++i) a[i] = m0 + i < p.rows ? load_io(x + i * p.xs + k) : 0.f;
#pragma unroll
        for (int i = 0; i < kFewM; ++i)
#pragma unroll
            for (int j = 0; j < kFewN; ++j) acc[i * kFewN + j] = fmaf(a[i], b[j], acc[i * kFewN + j]);
    }
    // the sum of output o to lane o of each warp, and over the warps
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int u = 0; u < m; ++u) {
            const float give = up ? acc[u] : acc[u + m], keep = up ? acc[u + m] : acc[u];
            acc[u] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
    part[threadIdx.x >> 5][lane] = acc[0];
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int64_t m = m0 + lane / kFewN;
    const int n = n0 + lane % kFewN;
    if (m >= p.rows || n >= p.n) return;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kFewThreads / 32; ++i) v += part[i][lane];
    finish<OUT>(p, m, n, v, p.bias ? load_io(static_cast<const IO *>(p.bias) + n) : 0.f);
}

template <typename IO, typename OUT>
cudaError_t launch(const Linear &p)
{
    // A step of a round of tiles takes 58 ns, whatever part of it is used; the others do 3.5e12 products a second: 1,025
    // inputs, 1,003 outputs, fp32, us: 16 rows 8.4 and (tiles) 65, 64 rows 20.7, 68, 128 rows 37.9, 68.
    const int64_t rounds = ((p.rows + kTileM - 1) / kTileM * ((p.n + kTileN - 1) / kTileN) + 151) / 152;
    const bool few = p.rows * p.n <= 200000 * rounds;
    const int tile_m = few ? kFewM : kTileM, tile_n = few ? kFewN : kTileN, tiles_n = (p.n + tile_n - 1) / tile_n;
    const int64_t blocks = (p.rows + tile_m - 1) / tile_m * tiles_n;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    static int configured = -1;
    const cudaError_t err = tc::allow_smem(linear_tile_kernel<IO, OUT>, kTileSmem<IO>, &configured);
    if (err != cudaSuccess) return err;
    return few ? latent_launch(linear_few_simt_kernel<IO, OUT>, dim3((unsigned)blocks), kFewThreads, 0, p.stream, 1, p, tiles_n)
               : latent_launch(linear_tile_kernel<IO, OUT>, dim3((unsigned)blocks), kThreads, kTileSmem<IO>, p.stream, 1, p, tiles_n);
}

}  // namespace

cudaError_t launch_linear_simt(const Linear &p)
{
    return p.dtype == KDA_DTYPE_F32       ? launch<float, float>(p)
           : p.out_dtype == KDA_DTYPE_F32 ? launch<__nv_bfloat16, float>(p)
                                          : launch<__nv_bfloat16, __nv_bfloat16>(p);
}

}  // namespace kda
