// latent.cuh -- latent attention (one shared latent vector and one position key per token):
// problem descriptions, the split of the absorbed decode over the CTAs, and device helpers
// shared by its kernels.
#pragma once

#include "common.cuh"

namespace kda {

// Device-side error bits beside those of common.cuh.
enum : uint32_t {
    DEV_ERR_POSITION = 32u,  // a position outside the rotation table
    DEV_ERR_PAGE = 64u,      // a page index outside the latent cache
};

// The supported widths (other values are refused by the entry points).
constexpr int kLatR = KDA_LATENT_DIM;         // latent channels; the values of the absorbed form
constexpr int kLatP = KDA_LATENT_PE_DIM;      // position channels
constexpr int kLatC = kLatR + kLatP;          // channels of a cache row = absorbed key width
constexpr int kLatN = KDA_LATENT_HEAD_DIM;    // expanded key channels without position; value channels
constexpr int kLatQK = kLatN + kLatP;         // expanded key width
constexpr float kLn2 = 0.6931471805599453f;   // ln 2: log-sum-exp from log2 units
constexpr float kLatLog2e = 1.4426950408889634f;

struct LatentAppend {
    const void *latent, *k_pe, *norm_weight, *q_pe;  // norm_weight, q_pe may be null
    int64_t latent_stride, k_pe_stride, q_ts, q_hs, qo_ts, qo_hs, lo_stride, ko_stride;  // elements
    float eps;
    const float *cos_sin;  // [num_positions, 64]: 32 cosines, 32 sines; null: no rotation
    const int32_t *positions, *slots;
    int num_positions, tokens, heads;
    void *q_pe_out, *latent_out, *k_pe_out, *cache;  // the outputs but the cache may be null
    int64_t num_slots;
    bool interleaved;
    kda_dtype_t dtype;
    uint32_t *errors;
    cudaStream_t stream;
};

struct LatentDecode {
    const void *q, *cache;
    int64_t q_bs, q_hs;  // elements
    int64_t num_pages, table_stride;
    int page_size, table_width;
    const int32_t *table, *lens;
    int batch, heads;
    float scale_log2;  // softmax scale x log2(e)
    void *o;
    float *lse;        // may be null
    char *workspace;
    kda_dtype_t dtype;
    uint32_t *errors;
    cudaStream_t stream;
};

struct LatentPrefill {
    const void *q, *k_nope, *k_pe, *v;
    int64_t q_ts, q_hs, kn_ts, kn_hs, kp_ts, v_ts, v_hs;  // elements
    const int32_t *cu_q, *cu_k;  // both null: one sequence
    int num_seqs;
    int64_t q_tokens, k_tokens;
    int heads;
    float scale_log2;
    bool causal;
    void *o;
    float *lse;  // may be null
    kda_dtype_t dtype;
    uint32_t *errors;
    cudaStream_t stream;
};

kda_status_t check_device();  // kda_api.cu

// Launch of a kernel that waits (griddepcontrol.wait) before its first access to global memory: it may be
// set up while the kernel before it on the stream ends.  cluster: CTAs per cluster (1: none).
template <class... P, class... A>
inline cudaError_t latent_launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                                 A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<A &&>(args)...);
}

cudaError_t launch_latent_append(const LatentAppend &p);
cudaError_t launch_latent_decode_simt(const LatentDecode &p);
cudaError_t launch_latent_prefill_simt(const LatentPrefill &p);
cudaError_t launch_latent_prefill_tc(const LatentPrefill &p);  // bf16
cudaError_t launch_latent_decode_tc(const LatentDecode &p);  // bf16
size_t latent_decode_simt_ws_bytes();
size_t latent_decode_tc_ws_bytes(int heads);

// ---------------------------------------------------------------- absorbed decode: work split
// The cache rows of all (head group, sequence) units, cut into tiles, are one list of W tiles
// (head group outermost, so that CTAs working on the same cache rows for different head groups
// do so at the same time and share them in L2).  CTA c of G' = min(G, W) takes the tiles
// [c W / G', (c + 1) W / G'): every CTA reads the same number of cache rows whatever the lengths,
// and the host needs to know no length.  A unit cut by a CTA boundary leaves partial results
// (the running maximum and sum, and the unnormalised output, fp32): slot 2c for the first unit
// of CTA c, 2c + 1 for its last.  Records tell the joining kernel which CTAs hold a unit's parts, to
// be joined in the order of the cache rows: one record per unit where there are no more units than
// CTAs (few joins, of many parts), else one per CTA boundary (at its first boundary inside a unit).
constexpr int kLatMaxGrid = 320;  // bound on the decode grid (two CTAs on each of 152 SMs, rounded up)
constexpr int kLatHeadTile = 64;  // most heads in one tile

struct LatentJoin {  // at the head of the workspace
    int b, h0;            // sequence and first head; b < 0: nothing to join
    int c_first, c_last;  // CTAs that hold parts
    int first_slot;       // slot of the first part; the others' are 2 c
    int pad[3];
};

constexpr size_t kLatJoinBytes = ((size_t)kLatMaxGrid * sizeof(LatentJoin) + 255) / 256 * 256;

// per slot and head: (maximum in log2 units, sum), then the slots' outputs
__host__ __device__ inline float *latent_ml(char *ws) { return reinterpret_cast<float *>(ws + kLatJoinBytes); }
__host__ __device__ inline float *latent_part(char *ws, int head_tile)
{
    return latent_ml(ws) + (size_t)2 * kLatMaxGrid * head_tile * 2;
}
inline size_t latent_ws_bytes(int head_tile, int grid)
{
    return kLatJoinBytes + (size_t)2 * kLatMaxGrid * head_tile * 2 * sizeof(float) +
           (size_t)2 * grid * head_tile * kLatR * sizeof(float);
}
// Joins the parts of the split units; `head_tile` heads per slot.
cudaError_t launch_latent_join(const LatentDecode &p, int head_tile, int grid);
// Whether records are per unit (see above).
__host__ __device__ inline bool latent_join_by_unit(int batch, int heads, int head_tile, int grid)
{
    return (int64_t)batch * ((heads + head_tile - 1) / head_tile) <= grid;
}

#ifdef __CUDACC__
// ---------------------------------------------------------------- expanded prefill: query tiles
// A tile of one sequence's queries: rows from query q0 (global), the sequence's keys from k0
// (global) and their count, how many of them the tile's last row sees, and the last key (counted
// from k0) that its first row sees when causal.  rows 0: no tile has this number.
struct LatentTile {
    int q0, k0, rows, klen, keys, off;
};

// Token range [t0, t1) of sequence n, held to the buffer (int: the token counts are below 2^31).
__device__ __forceinline__ void latent_range(const int32_t *cu, int n, int total, int &t0, int &t1)
{
    int64_t a, b;
    seq_range(cu, n, total, a, b);
    t0 = (int)a;
    t1 = (int)b;
}

// The query tiles of m rows in the order in which they are worked on, by a whole warp, without a table.
//  Up to 32 sequences (a lane each): the tiles with the highest index in their sequence first, so that
//  those with the most keys (causal) start first and the numbers without a tile come last.  With C(x) the
//  tiles of index x and more over all sequences, the index is the largest x with C(x) > order.
//  More: sequence n's tiles are numbered from cu_q[n] / m + n, which increases with n and leaves room for
//  all of them, and searched 32 candidates at a time (65,535 sequences: four rounds of one load, the first
//  of them here); late numbers first.
// A malformed cu_q or cu_k is reported and held to the buffers.
struct LatentLane {
    int q0, q1, k0, k1;  // up to 32 sequences: the lane's
    int first;           // more: the number of the first tile of the lane's candidate in the first round
};
__device__ __forceinline__ LatentLane latent_lane(const LatentPrefill &p, int m, int lane)
{
    LatentLane l{};
    const int step = (p.num_seqs + 31) / 32, at = lane * step;
    if (at < p.num_seqs) {
        latent_range(p.cu_q, at, (int)p.q_tokens, l.q0, l.q1);
        if (step == 1) latent_range(p.cu_k, at, (int)p.k_tokens, l.k0, l.k1);
        l.first = l.q0 / m + at;
    } else {
        l.first = 0x7fffffff;
    }
    return l;
}

// The order-th of `count` numbers.
__device__ __forceinline__ LatentTile latent_tile(const LatentPrefill &p, const LatentLane &l, int order, int count,
                                                  int m, int lane)
{
    int q0 = l.q0, q1 = l.q1, k0 = l.k0, k1 = l.k1, from, index;  // (from: the lane that has the sequence)
    if (p.num_seqs <= 32) {
        const int tiles = (q1 - q0 + m - 1) / m;
        auto above = [&](int x) { return (int)__reduce_add_sync(0xffffffffu, (unsigned)max(0, tiles - x)); };
        int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)tiles);  // C(hi) = 0
        while (lo + 1 < hi) {
            const int mid = (lo + hi) >> 1;
            if (above(mid) > order) lo = mid;
            else hi = mid;
        }
        index = lo;
        const int rank = order - above(index + 1);  // among the sequences that have such a tile
        const uint32_t have = __ballot_sync(0xffffffffu, tiles > index);
        const uint32_t at = __ballot_sync(0xffffffffu, tiles > index && __popc(have & ((1u << lane) - 1u)) == rank);
        if (!at) return LatentTile{0, 0, 0, 0, 0, 0};
        from = __ffs(at) - 1;
    } else {
        const int tile = count - 1 - order;
        // the last sequence whose first tile is not after `tile` is in [n, n + step)
        int step = (p.num_seqs + 31) / 32;
        from = 31 - __clz(__ballot_sync(0xffffffffu, l.first <= tile) | 1u);
        int n = from * step, left = min(step, p.num_seqs - n), first = 0;
        while (left > 1 || step > 1) {
            step = (left + 31) / 32;
            const int at = n + lane * step;
            bool before = false;
            if (lane * step < left) {
                latent_range(p.cu_q, at, (int)p.q_tokens, q0, q1);
                if (step == 1) latent_range(p.cu_k, at, (int)p.k_tokens, k0, k1);
                first = q0 / m + at;
                before = first <= tile;
            }
            from = 31 - __clz(__ballot_sync(0xffffffffu, before) | 1u);
            n += from * step;
            left = min(step, left - from * step);
        }
        index = max(0, tile - __shfl_sync(0xffffffffu, first, from));
    }
    q0 = __shfl_sync(0xffffffffu, q0, from);
    q1 = __shfl_sync(0xffffffffu, q1, from);
    k0 = __shfl_sync(0xffffffffu, k0, from);
    k1 = __shfl_sync(0xffffffffu, k1, from);
    LatentTile t;
    t.q0 = q0 + index * m;
    t.k0 = k0;
    t.klen = k1 - k0;
    t.rows = max(0, min(m, q1 - t.q0));
    t.off = (t.q0 - q0) + t.klen - (q1 - q0);
    t.keys = p.causal ? max(0, min(t.klen, t.off + t.rows)) : t.klen;
    return t;
}

// Reports a cu array that is not a prefix sum ending at `total`: the lanes of one warp call it.
__device__ __forceinline__ void latent_check_cu(const int32_t *cu, int num_seqs, int64_t total, uint32_t *errors)
{
    if (!cu || !errors) return;
    bool bad = cu[0] != 0 || cu[num_seqs] != total;
    for (int n = threadIdx.x & 31; n < num_seqs; n += 32) bad |= cu[n + 1] < cu[n];
    if (bad) atomicOr(errors, DEV_ERR_SEQLENS);
}

// ---------------------------------------------------------------- absorbed decode: the walk
// A sequence's length, held to what its page table can hold; `bad` when that changed it.
__device__ __forceinline__ int latent_len(const int32_t *lens, int b, int64_t capacity, bool &bad)
{
    const int64_t n = lens[b];
    if (n >= 0 && n <= capacity) return (int)n;
    bad = true;
    return n < 0 ? 0 : (int)capacity;
}

// a / b for non-negative a and positive b; in 32 bits where both fit (a 64-bit division costs some 300
// cycles, and these stand before the first copy).
__device__ __forceinline__ int64_t latent_div(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// Position of a CTA in the tile list.  W = base G' + rem: CTA c starts at floor(c W / G'), so that with two
// head groups CTA c and CTA c + G' / 2 read the same cache rows at the same time.
struct LatentWalk {
    int64_t g, g_end;   // tile list range of this CTA
    int64_t base;
    int rem;
    int cta, ctas;      // c, G'
    int hg, b, tile;    // head group, sequence and tile of g
    int64_t total;      // W
    __device__ __forceinline__ int64_t start_of(int c) const { return c * base + (uint32_t)(c * rem) / (uint32_t)ctas; }
    __device__ __forceinline__ int cta_of(int64_t x) const { return (int)latent_div((x + 1) * ctas - 1, total); }
};

// Called by all NT threads of the CTA (contains barriers); s_scan: NT / 32 + 2 ints of shared memory.
// The CTAs also clear the outputs of the sequences without cache rows, and write the records that say
// that there is nothing to join.  The tiles of all sequences are below 2^31 (the entry point sees to it).
template <int NT, typename IO>
__device__ __forceinline__ LatentWalk latent_walk(const LatentDecode &p, int tile_rows, int head_tile, int *s_scan)
{
    const int tid = threadIdx.x, batch = p.batch, heads = p.heads, head_groups = (heads + head_tile - 1) / head_tile;
    const int64_t capacity = (int64_t)p.table_width * p.page_size;
    const int32_t *lens = p.lens;
    uint32_t *errors = p.errors;
    IO *o = static_cast<IO *>(p.o);
    float *lse = p.lse;
    LatentJoin *records = reinterpret_cast<LatentJoin *>(p.workspace);
    const bool by_unit = latent_join_by_unit(batch, heads, head_tile, gridDim.x);
    const int chunk = (batch + NT - 1) / NT;
    const int lo = min(tid * chunk, batch), hi = min(lo + chunk, batch);
    bool bad = false;
    int sum = 0;
    for (int b = lo; b < hi; ++b) sum += (latent_len(lens, b, capacity, bad) + tile_rows - 1) / tile_rows;
    if (bad && errors && blockIdx.x == 0) atomicOr(errors, DEV_ERR_SEQLENS);
    int inc = sum;  // inclusive scan: within the warp, then over the warps
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, m);
        if ((tid & 31) >= m) inc += up;
    }
    if ((tid & 31) == 31) s_scan[tid >> 5] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const int x = s_scan[w];
        before += w < (tid >> 5) ? x : 0;
        all += x;
    }
    const int first = before + inc - sum;  // tiles before this thread's sequences
    const int64_t total = (int64_t)all * head_groups;
    LatentWalk k;
    k.cta = blockIdx.x;
    k.ctas = (int)min((int64_t)gridDim.x, total);
    k.hg = k.b = k.tile = 0;
    k.g = k.g_end = k.base = k.rem = 0;
    k.total = total;
    if (k.cta < k.ctas) {
        k.base = latent_div(total, k.ctas);
        k.rem = (int)(total - k.base * k.ctas);
        k.g = k.start_of(k.cta);
        k.g_end = k.start_of(k.cta + 1);
        k.hg = (int)latent_div(k.g, all);
        int r = (int)(k.g - (int64_t)k.hg * all);
        if (r >= first && r < first + sum) {
            r -= first;
            bool ignore = false;
            int b = lo;
            for (; b < hi - 1; ++b) {
                const int n = (latent_len(lens, b, capacity, ignore) + tile_rows - 1) / tile_rows;
                if (r < n) break;
                r -= n;
            }
            s_scan[NT / 32] = b;
            s_scan[NT / 32 + 1] = r;
        }
    }
    __syncthreads();
    if (k.cta < k.ctas) {
        k.b = s_scan[NT / 32];
        k.tile = s_scan[NT / 32 + 1];
    }
    for (int b = blockIdx.x; b < batch; b += gridDim.x) {
        bool ignore = false;
        if (latent_len(lens, b, capacity, ignore) > 0) continue;
        for (int64_t e = tid; e < (int64_t)heads * kLatR; e += NT) store_io(o + (size_t)b * heads * kLatR + e, 0.f);
        if (lse)
            for (int h = tid; h < heads; h += NT) lse[(size_t)b * heads + h] = -INFINITY;
        if (by_unit)
            for (int g = tid; g < head_groups; g += NT) records[g * batch + b].b = -1;
    }
    if (!by_unit && tid == 0 && !(k.cta < k.ctas && k.tile > 0)) records[blockIdx.x].b = -1;
    return k;
}

// One thread, for each of this CTA's units: the record for the joining kernel, where it is this CTA's
// to write.  k: the walk at the unit (k.tile its first tile here), n: the unit's tiles, tiles: those of
// this CTA.
__device__ __forceinline__ void latent_record_join(const LatentDecode &p, const LatentWalk &k, int64_t g, int tile0, int n,
                                                   int tiles, bool first, int head_tile)
{
    const bool by_unit = latent_join_by_unit(p.batch, p.heads, head_tile, gridDim.x);
    LatentJoin *r = reinterpret_cast<LatentJoin *>(p.workspace);
    if (by_unit) {
        if (tile0 > 0) return;  // written by the CTA of the unit's first tile
        r += k.hg * p.batch + k.b;
    } else {
        if (!first || tile0 == 0) return;  // (latent_walk wrote that there is nothing)
        r += blockIdx.x;
    }
    const int64_t a = g - tile0;  // the unit's first tile in the list
    const int cf = by_unit ? k.cta : k.cta_of(a);
    LatentJoin j = {-1, 0, 0, 0, 0, {0, 0, 0}};
    if (by_unit ? tiles < n : cf == k.cta - 1) {
        j.b = k.b;
        j.h0 = k.hg * head_tile;
        j.c_first = cf;
        j.c_last = k.cta_of(a + n - 1);
        j.first_slot = k.start_of(cf) >= a ? 2 * cf : 2 * cf + 1;
    }
    *r = j;
}
#endif

}  // namespace kda
