// latent_api.cu -- the extern "C" entry points of latent attention: argument validation and
// launches.  No compute happens here.
#include <math.h>

#include "latent.cuh"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A stride in elements: not negative and a whole number of 16-byte pieces.
bool stride_ok(int64_t s, size_t es) { return s >= 0 && s <= (int64_t)1 << 38 && (size_t)s * es % 16 == 0; }

// Whether no two of the rows of `width` elements at i s0 + j s1 (i < n0, j < n1) share an element, as far as
// nested strides show it: one dimension's whole extent lies within a step of the other's.
bool rows_apart(int64_t s0, int64_t n0, int64_t s1, int64_t n1, int64_t width)
{
    if (n0 <= 1) return n1 <= 1 || s1 >= width;
    if (n1 <= 1) return s0 >= width;
    const bool first = s0 <= s1;
    const int64_t inner = first ? s0 : s1, outer = first ? s1 : s0, steps = (first ? n0 : n1) - 1;
    return inner >= width && (outer - width) / steps >= inner;
}

// Packed tokens are counted in int32, rounded up to tiles.
constexpr int64_t kMaxTokens = INT32_MAX - 4096;

size_t elem_size(kda_dtype_t dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

bool dtype_ok(kda_dtype_t dtype) { return dtype == KDA_DTYPE_BF16 || dtype == KDA_DTYPE_F32; }

size_t workspace_bytes_of(int32_t heads, kda_dtype_t dtype)
{
    return dtype == KDA_DTYPE_BF16 ? kda::latent_decode_tc_ws_bytes(heads) : kda::latent_decode_simt_ws_bytes();
}

}  // namespace

extern "C" {

kda_status_t kda_latent_append(const void *latent, int64_t latent_stride, const void *k_pe, int64_t k_pe_stride,
                               const void *norm_weight, float norm_eps, const float *cos_sin,
                               int32_t num_positions, const int32_t *positions, const void *q_pe,
                               int64_t q_token_stride, int64_t q_head_stride, void *q_pe_out,
                               int64_t out_token_stride, int64_t out_head_stride, void *latent_out,
                               int64_t latent_out_stride, void *k_pe_out, int64_t k_pe_out_stride,
                               int32_t num_tokens, int32_t num_heads, int32_t d_latent, int32_t d_pe,
                               kda_dtype_t dtype, void *cache, int64_t num_slots, const int32_t *slots,
                               uint32_t *device_errors, void *stream, uint32_t flags)
{
    if (flags & ~KDA_LATENT_INTERLEAVED) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || d_latent <= 0 || d_pe <= 0) return KDA_ERR_INVALID_ARG;
    if (d_latent != KDA_LATENT_DIM || d_pe != KDA_LATENT_PE_DIM) return KDA_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_heads < 0 || num_slots < 0) return KDA_ERR_INVALID_ARG;
    if ((int64_t)num_tokens * (1 + (num_heads + 7) / 8) > INT32_MAX) return KDA_ERR_UNSUPPORTED;  // units of work
    if (num_tokens == 0) return KDA_OK;
    const size_t es = elem_size(dtype);
    if (!latent || !k_pe || !cache || !slots || !q_pe != !q_pe_out || (cos_sin && (!positions || num_positions <= 0)) ||
        (q_pe && num_heads == 0) || !(norm_eps >= 0.f))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(latent, 16) || !aligned(k_pe, 16) || !aligned(norm_weight, 16) || !aligned(cos_sin, 16) ||
        !aligned(positions, 4) || !aligned(q_pe, 16) || !aligned(q_pe_out, 16) || !aligned(latent_out, 16) ||
        !aligned(k_pe_out, 16) || !aligned(cache, 16) || !aligned(slots, 4) || !aligned(device_errors, 4))
        return KDA_ERR_INVALID_ARG;
    if (!stride_ok(latent_stride, es) || !stride_ok(k_pe_stride, es) ||
        (q_pe && (!stride_ok(q_token_stride, es) || !stride_ok(q_head_stride, es) ||
                  !stride_ok(out_token_stride, es) || !stride_ok(out_head_stride, es))) ||
        (latent_out && !stride_ok(latent_out_stride, es)) || (k_pe_out && !stride_ok(k_pe_out_stride, es)))
        return KDA_ERR_INVALID_ARG;
    // rows are written by different warps, and where an output is its input a row is read as often as it is
    // written: in shared rows the result would depend on the order
    if ((q_pe && !rows_apart(out_token_stride, num_tokens, out_head_stride, num_heads, d_pe)) ||
        (latent_out && !rows_apart(latent_out_stride, num_tokens, 0, 1, d_latent)) ||
        (k_pe_out && !rows_apart(k_pe_out_stride, num_tokens, 0, 1, d_pe)))
        return KDA_ERR_INVALID_ARG;
    const kda_status_t st = kda::check_device();
    if (st != KDA_OK) return st;
    kda::LatentAppend p;
    p.latent = latent; p.k_pe = k_pe; p.norm_weight = norm_weight; p.q_pe = q_pe;
    p.latent_stride = latent_stride; p.k_pe_stride = k_pe_stride;
    p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.qo_ts = out_token_stride; p.qo_hs = out_head_stride;
    p.lo_stride = latent_out_stride; p.ko_stride = k_pe_out_stride;
    p.eps = norm_eps; p.cos_sin = cos_sin; p.positions = positions; p.slots = slots;
    p.num_positions = num_positions; p.tokens = num_tokens; p.heads = num_heads;
    p.q_pe_out = q_pe_out; p.latent_out = latent_out; p.k_pe_out = k_pe_out; p.cache = cache;
    p.num_slots = num_slots; p.interleaved = (flags & KDA_LATENT_INTERLEAVED) != 0; p.dtype = dtype;
    p.errors = device_errors; p.stream = static_cast<cudaStream_t>(stream);
    return kda::launch_latent_append(p) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_latent_decode_workspace_size(int32_t num_heads, kda_dtype_t dtype)
{
    if (num_heads <= 0 || !dtype_ok(dtype)) return 0;
    return workspace_bytes_of(num_heads, dtype);
}

kda_status_t kda_latent_decode(const void *q, int64_t q_batch_stride, int64_t q_head_stride, const void *cache,
                               int64_t num_pages, int32_t page_size, const int32_t *page_table,
                               int64_t page_table_stride, int32_t max_pages, const int32_t *seq_lens,
                               int32_t batch, int32_t num_heads, int32_t d_latent, int32_t d_pe,
                               kda_dtype_t dtype, float scale, void *o, float *lse, void *workspace,
                               size_t workspace_bytes, uint32_t *device_errors, void *stream)
{
    if (!dtype_ok(dtype) || d_latent <= 0 || d_pe <= 0) return KDA_ERR_INVALID_ARG;
    if (d_latent != KDA_LATENT_DIM || d_pe != KDA_LATENT_PE_DIM) return KDA_ERR_UNSUPPORTED;
    if (batch < 0 || num_heads <= 0 || num_pages < 0 || page_size <= 0 || max_pages < 0 || page_table_stride < 0 ||
        !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    // a cache row's index is a TMA coordinate; the tiles of all sequences are counted in an int
    if (page_size % 8 != 0 || num_pages > INT32_MAX / page_size || num_heads > 65535 ||
        (int64_t)max_pages * page_size > INT32_MAX ||
        (int64_t)batch * (((int64_t)max_pages * page_size + 31) / 32) > INT32_MAX || batch > (1 << 24))
        return KDA_ERR_UNSUPPORTED;
    if (batch == 0) return KDA_OK;
    const size_t es = elem_size(dtype);
    if (!q || !seq_lens || !o || !workspace || (max_pages > 0 && (!page_table || (num_pages > 0 && !cache))))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256) || !aligned(device_errors, 4))
        return KDA_ERR_INVALID_ARG;
    if (!stride_ok(q_batch_stride, es) || !stride_ok(q_head_stride, es) || (num_heads > 1 && q_head_stride == 0))
        return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < workspace_bytes_of(num_heads, dtype)) return KDA_ERR_INVALID_ARG;
    const kda_status_t st = kda::check_device();
    if (st != KDA_OK) return st;
    kda::LatentDecode p;
    p.q = q; p.cache = cache; p.q_bs = q_batch_stride; p.q_hs = q_head_stride;
    p.num_pages = num_pages; p.table_stride = page_table_stride;
    p.page_size = page_size; p.table_width = max_pages; p.table = page_table; p.lens = seq_lens;
    p.batch = batch; p.heads = num_heads; p.scale_log2 = scale * kda::kLatLog2e;
    p.o = o; p.lse = lse; p.workspace = static_cast<char *>(workspace); p.dtype = dtype;
    p.errors = device_errors; p.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t err = dtype == KDA_DTYPE_BF16 ? kda::launch_latent_decode_tc(p) : kda::launch_latent_decode_simt(p);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_latent_prefill(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k_nope,
                                int64_t k_token_stride, int64_t k_head_stride, const void *k_pe,
                                int64_t k_pe_stride, const void *v, int64_t v_token_stride,
                                int64_t v_head_stride, const int32_t *cu_q, const int32_t *cu_k,
                                int32_t num_seqs, int64_t q_tokens, int64_t k_tokens, int32_t num_heads,
                                int32_t d_nope, int32_t d_pe, int32_t d_v, kda_dtype_t dtype, float scale,
                                void *o, float *lse, uint32_t *device_errors, void *stream, uint32_t flags)
{
    if (flags & ~KDA_LATENT_FULL) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || d_nope <= 0 || d_pe <= 0 || d_v <= 0) return KDA_ERR_INVALID_ARG;
    if (d_nope != KDA_LATENT_HEAD_DIM || d_v != KDA_LATENT_HEAD_DIM || d_pe != KDA_LATENT_PE_DIM)
        return KDA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || q_tokens < 0 || k_tokens < 0 || num_heads <= 0 || !isfinite(scale)) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 && (q_tokens != 0 || k_tokens != 0)) return KDA_ERR_INVALID_ARG;
    if (!cu_q && (cu_k || (num_seqs != 1 && num_seqs != 0))) return KDA_ERR_INVALID_ARG;
    if (cu_q && !cu_k && q_tokens != k_tokens) return KDA_ERR_INVALID_ARG;
    if (num_seqs > 65535 || num_heads > 65535 || q_tokens > kMaxTokens || k_tokens > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    if (q_tokens == 0) return KDA_OK;
    const size_t es = elem_size(dtype);
    if (!q || !o || (k_tokens > 0 && (!k_nope || !k_pe || !v))) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_nope, 16) || !aligned(k_pe, 16) || !aligned(v, 16) || !aligned(cu_q, 4) ||
        !aligned(cu_k, 4) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(device_errors, 4))
        return KDA_ERR_INVALID_ARG;
    if (!stride_ok(q_token_stride, es) || !stride_ok(q_head_stride, es) || !stride_ok(k_token_stride, es) ||
        !stride_ok(k_head_stride, es) || !stride_ok(k_pe_stride, es) || !stride_ok(v_token_stride, es) ||
        !stride_ok(v_head_stride, es) || (q_tokens > 1 && q_token_stride == 0) ||
        (k_tokens > 1 && (k_token_stride == 0 || k_pe_stride == 0 || v_token_stride == 0)))
        return KDA_ERR_INVALID_ARG;
    const kda_status_t st = kda::check_device();
    if (st != KDA_OK) return st;
    kda::LatentPrefill p;
    p.q = q; p.k_nope = k_nope; p.k_pe = k_pe; p.v = v;
    p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.kn_ts = k_token_stride; p.kn_hs = k_head_stride;
    p.kp_ts = k_pe_stride; p.v_ts = v_token_stride; p.v_hs = v_head_stride;
    p.cu_q = cu_q; p.cu_k = cu_k ? cu_k : cu_q; p.num_seqs = num_seqs;
    p.q_tokens = q_tokens; p.k_tokens = k_tokens; p.heads = num_heads; p.scale_log2 = scale * kda::kLatLog2e;
    p.causal = !(flags & KDA_LATENT_FULL); p.o = o; p.lse = lse; p.dtype = dtype;
    p.errors = device_errors; p.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t err = dtype == KDA_DTYPE_BF16 ? kda::launch_latent_prefill_tc(p) : kda::launch_latent_prefill_simt(p);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
