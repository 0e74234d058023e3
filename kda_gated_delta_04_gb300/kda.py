"""Python binding of libkda (ctypes).  Argument marshalling only.

The raw functions ``kda_prefill``, ``kda_decode_step``,
``kda_prefill_workspace_size``, ``kda_read_device_status`` and
``kda_status_string`` are the C entry points of ``include/kda.h`` with the same
names and arguments (pointers as integers).  ``prefill`` and ``decode_step``
take torch CUDA tensors, allocate outputs with torch when none are given, and
call the same entry points.  Every step of the computation runs in libkda's
kernels; there is no fallback: if ``libkda.so`` is missing or the tensors are
not on a CUDA device, these functions raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, \
    KDA_ERR_DECAY_RANGE, KDA_ERR_VALUE_RANGE = range(7)
KDA_DTYPE_BF16, KDA_DTYPE_F32 = 0, 1
KDA_FLAG_SCALAR_GATE = 1
KDA_FLAG_QK_L2NORM = 2
KDA_FLAG_NO_SEQ_SPLIT = 4
KDA_FLAG_NO_STREAM = 8
KDA_FLAG_STREAM = 16
KDA_PATH_CUDA_CORE, KDA_PATH_FUSED, KDA_PATH_TWO_KERNEL, KDA_PATH_SEQ_SPLIT, KDA_PATH_SEGMENTED, \
    KDA_PATH_STREAMED = range(6)
CHUNK = 64
KDA_STREAM_RING_MIN = 8
KDA_LATENT_DIM, KDA_LATENT_PE_DIM, KDA_LATENT_HEAD_DIM = 512, 64, 128
KDA_LATENT_INTERLEAVED, KDA_LATENT_FULL = 1, 2
KDA_LATENT_DECODE_WORKSPACE_MAX = 50331648

_lib = None
_lock = threading.Lock()

_c = ctypes
_VP = _c.c_void_p
_PREFILL_ARGS = [_VP, _VP, _VP, _VP, _VP, _VP, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                 _c.c_int32, _c.c_int, _VP, _VP, _VP, _VP, _c.c_size_t, _VP]
_DECODE_ARGS = [_VP, _VP, _VP, _VP, _VP, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int,
                _VP, _VP, _VP]
EXPORTS = {
    "kda_prefill_workspace_size": (_c.c_size_t, [_c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                                 _c.c_int32, _c.c_int]),
    "kda_prefill_workspace_size_segmented": (_c.c_size_t, [_c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                                           _c.c_int32, _c.c_int, _c.c_int64]),
    "kda_prefill_workspace_size_streamed": (_c.c_size_t, [_c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                                          _c.c_int32, _c.c_int, _c.c_int64]),
    "kda_prefill_path": (_c.c_int32, [_c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int,
                                       _c.c_size_t, _c.c_uint32]),
    "kda_prefill": (_c.c_int, _PREFILL_ARGS),
    "kda_decode_step": (_c.c_int, _DECODE_ARGS),
    "kda_read_device_status": (_c.c_int, [_VP, _VP]),
    "kda_status_string": (_c.c_char_p, [_c.c_int]),
    "kda_prefill_no_alloc": (_c.c_int, _PREFILL_ARGS[:15] + [_VP, _VP]),
    "kda_prefill_events": (_c.c_int, _PREFILL_ARGS + [_c.POINTER(_VP), _c.c_int32]),
    "kda_prefill_events_ex": (_c.c_int, _PREFILL_ARGS + [_c.POINTER(_VP), _c.c_int32, _c.c_uint32]),
    "kda_selftest_bounded_wait": (_c.c_int, [_VP, _c.c_uint64, _VP]),
    "kda_prefill_ex": (_c.c_int, _PREFILL_ARGS + [_c.c_uint32]),
    "kda_diag_tensor_phases": (_c.c_int, [_c.c_int32, _c.c_int32, _VP, _VP, _c.POINTER(_c.c_double)]),
    "kda_prefill_host": (_c.c_int, _PREFILL_ARGS + [_c.c_uint32]),
    "kda_prefill_host_buffer_size": (_c.c_size_t, [_VP, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                                   _c.c_int32, _c.c_int]),
    "kda_prefill_host_segments": (_c.c_int32, [_VP, _c.c_int32, _c.c_int64, _VP, _c.c_int32]),
    "kda_decode_step_ex": (_c.c_int, _DECODE_ARGS + [_c.c_uint32]),
    "kda_decode_step_slots": (_c.c_int, [_VP, _VP, _VP, _VP, _VP, _c.c_int32, _c.c_int32, _c.c_int32,
                                         _c.c_int32, _c.c_int, _VP, _c.c_int32, _VP, _VP, _VP, _VP,
                                         _c.c_uint32]),
    "kda_latent_append": (_c.c_int, [_VP, _c.c_int64, _VP, _c.c_int64, _VP, _c.c_float, _VP, _c.c_int32, _VP,
                                     _VP, _c.c_int64, _c.c_int64, _VP, _c.c_int64, _c.c_int64, _VP, _c.c_int64,
                                     _VP, _c.c_int64, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int,
                                     _VP, _c.c_int64, _VP, _VP, _VP, _c.c_uint32]),
    "kda_latent_decode_workspace_size": (_c.c_size_t, [_c.c_int32, _c.c_int]),
    "kda_latent_decode": (_c.c_int, [_VP, _c.c_int64, _c.c_int64, _VP, _c.c_int64, _c.c_int32, _VP, _c.c_int64,
                                     _c.c_int32, _VP, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int,
                                     _c.c_float, _VP, _VP, _VP, _c.c_size_t, _VP, _VP]),
    "kda_latent_prefill": (_c.c_int, [_VP, _c.c_int64, _c.c_int64, _VP, _c.c_int64, _c.c_int64, _VP, _c.c_int64,
                                      _VP, _c.c_int64, _c.c_int64, _VP, _VP, _c.c_int32, _c.c_int64, _c.c_int64,
                                      _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int, _c.c_float, _VP,
                                      _VP, _VP, _VP, _c.c_uint32]),
    "kda_prefill_slots": (_c.c_int, _PREFILL_ARGS[:12] + [_VP, _c.c_int32, _VP, _VP, _VP, _VP,
                                                          _c.c_size_t, _VP, _c.c_uint32]),
}


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def lib():
    """The loaded libkda (ctypes.CDLL).  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libkda.so not found at {LIB_PATH}; build it with "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in EXPORTS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


# ------------------------------------------------------------------ raw C entry points
def kda_prefill_workspace_size(num_seqs, total_tokens, num_heads, d_k, d_v, dtype):
    return lib().kda_prefill_workspace_size(num_seqs, total_tokens, num_heads, d_k, d_v, dtype)


def kda_prefill_workspace_size_segmented(num_seqs, total_tokens, num_heads, d_k, d_v, dtype,
                                         segment_chunks):
    return lib().kda_prefill_workspace_size_segmented(num_seqs, total_tokens, num_heads, d_k, d_v,
                                                      dtype, segment_chunks)


def kda_prefill_workspace_size_streamed(num_seqs, total_tokens, num_heads, d_k, d_v, dtype, ring_chunks):
    return lib().kda_prefill_workspace_size_streamed(num_seqs, total_tokens, num_heads, d_k, d_v, dtype,
                                                     ring_chunks)


def kda_prefill_path(num_seqs, total_tokens, num_heads, d_k, d_v, dtype, workspace_bytes, flags=0):
    return lib().kda_prefill_path(num_seqs, total_tokens, num_heads, d_k, d_v, dtype, workspace_bytes, flags)


def kda_prefill(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads, d_k,
                d_v, dtype, init_state, o, final_state, workspace, workspace_bytes, stream):
    return lib().kda_prefill(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens,
                             num_heads, d_k, d_v, dtype, init_state, o, final_state, workspace,
                             workspace_bytes, stream)


def kda_prefill_ex(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads, d_k,
                   d_v, dtype, init_state, o, final_state, workspace, workspace_bytes, stream, flags):
    return lib().kda_prefill_ex(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens,
                                num_heads, d_k, d_v, dtype, init_state, o, final_state, workspace,
                                workspace_bytes, stream, flags)


def kda_decode_step_ex(q, k, v, log_alpha, beta, batch, num_heads, d_k, d_v, dtype, state, o, stream,
                       flags):
    return lib().kda_decode_step_ex(q, k, v, log_alpha, beta, batch, num_heads, d_k, d_v, dtype,
                                    state, o, stream, flags)


def kda_decode_step(q, k, v, log_alpha, beta, batch, num_heads, d_k, d_v, dtype, state, o, stream):
    return lib().kda_decode_step(q, k, v, log_alpha, beta, batch, num_heads, d_k, d_v, dtype,
                                 state, o, stream)


def kda_prefill_no_alloc(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads,
                         d_k, d_v, dtype, init_state, o, final_state, device_errors, stream):
    """kda_prefill with its workspace in a fixed array inside libkda, for callers that
    cannot allocate device memory at call time (see include/kda.h)."""
    return lib().kda_prefill_no_alloc(q, k, v, log_alpha, beta, cu_seqlens, num_seqs,
                                      total_tokens, num_heads, d_k, d_v, dtype, init_state, o,
                                      final_state, device_errors, stream)


def kda_prefill_events(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads,
                       d_k, d_v, dtype, init_state, o, final_state, workspace, workspace_bytes,
                       stream, events):
    """kda_prefill that also records four CUDA events (handles as ints) on `stream` around
    its stages: before the schedule kernel, after it, after the chunk-local kernel, after
    the last kernel (see include/kda.h)."""
    arr = (_VP * len(events))(*events)
    return lib().kda_prefill_events(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens,
                                    num_heads, d_k, d_v, dtype, init_state, o, final_state,
                                    workspace, workspace_bytes, stream, arr, len(events))


def kda_prefill_events_ex(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads,
                          d_k, d_v, dtype, init_state, o, final_state, workspace, workspace_bytes,
                          stream, events, flags):
    """kda_prefill_events with option flags (as kda_prefill_ex)."""
    arr = (_VP * len(events))(*events)
    return lib().kda_prefill_events_ex(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens,
                                       num_heads, d_k, d_v, dtype, init_state, o, final_state,
                                       workspace, workspace_bytes, stream, arr, len(events), flags)


def kda_decode_step_slots(q, k, v, log_alpha, beta, batch, num_heads, d_k, d_v, dtype, state_pool,
                          num_slots, slots, o, device_errors, stream, flags):
    return lib().kda_decode_step_slots(q, k, v, log_alpha, beta, batch, num_heads, d_k, d_v, dtype,
                                       state_pool, num_slots, slots, o, device_errors, stream, flags)


def kda_prefill_slots(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads, d_k,
                      d_v, dtype, state_pool, num_slots, init_slots, final_slots, o, workspace,
                      workspace_bytes, stream, flags):
    return lib().kda_prefill_slots(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens,
                                   num_heads, d_k, d_v, dtype, state_pool, num_slots, init_slots,
                                   final_slots, o, workspace, workspace_bytes, stream, flags)


def kda_prefill_host(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads, d_k, d_v,
                     dtype, init_state, o, final_state, device_buffer, device_bytes, stream, flags):
    return lib().kda_prefill_host(q, k, v, log_alpha, beta, cu_seqlens, num_seqs, total_tokens, num_heads,
                                  d_k, d_v, dtype, init_state, o, final_state, device_buffer, device_bytes,
                                  stream, flags)


def kda_prefill_host_buffer_size(cu_seqlens, num_seqs, total_tokens, num_heads, d_k, d_v, dtype):
    return lib().kda_prefill_host_buffer_size(cu_seqlens, num_seqs, total_tokens, num_heads, d_k, d_v, dtype)


def kda_prefill_host_segments(cu_seqlens, num_seqs, total_tokens, bounds, max_bounds):
    return lib().kda_prefill_host_segments(cu_seqlens, num_seqs, total_tokens, bounds, max_bounds)


def kda_latent_append(*args):
    """The C entry point; arguments as in include/kda.h."""
    return lib().kda_latent_append(*args)


def kda_latent_decode_workspace_size(num_heads, dtype):
    return lib().kda_latent_decode_workspace_size(num_heads, dtype)


def kda_latent_decode(*args):
    """The C entry point; arguments as in include/kda.h."""
    return lib().kda_latent_decode(*args)


def kda_latent_prefill(*args):
    """The C entry point; arguments as in include/kda.h."""
    return lib().kda_latent_prefill(*args)


def kda_diag_tensor_phases(pass_, reps, workspace, stream, tflops):
    return lib().kda_diag_tensor_phases(pass_, reps, workspace, stream, tflops)


def diag_tensor_phases(pass_, reps, workspace, stream=None):
    """Executed TFLOP/s of the chunk kernel's (pass_ = 0), the state kernel's (pass_ = 1) or
    the streamed kernel's walk (pass_ = 2) tensor-core product groups run on their own (see
    include/kda.h)."""
    out = _c.c_double(0.0)
    st = lib().kda_diag_tensor_phases(pass_, reps, _ptr(workspace, "workspace"),
                                      _stream_handle(stream, workspace.device), _c.byref(out))
    if st != KDA_OK:
        raise KdaError(st, "kda_diag_tensor_phases")
    return out.value


def kda_selftest_bounded_wait(workspace, limit_ns, stream):
    """Runs the device-side bounded-wait self-test (see include/kda.h)."""
    return lib().kda_selftest_bounded_wait(workspace, limit_ns, stream)


def kda_read_device_status(workspace, stream):
    return lib().kda_read_device_status(workspace, stream)


def status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


kda_status_string = status_string


# ------------------------------------------------------------------ torch convenience
def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError(f"q/k/v must be bf16 or fp32, got {t.dtype}")


def _ptr(t, name, dtype=None):
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _flags(log_alpha, qk_l2norm, seq_split=True, streamed=None):
    """Option bits: a log_alpha without a channel axis is the scalar gate; streamed None leaves
    the streamed form to the library, True asks for it (KDA_FLAG_STREAM), False rules it out
    (KDA_FLAG_NO_STREAM)."""
    return ((KDA_FLAG_SCALAR_GATE if log_alpha.dim() == 2 else 0) |
            (KDA_FLAG_QK_L2NORM if qk_l2norm else 0) | (0 if seq_split else KDA_FLAG_NO_SEQ_SPLIT) |
            (0 if streamed is None else (KDA_FLAG_STREAM if streamed else KDA_FLAG_NO_STREAM)))


def _stream_handle(stream, device):
    """The handle of the given stream, or of the current one; the entry points launch on the current
    device, so `device`, where the tensors are, has to be that."""
    torch = _torch()
    now = torch.cuda.current_device()
    if device.index not in (None, now):
        raise ValueError(f"the tensors are on {device}, but the current device is cuda:{now}")
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def workspace_for(num_seqs, total_tokens, num_heads, d, dtype_code, device):
    torch = _torch()
    nbytes = kda_prefill_workspace_size(num_seqs, total_tokens, num_heads, d, d, dtype_code)
    # every byte the kernels read is written first in the same call
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def segmented_workspace_for(num_seqs, total_tokens, num_heads, d, dtype_code, device, segment_chunks):
    """A workspace whose per-chunk records cover at most `segment_chunks` packed chunks: the
    two-kernel prefill then runs segment by segment (kda_prefill_workspace_size_segmented)."""
    torch = _torch()
    nbytes = kda_prefill_workspace_size_segmented(num_seqs, total_tokens, num_heads, d, d, dtype_code,
                                                  segment_chunks)
    if nbytes == 0:
        raise KdaError(KDA_ERR_UNSUPPORTED, "kda_prefill_workspace_size_segmented")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def streamed_workspace_for(num_seqs, total_tokens, num_heads, d, dtype_code, device, ring_chunks):
    """A workspace whose records cover a ring of `ring_chunks` packed chunks: where the call
    streams, the streamed prefill then reuses their slots (kda_prefill_workspace_size_streamed)."""
    torch = _torch()
    nbytes = kda_prefill_workspace_size_streamed(num_seqs, total_tokens, num_heads, d, d, dtype_code, ring_chunks)
    if nbytes == 0:
        raise KdaError(KDA_ERR_UNSUPPORTED, "kda_prefill_workspace_size_streamed")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def min_workspace_bytes(num_seqs):
    """KDA_PREFILL_MIN_WORKSPACE(num_seqs): the smallest workspace kda_prefill accepts
    (it then runs the single fused kernel for bf16, d = 128)."""
    return 256 + ((num_seqs * 4 + 1 + 255) // 256) * 256


def prefill(q, k, v, log_alpha, beta, cu_seqlens=None, init_state=None, *, o=None,
            final_state=None, workspace=None, stream=None, check_status=False, outputs=True,
            qk_l2norm=False, seq_split=True, streamed=None):
    """KDA prefill over packed sequences.  q, k: [T, H, d]; v: [T, H, d]; log_alpha: [T, H, d]
    fp32; beta: [T, H] fp32; cu_seqlens: int32 [N+1] CUDA tensor or None (one sequence);
    init_state: [N, H, d, d] fp32 or None.  Returns (o, final_state); with outputs=False
    only the final states are computed and o is None.  A log_alpha of shape [T, H] is the
    scalar-gate (Gated DeltaNet) variant: one decay per token-head for every key channel.
    qk_l2norm=True: q and k are raw and the kernels L2-normalise their rows.  seq_split=False
    keeps each sequence's state pass in one piece (KDA_FLAG_NO_SEQ_SPLIT).  streamed: None (the
    default) leaves it to the library whether the chunk work and the state walk share one launch
    (it does so where that is the faster form); True asks for that whenever the launch holds it
    (KDA_FLAG_STREAM); False runs the chunk kernel and the state pass one after the other
    (KDA_FLAG_NO_STREAM)."""
    torch = _torch()
    T, H, d = q.shape
    dt = _dtype_code(q)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if o is None and outputs:
        o = torch.empty((T, H, v.shape[2]), dtype=q.dtype, device=q.device)
    if not outputs:
        o = None
    if final_state is None:
        final_state = torch.empty((N, H, d, v.shape[2]), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(N, T, H, d, dt, q.device)
    flags = _flags(log_alpha, qk_l2norm, seq_split, streamed)
    st = kda_prefill_ex(_ptr(q, "q", q.dtype), _ptr(k, "k", q.dtype), _ptr(v, "v", q.dtype),
                     _ptr(log_alpha, "log_alpha", torch.float32), _ptr(beta, "beta", torch.float32),
                     _ptr(cu_seqlens, "cu_seqlens", torch.int32), N, T, H, d, v.shape[2], dt,
                     _ptr(init_state, "init_state", torch.float32),
                     None if o is None else _ptr(o, "o", q.dtype),
                     _ptr(final_state, "final_state", torch.float32), _ptr(workspace, "workspace"),
                     workspace.numel() * workspace.element_size(),
                     _stream_handle(stream, q.device), flags)
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill")
    if check_status:
        st = kda_read_device_status(workspace.data_ptr(), _stream_handle(stream, q.device))
        if st != KDA_OK:
            raise KdaError(st, "kda_prefill (device)")
    return o, final_state


def prefill_slots(q, k, v, log_alpha, beta, cu_seqlens, state_pool, final_slots, init_slots=None, *,
                  o=None, workspace=None, stream=None, check_status=False, outputs=True,
                  qk_l2norm=False, seq_split=True, streamed=None):
    """Prefill into a paged state cache: sequence n starts from state_pool[init_slots[n]]
    (zero when init_slots is None or the entry is -1) and its final state is written to
    state_pool[final_slots[n]].  state_pool [S, H, d, d] fp32; slots int32 CUDA tensors [N].
    Other arguments as prefill.  Returns o (None with outputs=False)."""
    torch = _torch()
    T, H, d = q.shape
    dt = _dtype_code(q)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if o is None and outputs:
        o = torch.empty((T, H, v.shape[2]), dtype=q.dtype, device=q.device)
    if not outputs:
        o = None
    if workspace is None:
        workspace = workspace_for(N, T, H, d, dt, q.device)
    flags = _flags(log_alpha, qk_l2norm, seq_split, streamed)
    st = kda_prefill_slots(_ptr(q, "q", q.dtype), _ptr(k, "k", q.dtype), _ptr(v, "v", q.dtype),
                           _ptr(log_alpha, "log_alpha", torch.float32),
                           _ptr(beta, "beta", torch.float32),
                           _ptr(cu_seqlens, "cu_seqlens", torch.int32), N, T, H, d, v.shape[2], dt,
                           _ptr(state_pool, "state_pool", torch.float32), state_pool.shape[0],
                           _ptr(init_slots, "init_slots", torch.int32),
                           _ptr(final_slots, "final_slots", torch.int32),
                           None if o is None else _ptr(o, "o", q.dtype), _ptr(workspace, "workspace"),
                           workspace.numel() * workspace.element_size(),
                           _stream_handle(stream, q.device), flags)
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_slots")
    if check_status:
        st = kda_read_device_status(workspace.data_ptr(), _stream_handle(stream, q.device))
        if st != KDA_OK:
            raise KdaError(st, "kda_prefill_slots (device)")
    return o


def _hptr(t, name, dtype=None):
    """Address of a contiguous CPU tensor (None passes through)."""
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f"{name} must be a CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def prefill_host(q, k, v, log_alpha, beta, cu_seqlens=None, init_state=None, *, o=None, final_state=None,
                 device_buffer=None, device=None, stream=None, outputs=True, qk_l2norm=False, seq_split=True,
                 streamed=None):
    """kda_prefill_host: q, k, v, log_alpha, beta, cu_seqlens (int32), init_state and the outputs
    in host memory (pin them for the copies to overlap with the prefill).  Returns (o, final_state)
    as host tensors, valid once `stream` has been synchronised."""
    torch = _torch()
    T, H, d = q.shape
    dt = _dtype_code(q)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    device = device or torch.device("cuda", torch.cuda.current_device())
    if o is None and outputs:
        o = torch.empty((T, H, v.shape[2]), dtype=q.dtype).pin_memory()
    if not outputs:
        o = None
    if final_state is None:
        final_state = torch.empty((N, H, d, v.shape[2]), dtype=torch.float32).pin_memory()
    cu = _hptr(cu_seqlens, "cu_seqlens", torch.int32)
    if device_buffer is None:
        nbytes = kda_prefill_host_buffer_size(cu, N, T, H, d, v.shape[2], dt)
        if nbytes == 0:
            raise KdaError(KDA_ERR_INVALID_ARG, "kda_prefill_host_buffer_size")
        device_buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
    st = kda_prefill_host(_hptr(q, "q", q.dtype), _hptr(k, "k", q.dtype), _hptr(v, "v", q.dtype),
                          _hptr(log_alpha, "log_alpha", torch.float32), _hptr(beta, "beta", torch.float32),
                          cu, N, T, H, d, v.shape[2], dt, _hptr(init_state, "init_state", torch.float32),
                          _hptr(o, "o", q.dtype), _hptr(final_state, "final_state", torch.float32),
                          _ptr(device_buffer, "device_buffer"),
                          device_buffer.numel() * device_buffer.element_size(),
                          _stream_handle(stream, device_buffer.device),
                          _flags(log_alpha, qk_l2norm, seq_split, streamed))
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_host")
    return o, final_state


def decode_step_slots(q, k, v, log_alpha, beta, state_pool, slots, *, o=None, errors=None,
                      stream=None, qk_l2norm=False):
    """One decode step on a paged state cache: state_pool [S, H, d, d] fp32 (updated in
    place), slots int32 [B] CUDA tensor of distinct slot indices.  Returns o [B, H, d].
    A log_alpha of shape [B, H] is the scalar-gate variant."""
    torch = _torch()
    B, H, d = q.shape
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty((B, H, v.shape[2]), dtype=q.dtype, device=q.device)
    flags = _flags(log_alpha, qk_l2norm)
    st = kda_decode_step_slots(_ptr(q, "q", q.dtype), _ptr(k, "k", q.dtype), _ptr(v, "v", q.dtype),
                               _ptr(log_alpha, "log_alpha", torch.float32),
                               _ptr(beta, "beta", torch.float32), B, H, d, v.shape[2], dt,
                               _ptr(state_pool, "state_pool", torch.float32), state_pool.shape[0],
                               _ptr(slots, "slots", torch.int32), _ptr(o, "o", q.dtype),
                               None if errors is None else _ptr(errors, "errors", torch.int32),
                               _stream_handle(stream, q.device), flags)
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step_slots")
    return o


def decode_step(q, k, v, log_alpha, beta, state, *, o=None, stream=None, qk_l2norm=False):
    """One decode step; state [B, H, d, d] fp32 is updated in place.  Returns o [B, H, d].
    A log_alpha of shape [B, H] is the scalar-gate variant."""
    torch = _torch()
    B, H, d = q.shape
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty((B, H, v.shape[2]), dtype=q.dtype, device=q.device)
    flags = _flags(log_alpha, qk_l2norm)
    st = kda_decode_step_ex(_ptr(q, "q", q.dtype), _ptr(k, "k", q.dtype), _ptr(v, "v", q.dtype),
                            _ptr(log_alpha, "log_alpha", torch.float32),
                            _ptr(beta, "beta", torch.float32), B, H, d, v.shape[2], dt,
                            _ptr(state, "state", torch.float32), _ptr(o, "o", q.dtype),
                            _stream_handle(stream, q.device), flags)
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step")
    return o


# ------------------------------------------------------------------ latent attention
# These calls are made once per layer and generated token, where the host's time counts: a tensor
# that is as it should be is checked with a handful of comparisons, and only one that is not is
# looked at again for the message.
# Where latent_args.cpp has been built (against the torch that runs), a call whose every argument is as
# it should be goes through it; the checks here are then for naming what is not.
_torch_module = None
_native = None


def _load_torch():
    """torch, and the native argument passing when it fits."""
    global _torch_module, _native
    torch = _torch()
    path = os.path.join(PKG, "_latent_args.so")
    if os.path.exists(path) and torch.cuda.is_available():
        import importlib.machinery
        import importlib.util
        lib()
        loader = importlib.machinery.ExtensionFileLoader("_latent_args", path)
        try:
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_latent_args", loader))
        except ImportError:  # built against another torch
            module = None
        if module is not None and module.torch_version == torch.__version__.split("+")[0]:
            _native = module
    _torch_module = torch
    return torch


def _refuse(t, name, dtype, dev, shape):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous{' in its last dimension' if t.stride(-1) != 1 else ''}")


def _rows3(t, name, dtype, dev, shape):
    """Address and leading strides (0 where there is one entry only) of a CUDA tensor of three
    dimensions whose last one is contiguous."""
    try:
        a, b, c = t.stride()
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and c == 1:
            return t.data_ptr(), a if shape[0] > 1 else 0, b if shape[1] > 1 else 0
    except (AttributeError, ValueError):
        pass
    _refuse(t, name, dtype, dev, shape)


def _rows2(t, name, dtype, dev, shape):
    """The same of two dimensions."""
    try:
        a, c = t.stride()
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and (c == 1 or shape[1] <= 1):
            return t.data_ptr(), a if shape[0] > 1 else 0
    except (AttributeError, ValueError):
        pass
    _refuse(t, name, dtype, dev, shape)


def _flat(t, name, dtype, dev, shape):
    """Address of a contiguous CUDA tensor."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, dev, shape)


def _latent_like(t, name, dims):
    """Type code, type and device index that every other tensor of the call shares with t: the current
    device, on which the entry points launch."""
    torch = _torch_module or _load_torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    dt, dev = t.dtype, t.get_device()
    now = torch._C._cuda_getDevice()  # torch.cuda.current_device()
    if dev != now:
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{now}")
    return KDA_DTYPE_BF16 if dt is torch.bfloat16 else _dtype_code(t), dt, dev


def _raw_stream(stream, dev):
    if stream is not None:
        return stream.cuda_stream
    return _torch_module._C._cuda_getCurrentRawStream(dev)  # torch.cuda.current_stream(dev).cuda_stream


def _empty(shape, dtype, dev, stream):
    """torch.empty, owned by the stream that will use it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def latent_append(latent, k_pe, cache, slots, *, norm_weight=None, norm_eps=1e-6, cos_sin=None, positions=None,
                  interleaved=False, q_pe=None, q_pe_out=None, latent_out=None, k_pe_out=None, errors=None,
                  stream=None):
    """The tokens' rows into the latent cache: latent [T, 512] normalised (RMSNorm with norm_weight
    [512]; stored as it is when that is None), k_pe [T, 64] rotated by cos_sin[positions] (cos_sin
    [M, 64] fp32: 32 cosines, 32 sines; positions int32 [T]; None: no rotation), to row slots[t] of
    cache [pages, page_size, 576] (slots int32 [T], distinct; -1: not cached).  q_pe [T, H, 64], the
    queries' position channels, is rotated in the same launch into q_pe_out (None: in place).
    latent_out [T, 512] and k_pe_out [T, 64] receive the normalised latent and the rotated key
    again.  Rows may be strided; all are bf16 or all fp32.  interleaved: the rotated pairs are
    (2i, 2i + 1) instead of (i, i + 32).  errors: int32 [1] that collects KDA_DEVICE_ERR_* bits.
    The tensors are on the current device (this holds for every latent call)."""
    torch = _torch_module or _load_torch()
    if _native is not None:
        st = _native.append(latent, k_pe, cache, slots, norm_weight, norm_eps, cos_sin, positions, interleaved, q_pe,
                            q_pe_out, latent_out, k_pe_out, errors, None if stream is None else stream.cuda_stream)
        if st == KDA_OK:
            return
        if st > 0:
            raise KdaError(st, "kda_latent_append")
    if (cos_sin is None) != (positions is None):
        raise ValueError("cos_sin and positions go together")
    if q_pe is None and q_pe_out is not None:
        raise ValueError("q_pe_out without q_pe")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    code, dt, dev = _latent_like(latent, "latent", 2)
    i32 = torch.int32
    T = latent.shape[0]
    x, xs = _rows2(latent, "latent", dt, dev, (T, 512))
    k, ks = _rows2(k_pe, "k_pe", dt, dev, (T, 64))
    H = qt = qh = ot = oh = lo_s = ko_s = num_positions = 0
    q = qo = lo = ko = cs = pos = None
    if q_pe is not None:
        H = q_pe.shape[1] if q_pe.dim() == 3 else -1
        q, qt, qh = _rows3(q_pe, "q_pe", dt, dev, (T, H, 64))
        qo, ot, oh = (q, qt, qh) if q_pe_out is None else _rows3(q_pe_out, "q_pe_out", dt, dev, (T, H, 64))
    if latent_out is not None:
        lo, lo_s = _rows2(latent_out, "latent_out", dt, dev, (T, 512))
    if k_pe_out is not None:
        ko, ko_s = _rows2(k_pe_out, "k_pe_out", dt, dev, (T, 64))
    if cos_sin is not None:
        num_positions = cos_sin.shape[0]
        cs = _flat(cos_sin, "cos_sin", torch.float32, dev, (num_positions, 64))
        pos = _flat(positions, "positions", i32, dev, (T,))
    pages, page = cache.shape[:2] if cache.dim() == 3 else (-1, -1)
    st = (_lib or lib()).kda_latent_append(
        x, xs, k, ks, None if norm_weight is None else _flat(norm_weight, "norm_weight", dt, dev, (512,)), norm_eps,
        cs, num_positions, pos, q, qt, qh, qo, ot, oh, lo, lo_s, ko, ko_s, T, H, 512, 64, code,
        _flat(cache, "cache", dt, dev, (pages, page, 576)), pages * page, _flat(slots, "slots", i32, dev, (T,)),
        None if errors is None else _flat(errors, "errors", i32, dev, (1,)), _raw_stream(stream, dev),
        KDA_LATENT_INTERLEAVED if interleaved else 0)
    if st != KDA_OK:
        raise KdaError(st, "kda_latent_append")


def latent_decode_workspace_for(num_heads, dtype_code, device):
    """The scratch buffer of latent_decode, for any batch and lengths."""
    torch = _torch()
    return torch.empty(kda_latent_decode_workspace_size(num_heads, dtype_code), dtype=torch.uint8, device=device)


def latent_decode(q, cache, page_table, seq_lens, scale, *, o=None, lse=None, workspace=None, errors=None,
                  stream=None):
    """Absorbed latent attention, one token per sequence over the paged cache: q [B, H, 576]
    (batch and head dimensions may be strided), cache [pages, page_size, 576], page_table int32
    [B, W] (rows may be strided), seq_lens int32 [B] on the device.  Returns (o [B, H, 512],
    lse [B, H] fp32); a sequence of length 0 gives zeros and -inf.  bf16 or fp32.  The scratch
    buffer (latent_decode_workspace_for) may be kept by the caller; errors as latent_append."""
    torch = _torch_module or _load_torch()
    if o is None or lse is None or workspace is None:
        code, dt, dev = _latent_like(q, "q", 3)
        B, H = q.shape[:2]
        o = _empty((B, H, 512), dt, dev, stream) if o is None else o
        lse = _empty((B, H), torch.float32, dev, stream) if lse is None else lse
        if workspace is None:
            workspace = _empty((kda_latent_decode_workspace_size(H, code),), torch.uint8, dev, stream)
    if _native is not None:
        st = _native.decode(q, cache, page_table, seq_lens, scale, o, lse, workspace, errors,
                            None if stream is None else stream.cuda_stream)
        if st == KDA_OK:
            return o, lse
        if st > 0:
            raise KdaError(st, "kda_latent_decode")
    code, dt, dev = _latent_like(q, "q", 3)
    i32, f32 = torch.int32, torch.float32
    B, H = q.shape[:2]
    qp, qb, qh = _rows3(q, "q", dt, dev, (B, H, 576))
    pages, page = cache.shape[:2] if cache.dim() == 3 else (-1, -1)
    width = page_table.shape[-1]
    table, ts = _rows2(page_table, "page_table", i32, dev, (B, width))
    st = (_lib or lib()).kda_latent_decode(
        qp, qb, qh, _flat(cache, "cache", dt, dev, (pages, page, 576)), pages, page, table, ts, width,
        _flat(seq_lens, "seq_lens", i32, dev, (B,)), B, H, 512, 64, code, scale, _flat(o, "o", dt, dev, (B, H, 512)),
        _flat(lse, "lse", f32, dev, (B, H)), _flat(workspace, "workspace", workspace.dtype, dev, workspace.shape),
        workspace.nbytes, None if errors is None else _flat(errors, "errors", i32, dev, (1,)), _raw_stream(stream, dev))
    if st != KDA_OK:
        raise KdaError(st, "kda_latent_decode")
    return o, lse


def latent_prefill(q, k_nope, k_pe, v, scale, cu_q=None, cu_k=None, *, causal=True, o=None, lse=None, errors=None,
                   stream=None):
    """Expanded latent attention over packed sequences: q [Tq, H, 192], k_nope [Tk, H, 128], k_pe
    [Tk, 64] (shared by the heads), v [Tk, H, 128], all but the last dimension strided as they
    come; cu_q, cu_k int32 [N + 1] CUDA offsets (cu_k None: cu_q; both None: one sequence).
    Causal, aligned at each sequence's end: with lk > lq keys the queries are the last lq
    positions.  causal=False: every query sees all keys of its sequence.  Returns (o [Tq, H, 128],
    lse [Tq, H] fp32); a query without keys gives zeros and -inf.  errors as latent_append."""
    torch = _torch_module or _load_torch()
    if cu_q is None and cu_k is not None:
        raise ValueError("cu_k without cu_q")
    if o is None or lse is None:
        _, dt, dev = _latent_like(q, "q", 3)
        o = _empty((*q.shape[:2], 128), dt, dev, stream) if o is None else o
        lse = _empty(tuple(q.shape[:2]), torch.float32, dev, stream) if lse is None else lse
    if _native is not None:
        st = _native.prefill(q, k_nope, k_pe, v, scale, cu_q, cu_k, causal, o, lse, errors,
                             None if stream is None else stream.cuda_stream)
        if st == KDA_OK:
            return o, lse
        if st > 0:
            raise KdaError(st, "kda_latent_prefill")
    code, dt, dev = _latent_like(q, "q", 3)
    i32, f32 = torch.int32, torch.float32
    Tq, H = q.shape[:2]
    Tk = k_pe.shape[0]
    N = 1 if cu_q is None else cu_q.shape[0] - 1
    qp, qt, qh = _rows3(q, "q", dt, dev, (Tq, H, 192))
    kn, kt, kh = _rows3(k_nope, "k_nope", dt, dev, (Tk, H, 128))
    kp, kps = _rows2(k_pe, "k_pe", dt, dev, (Tk, 64))
    vp, vt, vh = _rows3(v, "v", dt, dev, (Tk, H, 128))
    st = (_lib or lib()).kda_latent_prefill(
        qp, qt, qh, kn, kt, kh, kp, kps, vp, vt, vh,
        None if cu_q is None else _flat(cu_q, "cu_q", i32, dev, (N + 1,)),
        None if cu_k is None else _flat(cu_k, "cu_k", i32, dev, (N + 1,)), N, Tq, Tk, H, 128, 64, 128, code, scale,
        _flat(o, "o", dt, dev, (Tq, H, 128)), _flat(lse, "lse", f32, dev, (Tq, H)),
        None if errors is None else _flat(errors, "errors", i32, dev, (1,)), _raw_stream(stream, dev),
        0 if causal else KDA_LATENT_FULL)
    if st != KDA_OK:
        raise KdaError(st, "kda_latent_prefill")
    return o, lse
