"""Python binding of ``libhils.so`` (the C ABI declared in include/hils.h).

Argument marshalling only: every step of the HiLS forward pass runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhils.so")

BF16, FP32 = 0, 1
CHUNK = 64
STATUS_NAMES = {0: "HILS_OK", 1: "HILS_ERR_INVALID_ARGUMENT", 2: "HILS_ERR_UNSUPPORTED", 3: "HILS_ERR_CUDA",
                4: "HILS_ERR_WORKSPACE_TOO_SMALL", 5: "HILS_ERR_DEVICE_TIMEOUT", 6: "HILS_ERR_DEVICE_BOUNDS"}
EXPORTS = ("hils_landmark_summary", "hils_kprime_mma_bytes", "hils_select", "hils_prefill_workspace_bytes",
           "hils_attn_prefill",
           "hils_decode_workspace_bytes", "hils_attn_decode", "hils_attn_decode_fixed_scratch",
           "hils_landmark_summary_paged", "hils_attn_decode_paged", "hils_query_calibrate", "hils_attn_decode_qcal",
           "hils_attn_backward_workspace_bytes", "hils_attn_backward",
           "hils_kv_append_paged", "hils_kv_append_quant", "hils_quant_page_bytes", "hils_kv_read_quant",
           "hils_landmark_summary_append", "hils_landmark_summary_quant",
           "hils_decode_quant_workspace_bytes", "hils_attn_decode_quant",
           "hils_get_status", "hils_selftest_bounded_wait", "hils_strerror", "hils_kernel_launches")
DECODE_FIXED_SCRATCH_BYTES = 16 << 20


class HilsError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call} failed: {STATUS_NAMES.get(status, status)} ({strerror(status)})")
        self.status = status


class hils_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("chunk", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("seqlen", ctypes.c_int64), ("dtype", ctypes.c_int32), ("window", ctypes.c_int32)]


class hils_tokens(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("cu_tokens", ctypes.c_void_p), ("seqlens", ctypes.c_void_p)]


class hils_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class hils_rotary(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


_lib = None


def lib():
    """Load libhils.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m chunk_wise_sparse_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        D = ctypes.POINTER(hils_dims)
        L.hils_landmark_summary.argtypes = [D, P, P, I64, I64, P, P, P, P]
        L.hils_kprime_mma_bytes.argtypes = [D]
        L.hils_kprime_mma_bytes.restype = SZ
        L.hils_select.argtypes = [D, P, P, P, P, P, I64, P, P, P]
        L.hils_prefill_workspace_bytes.argtypes = [D]
        L.hils_prefill_workspace_bytes.restype = SZ
        L.hils_attn_prefill.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_decode_workspace_bytes.argtypes = [D]
        L.hils_decode_workspace_bytes.restype = SZ
        L.hils_attn_decode.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_attn_decode_fixed_scratch.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P]
        L.hils_landmark_summary_paged.argtypes = [D, P, P, I64, P, I64, I64, P, P, P, P]
        L.hils_attn_decode_paged.argtypes = [D, P, P, P, P, I64, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_query_calibrate.argtypes = [D, P, I64, P, P, ctypes.c_int32, P, P]
        L.hils_attn_decode_qcal.argtypes = [D, P, P, P, P, P, I64, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_attn_backward_workspace_bytes.argtypes = [D]
        L.hils_attn_backward_workspace_bytes.restype = SZ
        L.hils_attn_backward.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_kv_append_paged.argtypes = [D, P, P, P, P, P, P, P, P, P, I64, P]
        L.hils_kv_append_quant.argtypes = [D, P, P, P, P, P, P, P, P, P, I64, P]
        L.hils_quant_page_bytes.argtypes = [D]
        L.hils_quant_page_bytes.restype = SZ
        L.hils_kv_read_quant.argtypes = [D, P, P, P, P, I64, P, P, P]
        L.hils_landmark_summary_append.argtypes = [D, P, P, P, I64, P, P, P, P, P]
        L.hils_landmark_summary_quant.argtypes = [D, P, P, P, I64, P, P, P, P, P]
        L.hils_decode_quant_workspace_bytes.argtypes = [D]
        L.hils_decode_quant_workspace_bytes.restype = SZ
        L.hils_attn_decode_quant.argtypes = [D, P, P, P, P, P, I64, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_get_status.argtypes = [ctypes.POINTER(ctypes.c_int32), P]
        L.hils_selftest_bounded_wait.argtypes = [ctypes.c_int32, P]
        L.hils_strerror.argtypes = [ctypes.c_int]
        L.hils_strerror.restype = ctypes.c_char_p
        L.hils_kernel_launches.restype = ctypes.c_uint64
        for name in EXPORTS:
            getattr(L, name).restype = getattr(L, name).restype or ctypes.c_int
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().hils_strerror(int(status)).decode()


def _on_current_device(t):
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device} but the current device is cuda:{torch.cuda.current_device()}")


def _ptr(t):
    """Device address of a tensor argument (a raw int is passed as is).  Every
    buffer the library reads or writes is dense device memory of the current
    GPU in the layout its header states: a host tensor, one on another GPU or
    a strided view is refused here, before any call."""
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device} but the current device is cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"expected a contiguous tensor, got strides {t.stride()} for shape {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(call, rc):
    if rc != 0:
        raise HilsError(call, rc)


def make_dims(batch, heads_q, heads_kv, head_dim, seqlen, topk, dtype, chunk=CHUNK, window=0) -> hils_dims:
    """window: local window in tokens (0 = the own chunk alone; else a multiple
    of the chunk, at most 16 chunks)."""
    if isinstance(dtype, torch.dtype):
        dtype = BF16 if dtype == torch.bfloat16 else FP32 if dtype == torch.float32 else -1
    return hils_dims(batch, heads_q, heads_kv, head_dim, chunk, topk, seqlen, dtype, window)


def dims_for(q, k, topk, window=0) -> hils_dims:
    """Dims of a prefill from q [B,Hq,N,d] and k [B,Hkv,N,d]."""
    B, Hq, N, d = q.shape
    return make_dims(B, Hq, k.shape[1], d, N, topk, q.dtype, window=window)


# ---------------------------------------------------------------------------
# The C entry points, one Python function each (same names).

def hils_landmark_summary(dims, k, lq, chunk_begin, chunk_end, kprime, bprime, kprime_mma=None, stream=None):
    _check("hils_landmark_summary",
           lib().hils_landmark_summary(ctypes.byref(dims), _ptr(k), _ptr(lq), int(chunk_begin), int(chunk_end),
                                       _ptr(kprime), _ptr(bprime), _ptr(kprime_mma), _stream(stream)))


def hils_kprime_mma_bytes(dims) -> int:
    return int(lib().hils_kprime_mma_bytes(ctypes.byref(dims)))


def hils_select(dims, q, kprime, bprime, kprime_mma, row_pos, n_rows, ids, scores=None, stream=None):
    """row_pos None (n_rows 0): every position; else a device int64 tensor of
    n_rows query positions, ids / scores [B, Hq, n_rows, K]."""
    _check("hils_select", lib().hils_select(ctypes.byref(dims), _ptr(q), _ptr(kprime), _ptr(bprime),
                                            _ptr(kprime_mma), _ptr(row_pos), int(n_rows), _ptr(ids), _ptr(scores),
                                            _stream(stream)))


def hils_prefill_workspace_bytes(dims) -> int:
    return int(lib().hils_prefill_workspace_bytes(ctypes.byref(dims)))


def hils_attn_prefill(dims, q, k, v, kprime, bprime, kprime_mma, ids, scores, o, lse_own=None, workspace=None,
                      workspace_bytes=None, stream=None):
    """scores None: the chunk scores of the kept ids are recomputed from q and
    the summaries (kprime_mma for bf16, kprime and bprime for fp32)."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("hils_attn_prefill", lib().hils_attn_prefill(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(kprime),
                                                        _ptr(bprime), _ptr(kprime_mma), _ptr(ids), _ptr(scores),
                                                        _ptr(o), _ptr(lse_own), _ptr(workspace),
                                                        int(workspace_bytes), _stream(stream)))


def prefill_workspace(dims, device):
    """A device workspace for hils_attn_prefill (None when none is needed)."""
    n = hils_prefill_workspace_bytes(dims)
    return torch.empty((n,), dtype=torch.uint8, device=device) if n else None


def hils_decode_workspace_bytes(dims) -> int:
    return int(lib().hils_decode_workspace_bytes(ctypes.byref(dims)))


def hils_attn_decode(dims, q, k_cache, v_cache, kprime, bprime, kprime_mma, seqlens, o, ids_out, scores_out,
                     workspace, workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("hils_attn_decode",
           lib().hils_attn_decode(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kprime),
                                  _ptr(bprime), _ptr(kprime_mma), _ptr(seqlens), _ptr(o), _ptr(ids_out),
                                  _ptr(scores_out), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def hils_attn_decode_fixed_scratch(dims, q, k_cache, v_cache, kprime, bprime, kprime_mma, seqlens, o, ids_out,
                                   scores_out, stream=None):
    """hils_attn_decode without a workspace, for callers that cannot allocate
    device memory (a host engine that owns all device memory, or a decode loop
    that must not pay cudaMalloc's implicit synchronisation).  Scratch is the
    library's fixed 16 MiB device array; overlapping calls race on it."""
    _check("hils_attn_decode_fixed_scratch",
           lib().hils_attn_decode_fixed_scratch(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                                _ptr(kprime), _ptr(bprime), _ptr(kprime_mma), _ptr(seqlens),
                                                _ptr(o), _ptr(ids_out), _ptr(scores_out), _stream(stream)))


def hils_landmark_summary_paged(dims, k_pages, page_table, n_pages, lq, chunk_begin, chunk_end, kprime, bprime,
                                kprime_mma=None, stream=None):
    _check("hils_landmark_summary_paged",
           lib().hils_landmark_summary_paged(ctypes.byref(dims), _ptr(k_pages), _ptr(page_table), int(n_pages),
                                             _ptr(lq), int(chunk_begin), int(chunk_end), _ptr(kprime), _ptr(bprime),
                                             _ptr(kprime_mma), _stream(stream)))


def hils_attn_decode_paged(dims, q, k_pages, v_pages, page_table, n_pages, kprime, bprime, kprime_mma, seqlens, o,
                           ids_out, scores_out, workspace, workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check("hils_attn_decode_paged",
           lib().hils_attn_decode_paged(ctypes.byref(dims), _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                        int(n_pages), _ptr(kprime), _ptr(bprime), _ptr(kprime_mma), _ptr(seqlens),
                                        _ptr(o), _ptr(ids_out), _ptr(scores_out), _ptr(workspace), int(nbytes),
                                        _stream(stream)))


def hils_query_calibrate(dims, q, n_pos, w_down, w_up, rank, q_hat, stream=None):
    _check("hils_query_calibrate",
           lib().hils_query_calibrate(ctypes.byref(dims), _ptr(q), int(n_pos), _ptr(w_down), _ptr(w_up), int(rank),
                                      _ptr(q_hat), _stream(stream)))


def hils_attn_decode_qcal(dims, q, q_score, k_cache, v_cache, page_table, n_pages, kprime, bprime, kprime_mma,
                          seqlens, o, ids_out, scores_out, workspace, workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check("hils_attn_decode_qcal",
           lib().hils_attn_decode_qcal(ctypes.byref(dims), _ptr(q), _ptr(q_score), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(page_table), int(n_pages), _ptr(kprime), _ptr(bprime), _ptr(kprime_mma),
                                       _ptr(seqlens), _ptr(o), _ptr(ids_out), _ptr(scores_out), _ptr(workspace),
                                       int(nbytes), _stream(stream)))


def hils_attn_backward_workspace_bytes(dims) -> int:
    return int(lib().hils_attn_backward_workspace_bytes(ctypes.byref(dims)))


def hils_attn_backward(dims, q, q_score, k, v, lq, kprime, ids, scores, lse_own, o, d_o, dq, dq_score, dk, dv, dlq,
                       workspace, workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check("hils_attn_backward",
           lib().hils_attn_backward(ctypes.byref(dims), _ptr(q), _ptr(q_score), _ptr(k), _ptr(v), _ptr(lq),
                                    _ptr(kprime), _ptr(ids), _ptr(scores), _ptr(lse_own), _ptr(o), _ptr(d_o),
                                    _ptr(dq), _ptr(dq_score), _ptr(dk), _ptr(dv), _ptr(dlq), _ptr(workspace),
                                    int(nbytes), _stream(stream)))


# The serving calls below run once per layer and token: their arguments are marshalled with one device query per call
# and packed structs.

_PACK_TOKENS, _PACK_ROWS, _PACK_ROTARY = struct.Struct("@qPP"), struct.Struct("@Pqq"), struct.Struct("@Pqii")


def _device(t):
    """The index of the current device, on which t has to be."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _on_current_device(t)
    return dev


def _dense(t, dev):
    """Address of a dense tensor on device dev (None is passed on, a raw address as it is)."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != dev or not t.is_contiguous():
        return _ptr(t)
    return t.data_ptr()


def _rows(t, dev):
    """hils_rows of a tensor [T, heads, d] whose last dimension is dense (None is passed on)."""
    if t is None:
        return None
    if t.get_device() != dev:
        _on_current_device(t)
    st = t.stride()
    if len(st) != 3 or st[2] != 1:
        raise ValueError(f"expected rows [T, heads, d] with a dense last dimension, got shape {tuple(t.shape)} with "
                         f"strides {st}")
    return _PACK_ROWS.pack(t.data_ptr(), st[0], st[1])


def _tokens(seqlens, n_tokens, cu_tokens, dev):
    return _PACK_TOKENS.pack(n_tokens, _dense(cu_tokens, dev) or 0, _dense(seqlens, dev) or 0)


def _rotary(r, dev):
    if r is None:
        return None
    n_pos, rot = r.table.shape
    return _PACK_ROTARY.pack(_dense(r.table, dev), n_pos, rot, r.interleaved)


def _on_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def hils_kv_append_paged(dims, seqlens, n_tokens, cu_tokens, rotary, q, q_out, k, v, k_pages, v_pages, page_table,
                         n_pages, stream=None):
    """rotary: a Rotary or None; q, q_out, k, v: rows [T, heads, d] with any token and head stride."""
    dev = _device(k_pages)
    _check("hils_kv_append_paged",
           lib().hils_kv_append_paged(ctypes.byref(dims), _tokens(seqlens, n_tokens, cu_tokens, dev),
                                      _rotary(rotary, dev), _rows(q, dev), _rows(q_out, dev), _rows(k, dev),
                                      _rows(v, dev), _dense(k_pages, dev), _dense(v_pages, dev),
                                      _dense(page_table, dev), n_pages, _on_stream(stream, dev)))


def hils_kv_append_quant(dims, seqlens, n_tokens, cu_tokens, rotary, q, q_out, k, v, k_pages, v_pages, page_table,
                         n_pages, stream=None):
    dev = _device(k_pages)
    _check("hils_kv_append_quant",
           lib().hils_kv_append_quant(ctypes.byref(dims), _tokens(seqlens, n_tokens, cu_tokens, dev),
                                      _rotary(rotary, dev), _rows(q, dev), _rows(q_out, dev), _rows(k, dev),
                                      _rows(v, dev), _dense(k_pages, dev), _dense(v_pages, dev),
                                      _dense(page_table, dev), n_pages, _on_stream(stream, dev)))


def hils_quant_page_bytes(dims) -> int:
    return int(lib().hils_quant_page_bytes(ctypes.byref(dims)))


def hils_kv_read_quant(dims, seqlens, n_tokens, cu_tokens, k_pages, v_pages, page_table, n_pages, k, v, stream=None):
    dev = _device(page_table)
    _check("hils_kv_read_quant",
           lib().hils_kv_read_quant(ctypes.byref(dims), _tokens(seqlens, n_tokens, cu_tokens, dev),
                                    _dense(k_pages, dev), _dense(v_pages, dev), _dense(page_table, dev), n_pages,
                                    _rows(k, dev), _rows(v, dev), _on_stream(stream, dev)))


def hils_landmark_summary_append(dims, seqlens, n_tokens, cu_tokens, k_pages, page_table, n_pages, lq, kprime, bprime,
                                 kprime_mma=None, stream=None):
    dev = _device(k_pages)
    _check("hils_landmark_summary_append",
           lib().hils_landmark_summary_append(ctypes.byref(dims), _tokens(seqlens, n_tokens, cu_tokens, dev),
                                              _dense(k_pages, dev), _dense(page_table, dev), n_pages, _dense(lq, dev),
                                              _dense(kprime, dev), _dense(bprime, dev), _dense(kprime_mma, dev),
                                              _on_stream(stream, dev)))


def hils_landmark_summary_quant(dims, seqlens, n_tokens, cu_tokens, k_pages, page_table, n_pages, lq, kprime, bprime,
                                kprime_mma=None, stream=None):
    dev = _device(k_pages)
    _check("hils_landmark_summary_quant",
           lib().hils_landmark_summary_quant(ctypes.byref(dims), _tokens(seqlens, n_tokens, cu_tokens, dev),
                                             _dense(k_pages, dev), _dense(page_table, dev), n_pages, _dense(lq, dev),
                                             _dense(kprime, dev), _dense(bprime, dev), _dense(kprime_mma, dev),
                                             _on_stream(stream, dev)))


def hils_decode_quant_workspace_bytes(dims) -> int:
    return int(lib().hils_decode_quant_workspace_bytes(ctypes.byref(dims)))


def hils_attn_decode_quant(dims, q, q_score, k_pages, v_pages, page_table, n_pages, kprime, bprime, kprime_mma,
                           seqlens, o, ids_out, scores_out, workspace, workspace_bytes=None, stream=None):
    dev = _device(q)
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check("hils_attn_decode_quant",
           lib().hils_attn_decode_quant(ctypes.byref(dims), _dense(q, dev), _dense(q_score, dev), _dense(k_pages, dev),
                                        _dense(v_pages, dev), _dense(page_table, dev), n_pages, _dense(kprime, dev),
                                        _dense(bprime, dev), _dense(kprime_mma, dev), _dense(seqlens, dev),
                                        _dense(o, dev), _dense(ids_out, dev), _dense(scores_out, dev),
                                        _dense(workspace, dev), nbytes, _on_stream(stream, dev)))


def hils_get_status(stream=None) -> int:
    v = ctypes.c_int32(0)
    _check("hils_get_status", lib().hils_get_status(ctypes.byref(v), _stream(stream)))
    return int(v.value)


def hils_selftest_bounded_wait(limit_ms: int = 50, stream=None):
    _check("hils_selftest_bounded_wait", lib().hils_selftest_bounded_wait(int(limit_ms), _stream(stream)))


def hils_kernel_launches() -> int:
    return int(lib().hils_kernel_launches())


# ---------------------------------------------------------------------------
# Convenience layer: allocate outputs with torch and chain the calls.

class Summary:
    """Landmark summaries of one KV sequence set: fp32 k', b' and the bf16
    scoring operand (bf16 only)."""

    def __init__(self, dims, device):
        B, H, nc, d = dims.batch, dims.heads_kv, dims.seqlen // CHUNK, dims.head_dim
        self.kprime = torch.empty((B, H, nc, d), dtype=torch.float32, device=device)
        self.bprime = torch.empty((B, H, nc), dtype=torch.float32, device=device)
        self.kprime_mma = None
        if dims.dtype == BF16:
            n = hils_kprime_mma_bytes(dims)
            self.kprime_mma = torch.empty((n // 2,), dtype=torch.bfloat16, device=device)

    @classmethod
    def of(cls, kprime, bprime, kprime_mma=None):
        """The summaries in tensors that the caller holds: fp32 [B,Hkv,nc,d] and [B,Hkv,nc], and for bf16 the scoring
        operand [B,Hkv,nc,d+16] (or flat)."""
        self = cls.__new__(cls)
        self.kprime, self.bprime, self.kprime_mma = kprime, bprime, kprime_mma
        return self


def landmark_summary(k, lq, topk=1, chunk_begin=0, chunk_end=None, out: Summary | None = None, stream=None):
    B, H, N, d = k.shape
    dims = make_dims(B, H, H, d, N, topk, k.dtype)
    out = out or Summary(dims, k.device)
    chunk_end = N // CHUNK if chunk_end is None else chunk_end
    hils_landmark_summary(dims, k, lq, chunk_begin, chunk_end, out.kprime, out.bprime, out.kprime_mma, stream)
    return out


def select(q, summ: Summary, heads_kv, topk, stream=None, window=0, row_pos=None, with_scores=True):
    """ids (and scores, or None) of every position, or of the positions in
    row_pos (a device int64 tensor): [B, Hq, rows, K]."""
    B, Hq, N, d = q.shape
    dims = make_dims(B, Hq, heads_kv, d, N, topk, q.dtype, window=window)
    n_rows = N if row_pos is None else row_pos.numel()
    ids = torch.empty((B, Hq, n_rows, topk), dtype=torch.int32, device=q.device)
    scores = torch.empty((B, Hq, n_rows, topk), dtype=torch.float32, device=q.device) if with_scores else None
    hils_select(dims, q, summ.kprime, summ.bprime, summ.kprime_mma, row_pos, 0 if row_pos is None else n_rows, ids,
                scores, stream)
    return ids, scores


def prefill(q, k, v, lq, topk, stream=None, return_all=False, window=0, scores_buffer=True):
    """Full HiLS prefill: summary -> select -> sparse attention.  Returns O
    (and, with return_all, the summary, ids, scores and the local branch's
    log-sum-exp).  scores_buffer False: the selection writes no scores and
    the attention recomputes them."""
    dims = dims_for(q, k, topk, window)
    summ = landmark_summary(k, lq, topk, stream=stream)
    ids, scores = select(q, summ, k.shape[1], topk, stream, window, with_scores=scores_buffer)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    hils_attn_prefill(dims, q, k, v, summ.kprime, summ.bprime, summ.kprime_mma, ids, scores, o, lse,
                      prefill_workspace(dims, q.device), stream=stream)
    if return_all:
        return o, dict(summary=summ, ids=ids, scores=scores, lse_own=lse)
    return o


def query_calibrate(q, w_down, w_up, out=None, stream=None):
    """Q-Cal: q^ = q + W_up (W_down q) per query head, for q [B,Hq,N,d] (a
    prefill) or [B,Hq,d] (a decode step); w_down [Hq,r,d], w_up [Hq,d,r]."""
    n_pos = q.shape[2] if q.dim() == 4 else 1
    B, Hq, d = q.shape[0], q.shape[1], q.shape[-1]
    Hq_w, r, _ = w_down.shape
    dims = make_dims(B, Hq, Hq, d, CHUNK, 1, q.dtype)
    out = torch.empty_like(q) if out is None else out
    hils_query_calibrate(dims, q, n_pos, w_down, w_up, r, out, stream)
    return out


def prefill_qcal(q, k, v, lq, topk, w_down, w_up, stream=None, return_all=False, window=0):
    """HiLS prefill with Q-Cal: summary -> calibrate -> select on q^ ->
    sparse attention with q."""
    dims = dims_for(q, k, topk, window)
    summ = landmark_summary(k, lq, topk, stream=stream)
    q_hat = query_calibrate(q, w_down, w_up, stream=stream)
    ids, scores = select(q_hat, summ, k.shape[1], topk, stream, window)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    hils_attn_prefill(dims, q, k, v, summ.kprime, summ.bprime, summ.kprime_mma, ids, scores, o, lse,
                      prefill_workspace(dims, q.device), stream=stream)
    if return_all:
        return o, dict(summary=summ, ids=ids, scores=scores, lse_own=lse, q_hat=q_hat)
    return o


def decode_step_qcal(q, q_score, k_cache, v_cache, summ: Summary, seqlens, topk, workspace=None, stream=None,
                     window=0):
    """One decode step with a separate scoring query q_score [B,Hq,d]."""
    B, Hq, d = q.shape
    Hkv, cap = k_cache.shape[1], k_cache.shape[2]
    dims = make_dims(B, Hq, Hkv, d, cap, topk, q.dtype, window=window)
    if workspace is None:
        workspace = torch.empty((hils_decode_workspace_bytes(dims),), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    ids = torch.empty((B, Hq, topk), dtype=torch.int32, device=q.device)
    scores = torch.empty((B, Hq, topk), dtype=torch.float32, device=q.device)
    hils_attn_decode_qcal(dims, q, q_score, k_cache, v_cache, None, 0, summ.kprime, summ.bprime, summ.kprime_mma,
                          seqlens, o, ids, scores, workspace, stream=stream)
    return o, ids, scores


def backward(q, k, v, lq, aux, o, d_o, topk, q_score=None, window=0, stream=None):
    """Gradients (fp32) of a prefill made by prefill()/prefill_qcal() with
    return_all=True: returns dict(dq, dq_score (with q_score), dk, dv, dlq)."""
    dims = dims_for(q, k, topk, window)
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    f32 = dict(dtype=torch.float32, device=q.device)
    g = dict(dq=torch.empty((B, Hq, N, d), **f32), dk=torch.empty((B, Hkv, N, d), **f32),
             dv=torch.empty((B, Hkv, N, d), **f32), dlq=torch.empty((B, Hkv, N // CHUNK, d), **f32))
    g["dq_score"] = torch.empty((B, Hq, N, d), **f32) if q_score is not None else None
    ws = torch.empty((hils_attn_backward_workspace_bytes(dims),), dtype=torch.uint8, device=q.device)
    hils_attn_backward(dims, q, q_score, k, v, lq, aux["summary"].kprime, aux["ids"], aux["scores"], aux["lse_own"], o,
                       d_o, g["dq"], g["dq_score"], g["dk"], g["dv"], g["dlq"], ws, stream=stream)
    return g


def decode_step(q, k_cache, v_cache, summ: Summary, seqlens, topk, workspace=None, stream=None, window=0):
    """One decode step for q [B,Hq,d] against caches [B,Hkv,cap,d]."""
    B, Hq, d = q.shape
    Hkv, cap = k_cache.shape[1], k_cache.shape[2]
    dims = make_dims(B, Hq, Hkv, d, cap, topk, q.dtype, window=window)
    if workspace is None:
        workspace = torch.empty((hils_decode_workspace_bytes(dims),), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    ids = torch.empty((B, Hq, topk), dtype=torch.int32, device=q.device)
    scores = torch.empty((B, Hq, topk), dtype=torch.float32, device=q.device)
    hils_attn_decode(dims, q, k_cache, v_cache, summ.kprime, summ.bprime, summ.kprime_mma, seqlens, o, ids, scores,
                     workspace, stream=stream)
    return o, ids, scores


# ---------------------------------------------------------------------------
# Serving from a chunk-paged cache: pages in bf16 / fp32 [n_pages,Hkv,64,d], or in 4 bits as uint8
# [n_pages,Hkv,64*(d/2+d/8)]; page_table int32 [B,nc].  A ragged batch of new tokens is packed [T]; seqlens int32 [B]
# are the lengths after the append, cu_tokens int32 [B+1] the sequences' places in it (None: T/B tokens each).
#
# stream: the kernels run there, and so are the outputs that a call makes; its inputs must be ready on it.

class Rotary:
    """A rotary position table fp32 [n_pos, rot_dim] (cosines, then sines of rot_dim/2 angles) and the pairing of
    dims: the halves of the first rot_dim dims, or neighbours (interleaved)."""
    __slots__ = ("table", "interleaved")

    def __init__(self, table, interleaved=False):
        if table.dim() != 2 or table.dtype is not torch.float32:
            raise ValueError(f"rotary table: expected fp32 [n_pos, rot_dim], got {table.dtype} {tuple(table.shape)}")
        self.table, self.interleaved = table, int(bool(interleaved))


def rotary_table(n_pos, rot_dim, base=10000.0, device="cuda"):
    """Cosines and sines of pos * base^(-2i/rot_dim) for a Rotary, angles computed in fp64 (far positions lose their
    phase in fp32)."""
    freq = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _need(t, name, dtype, shape):
    """Refuse a tensor of another type or shape (None: any extent)."""
    if t.dtype is dtype and t.shape == shape:
        return
    if t.dtype != dtype or t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name}: expected {dtype} {tuple('any' if n is None else n for n in shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")


def _page_kind(k_pages, v_pages, dtype):
    """(4-bit?, n_pages, Hkv, d) of a pair of pools (v_pages None: keys alone)."""
    shape, kind = k_pages.shape, k_pages.dtype
    if v_pages is not None and (v_pages.shape != shape or v_pages.dtype is not kind):
        raise ValueError(f"key pages {kind} {tuple(shape)} and value pages {v_pages.dtype} {tuple(v_pages.shape)} differ")
    if kind is torch.uint8:
        if len(shape) != 3 or shape[2] not in (40 * CHUNK, 80 * CHUNK):
            raise ValueError(f"4-bit pages are [n_pages, Hkv, 64 * (d/2 + d/8)], got {tuple(shape)}")
        return True, shape[0], shape[1], shape[2] // 40
    if len(shape) != 4 or shape[2] != CHUNK or kind is not dtype:
        raise ValueError(f"expected {dtype} pages [n_pages, Hkv, 64, d] or 4-bit ones, got {kind} {tuple(shape)}")
    return False, shape[0], shape[1], shape[3]


def _batch(page_table, seqlens, cu_tokens):
    """(B, nc) of a ragged batch."""
    if page_table.dim() != 2:
        raise ValueError(f"page_table: expected [B, nc], got {tuple(page_table.shape)}")
    B, nc = shape = page_table.shape
    _need(page_table, "page_table", torch.int32, shape)
    _need(seqlens, "seqlens", torch.int32, (B,))
    if cu_tokens is not None:
        _need(cu_tokens, "cu_tokens", torch.int32, (B + 1,))
    return B, nc


@functools.lru_cache(maxsize=1024)
def _dims_of(B, Hq, Hkv, d, nc, topk, dtype, window):
    return make_dims(B, Hq, Hkv, d, nc * CHUNK, topk, dtype, window=window)


@functools.lru_cache(maxsize=1024)
def _decode_quant_bytes(B, Hq, Hkv, d, nc, topk, dtype, window):
    return hils_decode_quant_workspace_bytes(_dims_of(B, Hq, Hkv, d, nc, topk, dtype, window))


def _new(like, shape, dtype, stream):
    """A new tensor on the stream that the kernels will run on, so that the caching allocator gives its memory to no
    other stream's work before they end."""
    if stream is None:
        if like.dtype is dtype and like.shape == shape:
            return torch.empty_like(like, memory_format=torch.contiguous_format)
        return like.new_empty(shape, dtype=dtype)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def quant_pages(n_pages, heads_kv, head_dim, device="cuda"):
    """A pool of 4-bit pages (of keys, or of values)."""
    dims = make_dims(1, heads_kv, heads_kv, head_dim, CHUNK, 1, BF16)
    n = hils_quant_page_bytes(dims)
    if not n:
        raise ValueError(f"head_dim {head_dim} is not supported")
    return torch.zeros((n_pages, heads_kv, n // heads_kv), dtype=torch.uint8, device=device)


def kv_append(k_pages, v_pages, page_table, k, v, seqlens, cu_tokens=None, rotary=None, q=None, q_out=None,
              stream=None):
    """Append the packed new keys and values k, v [T,Hkv,d] to a chunk-paged cache (bf16 / fp32 or 4-bit pages),
    rotating keys, and queries q [T,Hq,d], by their positions.  k, v, q may be views with any token and head stride.
    Returns the rotated queries (q_out, or a new [T,Hq,d]; None without q).  Rows of tokens that are skipped (behind
    the last sequence, or of a sequence that does not fit) are not written: q_out keeps what it held there, a new
    tensor holds anything."""
    dtype = k.dtype
    quant, n_pages, Hkv, d = _page_kind(k_pages, v_pages, dtype)
    B, nc = _batch(page_table, seqlens, cu_tokens)
    T, Hq = k.shape[0], Hkv
    _need(k, "k", dtype, (T, Hkv, d))
    _need(v, "v", dtype, (T, Hkv, d))
    if q is not None:
        Hq = q.shape[1]
        _need(q, "q", dtype, (T, Hq, d))
        if q_out is None:
            q_out = _new(q, (T, Hq, d), dtype, stream)
        else:
            _need(q_out, "q_out", dtype, (T, Hq, d))
    elif q_out is not None:
        raise ValueError("q_out without q")
    call = hils_kv_append_quant if quant else hils_kv_append_paged
    call(_dims_of(B, Hq, Hkv, d, nc, 1, dtype, 0), seqlens, T, cu_tokens, rotary, q, q_out, k, v, k_pages, v_pages,
         page_table, n_pages, stream)
    return q_out


def kv_read(k_pages, v_pages, page_table, seqlens, n_tokens, dtype, cu_tokens=None, k_out=None, v_out=None,
            stream=None):
    """The last n_b cached rows of every sequence of a 4-bit cache as (k, v) [T,Hkv,d] of `dtype`; k_out, v_out may
    have any token and head stride, e.g. cache[0].transpose(0, 1) of a contiguous cache [1,Hkv,N,d].  Rows of tokens
    that are skipped are not written: k_out and v_out keep what they held there, new tensors hold anything."""
    quant, n_pages, Hkv, d = _page_kind(k_pages, v_pages, dtype)
    if not quant:
        raise ValueError("kv_read reads 4-bit pages")
    B, nc = _batch(page_table, seqlens, cu_tokens)
    shape = (n_tokens, Hkv, d)
    if k_out is None:
        k_out = _new(k_pages, shape, dtype, stream)
    else:
        _need(k_out, "k_out", dtype, shape)
    if v_out is None:
        v_out = _new(k_pages, shape, dtype, stream)
    else:
        _need(v_out, "v_out", dtype, shape)
    hils_kv_read_quant(_dims_of(B, Hkv, Hkv, d, nc, 1, dtype, 0), seqlens, n_tokens, cu_tokens, k_pages, v_pages,
                       page_table, n_pages, k_out, v_out, stream)
    return k_out, v_out


def _need_summary(summ, B, Hkv, nc, d, dtype):
    _need(summ.kprime, "kprime", torch.float32, (B, Hkv, nc, d))
    _need(summ.bprime, "bprime", torch.float32, (B, Hkv, nc))
    if dtype == torch.bfloat16:
        m = summ.kprime_mma
        if m is None or m.dtype != torch.bfloat16 or m.numel() != B * Hkv * nc * (d + 16):
            raise ValueError(f"kprime_mma: expected the bf16 scoring operand of {B * Hkv * nc * (d + 16)} elements")


def landmark_summary_append(k_pages, page_table, lq, seqlens, n_tokens, summ: Summary, cu_tokens=None, stream=None):
    """Write the summaries of the chunks that an append of n_tokens packed tokens completed into summ; lq
    [B,Hkv,nc,d].  k_pages in lq's type or in 4 bits."""
    quant, n_pages, Hkv, d = _page_kind(k_pages, None, lq.dtype)
    B, nc = _batch(page_table, seqlens, cu_tokens)
    _need(lq, "lq", lq.dtype, (B, Hkv, nc, d))
    _need_summary(summ, B, Hkv, nc, d, lq.dtype)
    call = hils_landmark_summary_quant if quant else hils_landmark_summary_append
    call(_dims_of(B, Hkv, Hkv, d, nc, 1, lq.dtype, 0), seqlens, n_tokens, cu_tokens, k_pages, page_table, n_pages, lq,
         summ.kprime, summ.bprime, summ.kprime_mma, stream)
    return summ


def decode_step_quant(q, k_pages, v_pages, page_table, summ: Summary, seqlens, topk, q_score=None, workspace=None,
                      stream=None, window=0, out=None, with_selection=False):
    """One decode step for q [B,Hq,d] against a 4-bit chunk-paged cache; q_score: a separate scoring query (Q-Cal).
    Returns (o, ids, scores); ids and scores [B,Hq,topk] only with_selection, else None."""
    dtype = q.dtype
    quant, n_pages, Hkv, d = _page_kind(k_pages, v_pages, dtype)
    if not quant:
        raise ValueError("decode_step_quant reads 4-bit pages")
    B, nc = _batch(page_table, seqlens, None)
    Hq = q.shape[1]
    _need(q, "q", dtype, (B, Hq, d))
    if q_score is not None:
        _need(q_score, "q_score", dtype, (B, Hq, d))
    _need_summary(summ, B, Hkv, nc, d, dtype)
    key = (B, Hq, Hkv, d, nc, topk, dtype, window)
    if workspace is None:
        workspace = _new(q, (_decode_quant_bytes(*key),), torch.uint8, stream)
    if out is None:
        out = _new(q, (B, Hq, d), dtype, stream)
    else:
        _need(out, "out", dtype, (B, Hq, d))
    ids = scores = None
    if with_selection:
        ids = _new(q, (B, Hq, topk), torch.int32, stream)
        scores = _new(q, (B, Hq, topk), torch.float32, stream)
    hils_attn_decode_quant(_dims_of(*key), q, q_score, k_pages, v_pages, page_table, n_pages, summ.kprime, summ.bprime,
                           summ.kprime_mma, seqlens, out, ids, scores, workspace, workspace.nbytes, stream)
    return out, ids, scores
