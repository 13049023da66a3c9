"""ctypes binding of the fa512 C ABI (``include/fa512.h``).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the ``stream`` argument, and a non-zero status becomes a
:class:`Fa512Error`.  Every step of the computation runs in the library's
CUDA kernels; there is no fallback of any kind.  torch supplies device memory
(outputs and the decode workspace when the caller passes none) and streams.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

HEAD_DIM = 512
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libfa512.so"
_lock = threading.Lock()
_lib = None

_STATUS = {
    0: "FA512_OK",
    1: "FA512_ERR_INVALID_ARG",
    2: "FA512_ERR_UNSUPPORTED",
    3: "FA512_ERR_CUDA",
    4: "FA512_ERR_TIMEOUT",
    5: "FA512_ERR_WORKSPACE",
    6: "FA512_ERR_DEVICE_INDEX",
    7: "FA512_ERR_OUT_OF_PAGES",
}


class Fa512Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s (%d): %s" % (_STATUS.get(status, "?"), status, message))
        self.status = status


def library_path() -> str:
    return os.environ.get("FA512_LIBRARY", os.path.join(_HERE, _LIB_NAME))


def load_library():
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise Fa512Error(3, "CUDA library %s is missing; build it with "
                                "`python -c 'import __graft_entry__ as g; g.build()'`" % path)
        lib = ctypes.CDLL(path)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa512_prefill.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, I, P]
        lib.fa512_prefill.restype = I
        lib.fa512_prefill_d256.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, I, P]
        lib.fa512_prefill_d256.restype = I
        lib.fa512_prefill_paged.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F,
                                            I, I, P]
        lib.fa512_prefill_paged.restype = I
        lib.fa512_decode_paged.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I,
                                           P, Z, P]
        lib.fa512_decode_paged.restype = I
        lib.fa512_decode_paged_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I,
                                                   I, P]
        lib.fa512_decode_paged_noalloc.restype = I
        lib.fa512_decode_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.fa512_decode_workspace_bytes.restype = Z
        lib.fa512_decode_paged_q.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, I,
                                             P, Z, P]
        lib.fa512_decode_paged_q.restype = I
        lib.fa512_decode_paged_fp8.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, F,
                                               F, I, I, P, Z, P]
        lib.fa512_decode_paged_fp8.restype = I
        lib.fa512_decode_workspace_bytes_q.argtypes = [I, I, I, I, I, I, I]
        lib.fa512_decode_workspace_bytes_q.restype = Z
        lib.fa512_decode_auto_splits.argtypes = [I, I, I, I]
        lib.fa512_decode_auto_splits.restype = I
        lib.fa512_decode_auto_splits_fp8.argtypes = [I, I, I, I, I, I]
        lib.fa512_decode_auto_splits_fp8.restype = I
        lib.fa512_decode_workspace_bytes_fp8.argtypes = [I, I, I, I, I, I, I]
        lib.fa512_decode_workspace_bytes_fp8.restype = Z
        L = ctypes.c_int64
        lib.fa512_decode_paged_tree.argtypes = [P] * 9 + [I] * 8 + [F, I, I, I, P, Z, P]
        lib.fa512_decode_paged_tree.restype = I
        lib.fa512_decode_paged_tree_fp8.argtypes = [P] * 9 + [I] * 8 + [F, F, F, I, I, I, P, Z, P]
        lib.fa512_decode_paged_tree_fp8.restype = I
        lib.fa512_decode_auto_splits_tree.argtypes = [I] * 7
        lib.fa512_decode_auto_splits_tree.restype = I
        lib.fa512_decode_workspace_bytes_tree.argtypes = [I] * 8
        lib.fa512_decode_workspace_bytes_tree.restype = Z
        lib.fa512_cache_append.argtypes = [P, P, L, L, L, L, P, P, P, P, P] + [I] * 6 + [P]
        lib.fa512_cache_append.restype = I
        lib.fa512_cache_append_fp8.argtypes = [P, P, L, L, L, L, P, P, P, P, P, F, F] + [I] * 6 + [P]
        lib.fa512_cache_append_fp8.restype = I
        lib.fa512_cache_compact.argtypes = [P] * 8 + [I] * 9 + [P]
        lib.fa512_cache_compact.restype = I
        lib.fa512_cache_fork.argtypes = [P] * 9 + [I] * 8 + [P]
        lib.fa512_cache_fork.restype = I
        lib.fa512_cache_resize.argtypes = [P] * 6 + [I] * 4 + [P]
        lib.fa512_cache_resize.restype = I
        lib.fa512_device_status.argtypes = [P, I]
        lib.fa512_device_status.restype = I
        lib.fa512_status_string.argtypes = [I]
        lib.fa512_status_string.restype = ctypes.c_char_p
        lib.fa512_last_error_message.argtypes = []
        lib.fa512_last_error_message.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status != 0:
        lib = load_library()
        msg = lib.fa512_last_error_message()
        raise Fa512Error(status, msg.decode() if msg else "")


def _dptr(t: torch.Tensor | None, name: str, dtype=None) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise Fa512Error(1, "%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise Fa512Error(1, "%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise Fa512Error(1, "%s must be contiguous" % name)
    return t.data_ptr()


# The current stream's handle without building a Stream object (2.9 us of a
# call's host time against 0.1 us on the GB300's host), and the device.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, dev: int | None = None) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if dev is None else dev)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _side(stream):
    """The stream that a call is given as a torch stream; None where it is the current one."""
    if stream is None or _stream(stream) == _stream(None):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _new(side, shape, dtype, device, returned: bool = True) -> torch.Tensor:
    """A tensor that a call makes for itself.  It comes from the memory of the
    stream that writes it: a block of the current stream's may have a user that
    is still queued there, which the other stream does not wait for.  What is
    returned is not given back to that stream before the current one's work on
    it is done."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream())
    return t


def fa512_status_string(status: int) -> str:
    return load_library().fa512_status_string(int(status)).decode()


def fa512_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None, *,
                  q_offset: int = 0, scale: float | None = None, causal: bool = True,
                  window: int = 0, return_lse: bool = True, stream=None):
    """Attention forward of one prefill chunk; returns ``(out, lse)``.

    q [seqlen_q, n_q_heads, 512], k/v [seqlen_k, n_kv_heads, 512], bf16 CUDA.
    out is allocated when not given; lse [n_q_heads, seqlen_q] fp32 likewise
    (``return_lse=False`` passes NULL).
    """
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or k.shape != v.shape:
        raise Fa512Error(1, "q, k, v must be [seq, heads, 512] with k.shape == v.shape")
    sq, hq, d = q.shape
    sk, hk, _ = k.shape
    side = _side(stream)
    if out is None:
        out = _new(side, (sq, hq, d), torch.bfloat16, q.device)
    if lse is None and return_lse:
        lse = _new(side, (hq, sq), torch.float32, q.device)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    _check(lib.fa512_prefill(_dptr(q, "q", torch.bfloat16), _dptr(k, "k", torch.bfloat16),
                             _dptr(v, "v", torch.bfloat16), _dptr(out, "out", torch.bfloat16),
                             _dptr(lse, "lse", torch.float32), sq, sk, int(q_offset), hq, hk,
                             float(scale), 1 if causal else 0, int(window), _stream(stream)))
    return out, lse


def fa512_prefill_d256(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None, *,
                       q_offset: int = 0, scale: float | None = None, causal: bool = True,
                       window: int = 0, return_lse: bool = True, stream=None):
    """Attention forward of one prefill chunk with heads of 256 dimensions
    (the sliding-window local layers); returns ``(out, lse)``.

    q [seqlen_q, n_q_heads, 256], k/v [seqlen_k, n_kv_heads, 256], bf16 CUDA.
    """
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or k.shape != v.shape:
        raise Fa512Error(1, "q, k, v must be [seq, heads, 256] with k.shape == v.shape")
    sq, hq, d = q.shape
    sk, hk, dk = k.shape
    if d != 256 or dk != 256:
        raise Fa512Error(1, "fa512_prefill_d256 takes heads of 256 dimensions")
    side = _side(stream)
    if out is None:
        out = _new(side, (sq, hq, d), torch.bfloat16, q.device)
    if lse is None and return_lse:
        lse = _new(side, (hq, sq), torch.float32, q.device)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    _check(lib.fa512_prefill_d256(_dptr(q, "q", torch.bfloat16), _dptr(k, "k", torch.bfloat16),
                                  _dptr(v, "v", torch.bfloat16), _dptr(out, "out", torch.bfloat16),
                                  _dptr(lse, "lse", torch.float32), sq, sk, int(q_offset), hq, hk,
                                  float(scale), 1 if causal else 0, int(window), _stream(stream)))
    return out, lse


def fa512_prefill_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                        page_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                        seqused_k: torch.Tensor, out: torch.Tensor | None = None,
                        lse: torch.Tensor | None = None, *, max_seqlen_q: int,
                        scale: float | None = None, causal: bool = True, window: int = 0,
                        return_lse: bool = True, stream=None):
    """Attention forward of a batch of prefill chunks (varlen rows) over a
    paged KV cache; returns ``(out, lse)``.

    q [total_q, n_q_heads, 512] bf16; k_pages/v_pages [num_pages, page_size,
    n_kv_heads, 512] bf16; page_table [batch, max_pages_per_seq] int32;
    cu_seqlens_q [batch + 1] int32; seqused_k [batch] int32 (all CUDA).
    ``max_seqlen_q`` bounds the chunk lengths on the host.  out is allocated
    when not given; lse [n_q_heads, total_q] fp32 likewise.
    """
    if q.dim() != 3 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise Fa512Error(1, "q must be [total_q, heads, 512], pages [n, page, heads, 512]")
    if page_table.dim() != 2 or cu_seqlens_q.dim() != 1 or seqused_k.dim() != 1:
        raise Fa512Error(1, "page_table [batch, pages], cu_seqlens_q [batch + 1], seqused_k [batch]")
    total_q, hq, d = q.shape
    npages, psz, hk, _ = k_pages.shape
    bsz, mpps = page_table.shape
    if cu_seqlens_q.shape[0] != bsz + 1 or seqused_k.shape[0] != bsz:
        raise Fa512Error(1, "cu_seqlens_q must have batch + 1 entries and seqused_k batch")
    side = _side(stream)
    if out is None:
        out = _new(side, (total_q, hq, d), torch.bfloat16, q.device)
    if lse is None and return_lse:
        lse = _new(side, (hq, total_q), torch.float32, q.device)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    _check(lib.fa512_prefill_paged(
        _dptr(q, "q", torch.bfloat16), _dptr(k_pages, "k_pages", torch.bfloat16),
        _dptr(v_pages, "v_pages", torch.bfloat16), _dptr(page_table, "page_table", torch.int32),
        _dptr(cu_seqlens_q, "cu_seqlens_q", torch.int32),
        _dptr(seqused_k, "seqused_k", torch.int32), _dptr(out, "out", torch.bfloat16),
        _dptr(lse, "lse", torch.float32), bsz, total_q, int(max_seqlen_q), hq, hk, psz, npages,
        mpps, float(scale), 1 if causal else 0, int(window), _stream(stream)))
    return out, lse


def fa512_decode_workspace_bytes(batch: int, n_q_heads: int, n_kv_heads: int, page_size: int,
                                 max_kv_len: int, num_splits: int = 0) -> int:
    return int(load_library().fa512_decode_workspace_bytes(batch, n_q_heads, n_kv_heads,
                                                           page_size, max_kv_len, num_splits))


def fa512_decode_auto_splits(batch: int, n_kv_heads: int, page_size: int, max_kv_len: int) -> int:
    return int(load_library().fa512_decode_auto_splits(batch, n_kv_heads, page_size, max_kv_len))


def fa512_decode_auto_splits_fp8(batch: int, q_len: int, n_q_heads: int, n_kv_heads: int,
                                 page_size: int, max_kv_len: int) -> int:
    return int(load_library().fa512_decode_auto_splits_fp8(batch, q_len, n_q_heads, n_kv_heads,
                                                           page_size, max_kv_len))


def fa512_decode_workspace_bytes_fp8(batch: int, q_len: int, n_q_heads: int, n_kv_heads: int,
                                     page_size: int, max_kv_len: int, num_splits: int = 0) -> int:
    return int(load_library().fa512_decode_workspace_bytes_fp8(batch, q_len, n_q_heads, n_kv_heads,
                                                               page_size, max_kv_len, num_splits))


def fa512_decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                       page_table: torch.Tensor, kv_lens: torch.Tensor,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None, *,
                       max_kv_len: int | None = None, scale: float | None = None,
                       window: int = 0, num_splits: int = 0,
                       workspace: torch.Tensor | None = None, return_lse: bool = True,
                       stream=None):
    """One query token per sequence over a paged KV cache; returns ``(out, lse)``.

    q [batch, n_q_heads, 512]; k_pages/v_pages [num_pages, page_size,
    n_kv_heads, 512] bf16; page_table [batch, max_pages_per_seq] int32;
    kv_lens [batch] int32 (all CUDA).  ``max_kv_len`` bounds kv_lens on the
    host (default: the page table's capacity).
    """
    if q.dim() != 3 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise Fa512Error(1, "q must be [batch, heads, 512], pages [n, page, heads, 512]")
    bsz, hq, d = q.shape
    npages, psz, hk, _ = k_pages.shape
    if page_table.dim() != 2:
        raise Fa512Error(1, "page_table must be [batch, max_pages_per_seq]")
    mpps = page_table.shape[1]
    if max_kv_len is None:
        max_kv_len = mpps * psz
    side = _side(stream)
    if out is None:
        out = _new(side, (bsz, hq, d), torch.bfloat16, q.device)
    if lse is None and return_lse:
        lse = _new(side, (bsz, hq), torch.float32, q.device)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    need = int(lib.fa512_decode_workspace_bytes(bsz, hq, hk, psz, int(max_kv_len),
                                                int(num_splits)))
    if workspace is None:
        workspace = _new(side, max(need, 256), torch.uint8, q.device, returned=False)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.fa512_decode_paged(
        _dptr(q, "q", torch.bfloat16), _dptr(k_pages, "k_pages", torch.bfloat16),
        _dptr(v_pages, "v_pages", torch.bfloat16), _dptr(page_table, "page_table", torch.int32),
        _dptr(kv_lens, "kv_lens", torch.int32), _dptr(out, "out", torch.bfloat16),
        _dptr(lse, "lse", torch.float32), bsz, hq, hk, psz, npages, mpps, int(max_kv_len),
        float(scale), int(window), int(num_splits), _dptr(workspace, "workspace"), ws_bytes,
        _stream(stream)))
    return out, lse


def fa512_decode_paged_noalloc(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                               page_table: torch.Tensor, kv_lens: torch.Tensor,
                               out: torch.Tensor, lse: torch.Tensor | None = None, *,
                               max_kv_len: int | None = None, scale: float | None = None,
                               window: int = 0, num_splits: int = 0, stream=None):
    """fa512_decode_paged without a workspace: the split partials go to the
    library's static device array (for callers that cannot allocate).  The
    caller passes ``out`` (and ``lse``, or None); nothing is allocated here
    either.  Arguments as for :func:`fa512_decode_paged`."""
    if q.dim() != 3 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise Fa512Error(1, "q must be [batch, heads, 512], pages [n, page, heads, 512]")
    bsz, hq, d = q.shape
    npages, psz, hk, _ = k_pages.shape
    if page_table.dim() != 2:
        raise Fa512Error(1, "page_table must be [batch, max_pages_per_seq]")
    mpps = page_table.shape[1]
    if max_kv_len is None:
        max_kv_len = mpps * psz
    if scale is None:
        scale = d ** -0.5
    _check(load_library().fa512_decode_paged_noalloc(
        _dptr(q, "q", torch.bfloat16), _dptr(k_pages, "k_pages", torch.bfloat16),
        _dptr(v_pages, "v_pages", torch.bfloat16), _dptr(page_table, "page_table", torch.int32),
        _dptr(kv_lens, "kv_lens", torch.int32), _dptr(out, "out", torch.bfloat16),
        _dptr(lse, "lse", torch.float32), bsz, hq, hk, psz, npages, mpps, int(max_kv_len),
        float(scale), int(window), int(num_splits), _stream(stream)))
    return out, lse


def fa512_decode_paged_q(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                         page_table: torch.Tensor, kv_lens: torch.Tensor,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None, *,
                         max_kv_len: int | None = None, scale: float | None = None,
                         window: int = 0, num_splits: int = 0,
                         workspace: torch.Tensor | None = None, return_lse: bool = True,
                         stream=None):
    """q_len query tokens per sequence (its last q_len positions) over a paged
    KV cache; returns ``(out, lse)``.

    q [batch, q_len, n_q_heads, 512]; out like q; lse [batch, q_len, n_q_heads].
    Other arguments as :func:`fa512_decode_paged`.
    """
    if q.dim() != 4 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise Fa512Error(1, "q must be [batch, q_len, heads, 512], pages [n, page, heads, 512]")
    bsz, qlen, hq, d = q.shape
    npages, psz, hk, _ = k_pages.shape
    if page_table.dim() != 2:
        raise Fa512Error(1, "page_table must be [batch, max_pages_per_seq]")
    mpps = page_table.shape[1]
    if max_kv_len is None:
        max_kv_len = mpps * psz
    side = _side(stream)
    if out is None:
        out = _new(side, (bsz, qlen, hq, d), torch.bfloat16, q.device)
    if lse is None and return_lse:
        lse = _new(side, (bsz, qlen, hq), torch.float32, q.device)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    need = int(lib.fa512_decode_workspace_bytes_q(bsz, qlen, hq, hk, psz, int(max_kv_len),
                                                  int(num_splits)))
    if workspace is None:
        workspace = _new(side, max(need, 256), torch.uint8, q.device, returned=False)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.fa512_decode_paged_q(
        _dptr(q, "q", torch.bfloat16), _dptr(k_pages, "k_pages", torch.bfloat16),
        _dptr(v_pages, "v_pages", torch.bfloat16), _dptr(page_table, "page_table", torch.int32),
        _dptr(kv_lens, "kv_lens", torch.int32), _dptr(out, "out", torch.bfloat16),
        _dptr(lse, "lse", torch.float32), bsz, qlen, hq, hk, psz, npages, mpps, int(max_kv_len),
        float(scale), int(window), int(num_splits), _dptr(workspace, "workspace"), ws_bytes,
        _stream(stream)))
    return out, lse


def _e4m3_bytes(t: torch.Tensor, name: str) -> int | None:
    """Device pointer of an E4M3 cache given as uint8 codes or torch.float8_e4m3fn."""
    if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn:
        return _dptr(t, name)
    return _dptr(t, name, torch.uint8)


def fa512_decode_paged_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                           page_table: torch.Tensor, kv_lens: torch.Tensor,
                           out: torch.Tensor | None = None, lse: torch.Tensor | None = None, *,
                           k_scale: float = 1.0, v_scale: float = 1.0,
                           max_kv_len: int | None = None, scale: float | None = None,
                           window: int = 0, num_splits: int = 0,
                           workspace: torch.Tensor | None = None, return_lse: bool = True,
                           stream=None):
    """Decode over a paged KV cache stored in FP8 E4M3; returns ``(out, lse)``.

    q [batch, n_q_heads, 512] (one token) or [batch, q_len, n_q_heads, 512] bf16;
    k_pages / v_pages [num_pages, page_size, n_kv_heads, 512] as uint8 codes or
    torch.float8_e4m3fn; a key element is k_scale * e4m3, a value element
    v_scale * e4m3.  out / lse are shaped like q (lse without the head dim).
    Other arguments as :func:`fa512_decode_paged_q`.
    """
    single = q.dim() == 3
    q4 = q.unsqueeze(1) if single else q
    if q4.dim() != 4 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise Fa512Error(1, "q must be [batch, (q_len,) heads, 512], pages [n, page, heads, 512]")
    bsz, qlen, hq, d = q4.shape
    npages, psz, hk, _ = k_pages.shape
    if page_table.dim() != 2:
        raise Fa512Error(1, "page_table must be [batch, max_pages_per_seq]")
    mpps = page_table.shape[1]
    if max_kv_len is None:
        max_kv_len = mpps * psz
    side = _side(stream)
    if out is None:
        out = _new(side, q.shape, torch.bfloat16, q.device)
    if lse is None and return_lse:
        lse = _new(side, q.shape[:-1], torch.float32, q.device)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    need = int(lib.fa512_decode_workspace_bytes_fp8(bsz, qlen, hq, hk, psz, int(max_kv_len),
                                                    int(num_splits)))
    if workspace is None:
        workspace = _new(side, max(need, 256), torch.uint8, q.device, returned=False)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.fa512_decode_paged_fp8(
        _dptr(q, "q", torch.bfloat16), _e4m3_bytes(k_pages, "k_pages"),
        _e4m3_bytes(v_pages, "v_pages"), _dptr(page_table, "page_table", torch.int32),
        _dptr(kv_lens, "kv_lens", torch.int32), _dptr(out, "out", torch.bfloat16),
        _dptr(lse, "lse", torch.float32), bsz, qlen, hq, hk, psz, npages, mpps, int(max_kv_len),
        float(scale), float(k_scale), float(v_scale), int(window), int(num_splits),
        _dptr(workspace, "workspace"), ws_bytes, _stream(stream)))
    return out, lse


def _device(t: torch.Tensor, name: str) -> int:
    """Index of the CUDA device that ``t`` and all other tensors of a call must be on: the current one, on which the
    library works."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise Fa512Error(1, "%s must be a CUDA tensor" % name)
    dev = t.get_device()
    if dev != _current_device():
        raise Fa512Error(1, "%s is not on the current device" % name)
    return dev


def _arg(t: torch.Tensor | None, name: str, dtype, dev: int, shape=None) -> int | None:
    """Device pointer of a contiguous tensor of this type (one of these types), device and shape; None of None."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.is_contiguous()
            and (t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype))
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise Fa512Error(1, "%s must be a CUDA tensor" % name)
    if t.get_device() != dev:
        raise Fa512Error(1, "%s is on another device than the other tensors" % name)
    if not t.is_contiguous():
        raise Fa512Error(1, "%s must be contiguous" % name)
    if shape is not None and t.shape != shape:
        raise Fa512Error(1, "%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise Fa512Error(1, "%s must be %s, got %s" % (name, dtype, t.dtype))


_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_CACHE = (torch.bfloat16,) + _E4M3


def fa512_decode_auto_splits_tree(batch: int, q_len: int, n_q_heads: int, n_kv_heads: int,
                                  max_kv_len: int, window: int = 0, n_sinks: int = 0) -> int:
    return int(load_library().fa512_decode_auto_splits_tree(batch, q_len, n_q_heads, n_kv_heads,
                                                            max_kv_len, window, n_sinks))


def fa512_decode_workspace_bytes_tree(batch: int, q_len: int, n_q_heads: int, n_kv_heads: int,
                                      max_kv_len: int, window: int = 0, n_sinks: int = 0,
                                      num_splits: int = 0) -> int:
    return int(load_library().fa512_decode_workspace_bytes_tree(
        batch, q_len, n_q_heads, n_kv_heads, max_kv_len, window, n_sinks, num_splits))


def _decode_tree(fp8, q, k_pages, v_pages, page_table, kv_lens, tree_mask, out, lse, q_lens, k_scale,
                 v_scale, max_kv_len, scale, window, n_sinks, num_splits, workspace, return_lse, stream):
    qs, ks, ts = q.shape, k_pages.shape, page_table.shape
    if len(qs) != 4 or len(ks) != 4 or len(ts) != 2 or qs[3] != HEAD_DIM or ks[3] != HEAD_DIM:
        raise Fa512Error(1, "q must be [batch, q_len, heads, 512], pages [n, page, heads, 512], page_table "
                            "[batch, max_pages_per_seq]")
    bsz, qlen, hq, d = qs
    npages, psz, hk, _ = ks
    mpps = ts[1]
    dev = _device(q, "q")
    rows = (bsz, qlen, hq)
    max_kv_len = mpps * psz if max_kv_len is None else int(max_kv_len)
    window, n_sinks, num_splits = int(window), int(n_sinks), int(num_splits)
    lib = _lib or load_library()
    side = _side(stream)
    if out is None:
        out = _new(side, qs, _BF16, dev)
    if lse is None and return_lse:
        lse = _new(side, rows, _F32, dev)
    if workspace is None:
        # 0: a shape that the call below refuses
        ws_bytes = lib.fa512_decode_workspace_bytes_tree(bsz, qlen, hq, hk, max_kv_len, window, n_sinks,
                                                         num_splits) or 256
        workspace = _new(side, ws_bytes, torch.uint8, dev, returned=False)
        ws = workspace.data_ptr()
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws = _arg(workspace, "workspace", workspace.dtype, dev)
    kind = _E4M3 if fp8 else _BF16
    head = (_arg(q, "q", _BF16, dev), _arg(k_pages, "k_pages", kind, dev),
            _arg(v_pages, "v_pages", kind, dev, ks),
            _arg(page_table, "page_table", _I32, dev, (bsz, mpps)), _arg(kv_lens, "kv_lens", _I32, dev, (bsz,)),
            _arg(q_lens, "q_lens", _I32, dev, (bsz,)),
            _arg(tree_mask, "tree_mask", _I32, dev, (bsz, qlen, (qlen + 31) // 32)),
            _arg(out, "out", _BF16, dev, qs), _arg(lse, "lse", _F32, dev, rows), bsz, qlen, hq, hk,
            psz, npages, mpps, max_kv_len, d ** -0.5 if scale is None else float(scale))
    tail = (window, n_sinks, num_splits, ws, ws_bytes, _stream(stream, dev))
    if fp8:
        _check(lib.fa512_decode_paged_tree_fp8(*head, float(k_scale), float(v_scale), *tail))
    else:
        _check(lib.fa512_decode_paged_tree(*head, *tail))
    return out, lse


def fa512_decode_paged_tree(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                            page_table: torch.Tensor, kv_lens: torch.Tensor,
                            tree_mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, *, q_lens: torch.Tensor | None = None,
                            max_kv_len: int | None = None, scale: float | None = None, window: int = 0,
                            n_sinks: int = 0, num_splits: int = 0, workspace: torch.Tensor | None = None,
                            return_lse: bool = True, stream=None):
    """The drafted tokens of each sequence (its last ``q_lens[b]`` cached
    positions) over a paged KV cache; returns ``(out, lse)``.

    q [batch, q_len, n_q_heads, 512]; ``tree_mask`` [batch, q_len, ceil(q_len / 32)]
    int32, bit j of row t: token t sees token j (None: a plain run, token t
    sees tokens 0 .. t); ``q_lens`` [batch] int32 (None: q_len each).  With
    ``window`` > 0 the first ``n_sinks`` positions stay visible.  Rows of
    padding tokens get O = 0, LSE = -inf.  Other arguments as
    :func:`fa512_decode_paged_q`.
    """
    return _decode_tree(False, q, k_pages, v_pages, page_table, kv_lens, tree_mask, out, lse, q_lens, 1.0,
                        1.0, max_kv_len, scale, window, n_sinks, num_splits, workspace, return_lse, stream)


def fa512_decode_paged_tree_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                                page_table: torch.Tensor, kv_lens: torch.Tensor,
                                tree_mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                lse: torch.Tensor | None = None, *, q_lens: torch.Tensor | None = None,
                                k_scale: float = 1.0, v_scale: float = 1.0,
                                max_kv_len: int | None = None, scale: float | None = None,
                                window: int = 0, n_sinks: int = 0, num_splits: int = 0,
                                workspace: torch.Tensor | None = None, return_lse: bool = True,
                                stream=None):
    """:func:`fa512_decode_paged_tree` over a cache stored in FP8 E4M3 (uint8
    codes or torch.float8_e4m3fn; a key element is k_scale * e4m3, a value
    element v_scale * e4m3)."""
    return _decode_tree(True, q, k_pages, v_pages, page_table, kv_lens, tree_mask, out, lse, q_lens, k_scale,
                        v_scale, max_kv_len, scale, window, n_sinks, num_splits, workspace, return_lse,
                        stream)


def _new_rows(t: torch.Tensor, name: str, dev: int, shape):
    """(pointer, batch stride, token stride) of new rows whose heads are contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not _BF16 or t.shape != shape:
        raise Fa512Error(1, "%s must be a bf16 tensor of shape %s on the pages' device" % (name, tuple(shape)))
    b, n, h, d = t.stride()
    if d != 1 or (h != HEAD_DIM and shape[2] > 1):
        raise Fa512Error(1, "the heads of a token of %s must be contiguous" % name)
    # the stride of a dimension of one entry says nothing
    return t.data_ptr(), b if shape[0] > 1 else 0, n if shape[1] > 1 else 0


def _append(fp8, k_new, v_new, k_pages, v_pages, page_table, kv_lens, q_lens, k_scale, v_scale, stream):
    if k_new.dim() != 4 or k_pages.dim() != 4 or page_table.dim() != 2 or k_pages.shape[3] != HEAD_DIM:
        raise Fa512Error(1, "k_new, v_new must be [batch, q_len, heads, 512], pages [n, page, heads, 512], "
                            "page_table [batch, max_pages_per_seq]")
    npages, psz, hk, _ = k_pages.shape
    bsz, mpps = page_table.shape
    qlen = k_new.shape[1]
    shape = (bsz, qlen, hk, HEAD_DIM)
    dev = _device(k_pages, "k_pages")
    kp, kb, kt = _new_rows(k_new, "k_new", dev, shape)
    vp, vb, vt = _new_rows(v_new, "v_new", dev, shape)
    kind = _E4M3 if fp8 else _BF16
    head = (kp, vp, kb, kt, vb, vt, _arg(k_pages, "k_pages", kind, dev),
            _arg(v_pages, "v_pages", kind, dev, k_pages.shape), _arg(page_table, "page_table", _I32, dev),
            _arg(kv_lens, "kv_lens", _I32, dev, (bsz,)), _arg(q_lens, "q_lens", _I32, dev, (bsz,)))
    tail = (bsz, qlen, hk, psz, npages, mpps, _stream(stream, dev))
    lib = _lib or load_library()
    if fp8:
        _check(lib.fa512_cache_append_fp8(*head, float(k_scale), float(v_scale), *tail))
    else:
        _check(lib.fa512_cache_append(*head, *tail))
    return k_pages, v_pages


def fa512_cache_append(k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor,
                       v_pages: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, *,
                       q_lens: torch.Tensor | None = None, stream=None):
    """Writes the newest tokens' keys and values into the pages; returns
    ``(k_pages, v_pages)``, which are written in place.

    k_new / v_new [batch, q_len, n_kv_heads, 512] bf16, contiguous heads, any
    sequence and token strides that are multiples of 8; ``kv_lens`` counts the
    new tokens, ``q_lens`` [batch] int32 says how many there are (None: q_len).
    """
    return _append(False, k_new, v_new, k_pages, v_pages, page_table, kv_lens, q_lens, 1.0, 1.0, stream)


def fa512_cache_append_fp8(k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor,
                           v_pages: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, *,
                           q_lens: torch.Tensor | None = None, k_scale: float = 1.0,
                           v_scale: float = 1.0, stream=None):
    """:func:`fa512_cache_append` into an FP8 E4M3 cache (uint8 codes or
    torch.float8_e4m3fn): x is stored as the E4M3 value nearest to x / scale,
    beyond +-448 as +-448."""
    return _append(True, k_new, v_new, k_pages, v_pages, page_table, kv_lens, q_lens, k_scale, v_scale,
                   stream)


def _whole_cache(k_pages, v_pages):
    """(device, k pointer, v pointer, layers, pages, page size, heads, bytes) of a cache of one or several layers."""
    if k_pages.dim() not in (4, 5) or k_pages.dtype is not v_pages.dtype or k_pages.shape[-1] != HEAD_DIM:
        raise Fa512Error(1, "pages must be [(layers,) n, page, heads, 512], k_pages like v_pages")
    dev = _device(k_pages, "k_pages")
    shape = k_pages.shape
    layers = shape[0] if len(shape) == 5 else 1
    return (dev, _arg(k_pages, "k_pages", _CACHE, dev), _arg(v_pages, "v_pages", _CACHE, dev, shape), layers,
            shape[-4], shape[-3], shape[-2], k_pages.element_size())


def fa512_cache_compact(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                        kv_lens: torch.Tensor, accepted: torch.Tensor, n_accepted: torch.Tensor,
                        new_kv_lens: torch.Tensor | None = None, *, q_len: int,
                        q_lens: torch.Tensor | None = None, stream=None):
    """Moves the accepted drafted tokens' rows together; returns ``new_kv_lens``.

    k_pages / v_pages [(n_layers,) num_pages, page_size, n_kv_heads, 512], bf16
    or E4M3, changed in place; accepted [batch, max_accepted] int32, rising,
    the first n_accepted[b] of each row used; ``q_len`` drafted tokens per
    sequence (or ``q_lens`` [batch] int32, each at most q_len), which kv_lens
    counts.
    """
    dev, kp, vp, layers, npages, psz, hk, eb = _whole_cache(k_pages, v_pages)
    if page_table.dim() != 2 or accepted.dim() != 2:
        raise Fa512Error(1, "page_table must be [batch, pages], accepted [batch, max_accepted]")
    bsz, mpps = page_table.shape
    most = accepted.shape[1]
    one = (bsz,)
    if new_kv_lens is None:
        new_kv_lens = _new(_side(stream), one, _I32, dev)
    _check((_lib or load_library()).fa512_cache_compact(
        kp, vp, _arg(page_table, "page_table", _I32, dev), _arg(kv_lens, "kv_lens", _I32, dev, one),
        _arg(q_lens, "q_lens", _I32, dev, one), _arg(accepted, "accepted", _I32, dev, (bsz, most)),
        _arg(n_accepted, "n_accepted", _I32, dev, one), _arg(new_kv_lens, "new_kv_lens", _I32, dev, one),
        layers, bsz, int(q_len), most, hk, eb, psz, npages, mpps, _stream(stream, dev)))
    return new_kv_lens


def fa512_cache_fork(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                     kv_lens: torch.Tensor, parents: torch.Tensor, page_refs: torch.Tensor,
                     new_page_table: torch.Tensor | None = None,
                     new_kv_lens: torch.Tensor | None = None,
                     new_page_refs: torch.Tensor | None = None, *, stream=None):
    """Replaces the sequences of a cache by children of them; returns
    ``(new_page_table, new_kv_lens, new_page_refs)``.

    parents [n_children] int32; page_refs [num_pages] int32, 0 = free.  Whole
    pages are shared, a partly filled last page goes to its parent's first
    child and is copied (all layers) into a free page for every other one.
    ``new_page_refs`` may be ``page_refs`` itself.
    """
    dev, kp, vp, layers, npages, psz, hk, eb = _whole_cache(k_pages, v_pages)
    if page_table.dim() != 2 or parents.dim() != 1:
        raise Fa512Error(1, "page_table must be [batch, pages], parents [n_children]")
    bsz, mpps = page_table.shape
    kids = parents.shape[0]
    side = _side(stream)

    def out(t, shape):
        return _new(side, shape, _I32, dev) if t is None else t
    new_page_table = out(new_page_table, (kids, mpps))
    new_kv_lens = out(new_kv_lens, (kids,))
    new_page_refs = out(new_page_refs, (npages,))
    _check((_lib or load_library()).fa512_cache_fork(
        kp, vp, _arg(page_table, "page_table", _I32, dev), _arg(kv_lens, "kv_lens", _I32, dev, (bsz,)),
        _arg(parents, "parents", _I32, dev), _arg(page_refs, "page_refs", _I32, dev, (npages,)),
        _arg(new_page_table, "new_page_table", _I32, dev, (kids, mpps)),
        _arg(new_kv_lens, "new_kv_lens", _I32, dev, (kids,)),
        _arg(new_page_refs, "new_page_refs", _I32, dev, (npages,)), layers, bsz, kids, hk, eb, psz, npages,
        mpps, _stream(stream, dev)))
    return new_page_table, new_kv_lens, new_page_refs


def fa512_cache_resize(page_table: torch.Tensor, kv_lens: torch.Tensor, new_kv_lens: torch.Tensor,
                       page_refs: torch.Tensor, new_page_table: torch.Tensor | None = None,
                       new_page_refs: torch.Tensor | None = None, *, page_size: int, stream=None):
    """Gives each sequence the pages of its new length and takes back those
    behind it; returns ``(new_page_table, new_page_refs)``.

    page_table [batch, max_pages_per_seq]; page_refs [num_pages] int32, 0 =
    free.  The outputs may be the inputs themselves.  A sequence that is
    shortened to inside a page that others hold must not grow there: fork it
    into two children and end the first.
    """
    if page_table.dim() != 2 or page_refs.dim() != 1:
        raise Fa512Error(1, "page_table must be [batch, pages], page_refs [num_pages]")
    bsz, mpps = page_table.shape
    npages = page_refs.shape[0]
    dev = _device(page_table, "page_table")
    side = _side(stream)
    if new_page_table is None:
        new_page_table = _new(side, page_table.shape, _I32, dev)
    if new_page_refs is None:
        new_page_refs = _new(side, page_refs.shape, _I32, dev)
    _check((_lib or load_library()).fa512_cache_resize(
        _arg(page_table, "page_table", _I32, dev), _arg(kv_lens, "kv_lens", _I32, dev, (bsz,)),
        _arg(new_kv_lens, "new_kv_lens", _I32, dev, (bsz,)), _arg(page_refs, "page_refs", _I32, dev),
        _arg(new_page_table, "new_page_table", _I32, dev, (bsz, mpps)),
        _arg(new_page_refs, "new_page_refs", _I32, dev, (npages,)), bsz, int(page_size), npages, mpps,
        _stream(stream, dev)))
    return new_page_table, new_page_refs


def fa512_device_status(stream=None, clear: bool = True) -> int:
    """Synchronise ``stream`` and return (optionally clearing) the device error word."""
    return int(load_library().fa512_device_status(_stream(stream), 1 if clear else 0))
