"""The 4-bit key-value cache: append, read, attend (ctypes binding).

What a prefill leaves behind for generation: pages of 4-bit keys and values
(a bf16 scale and low for each token and 32 channels), attended to by new
tokens, densely or over listed blocks.  include/sbsa.h documents the format,
the layout and the description of a batch:

    cache      uint8 [n_pages, Hkv, 2, page_size, 5 d / 8]  (kv4.empty)
    page_table int32 [n_seqs, max_pages]
    seq_lens   int32 [n_seqs]      tokens of each sequence, the new ones counted
    cu_new     int32 [n_seqs + 1]  sequence b has rows cu_new[b]:cu_new[b + 1]

Rows are [heads, tokens, d] tensors of any strides with contiguous channels and
16-byte aligned rows; `x.transpose(0, 1)` of a [tokens, heads, d] projection
is taken as it is.  Calls allocate nothing but the workspace of `attend` (when
none is given) and run on `stream` (default: the current one of the tensors'
device).  As in `sbsa`, argument errors raise before anything is launched, and
what kernels meet is read with `sbsa.get_status`.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .sbsa import BF16, FP32, SbsaError, ERR_INVALID_ARG, _check, lib

SYMBOLS = ["sbsa_kv4_cache_bytes", "sbsa_kv4_append", "sbsa_kv4_read",
           "sbsa_kv4_attend_workspace_bytes", "sbsa_kv4_attend"]


class Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages", "max_pages",
                 "n_seqs", "n_tokens", "max_new", "dtype", "list_heads", "block_size",
                 "max_blocks")] + [("sm_scale", ctypes.c_float)]


_vp, _i64, _PP = ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(Params)
lib.sbsa_kv4_cache_bytes.argtypes = [_PP]
lib.sbsa_kv4_cache_bytes.restype = ctypes.c_size_t
lib.sbsa_kv4_append.argtypes = [_PP, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp,
                                _vp, _vp]
lib.sbsa_kv4_append.restype = ctypes.c_int
lib.sbsa_kv4_read.argtypes = [_PP, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.sbsa_kv4_read.restype = ctypes.c_int
lib.sbsa_kv4_attend_workspace_bytes.argtypes = [_PP]
lib.sbsa_kv4_attend_workspace_bytes.restype = ctypes.c_size_t
lib.sbsa_kv4_attend.argtypes = [_PP, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp,
                                _vp, _vp, ctypes.c_size_t, _vp]
lib.sbsa_kv4_attend.restype = ctypes.c_int

_DTYPE = {torch.bfloat16: BF16, torch.float32: FP32}


def empty(n_pages: int, n_kv_heads: int, page_size: int = 64, head_dim: int = 128,
          device="cuda") -> torch.Tensor:
    """A cache of zeroed pages: uint8 [n_pages, n_kv_heads, 2, page_size, 5 head_dim / 8]."""
    p = Params(n_q_heads=n_kv_heads, n_kv_heads=n_kv_heads, head_dim=head_dim,
               page_size=page_size, n_pages=n_pages, max_pages=1, max_new=1)
    if lib.sbsa_kv4_cache_bytes(ctypes.byref(p)) == 0:
        raise SbsaError(ERR_INVALID_ARG, "sbsa_kv4_cache_bytes")
    return torch.zeros(n_pages, n_kv_heads, 2, page_size, 5 * head_dim // 8, dtype=torch.uint8,
                       device=device)


def _on(t: torch.Tensor, name: str, device):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _batch(cache, page_table, seq_lens, cu_new) -> Params:
    """The parameters that every call has, from checked tensors."""
    dev = cache.device
    if dev.type != "cuda":
        raise ValueError("cache must be a CUDA tensor")
    if cache.dtype != torch.uint8 or cache.dim() != 5 or cache.shape[2] != 2 \
            or cache.shape[4] % 5 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 tensor of shape "
                         "[n_pages, n_kv_heads, 2, page_size, 5 * head_dim / 8]")
    n_seqs = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    for t, name, shape in ((page_table, "page_table", (n_seqs, page_table.shape[-1])),
                           (seq_lens, "seq_lens", (n_seqs,)), (cu_new, "cu_new", (n_seqs + 1,))):
        _on(t, name, dev)
        if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}, "
                             f"got {t.dtype} {tuple(t.shape)}")
    return Params(n_q_heads=cache.shape[1], n_kv_heads=cache.shape[1],
                  head_dim=cache.shape[4] // 5 * 8, page_size=cache.shape[3],
                  n_pages=cache.shape[0], max_pages=page_table.shape[1], n_seqs=n_seqs, max_new=1)


def _rows(p: Params, t: torch.Tensor, name: str, heads: int, dtype, device):
    """Pointer and strides of rows [heads, n_tokens, d]."""
    _on(t, name, device)
    if t.dtype != dtype or t.dim() != 3 or t.shape[0] != heads or t.shape[1] != p.n_tokens \
            or t.shape[2] != p.head_dim:
        raise ValueError(f"{name} must be {dtype} {(heads, p.n_tokens, p.head_dim)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if t.stride(2) != 1 and t.numel():
        raise ValueError(f"{name} must have contiguous channels")
    return t.data_ptr(), t.stride(1), t.stride(0)


def _plain(p: Params, t: Optional[torch.Tensor], name: str, dtype, device):
    """Pointer of a contiguous [Hkv, n_tokens, d] tensor, or None."""
    if t is None:
        return None
    _rows(p, t, name, p.n_kv_heads, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return _DTYPE[t.dtype]


def _call(fn, name: str, device, stream, *args):
    """The C call with the tensors' device current."""
    s = (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream
    if device.index == torch.cuda.current_device():
        _check(fn(*args, s), name)
    else:
        with torch.cuda.device(device):
            _check(fn(*args, s), name)


def append(cache, k, v, page_table, seq_lens, cu_new, k_stored=None, v_stored=None, stream=None):
    """Quantise the new rows k, v [Hkv, n_tokens, d] into the cache.  With k_stored / v_stored
    (contiguous, like k and v) also what the cache now stands for."""
    p, dev = _batch(cache, page_table, seq_lens, cu_new), cache.device
    p.dtype = _dtype(k, "k")
    p.n_tokens = k.shape[1] if k.dim() == 3 else -1
    kr = _rows(p, k, "k", p.n_kv_heads, k.dtype, dev)
    vr = _rows(p, v, "v", p.n_kv_heads, k.dtype, dev)
    _call(lib.sbsa_kv4_append, "sbsa_kv4_append", dev, stream, ctypes.byref(p), cache.data_ptr(),
          page_table.data_ptr(), seq_lens.data_ptr(), cu_new.data_ptr(), *kr, *vr,
          _plain(p, k_stored, "k_stored", k.dtype, dev), _plain(p, v_stored, "v_stored", k.dtype, dev))


def read(cache, page_table, seq_lens, cu_new, k_out=None, v_out=None, stream=None):
    """The same rows back into k_out and / or v_out [Hkv, n_tokens, d] (contiguous, bf16 or fp32).
    With cu_new the running sum of seq_lens: whole sequences."""
    p, dev = _batch(cache, page_table, seq_lens, cu_new), cache.device
    some = k_out if k_out is not None else v_out
    if some is None:
        raise ValueError("read needs k_out or v_out")
    p.dtype = _dtype(some, "k_out" if k_out is not None else "v_out")
    p.n_tokens = some.shape[1] if some.dim() == 3 else -1
    _call(lib.sbsa_kv4_read, "sbsa_kv4_read", dev, stream, ctypes.byref(p), cache.data_ptr(),
          page_table.data_ptr(), seq_lens.data_ptr(), cu_new.data_ptr(),
          _plain(p, k_out, "k_out", some.dtype, dev), _plain(p, v_out, "v_out", some.dtype, dev))


def attend(cache, q, page_table, seq_lens, cu_new, max_new: int, idx=None, cnt=None,
           block_size: int = 0, sm_scale: float = 0.0, out=None, workspace=None, stream=None):
    """o [Hq, n_tokens, d] (into `out` when given) of causal attention of the rows q over the
    cache, which holds their own tokens already.  max_new: at least the most rows of one sequence.  idx [n_seqs, heads,
    max_blocks] and cnt [n_seqs, heads] (heads = Hkv or Hq) restrict it to the listed blocks of
    block_size tokens.  workspace: uint8, at least attend_workspace_bytes (allocated when None)."""
    p, dev = _batch(cache, page_table, seq_lens, cu_new), cache.device
    p.dtype = _dtype(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [Hq, n_tokens, d]")
    p.n_q_heads, p.n_tokens, p.max_new, p.sm_scale = q.shape[0], q.shape[1], max_new, sm_scale
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.zeros_like(q)
    qr = _rows(p, q, "q", p.n_q_heads, q.dtype, dev)
    orow = _rows(p, out, "out", p.n_q_heads, q.dtype, dev)
    if (idx is None) != (cnt is None):
        raise ValueError("idx and cnt go together")
    if idx is not None:
        if idx.dim() != 3 or idx.dtype != torch.int32 or not idx.is_contiguous() \
                or idx.shape[0] != p.n_seqs or idx.shape[1] not in (p.n_kv_heads, p.n_q_heads):
            raise ValueError("idx must be contiguous int32 [n_seqs, Hkv or Hq, max_blocks]")
        if cnt.dtype != torch.int32 or not cnt.is_contiguous() \
                or tuple(cnt.shape) != tuple(idx.shape[:2]):
            raise ValueError(f"cnt must be contiguous int32 {tuple(idx.shape[:2])}")
        _on(idx, "idx", dev)
        _on(cnt, "cnt", dev)
        p.list_heads, p.max_blocks, p.block_size = idx.shape[1], idx.shape[2], block_size
    if workspace is None:
        # with the call's stream current, so that the memory is not given away before it has run
        with torch.cuda.stream(stream):
            workspace = torch.empty(attend_workspace_bytes(p), dtype=torch.uint8, device=dev)
    else:
        _on(workspace, "workspace", dev)
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
    _call(lib.sbsa_kv4_attend, "sbsa_kv4_attend", dev, stream, ctypes.byref(p), cache.data_ptr(),
          page_table.data_ptr(), seq_lens.data_ptr(), cu_new.data_ptr(), *qr, *orow,
          None if idx is None else idx.data_ptr(), None if cnt is None else cnt.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return out


def attend_workspace_bytes(p: Params) -> int:
    """Bytes of the workspace of `attend` (the same for every batch of one head_dim)."""
    n = lib.sbsa_kv4_attend_workspace_bytes(ctypes.byref(p))
    if n == 0:
        raise SbsaError(ERR_INVALID_ARG, "sbsa_kv4_attend_workspace_bytes")
    return int(n)
