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

_append, _read, _attend = lib.sbsa_kv4_append, lib.sbsa_kv4_read, lib.sbsa_kv4_attend
_workspace_bytes = lib.sbsa_kv4_attend_workspace_bytes

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


# The calls are short (a few microseconds on the GPU for a token), so the checks that every call
# passes are single expressions; what fails one is looked at again to say what is wrong.

def _bad_batch(cache, page_table, seq_lens, cu_new):
    if not cache.is_cuda:
        raise ValueError("cache must be a CUDA tensor")
    if cache.dtype != torch.uint8 or cache.dim() != 5 or cache.shape[2] != 2 \
            or cache.shape[4] % 5 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 tensor of shape "
                         "[n_pages, n_kv_heads, 2, page_size, 5 * head_dim / 8]")
    n_seqs = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    for t, name, shape in ((page_table, "page_table", (n_seqs, page_table.shape[-1])),
                           (seq_lens, "seq_lens", (n_seqs,)), (cu_new, "cu_new", (n_seqs + 1,))):
        if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous() \
                or t.device != cache.device:
            raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape} on "
                             f"{cache.device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    raise ValueError("inconsistent cache, page_table, seq_lens and cu_new")


_U8, _I32 = torch.uint8, torch.int32


def _batch(cache, page_table, seq_lens, cu_new):
    """Device index, shape of the cache, and of the page table, checked."""
    dev, shape, tab, lens = cache.get_device(), cache.shape, page_table.shape, seq_lens.shape
    if (dev < 0 or len(shape) != 5 or shape[2] != 2 or shape[4] % 5 or cache.dtype is not _U8
            or len(tab) != 2 or len(lens) != 1 or tab[0] != lens[0]
            or cu_new.shape != (lens[0] + 1,)
            or page_table.dtype is not _I32 or seq_lens.dtype is not _I32
            or cu_new.dtype is not _I32 or page_table.get_device() != dev
            or seq_lens.get_device() != dev or cu_new.get_device() != dev
            or not (cache.is_contiguous() and page_table.is_contiguous()
                    and seq_lens.is_contiguous() and cu_new.is_contiguous())):
        _bad_batch(cache, page_table, seq_lens, cu_new)
    return dev, shape, tab


def _rows(t: torch.Tensor, name: str, shape, dtype, dev: int):
    """Strides between tokens and heads of rows [heads, n_tokens, d]."""
    head, token, channel = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.shape != shape or t.dtype is not dtype or channel != 1 or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} with contiguous channels on "
                         f"cuda:{dev}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} "
                         f"on {t.device}")
    return token, head


def _plain(t: Optional[torch.Tensor], name: str, shape, dtype, dev: int):
    """Pointer of a contiguous [Hkv, n_tokens, d] tensor, or None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on cuda:{dev}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None or t.dim() != 3:
        raise ValueError(f"{name} must be a bfloat16 or float32 tensor [heads, tokens, d], got "
                         f"{t.dtype} {tuple(t.shape)}")
    return code


# The current stream's handle: directly where this torch has it (a sixth of the time).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(fn, name: str, dev: int, stream, *args):
    """The C call with the tensors' device current."""
    s = _current_stream(dev) if stream is None else stream.cuda_stream
    if dev == torch.cuda.current_device():
        code = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, s)
    if code:
        _check(code, name)


def append(cache, k, v, page_table, seq_lens, cu_new, k_stored=None, v_stored=None, stream=None):
    """Quantise the new rows k, v [Hkv, n_tokens, d] into the cache.  With k_stored / v_stored
    (contiguous, like k and v) also what the cache now stands for."""
    dev, c, tab = _batch(cache, page_table, seq_lens, cu_new)
    dt, code = k.dtype, _dtype(k, "k")
    heads, d, n = c[1], c[4] // 5 * 8, k.shape[1]
    shape = (heads, n, d)
    kr, vr = _rows(k, "k", shape, dt, dev), _rows(v, "v", shape, dt, dev)
    p = Params(heads, heads, d, c[3], c[0], tab[1], tab[0], n, 1, code)
    _call(_append, "sbsa_kv4_append", dev, stream, p, cache.data_ptr(), page_table.data_ptr(),
          seq_lens.data_ptr(), cu_new.data_ptr(), k.data_ptr(), *kr, v.data_ptr(), *vr,
          _plain(k_stored, "k_stored", shape, dt, dev),
          _plain(v_stored, "v_stored", shape, dt, dev))


def read(cache, page_table, seq_lens, cu_new, k_out=None, v_out=None, stream=None):
    """The same rows back into k_out and / or v_out [Hkv, n_tokens, d] (contiguous, bf16 or fp32).
    With cu_new the running sum of seq_lens: whole sequences."""
    dev, c, tab = _batch(cache, page_table, seq_lens, cu_new)
    some = v_out if k_out is None else k_out
    if some is None:
        raise ValueError("read needs k_out or v_out")
    dt, code = some.dtype, _dtype(some, "k_out or v_out")
    heads, d, n = c[1], c[4] // 5 * 8, some.shape[1]
    shape = (heads, n, d)
    p = Params(heads, heads, d, c[3], c[0], tab[1], tab[0], n, 1, code)
    _call(_read, "sbsa_kv4_read", dev, stream, p, cache.data_ptr(), page_table.data_ptr(),
          seq_lens.data_ptr(), cu_new.data_ptr(), _plain(k_out, "k_out", shape, dt, dev),
          _plain(v_out, "v_out", shape, dt, dev))


def attend(cache, q, page_table, seq_lens, cu_new, max_new: int, idx=None, cnt=None,
           block_size: int = 0, sm_scale: float = 0.0, out=None, workspace=None, stream=None):
    """o [Hq, n_tokens, d] (into `out` when given) of causal attention of the rows q over the
    cache, which holds their own tokens already.  max_new: at least the most rows of one sequence
    (it chooses the kernel for the whole call: single tokens and a prompt's chunk are faster apart).
    idx [n_seqs, heads, max_blocks] and cnt [n_seqs, heads] (heads = Hkv or Hq) restrict it to the
    listed blocks of block_size tokens.  workspace: uint8, at least attend_workspace_bytes
    (allocated when None)."""
    dev, c, tab = _batch(cache, page_table, seq_lens, cu_new)
    dt, code = q.dtype, _dtype(q, "q")
    heads, n, d = q.shape[0], q.shape[1], c[4] // 5 * 8
    shape = (heads, n, d)
    qr = _rows(q, "q", shape, dt, dev)
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.zeros_like(q)
    orow = _rows(out, "out", shape, dt, dev)
    p = Params(heads, c[1], d, c[3], c[0], tab[1], tab[0], n, max_new, code, 0, 0, 0, sm_scale)
    lists = (None, None)
    if idx is not None or cnt is not None:
        if idx is None or cnt is None:
            raise ValueError("idx and cnt go together")
        if idx.dim() != 3 or idx.dtype is not _I32 or not idx.is_contiguous() \
                or idx.shape[0] != tab[0] or idx.shape[1] not in (c[1], heads) \
                or idx.get_device() != dev:
            raise ValueError("idx must be contiguous int32 [n_seqs, Hkv or Hq, max_blocks] on "
                             f"cuda:{dev}")
        if cnt.dtype is not _I32 or not cnt.is_contiguous() or cnt.shape != idx.shape[:2] \
                or cnt.get_device() != dev:
            raise ValueError(f"cnt must be contiguous int32 {tuple(idx.shape[:2])} on cuda:{dev}")
        p.list_heads, p.max_blocks, p.block_size = idx.shape[1], idx.shape[2], block_size
        lists = (idx.data_ptr(), cnt.data_ptr())
    size = 0
    if workspace is None:
        size = _workspace_bytes(p)  # 0: none is needed (or the call below refuses p)
        if size:
            if stream is None:
                workspace = torch.empty(size, dtype=_U8, device=cache.device)
            else:  # with the call's stream current: the memory is not given away before it has run
                with torch.cuda.stream(stream):
                    workspace = torch.empty(size, dtype=_U8, device=cache.device)
    elif workspace.dtype is not _U8 or not workspace.is_contiguous() \
            or workspace.get_device() != dev:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{dev}")
    else:
        size = workspace.numel()
    _call(_attend, "sbsa_kv4_attend", dev, stream, p, cache.data_ptr(), page_table.data_ptr(),
          seq_lens.data_ptr(), cu_new.data_ptr(), q.data_ptr(), *qr, out.data_ptr(), *orow, *lists,
          None if workspace is None else workspace.data_ptr(), size)
    return out


def attend_workspace_bytes(p: Params) -> int:
    """Bytes of the workspace of `attend`; 0 where it needs none (or refuses p)."""
    return _workspace_bytes(p)
