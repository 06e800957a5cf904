"""Python binding of ``include/dspark_attention.h``: the cache side of a verify cycle.

``rotary_append`` rotates each sequence's new tokens and appends their keys and values to the
paged cache; ``block_attention`` attends them over it; ``rotary_frequencies`` makes the
rotary frequencies. As in ``binding.py`` the work runs in the CUDA library: this module checks
layouts, allocates results and workspace with PyTorch, and passes pointers and the current
stream of the tensors' device. The calls are not differentiable.

Rows come in one of two forms: a block ``[B, N, heads, head_dim]`` of which sequence b uses its
first ``n_new[b]`` rows (all N without ``n_new``), the form of ``mixed_accept``'s batch; or
packed rows ``[T, heads, head_dim]`` with ``q_start`` (int32 ``[B+1]``), sequence b's rows being
``q_start[b]`` to ``q_start[b+1] - 1``. Other rows are left as they were.
"""

from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Tuple

import torch

from .binding import DSPARK_OK, DsparkError, load_library

SEQ_BAD_PAGE = 32
CACHE_DTYPES = {torch.bfloat16: 0, torch.float16: 2}
ROTARY_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
# turns in the trained context that bound the ramp of each scaling, where the caller names none
_RAMP = {"yarn": (1.0, 32.0), "bands": (1.0, 4.0)}


class Heads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Rows(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("n_new", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_page_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
                ("max_pages", ctypes.c_int), ("kv_len", ctypes.c_void_p)]


def _lib() -> ctypes.CDLL:
    lib = load_library()
    if getattr(lib, "_cache_side", False):
        return lib
    vp, i32, sz, f32, f64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float,
                             ctypes.c_double)
    lib.dspark_rotary_frequencies.restype = i32
    lib.dspark_rotary_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
    lib.dspark_rotary_append.restype = i32
    lib.dspark_rotary_append.argtypes = [Heads, i32, Heads, Heads, Heads, i32, KvCache, Rows, vp,
                                         i32, i32, f32, vp, vp]
    lib.dspark_block_attention_workspace_bytes.restype = sz
    lib.dspark_block_attention_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.dspark_block_attention.restype = i32
    lib.dspark_block_attention.argtypes = [Heads, i32, Heads, i32, KvCache, Rows, f32, i32, i32,
                                           vp, vp, vp, sz, vp]
    lib.dspark_block_attention_withheld.restype = i32
    lib.dspark_block_attention_withheld.argtypes = lib.dspark_block_attention.argtypes
    lib._cache_side = True
    return lib


# The structs above are filled through `struct` (a tenth of the cost of their constructors: the
# calls on a few tokens are short).
_HEADS, _ROWS, _CACHE = struct.Struct("@Qqqq"), struct.Struct("@iiQQ"), struct.Struct("@QQ6q4iQqiQ")
_pack_heads, _heads_of = _HEADS.pack, Heads.from_buffer_copy
_pack_rows, _rows_of = _ROWS.pack, Rows.from_buffer_copy
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _int32(t: torch.Tensor, n: int, name: str, index: int) -> int:
    if t.dtype is not torch.int32 or t.shape != (n,) or t.get_device() != index or \
            (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on q's device")
    return t.data_ptr()


def _check_rows(q: torch.Tensor, kv_len: torch.Tensor, n_new: Optional[torch.Tensor],
                q_start: Optional[torch.Tensor], index: int) -> Tuple[int, int, int, int]:
    """The fields of Rows; `index` is q's device (-1: the CPU)."""
    if index < 0:
        raise RuntimeError("the cache-side calls run on CUDA tensors only")
    if q.dtype not in CACHE_DTYPES:
        raise ValueError("q must be bfloat16 or float16")
    shape = q.shape
    B = kv_len.shape[0] if kv_len.dim() == 1 else -1
    if q_start is not None:
        if n_new is not None:
            raise ValueError("n_new belongs to a block of rows, q_start to packed ones")
        if len(shape) != 3:
            raise ValueError("with q_start, q must be [T, heads, head_dim]")
        return B, shape[0], 0, _int32(q_start, B + 1, "q_start", index)
    if len(shape) != 4 or shape[0] != B:
        raise ValueError("q must be [B, N, heads, head_dim] (or packed, with q_start)")
    return B, shape[1], 0 if n_new is None else _int32(n_new, B, "n_new", index), 0


def _heads(t: torch.Tensor, shape: torch.Size, dtype: torch.dtype, index: int,
           name: str) -> Heads:
    """The head-row tensor t, of the given shape, element type and device."""
    stride = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or \
            (shape[-1] > 1 and stride[-1] != 1):
        raise ValueError(f"{name} must be {list(shape)} of q's dtype and device, its last "
                         "dimension contiguous")
    return _heads_of(_pack_heads(t.data_ptr(), stride[0] if len(stride) == 4 else 0, stride[-3],
                                 stride[-2]))


def _check_cache(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                 kv_len: torch.Tensor, head_dim: int, dtype: torch.dtype,
                 index: int) -> KvCache:
    shape, ks, vs = k_pages.shape, k_pages.stride(), v_pages.stride()
    if len(shape) != 4 or shape != v_pages.shape or shape[3] != head_dim:
        raise ValueError("k_pages and v_pages must be [pages, page_size, heads, head_dim] with "
                         "q's head_dim")
    if k_pages.dtype is not dtype or v_pages.dtype is not dtype or \
            k_pages.get_device() != index or v_pages.get_device() != index:
        raise ValueError("k_pages and v_pages must have q's dtype and device")
    if shape[3] > 1 and (ks[3] != 1 or vs[3] != 1):
        raise ValueError("the last dimension of the pages must be contiguous")
    B = kv_len.shape[0] if kv_len.dim() == 1 else -1
    kv_ptr = _int32(kv_len, B, "kv_len", index)
    ts, tstr = page_table.shape, page_table.stride()
    if page_table.dtype is not torch.int32 or len(ts) != 2 or ts[0] != B or \
            page_table.get_device() != index or (ts[1] > 1 and tstr[1] != 1):
        raise ValueError("page_table must be an int32 [B, max_pages] tensor on q's device with "
                         "contiguous rows")
    # (a table of one row has no row stride to speak of)
    return KvCache.from_buffer_copy(_CACHE.pack(
        k_pages.data_ptr(), v_pages.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
        *shape, page_table.data_ptr(), tstr[0] if B > 1 else ts[1], ts[1], kv_ptr))


def _run(index: int, fn, what: str, *args) -> None:
    """Call the library on the tensors' device and its current stream."""
    if index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != DSPARK_OK:
        raise DsparkError(rc, what)


def rotary_frequencies(rotary_dim: int, theta: float = 10000.0, *,
                       scaling: Optional[str] = None, factor: float = 1.0,
                       trained: float = 8192.0, low: Optional[float] = None,
                       high: Optional[float] = None) -> Tuple[torch.Tensor, float]:
    """The rotary frequencies (float32 ``[rotary_dim / 2]`` on the CPU) and the magnitude that
    ``rotary_append`` takes.

    ``scaling`` stretches them for contexts ``factor`` times the ``trained`` one: ``"linear"``
    (every frequency divided), ``"ntk"`` (a larger base), ``"yarn"`` (a ramp over the number of
    turns in the trained context, with a magnitude) or ``"bands"`` (low frequencies divided,
    high ones kept, a smooth band between). ``low`` and ``high`` bound the ramp in turns
    (1 and 32 for yarn, 1 and 4 for bands).
    """
    if scaling not in ROTARY_SCALINGS:
        raise ValueError("scaling must be None, 'linear', 'ntk', 'yarn' or 'bands'")
    lo, hi = _RAMP.get(scaling, (1.0, 4.0))
    freq = torch.empty(max(1, int(rotary_dim) // 2), dtype=torch.float32)
    mag = ctypes.c_float(1.0)
    rc = _lib().dspark_rotary_frequencies(
        int(rotary_dim), float(theta), ROTARY_SCALINGS[scaling], float(factor), float(trained),
        lo if low is None else float(low), hi if high is None else float(high),
        freq.data_ptr(), ctypes.addressof(mag))
    if rc != DSPARK_OK:
        raise DsparkError(rc, "dspark_rotary_frequencies")
    return freq, float(mag.value)


def rotary_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                  v_pages: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                  inv_freq: Optional[torch.Tensor], *, n_new: Optional[torch.Tensor] = None,
                  q_start: Optional[torch.Tensor] = None, interleaved: bool = False,
                  magnitude: float = 1.0, out: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate the new tokens' queries and keys and append keys and values to the paged cache.

    ``q`` has the rows of a block or packed rows (see the module), ``k`` and ``v`` the same rows
    with the cache's heads. ``k_pages`` and ``v_pages`` are ``[pages, page_size, heads,
    head_dim]`` (any strides with contiguous head_dim); new token i of sequence b goes to
    position ``kv_len[b] - n + i`` through ``page_table`` (int32 ``[B, max_pages]``): ``kv_len``
    (int32 ``[B]``) counts the new tokens. ``inv_freq`` (float32, on the device) rotates the
    first ``2 len(inv_freq)`` elements of each head, as halves or as ``interleaved`` pairs; None
    rotates nothing. Returns the rotated queries (``out``, which may be ``q``). ``status`` (int32
    ``[B]``) receives SEQ_BAD_PARAM / SEQ_BAD_PAGE bits. Any page_size, head_dim up to 1024 (what
    ``block_attention`` reads has narrower limits).
    """
    lib = _lib()
    index, dtype, shape = q.get_device(), q.dtype, q.shape
    rows = _check_rows(q, kv_len, n_new, q_start, index)
    cache = _check_cache(k_pages, v_pages, page_table, kv_len, shape[-1], dtype, index)
    R, freq = 0, None
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or \
                inv_freq.get_device() != index or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float32 vector on q's device")
        R, freq = 2 * inv_freq.shape[0], inv_freq.data_ptr()
        if R > shape[-1]:
            raise ValueError("inv_freq rotates more elements than a head has")
    st = None if status is None else _int32(status, rows[0], "status", index)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
    kv_shape = torch.Size((*shape[:-2], k_pages.shape[2], shape[-1]))
    _run(index, lib.dspark_rotary_append, "dspark_rotary_append",
         _heads(q, shape, dtype, index, "q"), shape[-2], _heads(out, shape, dtype, index, "out"),
         _heads(k, kv_shape, dtype, index, "k"), _heads(v, kv_shape, dtype, index, "v"),
         CACHE_DTYPES[dtype], cache, _rows_of(_pack_rows(*rows)), freq, R, int(interleaved),
         float(magnitude), st)
    return out


@functools.lru_cache(maxsize=256)
def block_attention_workspace_bytes(N: int, n_q_heads: int, n_heads: int, head_dim: int) -> int:
    """Bytes of workspace that block_attention needs (N: the block's tokens per sequence, or
    all packed ones); 0 for an unsupported shape."""
    return int(_lib().dspark_block_attention_workspace_bytes(N, n_q_heads, n_heads, head_dim))


def block_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    page_table: torch.Tensor, kv_len: torch.Tensor, *,
                    n_new: Optional[torch.Tensor] = None, q_start: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, causal: bool = True,
                    window: Optional[int] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    _withhold: bool = False) -> torch.Tensor:
    """Attention of the new tokens over the paged cache, which already holds their keys.

    ``q`` (a block or packed rows, see the module) is already rotated; query head h reads cache
    head ``h // (heads of q / heads of the cache)``. New token i of sequence b sits at position
    ``p = kv_len[b] - n + i`` and sees the positions below ``kv_len[b]`` that are ``<= p`` when
    ``causal`` (not: the whole block, as a block drafter does) and ``> p - window`` when a
    ``window`` is given. ``scale`` defaults to ``head_dim ** -0.5``. Returns ``out``, q's shape;
    a token that sees nothing gives zeros. head_dim is a multiple of 8 in 16..128, page_size a
    power of two in 8..1024. ``lse`` (float32, q's shape without head_dim) receives the logarithm
    of each row's sum of exponentials, ``status`` (int32 ``[B]``) the SEQ_* bits: SEQ_BAD_PARAM,
    SEQ_BAD_PAGE, and SEQ_TIMEOUT for all sequences of a call that gave up on a wait, whose
    results are incomplete. ``workspace``: at least ``block_attention_workspace_bytes(N, ...)`` bytes; by
    default one is taken from PyTorch's allocator for each call.
    """
    lib = _lib()
    index, dtype, shape = q.get_device(), q.dtype, q.shape
    rows = _check_rows(q, kv_len, n_new, q_start, index)
    cache = _check_cache(k_pages, v_pages, page_table, kv_len, shape[-1], dtype, index)
    Hq, D = shape[-2], shape[-1]
    if window is not None and window < 1:
        raise ValueError("window must be at least 1 (None: no window)")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != shape[:-1] or
                            lse.get_device() != index or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor of q's shape without head_dim")
    st = None if status is None else _int32(status, rows[0], "status", index)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
    if workspace is None:
        nbytes = block_attention_workspace_bytes(rows[1], Hq, k_pages.shape[2], D)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    fn = lib.dspark_block_attention_withheld if _withhold else lib.dspark_block_attention
    _run(index, fn, "dspark_block_attention", _heads(q, shape, dtype, index, "q"), Hq,
         _heads(out, shape, dtype, index, "out"), CACHE_DTYPES[dtype], cache,
         _rows_of(_pack_rows(*rows)), D ** -0.5 if scale is None else float(scale), int(causal),
         0 if window is None else min(int(window), 0x7fffffff),
         None if lse is None else lse.data_ptr(), st, workspace.data_ptr(),
         workspace.numel() * workspace.element_size())
    return out


def block_attention_withheld(*args, **kwargs) -> torch.Tensor:
    """block_attention with the first copy of keys of every CTA withheld, for tests of the timeout
    path only: its waits run out (about a second), the kernel gives up, ``pipeline_timeouts()``
    grows and the result is incomplete."""
    return block_attention(*args, _withhold=True, **kwargs)
