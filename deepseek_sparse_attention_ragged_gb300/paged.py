"""Positions and paged caches: the binding of ``ds_rows_rope``, ``ds_rows_append``,
``ds_rows_fetch``, ``ds_rows_indexer_score_paged``, ``ds_rows_sparse_attn_paged`` and
``ds_rows_prefix_attn``.

A ``Rope`` and a ``PagedCache`` are made once and kept: they hold the tensors that
the library reads and the C structures that describe them. The calls themselves
check tensor types, sizes and devices, and enqueue on the tensors' device.
"""

from __future__ import annotations

import ctypes
from array import array
from operator import add
from typing import Optional

import torch

from . import DIM, DS_OK, HEADS, INDEX_DIM, INDEX_HEADS, _check, load

PAGED_WORKSPACE_BYTES = 256  # DS_PAGED_WORKSPACE_BYTES
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # DS_BF16, DS_F16, DS_F32
_LAYOUTS = {"interleaved": 0, "half": 1}                           # DS_ROPE_*
_FORMATS = {"bf16": 0, "int4": 1, "fp8": 3}                        # DS_CACHE_*
_U32_MAX = 0xFFFFFFFF


class _Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("first", ctypes.c_uint32), ("rot_dim", ctypes.c_uint32),
                ("layout", ctypes.c_int), ("magnitude", ctypes.c_float)]


class _PagedCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("entries", ctypes.c_uint32),
                ("table_stride", ctypes.c_uint32), ("page_size", ctypes.c_uint32), ("num_pages", ctypes.c_uint32),
                ("dim", ctypes.c_uint32), ("format", ctypes.c_int)]


def declare(lib) -> None:
    """The argument types of this module's entry points."""
    vp, sz, i32, u32, u64, f32, f64 = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32,
                                       ctypes.c_uint64, ctypes.c_float, ctypes.c_double)
    rope, cache = ctypes.POINTER(_Rope), ctypes.POINTER(_PagedCache)
    lib.ds_rows_rope_turns.argtypes = [u32, f64, f64, u32, f64, f64, vp]
    lib.ds_rows_rope.argtypes = [rope, vp, u64, u64, vp, u64, u64, i32, u64, u32, u32, vp, i32, vp]
    lib.ds_rows_page_bytes.argtypes = [u32, u32, i32]
    lib.ds_rows_page_bytes.restype = sz
    lib.ds_rows_append.argtypes = [cache, vp, u64, i32, u64, vp, vp, rope, vp, vp, vp, vp]
    lib.ds_rows_fetch.argtypes = [cache, vp, vp, vp, u64, i32, u64, vp, vp]
    lib.ds_rows_indexer_score_paged.argtypes = [i32, vp, cache, vp, vp, vp, sz, vp]
    lib.ds_rows_sparse_attn_paged.argtypes = [i32, vp, cache, vp, vp, sz, vp, f32, vp, vp, vp, sz, vp]
    lib.ds_rows_prefix_attn_workspace_bytes.argtypes = [i32, vp, u32, i32]
    lib.ds_rows_prefix_attn_workspace_bytes.restype = sz
    lib.ds_rows_prefix_attn.argtypes = [i32, vp, u32, cache, vp, vp, sz, f32, vp, vp, vp, sz, vp]
    for f in (lib.ds_rows_rope_turns, lib.ds_rows_rope, lib.ds_rows_append, lib.ds_rows_fetch,
              lib.ds_rows_indexer_score_paged, lib.ds_rows_sparse_attn_paged, lib.ds_rows_prefix_attn):
        f.restype = i32


# ---------------------------------------------------------------------------
# argument checks
# ---------------------------------------------------------------------------

def _tensor(t, name: str, dtype, index: int, numel: int):
    """The address of `t`: a contiguous tensor of `dtype` on CUDA device `index` holding >= numel elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _cuda(t, name: str) -> int:
    """The index of a CUDA tensor's device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


# The current device, and the current stream's handle by device index without building a
# Stream object, where this torch has the calls for it (2 us of a call's host time).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_of(stream, index: int) -> int:
    if stream is None:
        return _current_raw_stream(index)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != index:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{index}")
        return stream.cuda_stream
    return int(stream)


def _call(index: int, fn, *args) -> None:
    """Call an entry point with the tensors' device as the current one."""
    if _current_device() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc != DS_OK:
        _check(load(), rc)


def _workspace_for(device: torch.device, raw_stream: int, size: int = PAGED_WORKSPACE_BYTES) -> torch.Tensor:
    """A workspace for one call on the stream `raw_stream`, taken from that stream's
    memory, so that it is not handed out again while the call still runs."""
    with torch.cuda.stream(torch.cuda.ExternalStream(raw_stream, device=device)):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _u32(value, name: str) -> int:
    """A whole number that a C uint32 holds (ctypes would cut it to 32 bits without a word)."""
    n = int(value)
    if n != value or not 0 <= n <= _U32_MAX:
        raise ValueError(f"{name} must be a whole number in 0 .. 2^32 - 1, got {value}")
    return n


def _code(table, value, name: str) -> int:
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(map(str, table))}, got {value}")
    return code


def _four(kv_len, width, index_offset, q_row):
    return kv_len, width, index_offset, q_row


def _rows(rows):
    """A row table as ds_row_t words, and its columns (kv_len, width, index_offset, q_row)."""
    if not isinstance(rows, (list, tuple)):
        rows = list(rows)
    try:
        try:
            words = array("I", [x for n, w, o, q in rows for x in (n, w, o, q)])  # four fields in every row
        except TypeError:  # Row structures, or objects with their fields
            words = array("I", [x for r in rows for x in
                                ((r.kv_len, r.width, r.index_offset, r.q_row) if hasattr(r, "kv_len") else _four(*r))])
    except (TypeError, ValueError):
        words = None
    if not words:
        raise ValueError("rows must be a nonempty list of (kv_len, width, index_offset, q_row)")
    return words, words[0::4], words[1::4], words[2::4], words[3::4]


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

class Rope:
    """A rotation of elements [first, first + rot_dim) of each row, by angles
    position * theta_i with theta_i = base^(-2 i / rot_dim).

    layout: "interleaved" pairs neighbours, "half" pairs element i with i + rot_dim / 2.
    factor > 1 stretches to longer contexts: linearly, or with original_len (the
    context the model was trained on) by YaRN's ramp between beta_fast and beta_slow
    turns. magnitude multiplies sine and cosine. Made once; `turns` is its table.
    """

    def __init__(self, rot_dim: int, *, first: int = 0, layout: str = "interleaved", base: float = 10000.0,
                 factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 magnitude: float = 1.0, device=None):
        lib = load()
        code = _code(_LAYOUTS, layout, "layout")
        rot_dim, first = _u32(rot_dim, "rot_dim"), _u32(first, "first")
        host = torch.zeros(DIM // 2, dtype=torch.int64)  # the longest table; the library checks rot_dim
        _check(lib, lib.ds_rows_rope_turns(rot_dim, float(base), float(factor), _u32(original_len, "original_len"),
                                           float(beta_fast), float(beta_slow), host.data_ptr()))
        host = host[: rot_dim // 2]
        self.turns = host.to(torch.device(device if device is not None else "cuda"))
        self.device_index = _cuda(self.turns, "the rotation's table")
        self.rot_dim, self.first, self.layout, self.magnitude = rot_dim, first, layout, float(magnitude)
        self._c = _Rope(self.turns.data_ptr(), self.first, self.rot_dim, code, self.magnitude)
        self._ref = ctypes.byref(self._c)


def ds_rows_rope(rope: Rope, x: torch.Tensor, positions: torch.Tensor, out: torch.Tensor, inverse: bool = False,
                 stream=None) -> None:
    """Rotate x [tokens, heads, dim] (or [tokens, dim]) into out; out may be x.

    bf16, fp16 or fp32; any strides whose last is 1 (the rows of out must not
    overlap). positions: int32 [tokens], negative for padding, whose rows of out
    stay as they are. inverse: the transposed rotation, which maps the gradient
    of out to that of x."""
    lib = load()
    dev = _cuda(x, "x")
    if _cuda(out, "out") != dev or rope.device_index != dev:
        raise ValueError(f"x is on {x.device}, out on {out.device} and the rotation on {rope.turns.device}")
    code = _code(_DTYPES, x.dtype, "the type of x")
    shape, xs, os_ = x.shape, x.stride(), out.stride()
    if out.shape != shape or out.dtype != x.dtype:
        raise ValueError("out must have the shape and type of x")
    if len(shape) == 3:
        tokens, heads, dim = shape
        xh, oh = xs[1], os_[1]
    elif len(shape) == 2:
        tokens, dim = shape
        heads, xh, oh = 1, 0, 0
    else:
        raise ValueError(f"x must be [tokens, heads, dim] or [tokens, dim], got {tuple(shape)}")
    if heads > _U32_MAX or dim > _U32_MAX:
        raise ValueError(f"x {tuple(shape)} has more than 2^32 - 1 heads or elements a head")
    if dim > 1 and (xs[-1] != 1 or os_[-1] != 1):
        raise ValueError("the elements of a row of x and out must be contiguous")
    ptr = _tensor(positions, "positions", torch.int32, dev, tokens)
    if tokens == 0 or heads == 0:
        return
    _call(dev, lib.ds_rows_rope, rope._ref, x.data_ptr(), xs[0], xh, out.data_ptr(), os_[0], oh, code, tokens, heads,
          dim, ptr, 1 if inverse else 0, _stream_of(stream, dev))


# ---------------------------------------------------------------------------
# paged caches
# ---------------------------------------------------------------------------

def ds_rows_page_bytes(page_size: int, dim: int, fmt: str) -> int:
    """Bytes of one page of `page_size` rows of `dim` (128 or 512) elements held as "bf16", "fp8" or "int4"."""
    lib = load()
    n = lib.ds_rows_page_bytes(_u32(page_size, "page_size"), _u32(dim, "dim"),
                               _code(_FORMATS, fmt, "the cache's format"))
    if n == 0:
        _check(lib, -1)
    return int(n)


class PagedCache:
    """A pool of pages and the page table of its entries (sequences).

    pages: a contiguous tensor of whole pages (any element type);
    page_table: int32 [entries, pages per entry], read by the device at each call,
    so it may be updated in place. Made once per pool; the tensors stay the same."""

    def __init__(self, pages: torch.Tensor, page_table: torch.Tensor, page_size: int, dim: int, fmt: str):
        size = ds_rows_page_bytes(page_size, dim, fmt)
        self.device_index = _cuda(pages, "pages")
        if not pages.is_contiguous():
            raise ValueError("pages must be contiguous")
        total = pages.numel() * pages.element_size()
        if total == 0 or total % size:
            raise ValueError(f"pages holds {total} bytes, not a whole number of {size}-byte pages")
        if page_table.dim() != 2 or page_table.numel() == 0:
            raise ValueError("page_table must be [entries, pages per entry]")
        _tensor(page_table, "page_table", torch.int32, self.device_index, 1)
        self.pages, self.page_table = pages, page_table
        self.page_size, self.dim, self.format, self.num_pages = int(page_size), int(dim), fmt, total // size
        entries, per_entry = (_u32(n, "a side of page_table") for n in page_table.shape)
        self._c = _PagedCache(pages.data_ptr(), page_table.data_ptr(), entries, per_entry, self.page_size,
                              self.num_pages, self.dim, _FORMATS[fmt])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_pages: int, page_table: torch.Tensor, page_size: int, dim: int, fmt: str) -> "PagedCache":
        """A cache over a new pool of `num_pages` pages on the page table's device."""
        size = ds_rows_page_bytes(page_size, dim, fmt)
        return cls(torch.zeros(num_pages, size, dtype=torch.uint8, device=page_table.device), page_table, page_size,
                   dim, fmt)


def ds_rows_append(cache: PagedCache, x: torch.Tensor, seq: torch.Tensor, slot: torch.Tensor,
                   rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                   values: Optional[torch.Tensor] = None, invalid: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Append row i of x [tokens, dim] as row slot[i] of entry seq[i] (-1: padding),
    rotated at positions[i] with `rope`, rounded to the cache's type.

    x: bf16, fp16 or fp32, its rows contiguous; seq, slot, positions: int32 [tokens].
    values (optional, bf16 [tokens, dim]) receives the rows as the cache now holds
    them; invalid (optional, int32 [tokens]) 1 where a row could not be written."""
    lib = load()
    dev = _cuda(x, "x")
    if cache.device_index != dev or (rope is not None and rope.device_index != dev):
        raise ValueError(f"x is on {x.device}, the cache on {cache.pages.device}"
                         + (f", the rotation on {rope.turns.device}" if rope is not None else ""))
    if x.dim() != 2 or x.shape[1] != cache.dim:
        raise ValueError(f"x must be [tokens, {cache.dim}], got {tuple(x.shape)}")
    row, element = x.stride()
    if element != 1 and x.shape[0]:  # no tokens: any strides (numpy's are 0)
        raise ValueError("the elements of a row of x must be contiguous")
    code = _code(_DTYPES, x.dtype, "the type of x")
    n = x.shape[0]
    i32 = torch.int32
    ps, pl = _tensor(seq, "seq", i32, dev, n), _tensor(slot, "slot", i32, dev, n)
    pp = _tensor(positions, "positions", i32, dev, n) if rope is not None else None
    pv = None if values is None else _tensor(values, "values", torch.bfloat16, dev, n * cache.dim)
    pi = None if invalid is None else _tensor(invalid, "invalid", i32, dev, n)
    if n == 0:
        return
    _call(dev, lib.ds_rows_append, cache._ref, x.data_ptr(), row if n > 1 else 0, code, n, ps, pl,
          None if rope is None else rope._ref, pp, pv, pi, _stream_of(stream, dev))


def ds_rows_fetch(cache: PagedCache, seq: torch.Tensor, slot: torch.Tensor, out: torch.Tensor,
                  invalid: Optional[torch.Tensor] = None, stream=None) -> None:
    """Read row slot[i] of entry seq[i] (-1: padding, left as it is) back into row i of out
    [tokens, dim]: bf16, fp16 or fp32, its rows contiguous. seq, slot: int32 [tokens].
    invalid (optional, int32 [tokens]) receives 1 where there is no such row; out is NaN there."""
    lib = load()
    dev = _cuda(out, "out")
    if cache.device_index != dev:
        raise ValueError(f"out is on {out.device}, the cache on {cache.pages.device}")
    if out.dim() != 2 or out.shape[1] != cache.dim:
        raise ValueError(f"out must be [tokens, {cache.dim}], got {tuple(out.shape)}")
    row, element = out.stride()
    if element != 1 and out.shape[0]:
        raise ValueError("the elements of a row of out must be contiguous")
    code = _code(_DTYPES, out.dtype, "the type of out")
    n = out.shape[0]
    ps, pl = _tensor(seq, "seq", torch.int32, dev, n), _tensor(slot, "slot", torch.int32, dev, n)
    pi = None if invalid is None else _tensor(invalid, "invalid", torch.int32, dev, n)
    if n == 0:
        return
    _call(dev, lib.ds_rows_fetch, cache._ref, ps, pl, out.data_ptr(), row, code, n, pi, _stream_of(stream, dev))


def ds_rows_indexer_score_paged(rows, q_index: torch.Tensor, w_index: torch.Tensor, keys: PagedCache,
                                scores: torch.Tensor, score_stride: Optional[int] = None, stream=None) -> None:
    """ds_rows_indexer_score with entry e's keys in entry e of a paged cache (dim 128)."""
    lib = load()
    dev = keys.device_index
    words, kv_len, _, _, q_row = _rows(rows)
    n, q_rows = len(kv_len), max(q_row) + 1
    if score_stride is None:
        score_stride = scores.shape[-1] if scores.dim() > 1 else max(kv_len)
    elif score_stride < 0:
        raise ValueError(f"score_stride must not be negative, got {score_stride}")
    pq = _tensor(q_index, "q_index", torch.bfloat16, dev, q_rows * INDEX_HEADS * INDEX_DIM)
    pw = _tensor(w_index, "w_index", torch.float32, dev, q_rows * INDEX_HEADS)
    po = _tensor(scores, "scores", torch.float32, dev, (n - 1) * score_stride + kv_len[-1])
    _call(dev, lib.ds_rows_indexer_score_paged, n, words.buffer_info()[0], keys._ref, pq, pw, po, score_stride,
          _stream_of(stream, dev))


def ds_rows_sparse_attn_paged(rows, q_attn: torch.Tensor, sinks: torch.Tensor, sinks_row_stride: int,
                              indices: torch.Tensor, scale: float, out: torch.Tensor, kv: PagedCache,
                              invalid: Optional[torch.Tensor] = None, workspace_t: Optional[torch.Tensor] = None,
                              stream=None) -> None:
    """ds_rows_sparse_attn with entry e's KV rows in entry e of a paged cache (dim 512).
    workspace_t (optional): any workspace of at least PAGED_WORKSPACE_BYTES; it holds the
    call's status word."""
    lib = load()
    dev = kv.device_index
    words, kv_len, width, offset, q_row = _rows(rows)
    n, q_rows = len(kv_len), max(q_row) + 1
    if sinks_row_stride < 0:
        raise ValueError(f"sinks_row_stride must not be negative, got {sinks_row_stride}")
    bf16 = torch.bfloat16
    pq = _tensor(q_attn, "q_attn", bf16, dev, q_rows * HEADS * DIM)
    po = _tensor(out, "out", bf16, dev, q_rows * HEADS * DIM)
    ps = _tensor(sinks, "sinks", torch.float32, dev,
                 HEADS if sinks_row_stride == 0 else (q_rows - 1) * sinks_row_stride + HEADS)
    px = _tensor(indices, "indices", torch.int32, dev, max(map(add, offset, width)))
    pi = None if invalid is None else _tensor(invalid, "invalid", torch.int32, dev, q_rows * HEADS)
    raw = _stream_of(stream, dev)
    if workspace_t is None:
        workspace_t = _workspace_for(kv.pages.device, raw)
    pw = _tensor(workspace_t, "workspace", torch.uint8, dev, 0)
    _call(dev, lib.ds_rows_sparse_attn_paged, n, words.buffer_info()[0], kv._ref, pq, ps, sinks_row_stride, px, scale,
          po, pi, pw, workspace_t.numel(), raw)


# ---------------------------------------------------------------------------
# attention over a shared prefix
# ---------------------------------------------------------------------------

def ds_rows_prefix_attn_workspace_bytes(rows, prefix_len: int, fmt: Optional[str] = None) -> int:
    """Workspace bytes that ds_rows_prefix_attn uses for these rows over a cache of `fmt` (None: of any)."""
    return _prefix_bytes(_rows(rows)[0], _u32(prefix_len, "prefix_len"),
                         -1 if fmt is None else _code(_FORMATS, fmt, "the cache's format"))


def _prefix_bytes(words, prefix_len: int, code: int) -> int:
    lib = load()
    n = lib.ds_rows_prefix_attn_workspace_bytes(len(words) // 4, words.buffer_info()[0], prefix_len, code)
    if n == 0:
        _check(lib, -1)
    return int(n)


def prefix_attn_workspace(rows, prefix_len: int, fmt: Optional[str] = None, device=None) -> torch.Tensor:
    """A workspace tensor for ds_rows_prefix_attn over a cache of `fmt`, or of any (uint8, 256-byte aligned by
    the caching allocator)."""
    return torch.empty(ds_rows_prefix_attn_workspace_bytes(rows, prefix_len, fmt), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def ds_rows_prefix_attn(rows, prefix_len: int, q_attn: torch.Tensor, sinks: torch.Tensor, sinks_row_stride: int,
                        scale: float, out: torch.Tensor, kv: PagedCache, invalid: Optional[torch.Tensor] = None,
                        workspace_t: Optional[torch.Tensor] = None, stream=None) -> None:
    """Sink-softmax attention of up to 64 rows over all their cached rows (dim 512): slots below
    prefix_len are those of entry 0 for every row, the others entry e's own.

    rows: (kv_len, width, index_offset, q_row) as elsewhere; width and index_offset are not
    looked at. workspace_t (optional): prefix_attn_workspace(rows, prefix_len, kv.format) or a larger one."""
    lib = load()
    dev = kv.device_index
    words, kv_len, _, _, q_row = _rows(rows)
    n, q_rows, prefix_len = len(kv_len), max(q_row) + 1, _u32(prefix_len, "prefix_len")
    if sinks_row_stride < 0:
        raise ValueError(f"sinks_row_stride must not be negative, got {sinks_row_stride}")
    pq = _tensor(q_attn, "q_attn", torch.bfloat16, dev, q_rows * HEADS * DIM)
    po = _tensor(out, "out", torch.bfloat16, dev, q_rows * HEADS * DIM)
    ps = _tensor(sinks, "sinks", torch.float32, dev,
                 HEADS if sinks_row_stride == 0 else (q_rows - 1) * sinks_row_stride + HEADS)
    pi = None if invalid is None else _tensor(invalid, "invalid", torch.int32, dev, q_rows * HEADS)
    raw = _stream_of(stream, dev)
    if workspace_t is None:
        workspace_t = _workspace_for(kv.pages.device, raw, _prefix_bytes(words, prefix_len, kv._c.format))
    pw = _tensor(workspace_t, "workspace", torch.uint8, dev, 0)
    _call(dev, lib.ds_rows_prefix_attn, n, words.buffer_info()[0], prefix_len, kv._ref, pq, ps, sinks_row_stride, scale,
          po, pi, pw, workspace_t.numel(), raw)
