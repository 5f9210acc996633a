"""Refusals and sizes of ds_rows_prefix_attn without a GPU (fake, aligned pointers: validation
fails before any of them is used)."""

import ctypes

import numpy as np
import pytest

import deepseek_sparse_attention_ragged_gb300 as ds
from test_paged_host import BAD_CACHES, FAKE, _cache, _err


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.load()


def _attn(lib, rows=((600, 1, 0, 0),), prefix=0, cache=None, q=FAKE, sinks=FAKE, stride=0, scale=0.04, out=FAKE,
          invalid=None, ws=FAKE, ws_bytes=1 << 30, table=True):
    tab, n = ds._table(rows)
    c = _cache() if cache is None else cache
    return lib.ds_rows_prefix_attn(n, tab if table else None, prefix, ctypes.byref(c), q, sinks, stride, scale, out, invalid,
                                   ws, ws_bytes, None)


@pytest.mark.parametrize("fmt", [0, 1, 3])
@pytest.mark.parametrize("kw,code,msg", [b for b in BAD_CACHES if "fmt" not in b[0]])
def test_cache_refusals(lib, fmt, kw, code, msg):
    assert _attn(lib, cache=_cache(fmt=fmt, **kw)) == code and msg in _err(lib)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(rows=[]), -1, "rows must be 1..=64"), (dict(rows=[(5, 1, 0, i) for i in range(65)]), -1, "rows must be 1..=64"),
    (dict(table=False), -1, "NULL"), (dict(rows=[(0, 1, 0, 0)]), -1, "nonzero"),
    (dict(rows=[(1 << 31, 1, 0, 0)], cache=_cache(stride=0xFFFFFFFF)), -2, "below 2^31"),
    (dict(rows=[(600, 1, 0, 0), (599, 1, 0, 1)], prefix=600), -1, "row 1: kv_len 599 is shorter than the prefix"),
    (dict(rows=[(6, 1, 0, 3), (7, 1, 0, 2), (8, 1, 0, 3)]), -1, "used twice"),
    (dict(rows=[(6, 1, 0, 0xFFFFFFFF)]), -2, "out of range"),
    (dict(rows=[(6, 1, 0, i) for i in range(9)]), -1, "8 entries for 9 rows"),
    (dict(rows=[(4097, 1, 0, 0)]), -1, "exceeds the 64 pages"), (dict(cache=_cache(dim=128)), -1, "512 wide"),
    (dict(cache=_cache(fmt=2)), -1, "format"),
    (dict(q=None), -1, "non-NULL"), (dict(q=FAKE + 8), -3, "16-B"), (dict(out=FAKE + 2), -3, "16-B"),
    (dict(out=None), -1, "non-NULL"), (dict(sinks=None), -1, "non-NULL"), (dict(sinks=FAKE + 2), -3, "4-B"),
    (dict(invalid=FAKE + 1), -3, "4-B"), (dict(stride=63), -1, "sinks_row_stride"), (dict(scale=0.0), -1, "scale"),
    (dict(scale=float("nan")), -1, "scale"), (dict(scale=float("inf")), -1, "scale"), (dict(scale=-1.0), -1, "scale"),
    (dict(ws=None), -1, "workspace"), (dict(ws=FAKE + 16), -3, "256-byte"), (dict(ws_bytes=1000), -2, "workspace holds"),
])
def test_refusals(lib, kw, code, msg):
    assert _attn(lib, **kw) == code and msg in _err(lib)


def test_width_and_index_offset_are_not_looked_at(lib):
    """The rows pass every check (the workspace, checked last, does not)."""
    assert _attn(lib, rows=[(6, 0, 0xFFFFFFFF, 0), (7, 0xFFFFFFFF, 0xFFFFFFFF, 1)], ws_bytes=0) == -2


def test_workspace_bytes(lib):
    part = 2 * 4 * (5 * 64 + 64 * 512)
    size = ds.ds_rows_prefix_attn_workspace_bytes
    assert size([(1, 1, 0, 0)], 0) >= 256 + part
    # The longest and most rows need no more than a part for every pair of processors and every segment.
    long = [((1 << 31) - 1, 1, 0, i) for i in range(64)], (1 << 31) - 200
    assert size(*long, "bf16") <= 512 + (76 + 96) * part
    # Packed rows that many entries share are also held as bf16, a kilobyte each, in whole tiles.
    shared = [(5000 + i, 1, 0, i) for i in range(6)], 5000
    for fmt in ("fp8", "int4", None):
        assert size(*shared, fmt) == size(*shared, "bf16") + (40 + 5) * 128 * 1024
        assert size([(1000, 1, 0, 0), (1001, 1, 0, 1)], 1000, fmt) == size([(1000, 1, 0, 0), (1001, 1, 0, 1)], 1000, "bf16")
    with pytest.raises(ValueError, match="one of"):
        size(*shared, "fp4")
    tab, n = ds._table([(5, 1, 0, 0)])
    assert lib.ds_rows_prefix_attn_workspace_bytes(n, tab, 5, 2) == 0 and "format" in _err(lib)
    assert size(iter([(9, 1, 0, 0)]), np.int64(9)) == size([(9, 1, 0, 0)], 9)
    for rows, prefix in (([], 0), ([(5, 1, 0, 0)], 6), ([(5, 1, 0, 0)] * 2, 0)):
        with pytest.raises((ValueError, ds.DsRowsError)):
            size(rows, prefix)
    for prefix in (-1, 0.5, 1 << 32):
        with pytest.raises(ValueError, match="whole number"):
            size([(5, 1, 0, 0)], prefix)
    tab, n = ds._table([(600, 1, 0, 0)])
    need = lib.ds_rows_prefix_attn_workspace_bytes(n, tab, 500, 1)
    assert _attn(lib, prefix=500, ws_bytes=need - 1) == -2 and f"needs {need}" in _err(lib)


def test_most_rows_match_the_header():
    assert ds.PREFIX_ROWS_MAX == 64
