"""Rotary positions and paged caches without a GPU: the oracle's own pins, the
rotation's table, page sizes, and every refusal of the C entry points (fake,
aligned pointers: validation fails before any of them is used)."""

import ctypes

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from deepseek_sparse_attention_ragged_gb300 import paged
from oracle import paged as ref

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.load()


def _err(lib):
    return lib.ds_rows_last_error().decode()


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def test_e4m3_rounds_as_torch_does():
    x = np.concatenate([ref.E4M3, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2,
                        np.random.default_rng(0).uniform(0, 448, 4000)]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.e4m3_byte(x), want)
    assert ref.e4m3_byte(np.float32(1e9)) == 0x7E and ref.E4M3[-1] == 448


@pytest.mark.parametrize("dim,page", [(128, 16), (128, 256), (512, 32)])
def test_int4_pages_round_trip(dim, page):
    rng = np.random.default_rng(dim + page)
    n, s = ref.int4_quantise(rng.standard_normal((page, dim)).astype(np.float32))
    data = np.zeros(ds.ds_rows_page_bytes(page, dim, "int4"), np.uint8)
    ref.write_int4_page(data, dim, page, n, s)
    n2, s2 = ref.read_int4_page(data, dim, page)
    np.testing.assert_array_equal(n, n2)
    np.testing.assert_array_equal(s, s2)
    # Every byte of the page belongs to exactly one row.
    v, sc = ref.row_places(dim, page)
    assert np.array_equal(np.sort(np.concatenate([v.ravel(), sc.ravel()])), np.arange(len(data)))


def test_int4_values_are_exact_in_bf16():
    n = np.arange(-7, 8)[:, None] * np.ones((1, 127))
    v = torch.from_numpy((n * ref.E4M3).astype(np.float32))
    assert torch.equal(v.to(torch.bfloat16).float(), v) and torch.equal(v.to(torch.float16).float(), v)


def test_rope_oracle_is_a_rotation_and_its_transpose():
    rng = np.random.default_rng(3)
    theta = ref.frequencies(64, factor=8.0, original_len=4096)
    x, g = rng.standard_normal((2, 5, 3, 128))
    pos = np.array([0, 1, 77, 100000, 2 ** 31 - 1])
    y = ref.rope(x, pos, theta, 32, "half", 1.3)
    # <g, R x> = <R^T g, x>, and the norm grows by the magnitude on the rotated half.
    back = ref.rope(g, pos, theta, 32, "half", 1.3, inverse=True)
    np.testing.assert_allclose((g * y).sum(), (back * x).sum(), rtol=1e-12)
    np.testing.assert_allclose(np.linalg.norm(y[..., 32:96]), 1.3 * np.linalg.norm(x[..., 32:96]), rtol=1e-12)
    np.testing.assert_array_equal(y[..., :32], x[..., :32])


# ---------------------------------------------------------------------------
# the rotation's table
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rot,base,factor,original,fast,slow", [
    (64, 10000.0, 1.0, 0, 32.0, 1.0), (128, 10000.0, 4.0, 0, 32.0, 1.0), (64, 10000.0, 16.0, 65536, 32.0, 1.0),
    (2, 10000.0, 40.0, 4096, 32.0, 1.0), (512, 500000.0, 8.0, 8192, 4.0, 1.0), (6, 2.0, 2.0, 17, 1.0, 1.0),
])
def test_turns(lib, rot, base, factor, original, fast, slow):
    t = np.zeros(rot // 2, np.uint64)
    assert lib.ds_rows_rope_turns(rot, base, factor, original, fast, slow, t.ctypes.data) == 0, _err(lib)
    want = ref.frequencies(rot, base, factor, original, fast, slow) / (2 * np.pi)
    # Both sides round in 64 bits: pow, two products and a sum, 2^-52 each; the table is
    # in steps of 2^-64, so it lies up to half a step off (the small angles' error).
    np.testing.assert_allclose(t.astype(np.float64) / 2.0 ** 64, want, rtol=8 * 2.0 ** -52, atol=2.0 ** -65)


@pytest.mark.parametrize("args,msg", [
    ((0, 1e4, 1.0, 0, 32.0, 1.0), "rot_dim"), ((7, 1e4, 1.0, 0, 32.0, 1.0), "rot_dim"),
    ((514, 1e4, 1.0, 0, 32.0, 1.0), "rot_dim"), ((64, 1.0, 1.0, 0, 32.0, 1.0), "base"),
    ((64, float("nan"), 1.0, 0, 32.0, 1.0), "base"), ((64, 1e4, 0.5, 0, 32.0, 1.0), "factor"),
    ((64, 1e4, float("inf"), 0, 32.0, 1.0), "factor"), ((64, 1e4, 2.0, 4096, 1.0, 2.0), "beta"),
    ((64, 1e4, 2.0, 4096, 1.0, 0.0), "beta"), ((64, 1e4, 2.0, 4096, float("nan"), 1.0), "beta"),
])
def test_turns_refusals(lib, args, msg):
    t = np.zeros(256, np.uint64)
    assert lib.ds_rows_rope_turns(*args, t.ctypes.data) == -1 and msg in _err(lib)


def test_turns_null(lib):
    assert lib.ds_rows_rope_turns(64, 1e4, 1.0, 0, 32.0, 1.0, None) == -1 and "NULL" in _err(lib)


# ---------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------

def _rope(lib, turns=FAKE, first=0, rot=64, layout=0, mag=1.0, x=FAKE, xs=(512, 64), out=FAKE + (1 << 30),
          os_=(512, 64), dtype=0, tokens=4, heads=8, dim=64, positions=FAKE, null=False):
    r = paged._Rope(turns, first, rot, layout, mag)
    return lib.ds_rows_rope(None if null else ctypes.byref(r), x, *xs, out, *os_, dtype, tokens, heads, dim, positions,
                            0, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(null=True), -1, "non-NULL"), (dict(turns=None), -1, "non-NULL"), (dict(turns=FAKE + 4), -3, "8-B"),
    (dict(layout=2), -1, "layout"), (dict(rot=63), -1, "rot_dim"), (dict(rot=0), -1, "rot_dim"),
    (dict(first=2), -1, "exceeds the row"), (dict(first=0xFFFFFFFE), -1, "exceeds the row"),
    (dict(first=1, rot=2), -1, "even element"), (dict(mag=0.0), -1, "magnitude"),
    (dict(mag=float("inf")), -1, "magnitude"), (dict(mag=float("nan")), -1, "magnitude"),
    (dict(positions=None), -1, "positions"), (dict(positions=FAKE + 2), -3, "positions"),
    (dict(x=None), -1, "non-NULL"), (dict(out=None), -1, "non-NULL"), (dict(x=FAKE + 1), -3, "element type"),
    (dict(out=FAKE + 2, dtype=2), -3, "element type"), (dict(dtype=3), -1, "dtype"), (dict(dim=0), -1, "dim"),
    (dict(dim=1025), -1, "dim"), (dict(heads=0), -1, "heads"), (dict(heads=65537), -1, "heads"),
    (dict(tokens=1 << 28), -2, "below 2^31"), (dict(xs=(1 << 40, 64)), -2, "stride"),
    (dict(os_=(512, 63)), -1, "overlap"), (dict(os_=(511, 64)), -1, "overlap"), (dict(os_=(0, 64)), -1, "overlap"),
    (dict(out=FAKE, os_=(1024, 64)), -1, "in place"), (dict(out=FAKE, os_=(512, 128)), -1, "in place"),
])
def test_rope_refusals(lib, kw, code, msg):
    assert _rope(lib, **kw) == code
    assert msg in _err(lib)


def test_rope_accepts_both_nestings_and_no_tokens(lib):
    # No tokens: checked, nothing enqueued (so no device is needed).
    assert _rope(lib, tokens=0) == 0
    assert _rope(lib, tokens=0, os_=(64, 256)) == 0
    # Heads outside tokens: the head stride spans the tokens.
    assert _rope(lib, os_=(64, 255)) == -1 and "overlap" in _err(lib)


# ---------------------------------------------------------------------------
# pages and append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("page,dim,fmt,size", [
    (16, 128, "int4", 1152), (64, 512, "int4", 18432), (256, 512, "bf16", 262144), (128, 128, "bf16", 32768)])
def test_page_bytes(page, dim, fmt, size):
    assert ds.ds_rows_page_bytes(page, dim, fmt) == size


@pytest.mark.parametrize("page,dim,fmt,msg", [(0, 128, 0, "page_size"), (8, 128, 0, "page_size"),
                                              (48, 128, 0, "page_size"), (512, 128, 0, "page_size"),
                                              (64, 64, 0, "wide"), (64, 512, 2, "format")])
def test_page_bytes_refusals(lib, page, dim, fmt, msg):
    assert lib.ds_rows_page_bytes(page, dim, fmt) == 0 and msg in _err(lib)


def _cache(pages=FAKE, table=FAKE, entries=8, stride=64, page=64, num=1000, dim=512, fmt=1):
    return paged._PagedCache(pages, table, entries, stride, page, num, dim, fmt)


BAD_CACHES = [
    (dict(pages=None), -1, "non-NULL"), (dict(table=None), -1, "non-NULL"), (dict(pages=FAKE + 8), -3, "16-B"),
    (dict(table=FAKE + 2), -3, "4-B"), (dict(entries=0), -1, "nonzero"), (dict(stride=0), -1, "nonzero"),
    (dict(num=0), -1, "nonzero"), (dict(page=65), -1, "page_size"), (dict(fmt=7), -1, "format"),
    (dict(dim=256), -1, "wide"), (dict(num=1 << 26), -2, "2^31"),
]


def _append(lib, cache=None, x=FAKE, xs=512, dtype=0, tokens=4, seq=FAKE, slot=FAKE, rope=None, positions=None,
            values=None, invalid=None, null=False):
    c = _cache() if cache is None else cache
    return lib.ds_rows_append(None if null else ctypes.byref(c), x, xs, dtype, tokens, seq, slot,
                              None if rope is None else ctypes.byref(rope), positions, values, invalid, None)


@pytest.mark.parametrize("kw,code,msg", BAD_CACHES)
def test_append_cache_refusals(lib, kw, code, msg):
    assert _append(lib, _cache(**kw)) == code and msg in _err(lib)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(null=True), -1, "NULL"), (dict(x=None), -1, "non-NULL"), (dict(x=FAKE + 1), -3, "element type"),
    (dict(dtype=-1), -1, "dtype"), (dict(tokens=1 << 31), -2, "below 2^31"), (dict(xs=1 << 40), -2, "x_stride"),
    (dict(seq=None), -1, "seq and slot"), (dict(slot=None), -1, "seq and slot"), (dict(seq=FAKE + 1), -3, "4-B"),
    (dict(slot=FAKE + 2), -3, "4-B"), (dict(values=FAKE + 8), -3, "values"), (dict(invalid=FAKE + 2), -3, "4-B"),
    (dict(rope=paged._Rope(FAKE, 449, 64, 1, 1.0), positions=FAKE), -1, "exceeds the row"),
    (dict(rope=paged._Rope(FAKE, 448, 64, 0, 1.0)), -1, "positions"),
    (dict(rope=paged._Rope(FAKE, 448, 64, 0, 1.0), positions=FAKE + 1), -3, "4-B"),
])
def test_append_refusals(lib, kw, code, msg):
    assert _append(lib, **kw) == code and msg in _err(lib)


def test_append_of_nothing(lib):
    assert _append(lib, tokens=0) == 0


# ---------------------------------------------------------------------------
# reads
# ---------------------------------------------------------------------------

def _scores(lib, rows=((600, 512, 0, 0),), cache=None, q=FAKE, w=FAKE, out=FAKE, stride=None):
    tab, n = ds._table(rows)
    c = _cache(dim=128) if cache is None else cache
    return lib.ds_rows_indexer_score_paged(n, tab, ctypes.byref(c), q, w, out,
                                           max(r[0] for r in rows) if stride is None else stride, None)


def _attn(lib, rows=((600, 512, 0, 0),), cache=None, q=FAKE, sinks=FAKE, stride=0, idx=FAKE, scale=0.04, out=FAKE,
          ws=FAKE, ws_bytes=1 << 30):
    tab, n = ds._table(rows)
    c = _cache() if cache is None else cache
    return lib.ds_rows_sparse_attn_paged(n, tab, ctypes.byref(c), q, sinks, stride, idx, scale, out, None, ws, ws_bytes,
                                         None)


@pytest.mark.parametrize("kw,code,msg", BAD_CACHES)
def test_read_cache_refusals(lib, kw, code, msg):
    assert _scores(lib, cache=_cache(**{"dim": 128, **kw})) == code and msg in _err(lib)
    assert _attn(lib, cache=_cache(**kw)) == code and msg in _err(lib)


def test_reads_need_the_right_width(lib):
    assert _scores(lib, cache=_cache(dim=512)) == -1 and "128 wide" in _err(lib)
    assert _attn(lib, cache=_cache(dim=128)) == -1 and "512 wide" in _err(lib)


def test_reads_need_entries_and_reach(lib):
    rows = [(10, 10, 16 * e, e) for e in range(8)]
    for call, dim in ((_scores, 128), (_attn, 512)):
        assert call(lib, rows, cache=_cache(dim=dim, entries=7)) == -1 and "7 entries for 8 rows" in _err(lib)
        # 64 pages of 64 rows hold 4096.
        assert call(lib, [(4097, 512, 0, 0)], cache=_cache(dim=dim)) == -1 and "exceeds the 64 pages" in _err(lib)
        huge = _cache(dim=dim, stride=0xFFFFFFFF)
        assert call(lib, [(1 << 31, 512, 0, 0)], cache=huge) == -2 and "below 2^31" in _err(lib)
        assert call(lib, [(0, 1, 0, 0)], cache=_cache(dim=dim)) == -1 and "nonzero" in _err(lib)
        assert call(lib, rows + rows, cache=_cache(dim=dim)) == -1 and "rows must be 1..=8" in _err(lib)


def test_score_refusals(lib):
    assert _scores(lib, q=None) == -1 and "q_index" in _err(lib)
    assert _scores(lib, q=FAKE + 8) == -3
    assert _scores(lib, w=None) == -1
    assert _scores(lib, out=None) == -1 and "scores is NULL" in _err(lib)
    assert _scores(lib, stride=599) == -1 and "score_stride" in _err(lib)


def test_attention_refusals(lib):
    assert _attn(lib, q=FAKE + 2) == -3
    assert _attn(lib, idx=None) == -1 and "indices" in _err(lib)
    assert _attn(lib, sinks=None) == -1
    assert _attn(lib, stride=63) == -1 and "sinks_row_stride" in _err(lib)
    for scale in (0.0, float("nan"), float("inf")):
        assert _attn(lib, scale=scale) == -1 and "scale" in _err(lib)
    assert _attn(lib, [(8, 8, 0, 3), (9, 9, 8, 3)]) == -1 and "used twice" in _err(lib)
    assert _attn(lib, ws_bytes=ds.PAGED_WORKSPACE_BYTES - 1) == -2 and "workspace holds" in _err(lib)
    assert _attn(lib, ws=FAKE + 16) == -3 and _attn(lib, ws=None) == -1


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        ds.PagedCache(torch.zeros(18432, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32), 64, 512, "int4")
    with pytest.raises(ValueError, match="one of"):
        ds.ds_rows_page_bytes(64, 512, "fp4")
    with pytest.raises(ValueError, match="layout"):
        ds.Rope(64, layout="neox", device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ds.Rope(64, device="cpu")
    with pytest.raises(ds.DsRowsError, match="rot_dim"):
        ds.Rope(63, device="cpu")


def test_row_tables_of_every_kind():
    want = [(600, 512, 0, 0), (7, 7, 512, 3)]
    for rows in (want, tuple(want), iter(want), [ds.Row(*r) for r in want], (ds.Row(*r) for r in want),
                 [list(r) for r in want]):
        words, *columns = paged._rows(rows)
        assert list(zip(*columns)) == want and len(words) == 8
    for bad in ([], [(1, 2), (3, 4)], [(1, 2, 3)], [(1, 2, 3, 4, 5)]):
        with pytest.raises(ValueError, match="nonempty list"):
            paged._rows(bad)
    with pytest.raises(OverflowError):
        paged._rows([(-1, 1, 0, 0)])
