"""GPU parity of the 8-bit pages and of ds_rows_fetch with the float64 oracle.

Tolerances: a fetched row is what the pages' bytes spell (exact in bf16 and fp32, one
rounding in fp16). An appended row without a rotation is exact; with one, the rotation's
bound (5e-7 of m (|a| + |b|), derived beside its own tests) comes on top of the type's half
step: 2^-4 of the value, or 2^-10 2^e below e4m3's normal numbers, where e is the
block's exponent (448 2^(e-1) < max, so 2^e < max / 224). Scores and attention carry the bits of
the contiguous calls; the scores' bound is the one derived beside the paged tests, and the
attention's output is a mean of rows, rounded to bf16: half a step of the largest value, and as
much again for its weights' and sums' roundings.
"""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
import oracle
from oracle import paged as ref
from parity import score_bound
from test_gpu_paged import (BF16, F32, ROPE_RTOL, SCALE, SCORE_RTOL, TYPES, attend, edge_rows, f64, i32, page_table, queries,
                            row_table)
from test_gpu_paged import make_cache as make_cache_4

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "fp8", "int4"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ds.build()
    ds.load()


def make_cache(rng, lens, dim, fmt, page, scale=1.0):
    """A cache whose entries hold random rows; returns it with the rows' values (float32, exact in bf16)."""
    if fmt != "fp8":
        return make_cache_4(rng, lens, dim, fmt, page, scale)
    table, total = page_table(rng, lens, page)
    pool = rng.integers(0, 256, (total, ds.ds_rows_page_bytes(page, dim, fmt)), dtype=np.uint8)
    v, sc = ref.fp8_places(dim, page)
    y = scale * rng.standard_normal((total * page, dim)) * np.exp(rng.uniform(-3, 3, (total * page, 1)))
    byte, ex = ref.fp8_quantise(y.astype(np.float32))
    pool_rows = ref.fp8_values(byte, ex).astype(np.float32).reshape(total, page, dim)
    pool[:, v], pool[:, sc] = byte.reshape(total, page, dim), ex.reshape(total, page, -1)
    cache = ds.PagedCache(torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(), page, dim, fmt)
    return cache, [pool_rows[table[e, : -(-n // page)]].reshape(-1, dim)[:n] for e, n in enumerate(lens)]


def read_fp8(cache, entry, slots):
    """Rows of an entry as the pages' bytes spell them (float64)."""
    page = cache.page_size
    table = cache.page_table.cpu().numpy()
    pool = cache.pages.cpu().numpy().reshape(cache.num_pages, -1)
    v, sc = ref.fp8_places(cache.dim, page)
    data = pool[table[entry, slots // page]]
    rows = np.arange(len(slots))[:, None]
    return ref.fp8_values(data[rows, v[slots % page]], data[rows, sc[slots % page]])


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def edge_blocks(rng, n, dim):
    """Random rows with blocks at the type's edges: exact bounds, saturation, tiny, zero and non-finite ones."""
    y = edge_rows(rng, n, dim)
    top = [448.0, 449.0, 448 * 128.0, 1e6, 3e38, 1e-38, 1e-44, 448 * 2.0 ** -100, 2.0 ** -108, 0.0, np.nan, np.inf, -np.inf]
    for i, t in enumerate(top):
        k = n - 1 - i
        y[k] = rng.uniform(-1, 1, dim) * (t if np.isfinite(t) else 1.0)
        y[k, (37 * i) % dim] = t
    # Halves between neighbouring e4m3 numbers (even on ties), and its subnormal steps.
    ties = np.r_[448.0, (ref.E4M3[:-1] + ref.E4M3[1:]) / 2]
    y[n - 14, :127] = np.r_[ties[:127]]
    return y.astype(np.float32)


@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", TYPES)
def test_append_without_rotation_is_exact(dim, page, dtype):
    rng = np.random.default_rng(page + dim)
    cache, _ = make_cache(rng, [300, 1, 77], dim, "fp8", page)
    before = cache.pages.cpu().numpy().reshape(cache.num_pages, -1).copy()
    y = torch.from_numpy(edge_blocks(rng, 40, dim)).to(dtype)
    seq = np.repeat([0, 2, 1, -1], [20, 15, 1, 4])
    slot = np.r_[np.arange(255, 275), np.arange(60, 75), 0, 5, -9, 2 ** 31 - 1, 0]
    order = rng.permutation(40)
    seq, slot = seq[order], slot[order]
    values = torch.full((40, dim), 9.0, dtype=BF16, device="cuda")
    invalid = torch.full((40,), 9, dtype=torch.int32, device="cuda")
    ds.ds_rows_append(cache, y.cuda(), i32(seq), i32(slot), values=values, invalid=invalid)
    assert not invalid.any()
    byte, ex = ref.fp8_quantise(y.float().numpy())
    want = ref.fp8_values(byte, ex)
    got = f64(values)
    now = cache.pages.cpu().numpy().reshape(cache.num_pages, -1)
    table = cache.page_table.cpu().numpy()
    v, sc = ref.fp8_places(dim, page)
    touched = np.zeros(now.shape, bool)
    for i in range(40):
        if seq[i] < 0:
            assert (got[i] == 9.0).all()
            continue
        np.testing.assert_array_equal(got[i], want[i])
        p, r = table[seq[i], slot[i] // page], slot[i] % page
        np.testing.assert_array_equal(now[p, sc[r]], ex[i])
        sound = np.repeat(ex[i] != 255, 128)  # a NaN block's values say nothing
        np.testing.assert_array_equal(now[p, v[r]][sound], byte[i][sound])
        touched[p, v[r]] = touched[p, sc[r]] = True
    np.testing.assert_array_equal(now[~touched], before[~touched])


@pytest.mark.parametrize("dim,rot,first,layout", [
    (512, 64, 448, "interleaved"), (128, 64, 0, "half"), (512, 512, 0, "half"), (128, 6, 50, "interleaved"),
    (128, 10, 17, "half"), (512, 86, 3, "half"), (128, 2, 126, "half"),
])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_rotates(dim, rot, first, layout, dtype):
    rng = np.random.default_rng(rot + first)
    n = 37
    cache, _ = make_cache(rng, [n], dim, "fp8", 16)
    x = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).to(dtype)
    pos = rng.integers(0, 1 << 20, n)
    rope = ds.Rope(rot, first=first, layout=layout, factor=4.0, original_len=4096, magnitude=1.1)
    values = torch.zeros(n, dim, dtype=BF16, device="cuda")
    ds.ds_rows_append(cache, x.cuda(), i32(np.zeros(n)), i32(np.arange(n)), rope=rope, positions=i32(pos), values=values)
    xd = x.double().numpy()
    want = ref.rope(xd, pos, ref.frequencies(rot, 10000.0, 4.0, 4096), first, layout, 1.1)
    a, b = ref.pairs(rot, first, layout)
    err = np.zeros_like(xd)
    err[:, a] = err[:, b] = ROPE_RTOL * 1.1 * (np.abs(xd[:, a]) + np.abs(xd[:, b]))
    held = f64(values)
    np.testing.assert_array_equal(read_fp8(cache, 0, np.arange(n)), held)
    top = np.repeat(np.abs(want).reshape(n, -1, 128).max(-1) * (1 + 1e-6), 128, 1)
    # Half a step at the rounded value's own size, which the error may have moved.
    assert np.all(np.abs(held - want) <= np.maximum((np.abs(want) + err) * 2.0 ** -4, top / 224 * 2.0 ** -10) + err)


def test_append_flags_what_it_cannot_write():
    rng = np.random.default_rng(4)
    cache, _ = make_cache(rng, [64, 20], 128, "fp8", 16)
    cache.page_table[0, 1] = cache.num_pages
    cache.page_table[1, 0] = -1
    before = cache.pages.clone()
    seq, slot = i32([0, 0, 1, 2, -2, 0, 0, -1]), i32([16, 31, 5, 0, 0, -1, 64 * 16, 3])
    invalid = torch.full((8,), 7, dtype=torch.int32, device="cuda")
    ds.ds_rows_append(cache, torch.ones(8, 128, device="cuda"), seq, slot, invalid=invalid)
    assert invalid.tolist() == [1, 1, 1, 1, 1, 1, 1, 0] and torch.equal(before, cache.pages)


# ---------------------------------------------------------------------------
# fetch
# ---------------------------------------------------------------------------

def fetched(values, seq, slot, dtype):
    return torch.from_numpy(np.stack([values[e][s] for e, s in zip(seq, slot)])).to(dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("dtype", TYPES)
def test_fetch(fmt, dim, page, dtype):
    rng = np.random.default_rng(page + dim)
    lens = [300, 1, 77]
    cache, values = make_cache(rng, lens, dim, fmt, page)
    for n in (1, 7, 300):
        seq = rng.integers(0, 3, n)
        slot = (rng.random(n) * np.array(lens)[seq]).astype(int)
        pad = rng.random(n) < 0.2
        out = torch.full((n, dim), 5.0, dtype=dtype, device="cuda")
        invalid = torch.full((n,), 9, dtype=torch.int32, device="cuda")
        ds.ds_rows_fetch(cache, i32(np.where(pad, -1, seq)), i32(slot), out, invalid=invalid)
        want = fetched(values, seq, slot, dtype)
        want[torch.from_numpy(pad)] = 5.0
        assert torch.equal(out.cpu(), want) and not invalid.any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_fetch_into_wider_rows(fmt, dtype, shift):
    """Rows inside wider rows, at offsets off 16 bytes too; memory around them stays as it was."""
    rng = np.random.default_rng(shift)
    cache, values = make_cache(rng, [50], 128, fmt, 16)
    base = torch.full((50, 200 + shift % 8), 3.0, dtype=dtype, device="cuda")
    ds.ds_rows_fetch(cache, i32(np.zeros(50)), i32(np.arange(50)), base[:, shift:shift + 128])
    assert torch.equal(base[:, shift:shift + 128].cpu(), torch.from_numpy(values[0]).to(dtype))
    rest = torch.ones(base.shape[1], dtype=torch.bool)
    rest[shift:shift + 128] = False
    assert (base[:, rest] == 3.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [128, 512])
def test_fetch_flags_what_it_cannot_read(fmt, dim):
    rng = np.random.default_rng(6)
    cache, values = make_cache(rng, [64, 20], dim, fmt, 16)
    cache.page_table[0, 1] = cache.num_pages
    cache.page_table[1, 0] = -5
    seq, slot = [0, 0, 1, 2, -2, 0, 0, -1, 0], [16, 31, 5, 0, 0, -1, 2 ** 31 - 1, 3, 47]
    out = torch.full((9, dim), 4.0, device="cuda")
    invalid = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    ds.ds_rows_fetch(cache, i32(seq), i32(slot), out, invalid=invalid)
    assert invalid.tolist() == [1, 1, 1, 1, 1, 1, 1, 0, 0]
    assert out[:7].isnan().all() and (out[7] == 4.0).all()
    assert torch.equal(out[8].cpu(), torch.from_numpy(values[0][47]))


def test_fetch_of_every_8_bit_code():
    """All 256 value bytes and all 256 exponents, in each type."""
    page, dim = 256, 128
    v, sc = ref.fp8_places(dim, page)
    pool = np.zeros((2, ds.ds_rows_page_bytes(page, dim, "fp8")), np.uint8)
    byte = np.stack([np.arange(256)[:, None] ^ (2 * np.arange(128)[None]) & 255] * 2).astype(np.uint8)
    ex = np.stack([np.arange(256)[:, None], np.full((256, 1), 127)]).astype(np.uint8)
    pool[:, v], pool[:, sc] = byte, ex
    cache = ds.PagedCache(torch.from_numpy(pool).cuda(), i32([[0, 1]]), page, dim, "fp8")
    want = ref.fp8_values(byte.reshape(-1, dim), ex.reshape(-1, 1))
    for dtype in TYPES:
        out = torch.zeros(512, dim, dtype=dtype, device="cuda")
        ds.ds_rows_fetch(cache, i32(np.zeros(512)), i32(np.arange(512)), out)
        np.testing.assert_array_equal(f64(out), f64(torch.from_numpy(want).to(dtype)))
        assert np.array_equal(np.signbit(f64(out)), np.signbit(want)) or np.isnan(want).any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_fetch_reads_what_append_held(fmt):
    """The rows come back as `values` gave them, and appended again they hold the same values."""
    rng = np.random.default_rng(8)
    n, dim, page = 500, 512, 32
    table, total = page_table(rng, [n], page)
    one, two = (ds.PagedCache.empty(total, torch.from_numpy(table).cuda(), page, dim, fmt) for _ in range(2))
    x = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).cuda()
    values, back = (torch.zeros(n, dim, dtype=BF16, device="cuda") for _ in range(2))
    seq, slot = i32(np.zeros(n)), i32(rng.permutation(n))
    ds.ds_rows_append(one, x, seq, slot, values=values)
    ds.ds_rows_fetch(one, seq, slot, back)
    assert torch.equal(values, back)
    if fmt != "int4":  # a group's largest value need not come back as 7 steps
        again = torch.zeros_like(back)
        ds.ds_rows_append(two, back, seq, slot)
        ds.ds_rows_fetch(two, seq, slot, again)
        assert torch.equal(values, again)


def test_fetch_past_32_bits():
    """A pool of more than 2^32 bytes, rows of out beyond 2^32 bytes, and padding in between."""
    page, dim = 256, 512
    pages = (1 << 32) // ds.ds_rows_page_bytes(page, dim, "fp8") + 3
    cache = ds.PagedCache.empty(pages, i32([[pages - 1, 0]]), page, dim, "fp8")
    x = torch.randn(page, dim, device="cuda")
    at = i32(range(page))
    values = torch.zeros(page, dim, dtype=BF16, device="cuda")
    ds.ds_rows_append(cache, x, i32(np.zeros(page)), at, values=values)
    out = torch.empty((1 << 30) * 2 + dim, dtype=BF16, device="cuda")
    rows = out.as_strided((3, dim), (1 << 30, 1))
    ds.ds_rows_fetch(cache, i32([0, -1, 0]), i32([255, 0, 3]), rows)
    assert torch.equal(rows[0], values[255]) and torch.equal(rows[2], values[3])


def test_append_and_fetch_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(9)
    cache, _ = make_cache(rng, [64], 512, "fp8", 16)
    x = torch.zeros(8, 512, device="cuda")
    seq, slot = i32(np.zeros(8)), i32(range(8))
    out = torch.zeros(8, 512, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ds.ds_rows_append(cache, x, seq, slot)
        ds.ds_rows_fetch(cache, seq, slot, out)
    for k in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal((8, 512)).astype(np.float32)))
        graph.replay()
        want = ref.fp8_values(*ref.fp8_quantise(x.cpu().numpy()))
        np.testing.assert_array_equal(f64(out), want)
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    ds.ds_rows_fetch(cache, seq, slot, out, stream=side)
    side.synchronize()
    np.testing.assert_array_equal(f64(out), want)
    with pytest.raises(TypeError):
        ds.ds_rows_fetch(cache, seq.long(), slot, out)
    with pytest.raises(ValueError, match="overlap|contiguous|must be"):
        ds.ds_rows_fetch(cache, seq, slot, out.t())
    with pytest.raises(ds.DsRowsError, match="overlap"):
        ds.ds_rows_fetch(cache, seq, slot, out[:1].expand(8, 512))
    with pytest.raises(ValueError, match="out must be"):
        ds.ds_rows_fetch(cache, seq, slot, out[:, :128])
    ds.ds_rows_fetch(cache, seq[:0], slot[:0], out[:0])


# ---------------------------------------------------------------------------
# the readers: the bits of the contiguous calls on the bf16 rows that the pages stand for
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17, 127, 128, 129, 255, 257], [1000, 3, 4097], [60000, 20001]])
def test_scores(page, lens):
    rng = np.random.default_rng(page + len(lens))
    cache, values = make_cache(rng, lens, 128, "fp8", page)
    q = queries(rng, len(lens), 128)
    w = torch.from_numpy(rng.standard_normal((len(lens), 64)).astype(np.float32) / 8).cuda()
    scores, plain = (torch.full((len(lens), max(lens) + 3), 123.0, device="cuda") for _ in range(2))
    ds.ds_rows_indexer_score_paged(row_table(lens), q, w, cache, scores)
    ds.ds_rows_indexer_score(row_table(lens), q, w, [torch.from_numpy(v).to(BF16).cuda() for v in values], plain)
    assert torch.equal(scores, plain)
    for e, n in enumerate(lens):
        args = f64(q[e]), f64(w[e]), values[e].astype(np.float64)
        assert np.all(np.abs(f64(scores[e, :n]) - oracle.indexer_score(*args)) <= SCORE_RTOL * score_bound(*args))
        assert (scores[e, n:] == 123.0).all()


@pytest.mark.parametrize("page", [16, 64, 256])
def test_scores_of_bad_pages_and_values(page):
    rng = np.random.default_rng(2)
    n = 700
    cache, values = make_cache(rng, [n], 128, "fp8", page)
    q, w = queries(rng, 1, 128), torch.ones(1, 64, device="cuda")
    last = (n - 1) // page
    cache.page_table[0, 0], cache.page_table[0, last] = -5, cache.num_pages
    row = page + 3
    one = torch.zeros(1, 128, device="cuda")
    one[0, 77] = float("nan")
    ds.ds_rows_append(cache, one, i32([0]), i32([row]))
    scores = torch.zeros(1, n, device="cuda")
    ds.ds_rows_indexer_score_paged(row_table([n]), q, w, cache, scores)
    gone = (np.arange(n) // page == 0) | (np.arange(n) // page == last) | (np.arange(n) == row)
    got = f64(scores[0])
    assert np.all(got[gone] == -np.inf)
    args = f64(q[0]), f64(w[0]), values[0].astype(np.float64)
    assert np.all(np.abs(got - oracle.indexer_score(*args))[~gone] <= (SCORE_RTOL * score_bound(*args))[~gone])


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("lens,widths", [([1], [1]), ([37, 130, 600], [37, 100, 512]),
                                         ([2000, 513, 128, 129, 5, 700, 511, 1024], [512, 512, 128, 129, 1, 384, 511, 3])])
def test_attention(page, lens, widths):
    rng = np.random.default_rng(page + len(lens))
    cache, values = make_cache(rng, lens, 512, "fp8", page)
    rows = [(n, w, 520 * e + 3, e) for e, (n, w) in enumerate(zip(lens, widths))]
    idx = np.full(520 * len(lens) + 3, -7, np.int64)
    for e, (n, w) in enumerate(zip(lens, widths)):
        pick = rng.permutation(n)[:w]
        if w > 4:
            pick[1] = pick[0]   # an index twice
            pick[3] = -1        # an empty slot
        idx[520 * e + 3: 520 * e + 3 + w] = pick
    q = queries(rng, len(lens) + 1, 512)
    sinks = torch.from_numpy(rng.standard_normal((len(lens) + 1, 70)).astype(np.float32)).cuda()
    out, plain, bad, bad_plain = attend(rows, q, sinks, 70, i32(idx), cache, values)
    assert torch.equal(out, plain) and torch.equal(bad, bad_plain) and not bad[:-1].any()
    assert (out[-1] == 4.0).all()
    want, _ = oracle.sparse_attention(f64(q[0]), values[0].astype(np.float64), idx[3: 3 + widths[0]], f64(sinks[0, :64]),
                                      SCALE)
    np.testing.assert_allclose(f64(out[0]), want, atol=2.0 ** -8 * np.abs(values[0]).max())


def test_attention_fails_closed():
    rng = np.random.default_rng(9)
    cache, values = make_cache(rng, [300] * 5, 512, "fp8", 32)
    cache.page_table[1, 4], cache.page_table[2, 4] = cache.num_pages, -1
    nan = torch.ones(2, 512, device="cuda")
    nan[:, 500] = float("inf")
    ds.ds_rows_append(cache, nan, i32([3, 4]), i32([10, 10]))
    idx = np.stack([np.arange(100)] * 5)
    idx[0, 7], idx[1, 0], idx[2, 99], idx[4, 10] = 300, 4 * 32 + 1, 5 * 32 - 1, 11
    rows = [(300, 100, 100 * e, e) for e in range(5)]
    q = queries(rng, 5, 512)
    out, bad = torch.full_like(q, 4.0), torch.zeros(5, 64, dtype=torch.int32, device="cuda")
    ds.ds_rows_sparse_attn_paged(rows, q, torch.zeros(64, device="cuda"), 0, i32(idx).reshape(-1), SCALE, out, cache,
                                 invalid=bad)
    assert not out[:4].any() and bad[:4].all() and out[4].any() and not bad[4].any()


@pytest.mark.parametrize("dim", [128, 512])
def test_reads_of_pools_past_32_bits(dim):
    """A row in the last page of a pool of more than 2^32 bytes reads as the same row in the first page."""
    rng = np.random.default_rng(dim)
    page = 256
    num = (1 << 32) // ds.ds_rows_page_bytes(page, dim, "fp8") + 3
    cache = ds.PagedCache.empty(num, i32([[0], [num - 1]]), page, dim, "fp8")
    x = torch.randn(page, dim, device="cuda")
    at = i32(range(page))
    for e in range(2):
        ds.ds_rows_append(cache, x, i32(np.full(page, e)), at)
    q = queries(rng, 1, dim)
    both = torch.cat([q, q])
    if dim == 128:
        scores = torch.zeros(2, page, device="cuda")
        ds.ds_rows_indexer_score_paged(row_table([page] * 2), both, torch.ones(2, 64, device="cuda"), cache, scores)
        assert torch.equal(scores[0], scores[1]) and scores.any()
    else:
        out = torch.zeros_like(both)
        rows = [(page, page, 0, 0), (page, page, page, 1)]
        idx = i32(np.r_[np.arange(page), np.arange(page)])
        ds.ds_rows_sparse_attn_paged(rows, both, torch.zeros(64, device="cuda"), 0, idx, SCALE, out, cache)
        assert torch.equal(out[0], out[1]) and out.any()
