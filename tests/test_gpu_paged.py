"""GPU parity of the rotary positions and the paged caches: ds_rows_rope,
ds_rows_append, ds_rows_indexer_score_paged and ds_rows_sparse_attn_paged against
the float64 oracle, and against the contiguous entry points on the bf16 rows that
a cache stands for.

Tolerances. Rotation: the remainder within a quarter turn is at most pi/4, rounded twice (2^-24 of
itself: 4.7e-8), the polynomials' last step rounds by 2^-25 to 2^-24 (6e-8), their next terms are
below 3e-8, and three roundings of 2^-24 follow (the magnitude, the product, the sum): 3.2e-7 of
m (|a| + |b|), taken as 5e-7, plus half a step of the output's type.
Scores: sums of 128 products and of 64 heads in fp32, 192 roundings of 2^-24 of
T = sum |w| sum |q k|: 1.2e-5 T. Attention: the bars of parity.check_out.
"""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
import oracle
from oracle import paged as ref
from parity import check_out, score_bound

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, F16, F32]
ROPE_RTOL = 5e-7
SCORE_RTOL = 192 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ds.build()
    ds.load()


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int64), dtype=torch.int32).cuda()


# ---------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------

def check_rope(got, x, pos, rope_kw, first, layout, inverse, magnitude, dtype):
    rot = rope_kw["rot_dim"]
    theta = ref.frequencies(**rope_kw)
    xd = f64(x)
    want = ref.rope(xd, pos, theta, first, layout, magnitude, inverse)
    a, b = ref.pairs(rot, first, layout)
    size = np.zeros_like(xd)
    size[..., a] = size[..., b] = magnitude * (np.abs(xd[..., a]) + np.abs(xd[..., b]))
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # a subnormal step
    bound = ROPE_RTOL * size + np.abs(want) * (torch.finfo(dtype).eps / 2) * (1 + 1e-6) + np.where(size > 0, tiny, 0)
    err = np.abs(f64(got) - want)
    live = np.asarray(pos) >= 0
    assert np.all(err[live] <= bound[live]), f"worst ratio {np.max(err[live] / np.maximum(bound[live], 1e-300))}"


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,heads,dim,rot,first", [
    (1, 1, 2, 2, 0), (3, 1, 64, 64, 0), (8, 64, 512, 64, 448), (5, 7, 128, 64, 64), (33, 2, 96, 86, 10),
    (2, 3, 130, 6, 4), (1, 5, 1024, 512, 512), (300, 16, 128, 128, 0), (17, 64, 64, 2, 62), (40, 9, 192, 48, 96),
    (2, 2, 1023, 510, 512), (1, 1, 1024, 512, 2),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_rope(layout, dtype, tokens, heads, dim, rot, first, inplace):
    g = torch.Generator(device="cuda").manual_seed(tokens * dim + rot)
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0 if tokens % 2 else 2 ** 31 - 1
    kw = dict(rot_dim=rot, base=10000.0, factor=16.0, original_len=65536)
    magnitude, inverse = 1.25, bool(heads % 2)
    rope = ds.Rope(rot, first=first, layout=layout, base=10000.0, factor=16.0, original_len=65536, magnitude=magnitude)
    keep = x.clone()
    out = x if inplace else torch.full_like(x, 7.0)
    ds.ds_rows_rope(rope, x, pos, out, inverse=inverse)
    check_rope(out, keep, f64(pos), kw, first, layout, inverse, magnitude, dtype)
    # Elements outside the range pass bit for bit.
    outside = torch.ones(dim, dtype=torch.bool)
    outside[first:first + rot] = False
    assert torch.equal(out[..., outside], keep[..., outside])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rope_strides_offsets_and_padding(layout, dtype):
    """Heads outside tokens, rows at odd offsets inside wider rows, a broadcast
    source, padding; memory around the rows stays as it was."""
    g = torch.Generator(device="cuda").manual_seed(5)
    pos = i32([4, -1, 99, -7, 123456, 0])
    kw = dict(rot_dim=16)
    rope = ds.Rope(16, first=2, layout=layout)
    for head_major in (False, True):
        for shift in (0, 1):
            shape = (3, 6, 41) if head_major else (6, 3, 41)
            base = torch.randn(shape, generator=g, device="cuda").to(dtype)
            view = base[..., shift:shift + 24]
            x = view.transpose(0, 1) if head_major else view
            out_base = torch.full(shape, 5.0, device="cuda", dtype=dtype)
            out = out_base[..., shift:shift + 24]
            out = out.transpose(0, 1) if head_major else out
            ds.ds_rows_rope(rope, x, pos, out)
            check_rope(out, x, f64(pos), kw, 2, layout, False, 1.0, dtype)
            assert torch.equal(out[[1, 3]], torch.full_like(out[[1, 3]], 5.0))
            rest = torch.ones(41, dtype=torch.bool)
            rest[shift:shift + 24] = False
            assert (out_base[..., rest] == 5.0).all()
            x2 = base.clone()[..., shift:shift + 24]
            x2 = x2.transpose(0, 1) if head_major else x2
            keep = x2.clone()
            ds.ds_rows_rope(rope, x2, pos, x2)
            assert torch.equal(x2[[0, 2, 4, 5]], out[[0, 2, 4, 5]]) and torch.equal(x2[[1, 3]], keep[[1, 3]])
    one = torch.randn(1, 1, 24, generator=g, device="cuda").to(dtype)
    out = torch.empty(6, 3, 24, device="cuda", dtype=dtype)
    ds.ds_rows_rope(rope, one.expand(6, 3, 24), pos, out)
    check_rope(out, one.expand(6, 3, 24), f64(pos), kw, 2, layout, False, 1.0, dtype)


def test_rope_two_dimensional_and_empty():
    rope = ds.Rope(64)
    x = torch.randn(9, 128, device="cuda")
    out = torch.empty_like(x)
    pos = i32(range(9))
    ds.ds_rows_rope(rope, x, pos, out)
    check_rope(out, x, f64(pos), dict(rot_dim=64), 0, "interleaved", False, 1.0, F32)
    ds.ds_rows_rope(rope, x[:0], pos[:0], out[:0])
    ds.ds_rows_rope(rope, x[:0, None], pos[:0], out[:0, None])


def test_rope_offsets_past_32_bits():
    """A token stride of 2^30 elements: the last row begins past 2^32 bytes."""
    base = torch.empty((1 << 30) * 2 + 64, dtype=BF16, device="cuda")
    x = torch.as_strided(base, (3, 1, 64), (1 << 30, 64, 1))
    x.copy_(torch.randn(3, 1, 64, device="cuda"))
    keep, pos = x.clone(), i32([3, 70000, 1 << 20])
    rope = ds.Rope(64, layout="half")
    ds.ds_rows_rope(rope, x, pos, x)
    check_rope(x, keep, f64(pos), dict(rot_dim=64), 0, "half", False, 1.0, BF16)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_gradient(layout):
    """The inverse is the gradient: against the formula's transpose in 64 bits and
    against differences of the forward pass (linear in x, so a central difference
    is exact but for the rounding of its two values)."""
    g = torch.Generator(device="cuda").manual_seed(11)
    x, grad = torch.randn(2, 5, 3, 32, generator=g, device="cuda")
    pos = i32([0, 1, 500, 65535, 1 << 20])
    rope = ds.Rope(16, first=8, layout=layout, magnitude=1.5)
    back = torch.empty_like(grad)
    ds.ds_rows_rope(rope, grad, pos, back, inverse=True)
    check_rope(back, grad, f64(pos), dict(rot_dim=16), 8, layout, True, 1.5, F32)
    out = [torch.empty_like(x) for _ in range(2)]
    for e in (0, 8, 13, 23, 31):
        step = torch.zeros_like(x)
        step[..., e] = 1.0
        ds.ds_rows_rope(rope, x + step, pos, out[0])
        ds.ds_rows_rope(rope, x - step, pos, out[1])
        diff = ((f64(out[0]) - f64(out[1])) / 2 * f64(grad)).sum(-1)
        # Each value is off by 5e-7 of m (|a| + |b|) <= 1.5 * 2 * (5 + 1), for two elements of a pair.
        bound = 2 * (ROPE_RTOL + 2.0 ** -24) * 1.5 * 2 * 6 * f64(grad.abs()).max()
        assert np.abs(diff - f64(back)[..., e]).max() <= bound


def test_rope_there_and_back_is_the_identity():
    x = torch.randn(64, 4, 128, device="cuda")
    pos = i32(np.random.default_rng(0).integers(0, 2 ** 31 - 1, 64))
    rope = ds.Rope(128)
    y, z = torch.empty_like(x), torch.empty_like(x)
    ds.ds_rows_rope(rope, x, pos, y)
    ds.ds_rows_rope(rope, y, pos, z, inverse=True)
    # Two rotations: each at most 5e-7 (|a| + |b|) plus a rounding, |a| + |b| <= sqrt(2) |pair|.
    assert (z - x).abs().max() <= 2 * (ROPE_RTOL + 2.0 ** -24) * 2 * x.abs().max() * 1.5


def test_rope_refusals_of_the_binding():
    rope, x = ds.Rope(64), torch.zeros(4, 2, 64, device="cuda")
    pos = i32(range(4))
    for args, err in (((x.cpu(), pos, x), ValueError), ((x, pos.long(), x), TypeError), ((x, pos[:3], x), ValueError),
                      ((x, pos, x[:3]), ValueError), ((x, pos, x.half()), ValueError),
                      ((x.double(), pos, x.double()), ValueError), ((x[0, 0], pos, x[0, 0]), ValueError),
                      ((x.transpose(1, 2), pos, x.transpose(1, 2)), ValueError),
                      ((x[..., :32], pos, x[..., :32]), ds.DsRowsError),
                      ((x, pos, x[:1].expand(4, 2, 64)), ds.DsRowsError)):
        with pytest.raises(err):
            ds.ds_rows_rope(rope, *args)


# ---------------------------------------------------------------------------
# caches
# ---------------------------------------------------------------------------

def page_table(rng, lens, page, extra=2, spare=1):
    """Pages in no order, `extra` unused ones, -1 in entries' unused places."""
    need = [-(-n // page) for n in lens]
    ids = rng.permutation(sum(need) + extra)
    table = np.full((len(lens), max(need) + spare), -1, np.int32)
    at = 0
    for e, n in enumerate(need):
        table[e, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + extra


def make_cache(rng, lens, dim, fmt, page, scale=1.0):
    """A cache whose entries hold random rows; returns it with the rows' values (float32, exact in bf16)."""
    table, total = page_table(rng, lens, page)
    size = ds.ds_rows_page_bytes(page, dim, fmt)
    if fmt == "int4":
        pool = rng.integers(0, 256, (total, size), dtype=np.uint8)  # what no row covers is noise
        pool_rows = np.zeros((total, page, dim), np.float32)
        for p in range(total):
            n, s = ref.int4_quantise(scale * rng.standard_normal((page, dim)).astype(np.float32))
            ref.write_int4_page(pool[p], dim, page, n, s)
            pool_rows[p] = ref.int4_values(n, s)
        pages = torch.from_numpy(pool).cuda()
    else:
        rows = torch.from_numpy(scale * rng.standard_normal((total, page, dim)).astype(np.float32)).to(BF16)
        pool_rows, pages = rows.float().numpy(), rows.cuda()
    cache = ds.PagedCache(pages, torch.from_numpy(table).cuda(), page, dim, fmt)
    values = [pool_rows[table[e, : -(-n // page)]].reshape(-1, dim)[:n] for e, n in enumerate(lens)]
    return cache, values


def read_cache(cache, entry, slots):
    """Rows of an entry as the pages' bytes spell them (float64)."""
    page, dim = cache.page_size, cache.dim
    table = cache.page_table.cpu().numpy()
    pool = cache.pages.contiguous().view(torch.uint8).cpu().numpy().reshape(cache.num_pages, -1)
    out = np.zeros((len(slots), dim))
    for i, s in enumerate(slots):
        data = pool[table[entry, s // page]]
        if cache.format == "bf16":
            bits = data.view(np.uint16).reshape(page, dim)[s % page]
            out[i] = oracle.bf16_to_f64(bits)
        else:
            v, sc = ref.row_places(dim, page)
            n = ref.int4_numbers(data[v[s % page]][None])
            out[i] = ref.int4_values(n, data[sc[s % page]][None])[0]
    return out


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def edge_rows(rng, n, dim):
    """Random rows with groups at the quantiser's edges."""
    y = rng.standard_normal((n, dim)).astype(np.float32) * np.exp(rng.uniform(-6, 6, (n, 1))).astype(np.float32)
    edges = [np.zeros(16), np.full(16, 1e-30), np.full(16, 3500.0), np.full(16, 1e30), np.full(16, 7 * 2.0 ** -10),
             np.full(16, 7 * 2.0 ** -9), np.arange(-7.5, 8.5), np.r_[7.0, np.arange(-7, 8) + 0.5],
             np.r_[7 * 1.0625, np.ones(15)], np.r_[np.nan, np.ones(15)], np.r_[np.ones(15), np.inf],
             np.r_[-np.inf, np.zeros(15)], np.full(16, -0.0), np.full(16, 448 * 7.0), np.full(16, 1e-45)]
    for i, g in enumerate(edges):
        if i < n:
            y[i, 16 * (i % (dim // 16)):][:16] = g
    return y


@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_append_without_rotation_is_exact(dim, page, dtype, fmt):
    rng = np.random.default_rng(page + dim)
    lens = [300, 1, 77]
    cache, _ = make_cache(rng, lens, dim, fmt, page)
    before = cache.pages.clone()
    y = torch.from_numpy(edge_rows(rng, 40, dim)).to(dtype)
    seq = np.repeat([0, 2, 1, -1], [20, 15, 1, 4])
    slot = np.r_[np.arange(255, 275), np.arange(60, 75), 0, 5, -9, 2 ** 31 - 1, 0]
    order = rng.permutation(40)
    seq, slot = seq[order], slot[order]
    values = torch.full((40, dim), 9.0, dtype=BF16, device="cuda")
    invalid = torch.full((40,), 9, dtype=torch.int32, device="cuda")
    ds.ds_rows_append(cache, y.cuda(), i32(seq), i32(slot), values=values, invalid=invalid)
    assert not invalid.any()
    yf = y.float().numpy()
    if fmt == "int4":
        n, s = ref.int4_quantise(yf)
        want = ref.int4_values(n, s)
    else:
        want = y.float().to(BF16).double().numpy()
    got = f64(values)
    for e in range(3):
        at = np.nonzero(seq == e)[0]
        np.testing.assert_array_equal(got[at], want[at])
        np.testing.assert_array_equal(read_cache(cache, e, slot[at]), want[at])
    assert (got[seq == -1] == 9.0).all()
    # Bytes of every other row stay as they were.
    table = cache.page_table.cpu().numpy()
    was = before.view(torch.uint8).cpu().numpy().reshape(cache.num_pages, -1)
    now = cache.pages.view(torch.uint8).cpu().numpy().reshape(cache.num_pages, -1)
    touched = np.zeros(was.shape, bool)
    for e, sl in zip(seq, slot):
        if e >= 0:
            p, r = table[e, sl // page], sl % page
            if fmt == "bf16":
                touched[p, r * 2 * dim:(r + 1) * 2 * dim] = True
            else:
                v, sc = ref.row_places(dim, page)
                touched[p, v[r]] = touched[p, sc[r]] = True
    np.testing.assert_array_equal(now[~touched], was[~touched])


@pytest.mark.parametrize("dim,rot,first,layout", [
    (512, 64, 448, "interleaved"), (128, 64, 0, "half"), (128, 128, 0, "half"), (512, 512, 0, "interleaved"),
    (512, 512, 0, "half"), (128, 6, 50, "interleaved"), (128, 10, 17, "half"), (512, 86, 3, "half"), (128, 2, 126, "half"),
])
@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_rotates(dim, rot, first, layout, fmt, dtype):
    rng = np.random.default_rng(rot + first)
    n = 37
    cache, _ = make_cache(rng, [n], dim, fmt, 16)
    x = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).to(dtype)
    pos = rng.integers(0, 1 << 20, n)
    rope = ds.Rope(rot, first=first, layout=layout, factor=4.0, original_len=4096, magnitude=1.1)
    values = torch.zeros(n, dim, dtype=BF16, device="cuda")
    ds.ds_rows_append(cache, x.cuda(), i32(np.zeros(n)), i32(np.arange(n)), rope=rope, positions=i32(pos),
                      values=values)
    xd = x.double().numpy()
    want = ref.rope(xd, pos, ref.frequencies(rot, 10000.0, 4.0, 4096), first, layout, 1.1)
    a, b = ref.pairs(rot, first, layout)
    err = np.zeros_like(xd)
    err[:, a] = err[:, b] = ROPE_RTOL * 1.1 * (np.abs(xd[:, a]) + np.abs(xd[:, b]))
    held = f64(values)
    np.testing.assert_array_equal(read_cache(cache, 0, np.arange(n)), held)
    if fmt == "bf16":
        assert np.all(np.abs(held - want) <= err + np.abs(want) * 2.0 ** -8 * (1 + 1e-5) + 2.0 ** -133)
        return
    # Half a step of the group's scale, which is the e4m3 next to max / 7 (2^-4 of it,
    # no subnormal here); 7.5 steps cover max, so nothing is clamped further away.
    top = np.abs(want).reshape(n, -1, 16).max(-1)
    s = np.repeat(top / 7 * (1 + 2.0 ** -4) * (1 + 1e-5), 16, 1)
    assert np.all(np.abs(held - want) <= s / 2 + err)


def test_append_flags_what_it_cannot_write():
    rng = np.random.default_rng(4)
    cache, _ = make_cache(rng, [64, 20], 512, "int4", 16)
    table = cache.page_table.clone()
    table[1, 1] = cache.num_pages       # out of the pool
    cache.page_table.copy_(table)
    before = cache.pages.clone()
    width = table.shape[1] * 16
    seq = [2, -2, 0, 0, 1, 0, -1, 0]
    slot = [0, 0, -1, width, 16, 64, 3, 7]  # slot 64 of entry 0: page -1
    pos = [0, 0, 0, 0, 0, 0, 0, -1]
    x = torch.ones(8, 512, device="cuda")
    invalid = torch.full((8,), 5, dtype=torch.int32, device="cuda")
    values = torch.full((8, 512), 3.0, dtype=BF16, device="cuda")
    ds.ds_rows_append(cache, x, i32(seq), i32(slot), rope=ds.Rope(64), positions=i32(pos), values=values,
                      invalid=invalid)
    assert invalid.tolist() == [1, 1, 1, 1, 1, 1, 0, 1]
    assert torch.equal(cache.pages, before) and (values == 3.0).all()


@pytest.mark.parametrize("shift", [0, 1])
def test_append_strided_source(shift):
    rng = np.random.default_rng(6)
    base = torch.randn(21, 600, device="cuda").to(BF16)
    x = base[:, shift:shift + 512]
    cache, _ = make_cache(rng, [32], 512, "int4", 32)
    values = torch.zeros(21, 512, dtype=BF16, device="cuda")
    ds.ds_rows_append(cache, x, i32(np.zeros(21)), i32(range(21)), values=values)
    n, s = ref.int4_quantise(x.float().cpu().numpy())
    np.testing.assert_array_equal(f64(values), ref.int4_values(n, s))


def test_append_refusals_of_the_binding():
    cache, _ = make_cache(np.random.default_rng(0), [32], 512, "int4", 32)
    x, s = torch.zeros(4, 512, device="cuda"), i32(range(4))
    for args, kw, err in (((x[:, :128], s, s), {}, ValueError), ((x.cpu(), s, s), {}, ValueError),
                          ((x.double(), s, s), {}, ValueError), ((x, s[:3], s), {}, ValueError),
                          ((x, s, s.long()), {}, TypeError), ((x, s, s), dict(rope=ds.Rope(64)), TypeError),
                          ((x, s, s), dict(values=x), TypeError), ((x.T.contiguous().T, s, s), {}, ValueError),
                          ((x, s, s), dict(rope=ds.Rope(64, first=449, layout="half"), positions=s), ds.DsRowsError)):
        with pytest.raises(err):
            ds.ds_rows_append(cache, *args, **kw)
    ds.ds_rows_append(cache, x[:0], s[:0], s[:0])


# ---------------------------------------------------------------------------
# indexer scores
# ---------------------------------------------------------------------------

def row_table(lens):
    return [(n, min(512, n), 512 * e, e) for e, n in enumerate(lens)]


def queries(rng, rows, dim):
    return torch.from_numpy(rng.standard_normal((rows, 64, dim)).astype(np.float32)).to(BF16).cuda()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17, 127, 128, 129, 255, 257], [1000, 3, 4097]])
def test_scores(fmt, page, lens):
    rng = np.random.default_rng(page + len(lens))
    cache, values = make_cache(rng, lens, 128, fmt, page)
    q = queries(rng, len(lens), 128)
    w = torch.from_numpy(rng.standard_normal((len(lens), 64)).astype(np.float32) / 8).cuda()
    stride = max(lens) + 3
    scores = torch.full((len(lens), stride), 123.0, device="cuda")
    ds.ds_rows_indexer_score_paged(row_table(lens), q, w, cache, scores)
    plain = torch.full_like(scores, 123.0)
    keys = [torch.from_numpy(v).to(BF16).cuda() for v in values]
    ds.ds_rows_indexer_score(row_table(lens), q, w, keys, plain)
    got = f64(scores)
    for e, n in enumerate(lens):
        args = f64(q[e]), f64(w[e]), values[e].astype(np.float64)
        err = np.abs(got[e, :n] - oracle.indexer_score(*args))
        assert np.all(err <= SCORE_RTOL * score_bound(*args))
        assert (got[e, n:] == 123.0).all()
    if fmt == "bf16":
        assert torch.equal(scores, plain)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_scores_of_many_tiles(fmt):
    """More tiles than multiprocessors and than a CTA's ring holds, entries sharing pages."""
    rng = np.random.default_rng(1)
    page, lens = 64, [60000, 59999, 40000]
    cache, values = make_cache(rng, [4096], 128, fmt, page)
    ids = rng.integers(0, cache.num_pages, (3, -(-60000 // page))).astype(np.int32)
    pool = [read_cache(ds.PagedCache(cache.pages, i32([[p]]), page, 128, fmt), 0, np.arange(page))
            for p in range(cache.num_pages)]
    cache = ds.PagedCache(cache.pages, torch.from_numpy(ids).cuda(), page, 128, fmt)
    q = queries(rng, 3, 128)
    w = torch.from_numpy(rng.standard_normal((3, 64)).astype(np.float32) / 8).cuda()
    scores = torch.zeros(3, 60000, device="cuda")
    ds.ds_rows_indexer_score_paged(row_table(lens), q, w, cache, scores)
    got = f64(scores)
    for e, n in enumerate(lens):
        by_page = [(oracle.indexer_score(f64(q[e]), f64(w[e]), k), score_bound(f64(q[e]), f64(w[e]), k)) for k in pool]
        want = np.concatenate([by_page[p][0] for p in ids[e]])[:n]
        bound = np.concatenate([by_page[p][1] for p in ids[e]])[:n]
        assert np.all(np.abs(got[e, :n] - want) <= SCORE_RTOL * bound)
        # A row of a joint call is bitwise the row alone.
        alone = torch.zeros(1, n, device="cuda")
        one = ds.PagedCache(cache.pages, cache.page_table[e:e + 1].contiguous(), page, 128, fmt)
        ds.ds_rows_indexer_score_paged([(n, 512, 0, e)], q, w, one, alone)
        assert torch.equal(alone[0], scores[e, :n])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_scores_of_bad_pages_and_values(fmt, page):
    rng = np.random.default_rng(2)
    n = 700
    cache, values = make_cache(rng, [n], 128, fmt, page)
    q, w = queries(rng, 1, 128), torch.ones(1, 64, device="cuda")
    table = cache.page_table.cpu().numpy()
    bad = [0, (n - 1) // page]
    table[0, 0], table[0, bad[1]] = -5, cache.num_pages
    cache.page_table.copy_(torch.from_numpy(table))
    # A NaN among the values of a key on a good page.
    row = page + 3 if page < 256 else 256 + 3
    one = torch.zeros(1, 128, device="cuda")
    one[0, 77] = float("nan")
    ds.ds_rows_append(cache, one, i32([0]), i32([row]))
    scores = torch.zeros(1, n, device="cuda")
    ds.ds_rows_indexer_score_paged(row_table([n]), q, w, cache, scores)
    got = f64(scores)[0]
    gone = np.isin(np.arange(n) // page, bad) | (np.arange(n) == row)
    assert np.all(np.isneginf(got[gone])) and np.all(np.isfinite(got[~gone]))
    k = values[0].astype(np.float64)
    args = f64(q[0]), f64(w[0]), k
    err = np.abs(got - oracle.indexer_score(*args))[~gone]
    assert np.all(err <= SCORE_RTOL * score_bound(*args)[~gone])


def test_every_scale_byte():
    """Keys and KV rows of one value n = 1 in every group, row r with scale byte r: the scores
    and outputs of the value, NaN (so -inf, and zero heads) from byte 0x7F on."""
    page, w = 256, torch.zeros(1, 64, device="cuda")
    w[0, 0] = 1.0
    for dim in (128, 512):
        data = np.zeros(ds.ds_rows_page_bytes(page, dim, "int4"), np.uint8)
        n = np.ones((page, dim), np.int64)
        ref.write_int4_page(data, dim, page, n, np.repeat(np.arange(256, dtype=np.uint8)[:, None], dim // 16, 1))
        cache = ds.PagedCache(torch.from_numpy(data).cuda(), i32([[0]]), page, dim, "int4")
        q = torch.zeros(1, 64, dim, dtype=BF16, device="cuda")
        q[0, 0, dim - 1] = 1.0
        if dim == 128:
            scores = torch.zeros(256, device="cuda")
            ds.ds_rows_indexer_score_paged([(256, 256, 0, 0)], q, w, cache, scores)
            got = f64(scores)
            np.testing.assert_array_equal(got[:127], ref.E4M3)
            assert np.all(np.isneginf(got[127:]))
            continue
        out = torch.zeros_like(q)
        for r in (0, 1, 7, 8, 63, 126, 127, 128, 200, 255):
            ds.ds_rows_sparse_attn_paged([(256, 1, 0, 0)], q, torch.full((64,), -1e30, device="cuda"), 0, i32([r]), SCALE,
                                         out, cache)
            want = ref.E4M3[r] if r < 127 else 0.0
            assert (out == want).all(), r


def test_scores_with_weights_off_16_bytes():
    rng = np.random.default_rng(3)
    cache, values = make_cache(rng, [200], 128, "int4", 32)
    q = queries(rng, 1, 128)
    w = torch.randn(65, device="cuda")[1:]
    scores = torch.zeros(200, device="cuda")
    ds.ds_rows_indexer_score_paged(row_table([200]), q, w, cache, scores)
    args = f64(q[0]), f64(w), values[0].astype(np.float64)
    assert np.all(np.abs(f64(scores) - oracle.indexer_score(*args)) <= SCORE_RTOL * score_bound(*args))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

SCALE = 512 ** -0.5


def attend(rows, q, sinks, stride, idx, cache, values):
    """The paged attention, and the contiguous one on the rows that the cache stands for."""
    out, plain = (torch.full_like(q, 4.0) for _ in range(2))
    bad, bad_plain = (torch.full((q.shape[0], 64), 4, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = ds.workspace(rows)
    ds.ds_rows_sparse_attn_paged(rows, q, sinks, stride, idx, SCALE, out, cache, invalid=bad, workspace_t=ws)
    assert ds.workspace_status(ws) == 0
    kv = [torch.from_numpy(v).to(BF16).cuda() for v in values]
    ds.ds_rows_sparse_attn(rows, q, sinks, stride, idx, SCALE, plain, kv, invalid=bad_plain, workspace_t=ws)
    return out, plain, bad, bad_plain


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("lens,widths", [([1], [1]), ([37, 130, 600], [37, 100, 512]),
                                         ([2000, 513, 128, 129, 5, 700, 511, 1024], [512, 512, 128, 129, 1, 384, 511, 3])])
def test_attention(fmt, page, lens, widths):
    rng = np.random.default_rng(page + len(lens))
    cache, values = make_cache(rng, lens, 512, fmt, page)
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
    assert torch.equal(out, plain) and torch.equal(bad, bad_plain)
    for e, (n, w) in enumerate(zip(lens, widths)):
        want, _ = oracle.sparse_attention(f64(q[e]), values[e].astype(np.float64), idx[520 * e + 3: 520 * e + 3 + w],
                                     f64(sinks[e, :64]), SCALE)
        check_out(f64(out[e]), want)
    assert (out[-1] == 4.0).all() and (bad[-1] == 4).all() and not bad[:-1].any()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_attention_of_an_empty_row(fmt):
    rng = np.random.default_rng(8)
    cache, values = make_cache(rng, [50, 50], 512, fmt, 16)
    rows = [(50, 50, 0, 0), (50, 50, 50, 1)]
    idx = np.r_[np.full(50, -1), rng.permutation(50)]
    out, plain, bad, _ = attend(rows, queries(rng, 2, 512), torch.zeros(64, device="cuda"), 0, i32(idx), cache, values)
    assert not out[0].any() and out[1].any() and not bad.any() and torch.equal(out, plain)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_attention_fails_closed(fmt):
    """An index or a page id out of range zeroes its entry; a non-finite row that is
    selected zeroes the heads of its entry, one that is not selected changes nothing."""
    rng = np.random.default_rng(9)
    lens = [300, 300, 300, 300, 300]
    cache, values = make_cache(rng, lens, 512, fmt, 32)
    table = cache.page_table.cpu().numpy()
    table[1, 4] = cache.num_pages
    table[2, 4] = -1
    cache.page_table.copy_(torch.from_numpy(table))
    nan = torch.ones(2, 512, device="cuda")
    nan[:, 5] = float("nan")
    ds.ds_rows_append(cache, nan, i32([3, 4]), i32([10, 10]))
    idx = np.stack([np.arange(100)] * 5)
    idx[0, 7] = 300
    idx[1, 0] = 4 * 32 + 1
    idx[2, 99] = 5 * 32 - 1
    idx[4, 10] = 11
    rows = [(300, 100, 100 * e, e) for e in range(5)]
    q = queries(rng, 5, 512)
    out = torch.full_like(q, 4.0)
    bad = torch.zeros(5, 64, dtype=torch.int32, device="cuda")
    ds.ds_rows_sparse_attn_paged(rows, q, torch.zeros(64, device="cuda"), 0, i32(idx).reshape(-1), SCALE, out, cache,
                                 invalid=bad)
    assert not out[:4].any() and bad[:4].all() and out[4].any() and not bad[4].any()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_a_decode_step_over_paged_caches(fmt):
    """Rotate and append a run of rows to both caches, then a decode step: rotated
    queries, scores, top-512, attention, the output rotated back; captured in a graph
    and replayed with the step's inputs and the page tables changed in place."""
    rng = np.random.default_rng(12)
    lens, page = [900, 513, 64], 64
    table, total = page_table(rng, lens, page)
    keys = ds.PagedCache.empty(total, torch.from_numpy(table).cuda(), page, 128, fmt)
    kv = ds.PagedCache.empty(total, torch.from_numpy(table).cuda(), page, 512, fmt)
    r_key = ds.Rope(64, first=64, layout="half", factor=4.0, original_len=4096)
    r_kv = ds.Rope(64, first=448, factor=4.0, original_len=4096)
    rows = row_table(lens)
    seq = i32(np.repeat(np.arange(3), lens))
    slot = i32(np.concatenate([np.arange(n) for n in lens]))
    pos = 4 * slot
    s = {}

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = dict(k=torch.randn(len(seq), 128, generator=g, device="cuda"),
                   v=torch.randn(len(seq), 512, generator=g, device="cuda"),
                   qi=torch.randn(3, 64, 128, generator=g, device="cuda").to(BF16),
                   qa=torch.randn(3, 64, 512, generator=g, device="cuda").to(BF16),
                   w=torch.randn(3, 64, generator=g, device="cuda") / 8)
        for name, t in new.items():
            s.setdefault(name, t).copy_(t)

    fill(1)
    at = i32([4 * (n - 1) + 3 for n in lens])
    s["sinks"] = torch.randn(64, device="cuda")
    s["keys_held"] = torch.zeros(len(seq), 128, dtype=BF16, device="cuda")
    s["kv_held"] = torch.zeros(len(seq), 512, dtype=BF16, device="cuda")
    s["qi_r"], s["qa_r"] = torch.empty_like(s["qi"]), torch.empty_like(s["qa"])
    s["scores"] = torch.zeros(3, max(lens), device="cuda")
    s["idx"] = torch.zeros(3 * 512, dtype=torch.int32, device="cuda")
    s["attn"], s["out"] = torch.empty_like(s["qa"]), torch.empty_like(s["qa"])
    ws = ds.workspace(rows)

    def step():
        ds.ds_rows_append(keys, s["k"], seq, slot, rope=r_key, positions=pos, values=s["keys_held"])
        ds.ds_rows_append(kv, s["v"], seq, slot, rope=r_kv, positions=pos, values=s["kv_held"])
        ds.ds_rows_rope(r_key, s["qi"], at, s["qi_r"])
        ds.ds_rows_rope(r_kv, s["qa"], at, s["qa_r"])
        ds.ds_rows_indexer_score_paged(rows, s["qi_r"], s["w"], keys, s["scores"])
        ds.ds_rows_topk(rows, s["scores"], max(lens), s["idx"], ws)
        ds.ds_rows_sparse_attn_paged(rows, s["qa_r"], s["sinks"], 0, s["idx"], SCALE, s["attn"], kv, workspace_t=ws)
        ds.ds_rows_rope(r_kv, s["attn"], at, s["out"], inverse=True)

    def check():
        assert ds.workspace_status(ws) == 0
        idx, start = s["idx"].cpu().numpy(), 0
        theta = ref.frequencies(64, 10000.0, 4.0, 4096)
        for e, n in enumerate(lens):
            k, v = f64(s["keys_held"][start:start + n]), f64(s["kv_held"][start:start + n])
            np.testing.assert_array_equal(read_cache(kv, e, [0, n // 2, n - 1]), v[[0, n // 2, n - 1]])
            start += n
            args = f64(s["qi_r"][e]), f64(s["w"][e]), k
            got = f64(s["scores"][e, :n])
            assert np.all(np.abs(got - oracle.indexer_score(*args)) <= SCORE_RTOL * score_bound(*args))
            sel = idx[512 * e: 512 * e + min(512, n)]
            np.testing.assert_array_equal(sel, oracle.topk(got, min(512, n)))
            want, _ = oracle.sparse_attention(f64(s["qa_r"][e]), v, sel, f64(s["sinks"]), SCALE)
            check_out(f64(s["attn"][e]), want)
            back = ref.rope(f64(s["attn"][e:e + 1]), f64(at[e:e + 1]), theta, 448, "interleaved", 1.0, True)[0]
            check_out(f64(s["out"][e]), back)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for seed in (2, 3):
        fill(seed)
        perm = torch.randperm(total, device="cuda").to(torch.int32)
        for c in (keys, kv):
            old = c.page_table.clone()
            c.page_table.copy_(torch.where(old >= 0, perm[old.clamp(min=0).long()], old))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("dim", [128, 512])
def test_pools_past_32_bits(fmt, dim):
    """Pages that begin past 4 GiB: appended rows read as from a small pool."""
    page, n = 64, 150
    size = ds.ds_rows_page_bytes(page, dim, fmt)
    total = (1 << 32) // size + 5
    x = torch.randn(n, dim, device="cuda")
    q, w = queries(np.random.default_rng(0), 1, dim), torch.ones(1, 64, device="cuda")
    got = []
    for num, ids in ((total, [total - 1, total - 3, total - 2]), (3, [0, 2, 1])):
        cache = ds.PagedCache(torch.empty(num, size, dtype=torch.uint8, device="cuda"), i32([ids]), page, dim, fmt)
        values = torch.zeros(n, dim, dtype=BF16, device="cuda")
        ds.ds_rows_append(cache, x, i32(np.zeros(n)), i32(range(n)), values=values)
        if dim == 128:
            out = torch.zeros(n, device="cuda")
            ds.ds_rows_indexer_score_paged([(n, n, 0, 0)], q, w, cache, out)
        else:
            out = torch.zeros_like(q)
            ds.ds_rows_sparse_attn_paged([(n, n, 0, 0)], q, torch.zeros(64, device="cuda"), 0, i32(range(n)), SCALE, out,
                                         cache)
        got.append((out, values))
        del cache
    assert got[0][0].any() and torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_the_longest_rows(fmt):
    """kv_len 2^31 - 1, one page under every place of the table: the page's scores over and
    over (the second row's begin past 2^33 bytes), and its rows under the last indices."""
    n, page = 2 ** 31 - 1, 256
    places = -(-n // page)
    rng = np.random.default_rng(15)
    table = torch.zeros(2, places, dtype=torch.int32, device="cuda")
    one, values = make_cache(rng, [page], 128, fmt, page)
    keys = ds.PagedCache(one.pages, table + one.page_table[0, 0], page, 128, fmt)
    q, w = queries(rng, 2, 128), torch.rand(2, 64, device="cuda")
    short = torch.zeros(2, page, device="cuda")
    both = ds.PagedCache(one.pages, one.page_table[:, :1].expand(2, 1).contiguous(), page, 128, fmt)
    ds.ds_rows_indexer_score_paged(row_table([page, page]), q, w, both, short)
    scores = torch.zeros(n + 1 + 999, device="cuda")
    ds.ds_rows_indexer_score_paged([(n, 512, 0, 0), (999, 512, 512, 1)], q, w, keys, scores, score_stride=n + 1)
    assert scores[n] == 0 and torch.equal(scores[n + 1:], short[1].repeat(4)[:999])
    assert torch.equal(scores[n - 255:n], short[0, :255])
    body = scores[:n - 255].view(-1, page)
    assert all(torch.equal(part, short[0].expand_as(part)) for part in body.split(1 << 20))
    del scores, body
    one, values = make_cache(rng, [page], 512, fmt, page)
    kv = ds.PagedCache(one.pages, table[:1] + one.page_table[0, 0], page, 512, fmt)
    idx = np.r_[n - 1 - rng.permutation(300)[:99], 0]
    q, sinks = queries(rng, 1, 512), torch.zeros(64, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.full((ds.PAGED_WORKSPACE_BYTES,), 255, dtype=torch.uint8, device="cuda")
    with pytest.raises(ds.DsRowsError, match="workspace holds"):
        ds.ds_rows_sparse_attn_paged([(n, 100, 0, 0)], q, sinks, 0, i32(idx), SCALE, out, kv, workspace_t=ws[:255])
    ds.ds_rows_sparse_attn_paged([(n, 100, 0, 0)], q, sinks, 0, i32(idx), SCALE, out, kv, workspace_t=ws)
    assert ds.workspace_status(ws) == 0 and (ws[4:] == 255).all()
    want, _ = oracle.sparse_attention(f64(q[0]), values[0].astype(np.float64), np.sort(idx) % page, f64(sinks), SCALE)
    check_out(f64(out[0]), want)


def test_two_streams_at_once():
    """Calls on two streams with their own outputs and workspaces, interleaved; one
    stream given as an argument, its workspace left to the binding."""
    rng = np.random.default_rng(13)
    lens = [3000, 700]
    rows = row_table(lens)
    cache, values = make_cache(rng, lens, 512, "int4", 64)
    idx = i32(np.concatenate([rng.permutation(n)[:512] for n in lens]))
    sinks = torch.zeros(64, device="cuda")
    qs = [queries(rng, 2, 512) for _ in range(2)]
    want = [attend(rows, q, sinks, 0, idx, cache, values)[0] for q in qs]
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for q, o, st in zip(qs, outs, streams):
            ds.ds_rows_sparse_attn_paged(rows, q, sinks, 0, idx, SCALE, o[i], cache, stream=st)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_captured_calls_of_two_graphs_without_a_workspace():
    """Two graphs whose workspaces the binding takes during capture, replayed in turn and
    on two streams at once."""
    rng = np.random.default_rng(14)
    lens = [900, 64]
    rows = row_table(lens)
    cache, values = make_cache(rng, lens, 512, "int4", 32)
    idx = i32(np.concatenate([np.r_[rng.permutation(n)[:512], np.full(max(0, 512 - n), -1)] for n in lens]))
    sinks = torch.zeros(64, device="cuda")
    qs = [queries(rng, 2, 512) for _ in range(2)]
    want = [attend(rows, q, sinks, 0, idx, cache, values)[0] for q in qs]
    outs = [torch.zeros_like(q) for q in qs]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for q, o, st in zip(qs, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(4):
                ds.ds_rows_sparse_attn_paged(rows, q, sinks, 0, idx, SCALE, o, cache)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(w, o) for w, o in zip(want, outs))


def test_cache_refusals_of_the_binding():
    pages = torch.zeros(18432 * 2, dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for args, err in (((pages[:-1], table, 64, 512, "int4"), ValueError), ((pages[:0], table, 64, 512, "int4"), ValueError),
                      ((pages, table.long(), 64, 512, "int4"), TypeError), ((pages, table[0], 64, 512, "int4"), ValueError),
                      ((pages, table.cpu(), 64, 512, "int4"), ValueError), ((pages[::2], table, 64, 512, "int4"), ValueError),
                      ((pages, table, 63, 512, "int4"), ds.DsRowsError)):
        with pytest.raises(err):
            ds.PagedCache(*args)
    cache = ds.PagedCache(pages, table, 64, 512, "int4")
    q, out = (torch.zeros(1, 64, 512, dtype=BF16, device="cuda") for _ in range(2))
    idx = torch.zeros(512, dtype=torch.int32, device="cuda")
    sinks = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="negative"):
        ds.ds_rows_sparse_attn_paged([(100, 10, 0, 0)], q, sinks, -64, idx, SCALE, out, cache)
    with pytest.raises(ValueError, match="negative"):
        ds.ds_rows_indexer_score_paged([(100, 100, 0, 0)] * 2, q, torch.zeros(1, 64, device="cuda"), cache,
                                       torch.zeros(100, device="cuda"), score_stride=-100)
    with pytest.raises(ds.DsRowsError, match="exceeds the 2 pages"):
        ds.ds_rows_sparse_attn_paged([(129, 10, 0, 0)], q, sinks, 0, idx, SCALE, out, cache)
    with pytest.raises(ValueError, match="q_attn"):
        ds.ds_rows_sparse_attn_paged([(100, 10, 0, 1)], q, sinks, 0, idx, SCALE, out, cache)
    with pytest.raises(ds.DsRowsError, match="128 wide"):
        ds.ds_rows_indexer_score_paged([(100, 100, 0, 0)], q, torch.zeros(1, 64, device="cuda"), cache,
                                       torch.zeros(100, device="cuda"))
