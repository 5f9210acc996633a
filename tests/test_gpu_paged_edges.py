"""Rotary positions and paged caches at the edges of what their documentation allows: shapes,
strides and streams that tests/test_gpu_paged.py leaves out."""

from decimal import Decimal

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from test_rope_table import TWO_PI, exact_turns

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ds.build()
    ds.load()


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int64), dtype=torch.int32).cuda()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(1, (1 << 32) + 8, 2), (1, 1, (1 << 32) + 64)])
def test_rope_refuses_shapes_past_32_bits(shape):
    """Cut to 32 bits, these would be 8 heads of 2, and one of 64."""
    x = torch.empty(shape, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="2\\^32"):
        ds.ds_rows_rope(ds.Rope(2), x, i32([5]), x)


def test_cache_refuses_tables_past_32_bits():
    pages = torch.zeros(ds.ds_rows_page_bytes(16, 128, "int4"), dtype=torch.uint8, device="cuda")
    table = torch.empty(1, (1 << 32) + 1, dtype=torch.int32, device="cuda")  # would have been one page an entry
    with pytest.raises(ValueError, match="side of page_table"):
        ds.PagedCache(pages, table, 16, 128, "int4")


# ---------------------------------------------------------------------------
# strides
# ---------------------------------------------------------------------------

def test_rope_of_a_lone_token_of_a_wide_buffer():
    """A token taken from a buffer whose tokens lie 2^32 elements apart, and one head of such a buffer."""
    rope, pos = ds.Rope(64), i32([77])
    data = torch.randn(4, 64, device="cuda")
    want = torch.empty(1, 4, 64, device="cuda")
    ds.ds_rows_rope(rope, data[None], pos, want)
    x = torch.as_strided(data, (1, 4, 64), (1 << 32, 64, 1))
    out = torch.empty_like(want)
    ds.ds_rows_rope(rope, x, pos, out)
    assert torch.equal(out, want)
    x = torch.as_strided(data, (4, 1, 64), (64, 1 << 32, 1))
    ds.ds_rows_rope(rope, x, pos.repeat(4), out.view(4, 1, 64))
    assert torch.equal(out, want)
    ds.ds_rows_rope(rope, torch.as_strided(data, (1, 4, 64), (1 << 40, 64, 1)), pos, data.view(1, 4, 64))
    assert torch.equal(data, want[0])


# ---------------------------------------------------------------------------
# many heads: a thread rotates several of them
# ---------------------------------------------------------------------------

ROPE_RTOL = 5e-7  # of m (|a| + |b|), derived at the head of tests/test_gpu_paged.py


def check_rotated(got, x, pos, rot, first, layout, magnitude, inverse, fill):
    """Every element of got against 64-bit arithmetic on x; rows of negative positions hold `fill`."""
    dtype, half = x.dtype, rot // 2
    theta = torch.from_numpy(10000.0 ** (-2.0 * np.arange(half) / rot)).cuda()
    angle = pos.double()[:, None, None] * theta * (-1.0 if inverse else 1.0)
    c, s = magnitude * angle.cos(), magnitude * angle.sin()
    at = torch.arange(half, device="cuda")
    a, b = (first + 2 * at, first + 2 * at + 1) if layout == "interleaved" else (first + at, first + half + at)
    xa, xb = x[..., a].double(), x[..., b].double()
    live = pos >= 0
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    size = ROPE_RTOL * magnitude * (xa.abs() + xb.abs()) + tiny
    for part, want in ((a, xa * c - xb * s), (b, xa * s + xb * c)):
        bound = size + want.abs() * (torch.finfo(dtype).eps / 2) * (1 + 1e-6)
        bad = (got[..., part].double() - want).abs() > bound
        assert not bad[live].any(), torch.nonzero(bad & live[:, None, None])[0].tolist()
    rest = torch.ones(x.shape[-1], dtype=torch.bool, device="cuda")
    rest[first:first + rot] = False
    assert torch.equal(got[live][..., rest], x[live][..., rest]) and torch.equal(got[~live], fill[~live])


# Shapes by what they reach on 152 SMs, where a thread takes twice the heads while 512 threads an SM
# are left: heads a thread, and whether the groups divide the heads.
@pytest.mark.parametrize("dtype,tokens,heads,dim,rot,first,shift", [
    (F32, 160, 33, 128, 64, 64, 0),      # 2 (out of place)
    (F32, 300, 64, 128, 128, 0, 0),      # 4
    (BF16, 700, 64, 128, 64, 64, 0),     # 8
    (BF16, 4900, 13, 128, 64, 64, 0),    # 16, one group of 13
    (BF16, 1300, 65, 128, 64, 0, 0),     # 16, the last one short; in place 4 or 8
    (F16, 2500, 65, 64, 64, 0, 0),       # 16; in place 8
    (F32, 1021, 64, 512, 64, 448, 0),    # 16; in place 4 or 8
    (BF16, 13000, 7, 96, 64, 32, 0),     # 8 (rows of 12 pieces: the half layout's out of place too)
    (BF16, 4000, 7, 41, 16, 2, 1),       # 8, element by element (in place 2)
    (F32, 2500, 13, 70, 64, 4, 1),       # 8, element by element
    (F16, 1300, 65, 129, 6, 122, 1),     # the same, most of a row copied
])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_of_many_heads(dtype, tokens, heads, dim, rot, first, shift, layout, inplace, inverse):
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    wide = dim + 8 if shift else dim
    x = torch.randn(tokens, heads, wide, generator=g, device="cuda").to(dtype)[..., shift:shift + dim]
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    pos[5::97] = -1
    rope = ds.Rope(rot, first=first, layout=layout, magnitude=1.25)
    keep = x.clone()
    out = x if inplace else torch.full((tokens, heads, wide), 7.0, dtype=dtype, device="cuda")[..., shift:shift + dim]
    fill = out.clone()
    ds.ds_rows_rope(rope, x, pos, out, inverse=inverse)
    check_rotated(out, keep, pos, rot, first, layout, 1.25, inverse, fill)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inplace", [False, True])
def test_rope_of_many_heads_outside_the_tokens(layout, inplace):
    """Heads that lie outside the tokens, rows inside wider ones, sixteen (in place eight) a thread."""
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(21, 3000, 192, generator=g, device="cuda").to(BF16).transpose(0, 1)[..., 32:160]
    pos = torch.randint(0, 1 << 20, (3000,), generator=g, device="cuda", dtype=torch.int32)
    pos[::41] = -9
    base = torch.full((21, 3000, 136), 7.0, dtype=BF16, device="cuda")
    keep = x.clone()
    out = x if inplace else base.transpose(0, 1)[..., 8:]
    fill = out.clone()
    ds.ds_rows_rope(ds.Rope(64, first=32, layout=layout), x, pos, out)
    check_rotated(out, keep, pos, 64, 32, layout, 1.0, False, fill)
    assert (base[..., :8] == 7.0).all()

# ---------------------------------------------------------------------------
# the largest calls
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("tokens,heads,dim", [(2 ** 31 - 1, 1, 2), (32767, 65536, 8), (2 ** 31 // 65535, 65535, 8)])
def test_rope_of_the_most_rows(layout, tokens, heads, dim):
    """2^31 - 1 rows at most, in place: the first and the last as in small calls, others between
    them; one row more is refused."""
    x = torch.ones(tokens, heads, dim, dtype=BF16, device="cuda")
    pos = torch.full((tokens,), 3, dtype=torch.int32, device="cuda")
    pos[-2:] = 77
    pos[-1] = -1
    rope = ds.Rope(dim, layout=layout)
    small = torch.ones(3, 1, dim, dtype=BF16, device="cuda")
    ds.ds_rows_rope(rope, small, i32([3, 77, -1]), small)
    ds.ds_rows_rope(rope, x, pos, x)
    assert torch.equal(x[-2], small[1].expand(heads, dim)) and torch.equal(x[-1], torch.ones_like(x[-1]))
    assert all((part == small[0]).all() for part in x[:-2].split(max(1, (1 << 28) // heads)))
    del x
    more = torch.empty(1, 1, dim, dtype=BF16, device="cuda").expand(2 ** 31 // heads + 1, heads, dim)
    with pytest.raises(ds.DsRowsError, match="below 2"):
        ds.ds_rows_rope(rope, more, torch.empty(more.shape[0], dtype=torch.int32, device="cuda"), more)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_append_of_the_most_rows(fmt):
    """2^31 - 1 rows from one broadcast row, all padding but the first and the last two."""
    n = 2 ** 31 - 1
    x = torch.randn(1, 128, device="cuda").to(BF16)
    seq = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slot = torch.zeros(n, dtype=torch.int32, device="cuda")
    seq[0] = seq[-2] = seq[-1] = 0
    slot[-2], slot[-1] = 17, 33
    pages = [torch.full((3, ds.ds_rows_page_bytes(16, 128, fmt)), 90, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = i32([[2, 0, 1]])
    invalid = torch.full((n,), 9, dtype=torch.int32, device="cuda")
    ds.ds_rows_append(ds.PagedCache(pages[0], table, 16, 128, fmt), x.expand(n, 128), seq, slot, invalid=invalid)
    assert not invalid.any()
    ds.ds_rows_append(ds.PagedCache(pages[1], table, 16, 128, fmt), x.expand(3, 128), i32([0, 0, 0]), i32([0, 17, 33]))
    assert torch.equal(pages[0], pages[1]) and (pages[0] != 90).any()


# ---------------------------------------------------------------------------
# angles
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("rot,base,factor", [(64, 1e4, 1.0), (64, 1e4, 40.0), (128, 5e6, 1.0), (512, 5e5, 8.0), (6, 1e4, 1.0)])
def test_sines_of_small_angles(layout, inverse, rot, base, factor):
    """Pairs (1, 0) at near positions: cosine and sine to 3e-7 of themselves, however small.
    The remainder is rounded twice and its constant once (two steps of 2^-24 and 2.8e-8: 1.5e-7 of
    r, so at most 1.5e-7 of a sine and 1.2e-7 of a cosine), the polynomial's last step 2^-24 of a
    sine and 4.2e-8 of a cosine, its inner steps 3e-8 and 5e-8, the terms left out 3e-9 and
    3.5e-8; products with 1 and 0 are exact: 2.5e-7 at most. 1e-16: the low word's rounding where
    the high one is -1."""
    pos = np.r_[np.arange(1, 40), 100, 1000, 4097, 30000]
    theta = base ** (-2.0 * np.arange(rot // 2) / rot) / factor
    angle = pos[:, None] * theta
    # Both sides round the angle in 64 bits: 2^-52 of it, whatever the size of its sine; the
    # table's half step is 2 pi 2^-65 a position.
    x = torch.zeros(len(pos), 1, rot, device="cuda")
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if layout == "interleaved" else (slice(0, rot // 2), slice(rot // 2, rot))
    x[..., a] = 1.0
    rope = ds.Rope(rot, layout=layout, base=base, factor=factor)
    for out in (torch.empty_like(x), x):
        ds.ds_rows_rope(rope, x, i32(pos), out, inverse=inverse)
        got = out[:, 0].double().cpu().numpy()
        for part, want in ((a, np.cos(angle)), (b, np.sin(-angle if inverse else angle))):
            err = np.abs(got[:, part] - want)
            bound = 3e-7 * np.abs(want) + 1e-16 + angle * 2.0 ** -52 + pos[:, None] * 2.0 ** -62
            assert np.all(err <= bound), np.max(err / np.abs(want))


@pytest.mark.parametrize("rot,kw", [(64, dict(base=1e4)), (512, dict(base=1e4)), (128, dict(base=5e5, factor=8.0)),
                                    (64, dict(base=1e4, factor=16.0, original_len=65536))])
def test_sines_at_the_last_positions(rot, kw):
    """The bound of test_sines_of_small_angles at positions up to 2^31 - 1, against angles reduced
    in 60 decimal digits; the table's half step is 2 pi 2^-65 a position (3.7e-10 at the last)."""
    pos = np.r_[2 ** 31 - 1 - np.arange(20), 2 ** 30 + 12345, 10 ** 9, 123456789, 2 ** 24 + 1]
    full = [int(t * 2 ** 128) for t in exact_turns(rot, kw["base"], kw.get("factor", 1.0), kw.get("original_len", 0))]
    turn = np.array([[float(Decimal(int(p) * f % 2 ** 128) / 2 ** 128) for f in full] for p in pos])
    near = np.round(4 * turn)  # quarter turns, and the rest in radians: each value to 2^-52 of itself
    angle = np.array([[float((Decimal(int(p) * f % 2 ** 128) / 2 ** 128 - Decimal(k / 4)) * TWO_PI)
                       for f, k in zip(full, ks)] for p, ks in zip(pos, near)])
    c, s = np.cos(angle), np.sin(angle)
    k = near.astype(int) % 4
    cos, sin = np.choose(k, [c, -s, -c, s]), np.choose(k, [s, c, -s, -c])
    x = torch.zeros(len(pos), 1, rot, device="cuda")
    x[..., : rot // 2] = 1.0
    ds.ds_rows_rope(ds.Rope(rot, layout="half", **kw), x, i32(pos), x)
    got = x[:, 0].double().cpu().numpy()
    for part, want in ((got[:, : rot // 2], cos), (got[:, rot // 2:], sin)):
        assert np.all(np.abs(part - want) <= 3e-7 * np.abs(want) + 1e-16 + pos[:, None] * 2.0 ** -62)


# ---------------------------------------------------------------------------
# indexer scores
# ---------------------------------------------------------------------------

def appended(lens, fmt, page, seed, dim=128):
    """A cache of random rows, its pages in no order, and the bf16 rows that it stands for."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    places = -(-max(lens) // page)
    table = torch.randperm(len(lens) * places, generator=g, device="cuda").to(torch.int32).view(len(lens), places)
    cache = ds.PagedCache.empty(len(lens) * places, table, page, dim, fmt)
    held = []
    for e, n in enumerate(lens):
        held.append(torch.empty(n, dim, dtype=BF16, device="cuda"))
        ds.ds_rows_append(cache, torch.randn(n, dim, generator=g, device="cuda"),
                          torch.full((n,), e, dtype=torch.int32, device="cuda"),
                          torch.arange(n, dtype=torch.int32, device="cuda"), values=held[-1])
    return cache, held, g


def row_table(lens):
    return [(n, min(512, n), 512 * e, e) for e, n in enumerate(lens)]


def scores_both_ways(cache, held, lens, q, w):
    out = [torch.full((len(lens), max(lens)), 123.0, device="cuda") for _ in range(2)]
    ds.ds_rows_indexer_score_paged(row_table(lens), q, w, cache, out[0])
    ds.ds_rows_indexer_score(row_table(lens), q, w, held, out[1])
    return out


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17, 127, 128, 129, 255, 257], [30000, 3, 4097]])
def test_scores_are_those_of_the_rows_held(fmt, page, lens):
    cache, held, g = appended(lens, fmt, page, 25)
    q = torch.randn(len(lens), 64, 128, generator=g, device="cuda").to(BF16)
    w = torch.randn(len(lens), 64, generator=g, device="cuda") / 8
    paged, plain = scores_both_ways(cache, held, lens, q, w)
    assert torch.equal(paged, plain) and torch.isfinite(paged).all()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("power", [1, -100, -124, -126, -130, -140, -148, 120, 126])
def test_scores_with_weights_of_any_size(fmt, power):
    """Bitwise the contiguous scores of the keys that the cache stands for, where products fall
    below the normal range, where weights themselves do, and where sums overflow."""
    lens = [3000, 129]
    cache, held, g = appended(lens, fmt, 64, 23)
    q = torch.randn(2, 64, 128, generator=g, device="cuda").to(BF16)
    w = (torch.randn(2, 64, generator=g, device="cuda").double() * 2.0 ** power).float()
    paged, plain = scores_both_ways(cache, held, lens, q, w)
    assert torch.equal(paged, plain)
    w[0, 5:] = 0  # one head alone, and one of ordinary size beside the small ones
    w[1, 7] = 1.0
    paged, plain = scores_both_ways(cache, held, lens, q, w)
    assert torch.equal(paged, plain)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_scores_of_products_that_overflow(fmt):
    """Dot products near the largest float (and infinite ones), under weights of every sign and zero."""
    lens = [1500]
    cache, held, g = appended(lens, fmt, 64, 24)
    q = torch.randn(1, 64, 128, generator=g, device="cuda") * 2.0 ** torch.randint(118, 128, (1, 64, 1), generator=g,
                                                                                 device="cuda")
    w = torch.randn(1, 64, generator=g, device="cuda") * 2.0 ** -8
    w[0, ::3] = 0
    for x in (q, q.clamp(-1e38, 1e38) / 16):
        paged, plain = scores_both_ways(cache, held, lens, x.to(BF16), w)
        assert torch.equal(paged, plain)
    assert torch.isfinite(plain).any() and torch.isneginf(paged).sum() < 1500


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("size", [1.0, 1e4, 1e37])
def test_attention_of_values_at_the_ends(fmt, size):
    """Queries, sinks and logits that are infinite, NaN, the lowest and past the range: bitwise the
    contiguous call on the rows held, flags among it."""
    lens = [700, 600, 129, 128, 127, 2, 1, 513]
    widths = [512, 385, 129, 128, 127, 2, 1, 384]
    cache, held, g = appended(lens, fmt, 32, 51, 512)
    rows = [(n, w, 512 * e, e) for e, (n, w) in enumerate(zip(lens, widths))]
    idx = torch.full((8 * 512,), -1, dtype=torch.int32, device="cuda")
    for e, (n, w) in enumerate(zip(lens, widths)):
        idx[512 * e: 512 * e + w] = torch.randperm(n, generator=g, device="cuda")[:w]
    idx[512 + 100: 512 + 385] = -1  # chunks with no row at all
    q = (torch.randn(8, 64, 512, generator=g, device="cuda") * size).to(BF16)
    inf, nan = float("inf"), float("nan")
    for e in range(8):
        q[e, e, 3], q[e, 9 + e, 500], q[e, 18 + e, 7] = nan, inf, -inf
    sinks = torch.randn(8, 64, generator=g, device="cuda")
    low = torch.finfo(F32).min
    sinks[:, 30:38] = torch.tensor([inf, -inf, nan, low, -low, 0.0, 1e30, -1e30], device="cuda")
    ws = ds.workspace(rows)
    for scale in (512 ** -0.5, 1e30, 1e-30):
        out, plain = (torch.full_like(q, 4.0) for _ in range(2))
        bad, bad_plain = (torch.full((8, 64), 4, dtype=torch.int32, device="cuda") for _ in range(2))
        ds.ds_rows_sparse_attn_paged(rows, q, sinks, 64, idx, scale, out, cache, invalid=bad, workspace_t=ws)
        assert ds.workspace_status(ws) == 0
        ds.ds_rows_sparse_attn(rows, q, sinks, 64, idx, scale, plain, held, invalid=bad_plain, workspace_t=ws)
        assert torch.equal(out, plain) and torch.equal(bad, bad_plain)
        assert torch.isfinite(out).all() and bad[0, [0, 30, 32]].all() and not out[0, 0].any()


# ---------------------------------------------------------------------------
# beside the contiguous calls
# ---------------------------------------------------------------------------

def test_contiguous_calls_behind_a_rotation_in_place():
    """A long rotation in place, whose last rows the next call of the stream takes as its query: the
    contiguous calls fetch their query early, and the rotation lets the next launch begin early."""
    g = torch.Generator(device="cuda").manual_seed(41)
    tokens, lens = 4096, [3000, 700, 64]
    first = tokens - len(lens)
    rows = [(n, min(n, 512), 512 * e, first + e) for e, n in enumerate(lens)]
    keys = [torch.randn(n, 128, generator=g, device="cuda").to(BF16) for n in lens]
    kv = [torch.randn(n, 512, generator=g, device="cuda").to(BF16) for n in lens]
    qi = torch.randn(tokens, 64, 128, generator=g, device="cuda").to(BF16)
    qa = torch.randn(tokens, 64, 512, generator=g, device="cuda").to(BF16)
    w = torch.randn(tokens, 64, generator=g, device="cuda") / 8
    sinks = torch.randn(64, generator=g, device="cuda")
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    ri, ra = ds.Rope(64, first=64, layout="half"), ds.Rope(64, first=448)
    ws = ds.workspace(rows)

    def results(pause):
        a, b = qi.clone(), qa.clone()
        scores = torch.zeros(3, 3000, device="cuda")
        idx = torch.full((3 * 512,), -1, dtype=torch.int32, device="cuda")
        out, attn = (torch.zeros_like(qa[first:]) for _ in range(2))
        full = [torch.zeros(tokens, 64, 512, dtype=BF16, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        ds.ds_rows_rope(ri, a, pos, a)
        pause()
        ds.ds_rows_indexer_score(rows, a, w, keys, scores)
        ds.ds_rows_rope(ra, b, pos, b)
        pause()
        ds.ds_rows_decode(rows, a, w, keys, b, kv, sinks, 0, 512 ** -0.5, full[0], indices=idx, workspace_t=ws)
        ds.ds_rows_rope(ra, b, pos, b, inverse=True)
        pause()
        ds.ds_rows_sparse_attn(rows, b, sinks, 0, idx, 512 ** -0.5, full[1], kv, workspace_t=ws)
        torch.cuda.synchronize()
        assert ds.workspace_status(ws) == 0
        out.copy_(full[0][first:]), attn.copy_(full[1][first:])
        return scores, idx, out, attn

    want = results(torch.cuda.synchronize)
    assert all(t.any() for t in want)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(results(lambda: None), want))
