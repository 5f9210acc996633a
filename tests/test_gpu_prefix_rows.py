"""ds_rows_prefix_attn on rows made to show one thing each: that every slot is counted once, that what was
accumulated is scaled when the maximum rises within a pair's run, and that logits of any finite size are sound.
"""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from test_gpu_fp8 import FORMATS
from test_gpu_paged import BF16, SCALE, f64, i32
from test_gpu_prefix import check, table

pytestmark = pytest.mark.gpu

PAIRS = 76  # of the chip's processors: with more tiles than these a pair has a run of several


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ds.build()
    ds.load()


def cache_of(rng, shared, own, fmt, page):
    """A cache of the rows [n, 512] that entries share and of each entry's own, whole pages of the first shared; returns it
    with the rows that each entry attends to, as the cache holds them."""
    prefix, whole = len(shared), len(shared) // page
    need = [max(-(-(prefix + len(x)) // page), 1) for x in own]
    ids = rng.permutation(whole + sum(n - whole for n in need) + 2)
    t, at = np.full((len(own), max(need)), -1), whole
    for e, n in enumerate(need):
        t[e, :whole] = ids[:whole]
        t[e, whole:n] = ids[at:at + n - whole]
        at += n - whole
    cache = ds.PagedCache.empty(len(ids), i32(t), page, 512, fmt)
    cache.pages.view(torch.uint8).fill_(0xFF)  # NaN wherever no row is

    def put(rows, entry, first):
        x = torch.as_tensor(rows, dtype=torch.float32).cuda()
        held = torch.zeros(len(x), 512, dtype=BF16, device="cuda")
        slot = i32(first + np.arange(len(x)))
        ds.ds_rows_append(cache, x, torch.full_like(slot, entry), slot, values=held)
        return held.float()
    head = put(shared, 0, 0)
    return cache, [torch.cat([head, put(x, e, prefix)]) if len(x) else head for e, x in enumerate(own)]


def attend(cache, prefix, tails, q, sinks, fmt):
    """The call, for packed rows with and without room to widen them beforehand: the same bits; no wait gives up."""
    rows, got = table(prefix, tails), []
    for f in dict.fromkeys(("bf16", fmt)):
        ws = ds.prefix_attn_workspace(rows, prefix, f)
        out, bad = torch.full_like(q, 4.0), torch.full(q.shape[:2], 9, dtype=torch.int32, device="cuda")
        ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 0, SCALE, out, cache, invalid=bad, workspace_t=ws)
        assert ds.workspace_status(ws) == 0
        got.append((out, bad))
    assert torch.equal(got[0][0].view(torch.int16), got[-1][0].view(torch.int16)) and torch.equal(got[0][1], got[-1][1])
    return got[0]


def tiles(prefix, tails):
    up = lambda n: -(-n // 128)  # noqa: E731
    return -(-len(tails) // 2) * up(prefix) + sum(map(up, tails))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("prefix,tails", [
    (20000, [0]), (20009, [1]), (30000, [0, 7]), (20000, [5, 0, 9]), (10299, [0]), (0, [9000, 1, 20000]),
    (130, [300 + i for i in range(64)]), (9999, [300] * 5), (3001, [1 + 7 * i for i in range(63)]), (6000, [1] * 8), (300, [1, 40]),
    (0, [1000, 8192, 3000, 5001, 1, 129, 127, 128]), (40000, [0] * 2), (12800, [128] * 7),
])
def test_every_slot_counts_once(fmt, page, prefix, tails):
    """With q = 0 every weight is 1. A row is 7 (exact in every type) at the dim of its tile, so an output is
    7 count / (slots + 1): whole numbers in fp32, one reciprocal and one product (2^-24 each, and half as much again
    for the reciprocal's use), rounded to bf16 (2^-8). A slot more or less in a tile of 128 changes it by 2^-7."""
    rng = np.random.default_rng(prefix + page)

    def marked(n, first):
        x = np.zeros((n, 512), np.float32)
        x[np.arange(n), (first + np.arange(n) // 128) % 512] = 7.0
        return x
    cache, held = cache_of(rng, marked(prefix, 0), [marked(n, 200 + 3 * e) for e, n in enumerate(tails)], fmt, page)
    n = len(tails)
    out, bad = attend(cache, prefix, tails, torch.zeros(n, 64, 512, dtype=BF16, device="cuda"),
                      torch.zeros(64, device="cuda"), fmt)
    assert not bad.any()
    for e in range(n):
        assert set(held[e].unique().tolist()) <= {0.0, 7.0}
        want = held[e].double().sum(0) / (len(held[e]) + 1)
        assert ((out[e].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -22)).all(), f"row {e}"


def spiked(rng, n, first):
    """Rows of a run whose first tile is number `first`: a slot of each tile stands out in dim (tile mod 8)."""
    x = rng.standard_normal((n, 512)).astype(np.float32)
    x[:, :16] = 0  # the spikes' dims, a group of the 4-bit type
    t = first + np.arange(n // 128)
    at = 128 * np.arange(n // 128)
    at += rng.integers(0, 128, len(at))
    x[at, t % 8] = np.where(t % 16 < 8, 1.0, 2.0)
    return x


def spiked_queries(n):
    """Heads 8 k + d see the spikes of dim d; the others' dims add little."""
    q = torch.zeros(n, 64, 512)
    q[:, torch.arange(64), torch.arange(64) % 8] = 9.5 / (SCALE * 1.4427)
    q[:, :, 16:] = 0.02 * torch.randn(n, 64, 496, generator=torch.Generator().manual_seed(1))
    return q.to(BF16).cuda()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("prefix,tails", [(40000, [0]), (0, [9000, 12000, 30000]), (20000, [300] * 5), (31000, [0, 9]),
                                          (4000, [1500] * 9), (0, [38000])])
def test_the_maximum_rises_within_a_run(fmt, prefix, tails):
    """Slots of nearly equal logits, and in a tile here and there one that stands 9.5 ln 2 (later 19 ln 2) above all before:
    it weighs as much as some hundred of the others, so both what was accumulated and what comes count."""
    assert tiles(prefix, tails) > 3 * PAIRS
    rng = np.random.default_rng(prefix + len(tails))

    cache, held = cache_of(rng, spiked(rng, prefix, 0), [spiked(rng, n, 5 * e) for e, n in enumerate(tails)], fmt, 64)
    n = len(tails)
    q = spiked_queries(n)
    out, bad = attend(cache, prefix, tails, q, torch.zeros(64, device="cuda"), fmt)
    assert not bad.any()
    check(out, q, held, torch.zeros(64, device="cuda"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("prefix,tails", [(300, [1, 17, 40]), (20000, [700, 3]), (0, [5000, 130, 12000])])
def test_logits_of_any_finite_size(fmt, prefix, tails):
    """Query vectors along one dim, from 2^20 to 2^110: the largest logit is further from the others than any weight
    reaches, and the output is its row, bit for bit (its weight is 1, the sum is 1)."""
    rng = np.random.default_rng(len(tails))

    def rows(n):
        x = rng.standard_normal((n, 512)).astype(np.float32)
        x[:, 0] = rng.uniform(-0.5, 0.5, n)
        x[:, 1:16] = 0.25 * np.clip(x[:, 1:16], -1, 1)  # the rest of the first dim's group of 16
        return x
    shared, own = rows(prefix), [rows(n) for n in tails]
    for x in own + [shared]:
        if len(x) > 1:
            low, high = rng.permutation(len(x))[:2]
            x[low, 0], x[high, 0] = -1.5 - 0.25 * (x is shared), 1.5 + 0.25 * (x is shared)
    cache, held = cache_of(rng, shared, own, fmt, 32)
    n = len(tails)
    size = 2.0 ** np.linspace(20, 110, 32).round()
    q = torch.zeros(n, 64, 512)
    q[:, :, 0] = torch.from_numpy(np.r_[size, -size])
    out, bad = attend(cache, prefix, tails, q.to(BF16).cuda(), torch.zeros(64, device="cuda"), fmt)
    assert not bad.any()
    for e in range(n):
        first = held[e][:, 0]
        for heads, at in ((slice(0, 32), first.argmax()), (slice(32, 64), first.argmin())):
            assert (first == first[at]).sum() == 1 and first[at].abs() > 1
            assert torch.equal(out[e, heads], held[e][at].to(BF16).expand(32, 512)), f"row {e}"


def test_a_call_of_several_seconds():
    """26 rows over 2^31 - 1 slots of the same four pages: a pair of processors works for seconds on a run of 2.9 million
    tiles. No wait gives up, and the sums come out: with weights and rows of ones they are whole numbers, and those of a
    piece of 512 tiles, 2^16, and of the pieces, multiples of it below 2^40, are exact in 32 bits."""
    slots, page, n = (1 << 31) - 1, 256, 26
    places = -(-slots // page)
    assert tiles(slots, [0] * n) > 2800000 * PAIRS
    table_ = torch.arange(places, dtype=torch.int32, device="cuda").remainder_(4).expand(n, places).contiguous()
    cache = ds.PagedCache(torch.ones(4, page, 512, dtype=BF16, device="cuda"), table_, page, 512, "bf16")
    rows = table(slots, [0] * n)
    ws = ds.prefix_attn_workspace(rows, slots, "bf16")
    out, bad = torch.zeros(n, 64, 512, dtype=BF16, device="cuda"), torch.full((n, 64), 9, dtype=torch.int32, device="cuda")
    ds.ds_rows_prefix_attn(rows, slots, torch.zeros_like(out), torch.zeros(64, device="cuda"), 0, SCALE, out, cache,
                           invalid=bad, workspace_t=ws)
    assert ds.workspace_status(ws) == 0
    assert not bad.any() and (out == 1).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_runs_of_several_pieces(fmt):
    """64 rows over 170003 shared slots: a pair's run is longer than the 512 tiles of a piece. Once with marked rows and
    weights of 1 (a slot more or less in a tile's dim, whose three tiles count 384, changes an output by 2^-8.6: the bound
    shows a tile, 2^-1.6), once with maxima that rise."""
    prefix, tails = 170003, [0] * 62 + [1, 300]
    assert tiles(prefix, tails) > 520 * PAIRS
    rng = np.random.default_rng(5)
    n, sinks = len(tails), torch.zeros(64, device="cuda")
    x = np.zeros((prefix, 512), np.float32)
    x[np.arange(prefix), np.arange(prefix) // 128 % 512] = 7.0
    own = [np.zeros((t, 512), np.float32) for t in tails]
    own[-1][:, 5] = 7.0
    cache, held = cache_of(rng, x, own, fmt, 128)
    out, bad = attend(cache, prefix, tails, torch.zeros(n, 64, 512, dtype=BF16, device="cuda"), sinks, fmt)
    assert not bad.any()
    for e in range(n):
        want = held[e].double().sum(0) / (len(held[e]) + 1)
        assert ((out[e].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -22)).all(), f"row {e}"
    del cache, held
    cache, held = cache_of(rng, spiked(rng, prefix, 0), [rng.standard_normal((t, 512)) for t in tails], fmt, 64)
    q = spiked_queries(n)
    out, bad = attend(cache, prefix, tails, q, sinks, fmt)
    assert not bad.any()
    check(out, q, held, sinks)


@pytest.mark.parametrize("fmt", FORMATS)
def test_in_place_and_captured_without_a_workspace(fmt):
    """The output over the queries gives the same bits; so do replays of a capture that takes its workspace from the
    graph's memory, between other captured work."""
    rng = np.random.default_rng(6)
    prefix, tails = 9000, [3, 700, 0, 1, 64]
    make = lambda n: rng.standard_normal((n, 512)).astype(np.float32)  # noqa: E731
    cache, held = cache_of(rng, make(prefix), [make(n) for n in tails], fmt, 64)
    n, sinks = len(tails), torch.randn(64, device="cuda")
    q = torch.randn(n, 64, 512, device="cuda").to(BF16)
    want, _ = attend(cache, prefix, tails, q, sinks, fmt)
    check(want, q, held, sinks)
    rows = table(prefix, tails)
    both = q.clone()
    ds.ds_rows_prefix_attn(rows, prefix, both, sinks, 0, SCALE, both, cache)
    assert torch.equal(both, want)
    out, kept, graph = torch.zeros_like(q), q.clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        scratch = torch.full((1 << 20,), 7.0, device="cuda")
        ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 0, SCALE, out, cache)
        more = scratch * 2  # may take the workspace's place, behind the call
        total = more.sum()
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want) and total.item() == 14.0 * (1 << 20)
        q.copy_(torch.randn_like(q))
        graph.replay()
        check(out, q, held, sinks)
        q.copy_(kept)
