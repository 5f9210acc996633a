"""GPU parity of ds_rows_prefix_attn with the formula in float64.

Tolerance, for an element with A = sum_j w_j |g_j| / den. Weights: half a bf16 step, 2^-8 A, and an fp32
error each: a logit is a sum of 512 products in fp32 (512 steps of 2^-22, for the tensor cores need not
round to nearest, of scale sum |q g|) and both its rounding in units of ln 2 and the
exponential's (2^-22) are relative to sizes below 128: dl in all, entering the numerator and the denominator.
Accumulation over n slots: n 2^-22 A. Output: half a bf16 step of itself.
"""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from test_gpu_fp8 import FORMATS, make_cache
from test_gpu_paged import BF16, SCALE, f64, i32, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ds.build()
    ds.load()


def formula(q, rows, sinks, scale):
    """q [64, 512], rows [n, 512], sinks [64] in float64 (on the GPU): the output and its tolerance."""
    l = q @ rows.T * scale
    top = torch.maximum(l.amax(1), sinks) if len(rows) else sinks
    w = (l - top[:, None]).exp()
    den = w.sum(1) + (sinks - top).exp()
    out, size = w @ rows / den[:, None], w @ rows.abs() / den[:, None]
    dl = 512 * 2.0 ** -22 * scale * (q.abs() @ rows.abs().T).amax(1) + 130 * 2.0 ** -22 if len(rows) else 0 * top
    bound = size * (2.0 ** -8 + 2 * dl[:, None] + len(rows) * 2.0 ** -22) + out.abs() * 2.0 ** -8 + 2.0 ** -133
    return out, bound


def gpu64(x):
    return torch.as_tensor(x).double().cuda()


def check(out, q, held, sinks, scale=SCALE, rows=None):
    """out [.., 64, 512] against each row's held rows (a list of [n, 512] arrays)."""
    for e, g in enumerate(held):
        r = e if rows is None else rows[e]
        want, bound = formula(q[r].double(), gpu64(g), gpu64(sinks if sinks.dim() == 1 else sinks[r, :64]), scale)
        err = (out[r].double() - want).abs()
        worst = (err / bound).max().item()
        assert worst <= 1.0, f"row {e}: {worst} of the bound"


def shared_cache(rng, prefix, tails, fmt, page, scale=1.0):
    """A cache of rows that share whole pages of a prefix; returns it with the rows that each attends to."""
    whole, rest = prefix // page, prefix % page
    cache, values = make_cache(rng, [prefix + tails[0]] + [max(rest + t, 1) for t in tails[1:]], 512, fmt, page, scale)
    old = cache.page_table.cpu().numpy()
    new = np.full((len(tails), whole + old.shape[1]), -1)
    new[0, : old.shape[1]] = old[0]
    new[1:, :whole], new[1:, whole:] = old[0, :whole], old[1:]
    cache = ds.PagedCache(cache.pages, i32(new), page, 512, fmt)
    return cache, [np.concatenate([values[0][:prefix], v[(prefix if e == 0 else rest):][:tails[e]]])
                   for e, v in enumerate(values)]


def table(prefix, tails):
    return [(prefix + t, 1, 0, e) for e, t in enumerate(tails)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("prefix,tails", [
    (0, [1]), (1, [0]), (127, [0, 1]), (128, [0, 128, 129]), (129, [127, 0, 2, 1]), (300, [1, 17, 40, 5, 6]),
    (0, [5, 700, 128]), (1000, [3, 300]), (2048, [0] * 8),
])
def test_prefix_attention(fmt, page, prefix, tails):
    rng = np.random.default_rng(page + prefix + len(tails))
    cache, held = shared_cache(rng, prefix, tails, fmt, page)
    n = len(tails)
    q = queries(rng, n + 1, 512)
    sinks = torch.from_numpy(rng.standard_normal(64).astype(np.float32)).cuda()
    out = torch.full_like(q, 4.0)
    bad = torch.full((n + 1, 64), 4, dtype=torch.int32, device="cuda")
    ws = ds.prefix_attn_workspace(table(prefix, tails), prefix)
    ds.ds_rows_prefix_attn(table(prefix, tails), prefix, q, sinks, 0, SCALE, out, cache, invalid=bad, workspace_t=ws)
    assert ds.workspace_status(ws) == 0
    check(out, q, held, sinks)
    assert (out[-1] == 4.0).all() and (bad[-1] == 4).all() and not bad[:-1].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("prefix,tails", [(9999, [300] * 5), (20000, [0]), (3001, [1 + 7 * i for i in range(63)]),
                                          (0, [9000, 1, 20000]), (130, [300 + i for i in range(64)]), (30000, [0, 7]),
                                          (20000, [5, 0, 9]), (7000, [0] * 4), (6000, [1] * 8), (512, [0] * 8)])
def test_many_tiles_and_rows(fmt, prefix, tails):
    """More tiles than pairs of processors: parts that begin and end inside segments; rows in any order,
    each with its own sinks; the same bits again."""
    rng = np.random.default_rng(prefix)
    cache, held = shared_cache(rng, prefix, tails, fmt, 128)
    n = len(tails)
    q = queries(rng, n + 2, 512)
    order = rng.permutation(n + 2)[:n].tolist()
    sinks = torch.from_numpy(rng.standard_normal((n + 2, 65)).astype(np.float32)).cuda()
    rows = [(prefix + t, 0, 77, r) for t, r in zip(tails, order)]
    out, again = torch.full_like(q, 4.0), torch.full_like(q, 4.0)
    ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 65, SCALE, out, cache)
    ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 65, SCALE, again, cache)
    check(out, q, held, sinks, rows=order)
    assert torch.equal(out, again)
    unused = [r for r in range(n + 2) if r not in order]
    assert (out[unused] == 4.0).all()


@pytest.mark.parametrize("scale", [1e-3, SCALE, 0.3, 2.0])
@pytest.mark.parametrize("growing", [False, True])
def test_peaked_and_flat_weights(scale, growing):
    """Logits from nearly equal to far apart, with the largest last in the second form: the running maximum
    rises again and again, and what was accumulated is scaled."""
    rng = np.random.default_rng(3)
    n = 3000
    cache, held = shared_cache(rng, n, [5, 9], "bf16", 64)
    q = queries(rng, 2, 512)
    if growing:
        by = np.argsort((held[0][:n] @ f64(q[0, 7]).T))
        sorted_rows = torch.from_numpy(held[0][:n][by]).to(BF16).cuda()
        at = i32(np.arange(n))
        ds.ds_rows_append(cache, sorted_rows, i32(np.zeros(n)), at)
        held = [np.concatenate([held[0][:n][by], h[n:]]) for h in held]
        # The page that the prefix shares with each row's own: entry 1 keeps its own copy.
    sinks = torch.tensor(np.linspace(-50, 200, 64), dtype=torch.float32).cuda()
    out = torch.zeros_like(q)
    ds.ds_rows_prefix_attn(table(n, [5, 9]), n, q, sinks, 0, scale, out, cache)
    check(out, q, held, sinks, scale)


def test_one_slot_is_that_row():
    rng = np.random.default_rng(4)
    cache, held = shared_cache(rng, 0, [1, 1], "bf16", 16)
    q = queries(rng, 2, 512)
    out = torch.zeros_like(q)
    ds.ds_rows_prefix_attn(table(0, [1, 1]), 0, q, torch.full((64,), -3e38, device="cuda"), 0, SCALE, out, cache)
    for e in range(2):
        assert torch.equal(out[e].cpu(), torch.from_numpy(held[e][0]).to(BF16).expand(64, 512))


@pytest.mark.parametrize("fmt", FORMATS)
def test_fails_closed(fmt):
    """A page id out of range, a non-finite row, query or sink zeroes what it reaches and nothing else."""
    rng = np.random.default_rng(5)
    prefix, tails, page = 500, [100, 200, 300, 40, 7], 32
    rows = table(prefix, tails)

    def run(change):
        cache, held = shared_cache(rng, prefix, tails, fmt, page)
        q = queries(rng, 5, 512)
        sinks = torch.from_numpy(rng.standard_normal((5, 64)).astype(np.float32)).cuda()
        zero = torch.zeros(5, 64, dtype=torch.bool)
        change(cache, q, sinks, zero)
        out, bad = torch.full_like(q, 4.0), torch.full((5, 64), 9, dtype=torch.int32, device="cuda")
        ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 64, SCALE, out, cache, invalid=bad)
        assert torch.equal(bad.cpu(), zero.int())
        assert not out.cpu()[zero].any()
        for e in range(5):
            good = ~zero[e]
            if good.any():
                want, bound = formula(q[e].double(), gpu64(held[e]), sinks[e].double(), SCALE)
                ok = (out[e].double() - want).abs() <= bound
                assert ok[good.cuda()].all()

    def own_page(cache, q, sinks, zero):
        cache.page_table[2, 17] = cache.num_pages
        zero[2] = True

    def negative_page(cache, q, sinks, zero):
        cache.page_table[4, 15] = -1  # the page that its copy of the prefix's end shares
        zero[4] = True

    def shared_page(cache, q, sinks, zero):
        cache.page_table[0, 3] = -2 ** 31
        zero[:] = True

    def page_of_another_row(cache, q, sinks, zero):
        cache.page_table[1:, 3] = -1      # the prefix is read through entry 0
        cache.page_table[3, 17:] = -1     # behind its 540 slots

    def bad_row(value, entry, slot):
        def change(cache, q, sinks, zero):
            x = torch.ones(1, 512, device="cuda")
            x[0, 500] = value
            ds.ds_rows_append(cache, x, i32([entry]), i32([slot]))
            zero[entry] = True
            if slot < prefix:
                zero[:] = True
        return change

    def behind(cache, q, sinks, zero):
        x = torch.full((1, 512), float("nan"), device="cuda")
        ds.ds_rows_append(cache, x, i32([3]), i32([540]))  # the first slot behind entry 3
        ds.ds_rows_append(cache, x, i32([3]), i32([499]))  # entry 3's own copy of the prefix's last row

    def query(cache, q, sinks, zero):
        q[1, 5, 100], q[4, 63, 511], q[2, 0, 0] = float("inf"), float("nan"), -float("inf")
        zero[1, 5] = zero[4, 63] = zero[2, 0] = True

    def sink(cache, q, sinks, zero):
        sinks[0, 3], sinks[1, 4], sinks[2, 5] = float("inf"), -float("inf"), float("nan")
        zero[0, 3] = zero[1, 4] = zero[2, 5] = True

    for change in (own_page, negative_page, shared_page, page_of_another_row, bad_row(float("nan"), 2, 700),
                   bad_row(float("inf"), 0, 13), behind, query, sink):
        run(change)


def test_overflowing_logits_zero_their_heads():
    rng = np.random.default_rng(6)
    cache, held = shared_cache(rng, 200, [1, 2, 3], "bf16", 16)
    q = queries(rng, 3, 512)
    q[1, 7] = 3e38
    out, bad = torch.full_like(q, 4.0), torch.zeros(3, 64, dtype=torch.int32, device="cuda")
    ds.ds_rows_prefix_attn(table(200, [1, 2, 3]), 200, q, torch.zeros(64, device="cuda"), 0, 1.0, out, cache, invalid=bad)
    assert bad.nonzero().tolist() == [[1, 7]] and not out[1, 7].any() and out[1, 6].any()
    # A scale that takes every logit past 32 bits.
    ds.ds_rows_prefix_attn(table(200, [1, 2, 3]), 200, q, torch.zeros(64, device="cuda"), 0, 3e38, out, cache, invalid=bad)
    assert bad.all() and not out.any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_graph_streams_and_workspaces(fmt):
    """Captured and replayed with inputs, page table and cache changed in place; on another stream with a
    workspace of its own."""
    rng = np.random.default_rng(7)
    prefix, tails = 700, [3, 150, 0]
    cache, held = shared_cache(rng, prefix, tails, fmt, 64)
    rows, ws = table(prefix, tails), ds.prefix_attn_workspace(table(prefix, tails), prefix)
    q, sinks = queries(rng, 3, 512), torch.zeros(64, device="cuda")
    out = torch.zeros_like(q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 0, SCALE, out, cache, workspace_t=ws)
    for _ in range(3):
        q.copy_(queries(rng, 3, 512))
        perm = torch.randperm(cache.num_pages, device="cuda").to(torch.int32)
        view = cache.pages.view(cache.num_pages, -1)
        moved = torch.empty_like(view)
        moved[perm.long()] = view
        view.copy_(moved)
        old = cache.page_table.clone()
        cache.page_table.copy_(torch.where(old >= 0, perm[old.clamp(min=0).long()], old))
        ws.fill_(255)
        out.zero_()
        graph.replay()
        check(out, q, held, sinks)
        assert ds.workspace_status(ws) == 0
    torch.cuda.synchronize()
    there = torch.zeros_like(q)
    torch.cuda.synchronize()
    for _ in range(5):  # without a workspace: one from the stream's own memory
        ds.ds_rows_prefix_attn(iter(rows), prefix, q, sinks, 0, SCALE, there, cache, stream=side)
        ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 0, SCALE, out, cache, workspace_t=ws)
    torch.cuda.synchronize()
    assert torch.equal(there, out)


def test_pools_past_32_bits():
    """Rows in the last pages of pools of more than 2^32 bytes, for every type."""
    rng = np.random.default_rng(8)
    page = 256
    for fmt in FORMATS:
        num = (1 << 32) // ds.ds_rows_page_bytes(page, 512, fmt) + 5
        cache = ds.PagedCache.empty(num, i32([[num - 1, num - 2], [num - 1, num - 3]]), page, 512, fmt)
        x = torch.randn(600, 512, device="cuda")
        held = torch.zeros(600, 512, dtype=BF16, device="cuda")
        seq = i32(np.r_[np.zeros(300), np.ones(300)])
        slot = i32(np.r_[np.arange(300), np.arange(300)])
        x[300:556] = x[:256]  # the page that they share
        ds.ds_rows_append(cache, x, seq, slot, values=held)
        q, sinks = queries(rng, 2, 512), torch.zeros(64, device="cuda")
        out = torch.zeros_like(q)
        ds.ds_rows_prefix_attn([(300, 1, 0, 0), (290, 1, 0, 1)], 256, q, sinks, 0, SCALE, out, cache)
        h = f64(held)
        check(out, q, [h[:300], h[300:590]], sinks)
        del cache


def test_a_decode_step_of_samples_of_one_prompt():
    """Samples of one prompt decode over 8-bit pages: the prompt's rows appended once into shared pages, each
    sample's behind them, queries rotated, attention, output rotated back; and the rows read back."""
    rng = np.random.default_rng(9)
    prompt, own, page, n = 333, [1, 2, 3, 70], 16, 4
    shared = prompt // page
    need = [-(-(prompt + t) // page) for t in own]
    ids = rng.permutation(400)
    t = np.full((n, max(need)), -1)
    t[:, :shared] = ids[:shared]
    at = shared
    for e in range(n):
        t[e, shared:need[e]] = ids[at:at + need[e] - shared]
        at += need[e] - shared
    cache = ds.PagedCache.empty(400, i32(t), page, 512, "fp8")
    rope = ds.Rope(64, first=448, factor=4.0, original_len=4096)
    x = torch.randn(prompt, 512, device="cuda").to(BF16)
    pos = i32(np.arange(prompt))
    ds.ds_rows_append(cache, x, i32(np.zeros(prompt)), pos, rope=rope, positions=pos)
    seq = np.repeat(np.arange(n), own)
    slot = np.concatenate([prompt + np.arange(k) for k in own])
    y = torch.randn(len(seq), 512, device="cuda").to(BF16)
    ds.ds_rows_append(cache, y, i32(seq), i32(slot), rope=rope, positions=i32(slot))
    q, sinks = queries(rng, n, 512), torch.randn(64, device="cuda")
    at = i32([prompt + k - 1 for k in own])
    ds.ds_rows_rope(rope, q, at, q)
    out, back = torch.zeros_like(q), torch.zeros_like(q)
    rows = [(prompt + k, 1, 0, e) for e, k in enumerate(own)]
    ds.ds_rows_prefix_attn(rows, prompt, q, sinks, 0, SCALE, out, cache)
    ds.ds_rows_rope(rope, out, at, back, inverse=True)
    held = []
    for e, k in enumerate(own):
        s = np.r_[np.zeros(prompt), np.full(k, e)]
        got = torch.zeros(prompt + k, 512, device="cuda")
        ds.ds_rows_fetch(cache, i32(s), i32(np.arange(prompt + k)), got)
        held.append(got)
        # Half an e4m3 step of what was appended (its length is kept by the rotation).
        raw = torch.cat([x, y[torch.from_numpy(seq == e).cuda()]]).float()
        assert (got.norm(dim=1) - raw.norm(dim=1)).abs().max() <= 2.0 ** -4 * raw.norm(dim=1).max()
    check(out, q, held, sinks)
    assert torch.isfinite(back).all() and back.any()


@pytest.mark.parametrize("fmt", ["fp8", "int4"])
@pytest.mark.parametrize("prefix,tails", [(5000, [0, 1, 127, 128, 129, 300]), (2560, [5] * 9), (2049, [3] * 64)])
def test_rows_widened_beforehand_give_the_same_bits(fmt, prefix, tails):
    """With the smaller workspace the packed rows are widened as they are used; a page id out of range zeroes the same
    heads both ways."""
    rng = np.random.default_rng(prefix)
    n, page = len(tails), 64
    cache, held = shared_cache(rng, prefix, tails, fmt, page)
    q, sinks = queries(rng, n, 512), torch.zeros(64, device="cuda")
    rows = table(prefix, tails)
    small, large = (ds.prefix_attn_workspace(rows, prefix, f) for f in ("bf16", fmt))
    assert large.numel() > small.numel()
    for change in (lambda: None, lambda: cache.page_table[n - 1, prefix // page].fill_(-1),
                   lambda: cache.page_table[0, 0].fill_(cache.num_pages)):
        change()
        got = []
        for ws in (small, large):
            out, bad = torch.full_like(q, 4.0), torch.full((n, 64), 9, dtype=torch.int32, device="cuda")
            ds.ds_rows_prefix_attn(rows, prefix, q, sinks, 0, SCALE, out, cache, invalid=bad, workspace_t=ws)
            assert ds.workspace_status(ws) == 0
            got.append((out, bad))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        if change is not None and not got[0][1].any():
            check(got[0][0], q, held, sinks)
    assert got[0][1].all() and not got[0][0].any()


def test_the_workspace_has_to_be_large_enough():
    cache, _ = shared_cache(np.random.default_rng(1), 300, [1, 2], "fp8", 16)
    q = queries(np.random.default_rng(2), 2, 512)
    ws = ds.prefix_attn_workspace(table(300, [1, 2]), 300, "bf16")
    with pytest.raises(ds.DsRowsError, match="workspace holds"):
        ds.ds_rows_prefix_attn(table(300, [1, 2]), 300, q, torch.zeros(64, device="cuda"), 0, SCALE, torch.zeros_like(q),
                               cache, workspace_t=ws[:-256])
    for wrong in (q.half(), q.cpu(), q[:1], q.transpose(1, 2)):
        with pytest.raises((TypeError, ValueError)):
            ds.ds_rows_prefix_attn(table(300, [1, 2]), 300, wrong, torch.zeros(64, device="cuda"), 0, SCALE,
                                   torch.zeros_like(q), cache, workspace_t=ws)


def test_extreme_sinks():
    """Finite sinks of any size: the heads are sound, and the largest leave nothing of the rows."""
    cache, held = shared_cache(np.random.default_rng(3), 200, [1, 70], "bf16", 16)
    q = queries(np.random.default_rng(4), 2, 512)
    big = torch.finfo(torch.float32).max
    sinks = torch.zeros(64, device="cuda")
    sinks[:6] = torch.tensor([big, -big, 2.5e38, -2.5e38, 1e-45, 3000.0])
    out, bad = torch.full_like(q, 4.0), torch.full((2, 64), 9, dtype=torch.int32, device="cuda")
    ds.ds_rows_prefix_attn(table(200, [1, 70]), 200, q, sinks, 0, SCALE, out, cache, invalid=bad)
    assert not bad.any()
    check(out, q, held, sinks)
    assert not out[:, [0, 2, 5]].any() and out[:, [1, 3, 4]].any()
