"""ds_rows_prefix_attn on rows made to show one thing each: that logits of any finite size are sound."""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from test_gpu_fp8 import FORMATS
from test_gpu_paged import BF16, SCALE, f64, i32
from test_gpu_prefix import table

pytestmark = pytest.mark.gpu

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
    return cache, [torch.cat([head, put(x, e, prefix)]) for e, x in enumerate(own)]


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
