"""Calls on 8-bit pages that the documentation allows and that are easy to get wrong: no tokens, and blocks with
non-finite values.
"""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from oracle import paged as ref
from test_gpu_fp8 import FORMATS, edge_blocks, make_cache
from test_gpu_paged import TYPES, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ds.build()
    ds.load()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [128, 512])
def test_no_tokens_of_any_strides(fmt, dim):
    """Zero rows from numpy have strides of 0; nothing is enqueued."""
    cache, _ = make_cache(np.random.default_rng(1), [5], dim, fmt, 16)
    before = cache.pages.clone()
    for x in (torch.from_numpy(np.zeros((0, dim), np.float32)).cuda(), torch.zeros(0, dim, device="cuda"),
              torch.zeros(dim, 0, device="cuda").T, torch.zeros(3, 2 * dim, device="cuda")[:0, ::2]):
        ds.ds_rows_append(cache, x, i32([]), i32([]))
        ds.ds_rows_fetch(cache, i32([]), i32([]), x)
    torch.cuda.synchronize()
    assert torch.equal(cache.pages.view(torch.uint8), before.view(torch.uint8))
    for wrong in (torch.zeros(dim, 3, device="cuda").T, torch.zeros(3, 2 * dim, device="cuda")[:, ::2]):
        for call in (lambda: ds.ds_rows_append(cache, wrong, i32([0] * 3), i32([0, 1, 2])),
                     lambda: ds.ds_rows_fetch(cache, i32([0] * 3), i32([0, 1, 2]), wrong)):
            with pytest.raises(ValueError, match="contiguous"):
                call()


@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_block_stored_as_nan_holds_zeros(dim, dtype):
    """Every byte that an append writes is the oracle's; e4m3's codes for NaN are not among them."""
    rng = np.random.default_rng(dim)
    n = 300
    cache, _ = make_cache(rng, [n], dim, "fp8", 32)
    y = edge_blocks(rng, n, dim)
    for k, bad in enumerate((np.nan, -np.nan, np.inf, -np.inf) * 8):
        y[k, rng.integers(0, dim)] = bad
    y = torch.from_numpy(y).to(dtype)
    ds.ds_rows_append(cache, y.cuda(), i32(np.zeros(n)), i32(np.arange(n)))
    byte, ex = ref.fp8_quantise(y.float().numpy())
    assert (ex == 255).any(1).sum() >= 32
    pool = cache.pages.cpu().numpy().reshape(cache.num_pages, -1)[cache.page_table.cpu().numpy()[0, np.arange(n) // 32]]
    v, sc = ref.fp8_places(dim, 32)
    rows, at = np.arange(n)[:, None], np.arange(n) % 32
    np.testing.assert_array_equal(pool[rows, v[at]], byte)
    np.testing.assert_array_equal(pool[rows, sc[at]], ex)
    assert not np.isin(pool[rows, v[at]], (0x7F, 0xFF)).any()
