"""Calls on 8-bit pages that the documentation allows and that are easy to get wrong: no tokens, and blocks with
non-finite values.
"""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from test_gpu_fp8 import FORMATS, make_cache
from test_gpu_paged import i32

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
