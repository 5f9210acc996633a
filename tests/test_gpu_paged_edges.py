"""Rotary positions and paged caches at the edges of what their documentation allows: shapes,
strides and streams that tests/test_gpu_paged.py leaves out."""

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds

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
