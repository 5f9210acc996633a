"""The paged binding's reading of its arguments, without a GPU."""

import numpy as np
import pytest

import deepseek_sparse_attention_ragged_gb300 as ds
from deepseek_sparse_attention_ragged_gb300 import paged


@pytest.mark.parametrize("bad", [
    [(600, 512, 0), (7, 7, 512, 3, 9)], [(1, 2, 3, 4), ()], [(1, 2, 3, 4), (1,), (5, 6, 7)], [ds.Row(1, 1, 0, 0), (1, 2)],
    [np.arange(3), np.arange(5)], [(1,) * 8, ()],
])
def test_every_row_has_four_fields(bad):
    """Uneven rows are refused even where their words make up whole rows."""
    with pytest.raises(ValueError, match="nonempty list"):
        paged._rows(bad)


def test_rows_of_numpy_words_and_mixed_kinds():
    want = [(600, 512, 0, 2), (7, 6, 512, 1)]
    for rows in (np.array(want), np.array(want, np.uint32), [ds.Row(*want[0]), want[1]], [list(want[0]), ds.Row(*want[1])],
                 [np.array(want[0]), ds.Row(*want[1])]):
        words, *columns = paged._rows(rows)
        assert list(zip(*columns)) == want and len(words) == 8
        assert all(type(x) is int for column in columns for x in column)  # sums of them cannot wrap
    for bad in ([(1.5, 1, 0, 0)], ["abcd"], [None], 7 * [3]):
        with pytest.raises(ValueError, match="nonempty list"):
            paged._rows(bad)


@pytest.mark.parametrize("kw", [dict(first=1 << 32), dict(first=-2), dict(first=0.5), dict(original_len=-1, factor=2.0),
                                dict(original_len=1 << 32, factor=2.0), dict(rot_dim=(1 << 32) + 64), dict(rot_dim=-64),
                                dict(rot_dim=63.5)])
def test_rotations_beyond_32_bits_are_refused(kw):
    """ctypes cuts what it is given to 32 bits: 2^32 would have been 0, -1 a context of 2^32 - 1."""
    ds.build()
    with pytest.raises(ValueError, match="whole number"):
        ds.Rope(kw.pop("rot_dim", 64), device="cpu", **kw)


@pytest.mark.parametrize("page,dim", [((1 << 32) + 64, 128), (64, (1 << 32) + 512), (-64, 128), (64.5, 128)])
def test_page_sizes_beyond_32_bits_are_refused(page, dim):
    ds.build()
    with pytest.raises(ValueError, match="whole number"):
        ds.ds_rows_page_bytes(page, dim, "bf16")
    assert ds.ds_rows_page_bytes(64.0, np.int64(128), "bf16") == 16384
