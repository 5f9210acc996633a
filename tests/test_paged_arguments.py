"""Arguments of the rotation, append and score entry points without a GPU (refused, or calls of no tokens: nothing enqueued)."""

import ctypes

import pytest

import deepseek_sparse_attention_ragged_gb300 as ds
from deepseek_sparse_attention_ragged_gb300 import paged

FAKE = 0x7F0000000000
FAR = 1 << 40


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.load()


def rope(lib, xs, os_, tokens, heads, out=FAKE + (1 << 30)):
    r = paged._Rope(FAKE, 0, 64, 0, 1.0)
    return lib.ds_rows_rope(ctypes.byref(r), FAKE, *xs, out, *os_, 0, tokens, heads, 64, FAKE, 0, None)


def test_strides_of_sides_of_one_are_not_looked_at(lib):
    assert rope(lib, (FAR, 64), (FAR, 64), 0, 8) == 0
    assert rope(lib, (64, FAR), (64, FAR), 0, 1) == 0
    assert rope(lib, (FAR, FAR), (7, 3), 0, 1, out=FAKE) == 0  # in place: nothing to differ
    assert rope(lib, (FAR, 64), (64, 64), 2, 1) == -2 and rope(lib, (64, FAR), (64, 64), 1, 2) == -2
    assert rope(lib, (64, 64), (64, 0), 0, 2) == -1 and "overlap" in lib.ds_rows_last_error().decode()


def test_append_of_a_lone_row_from_anywhere(lib):
    c = paged._PagedCache(FAKE, FAKE, 8, 64, 64, 1000, 512, 1)
    call = lambda tokens: lib.ds_rows_append(ctypes.byref(c), FAKE, FAR, 0, tokens, FAKE, FAKE, None, None, None,  # noqa: E731
                                             None, None)
    assert call(0) == 0
    assert call(2) == -2 and "x_stride" in lib.ds_rows_last_error().decode()


def test_reads_need_aligned_words(lib):
    """Words off 4 bytes would be misaligned accesses on the device."""
    tab, n = ds._table([(600, 512, 0, 0)])
    keys, kv = (paged._PagedCache(FAKE, FAKE, 8, 64, 64, 1000, dim, 1) for dim in (128, 512))
    for w, out in ((FAKE + 2, FAKE), (FAKE, FAKE + 1)):
        assert lib.ds_rows_indexer_score_paged(n, tab, ctypes.byref(keys), FAKE, w, out, 600, None) == -3
        assert "4-B" in lib.ds_rows_last_error().decode()
    for sinks, idx, invalid in ((FAKE + 2, FAKE, None), (FAKE, FAKE + 3, None), (FAKE, FAKE, FAKE + 2)):
        assert lib.ds_rows_sparse_attn_paged(n, tab, ctypes.byref(kv), FAKE, sinks, 0, idx, 0.04, FAKE, invalid, FAKE, 256,
                                             None) == -3
        assert "4-B" in lib.ds_rows_last_error().decode()
