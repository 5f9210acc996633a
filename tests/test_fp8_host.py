"""The 8-bit pages and reading rows back without a GPU: the oracle's own pins, page
sizes, and every refusal of ds_rows_fetch (fake, aligned pointers: validation fails
before any of them is used)."""

import ctypes

import numpy as np
import pytest
import torch

import deepseek_sparse_attention_ragged_gb300 as ds
from deepseek_sparse_attention_ragged_gb300 import paged
from oracle import paged as ref
from test_paged_host import BAD_CACHES, FAKE, _append, _cache, _err

FP8 = 3


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.load()


def test_fp8_values_are_those_of_torch_and_exact_in_bf16():
    rng = np.random.default_rng(0)
    y = (rng.standard_normal((40, 256)) * np.exp(rng.uniform(-30, 8, (40, 1)))).astype(np.float32)
    byte, ex = ref.fp8_quantise(y)
    e = torch.from_numpy(ex.astype(np.int32)) - 127
    v = torch.from_numpy(byte).view(torch.float8_e4m3fn).float().view(40, 2, 128)
    want = torch.ldexp(v, e[..., None]).view(40, 256)
    got = torch.from_numpy(ref.fp8_values(byte, ex))
    assert torch.equal(want.double(), got) and torch.equal(want.bfloat16().double(), got)
    scaled = torch.ldexp(torch.from_numpy(y).view(40, 2, 128), -e[..., None])
    assert torch.equal(scaled.to(torch.float8_e4m3fn).view(torch.uint8).view(40, 256), torch.from_numpy(byte))
    # Half a step: 2^-4 of a value, and 2^-10 2^e below e4m3's smallest normal number.
    step = np.repeat(2.0 ** (ex - 127.0), 128, 1)
    assert np.all(np.abs(got.numpy() - y) <= np.maximum(np.abs(y) * 2.0 ** -4, step * 2.0 ** -10))


@pytest.mark.parametrize("top,e", [(448.0, 0), (449.0, 1), (np.nextafter(np.float32(448), np.float32(1000)), 1), (1.0, -8),
                                   (1.75, -8), (1.7500001, -7), (0.0, -100), (1e-40, -100), (448 * 2.0 ** -100, -100),
                                   (450 * 2.0 ** -100, -99), (448 * 128.0, 7), (3e38, 7), (57000.0, 7), (28672.0, 6)])
def test_fp8_exponents(top, e):
    y = np.zeros((1, 128), np.float32)
    y[0, 77] = -top
    byte, ex = ref.fp8_quantise(y)
    assert ex[0, 0] == e + 127
    assert ref.fp8_values(byte, ex)[0, 77] >= -448 * 2.0 ** e


@pytest.mark.parametrize("dim,page", [(128, 16), (128, 256), (512, 32), (512, 128)])
def test_every_byte_of_a_page_belongs_to_one_row(dim, page):
    v, s = ref.fp8_places(dim, page)
    size = ds.ds_rows_page_bytes(page, dim, "fp8")
    assert size == page * (dim + dim // 128) and size % 16 == 0
    assert np.array_equal(np.sort(np.concatenate([v.ravel(), s.ravel()])), np.arange(size))


@pytest.mark.parametrize("kw,code,msg", [b for b in BAD_CACHES if "fmt" not in b[0]])
def test_caches_are_checked_in_8_bits_too(lib, kw, code, msg):
    assert _append(lib, _cache(fmt=FP8, **kw)) == code and msg in _err(lib)


def _fetch(lib, cache=None, seq=FAKE, slot=FAKE, out=FAKE + (1 << 30), stride=512, dtype=0, tokens=4, invalid=None,
           null=False):
    c = _cache(fmt=FP8) if cache is None else cache
    return lib.ds_rows_fetch(None if null else ctypes.byref(c), seq, slot, out, stride, dtype, tokens, invalid, None)


@pytest.mark.parametrize("kw,code,msg", BAD_CACHES)
def test_fetch_cache_refusals(lib, kw, code, msg):
    assert _fetch(lib, _cache(**kw)) == code and msg in _err(lib)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(null=True), -1, "NULL"), (dict(out=None), -1, "non-NULL"), (dict(out=FAKE + 1), -3, "element type"),
    (dict(dtype=2, out=FAKE + 2), -3, "element type"), (dict(dtype=3), -1, "dtype"), (dict(tokens=1 << 31), -2, "below 2^31"),
    (dict(stride=(1 << 31) + 1), -2, "out_stride"), (dict(stride=511), -1, "overlap"), (dict(stride=0), -1, "overlap"),
    (dict(seq=None), -1, "seq and slot"), (dict(slot=None), -1, "seq and slot"), (dict(seq=FAKE + 1), -3, "4-B"),
    (dict(slot=FAKE + 2), -3, "4-B"), (dict(invalid=FAKE + 2), -3, "4-B"),
])
def test_fetch_refusals(lib, kw, code, msg):
    assert _fetch(lib, **kw) == code and msg in _err(lib)


def test_fetch_of_nothing(lib):
    assert _fetch(lib, tokens=0) == 0
    assert _fetch(lib, tokens=0, stride=1 << 40) == 0  # no row: its stride says nothing


def test_binding_refuses_host_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ds.ds_rows_fetch(None, z, z, torch.zeros(4, 512))
    assert paged._FORMATS["fp8"] == FP8
