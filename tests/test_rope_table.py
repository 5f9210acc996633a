"""The rotation's table against its formula in 60 decimal digits (no GPU is used)."""

from decimal import Decimal, getcontext

import numpy as np
import pytest

import deepseek_sparse_attention_ragged_gb300 as ds

getcontext().prec = 60
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def exact_turns(rot, base, factor=1.0, original=0, fast=32.0, slow=1.0):
    """theta_i / (2 pi) as Decimals."""
    b, f = Decimal(base), Decimal(factor)
    theta = [(-2 * i * b.ln() / rot).exp() for i in range(rot // 2)]
    if factor != 1.0 and not original:
        theta = [t / f for t in theta]
    elif factor != 1.0:
        at = lambda beta: rot * (original / (TWO_PI * Decimal(beta))).ln() / (2 * b.ln())  # noqa: E731
        low = max(at(fast).__floor__(), 0)
        high = min(at(slow).__ceil__(), rot - 1)
        width = max(Decimal(high - low), Decimal(0.001))
        ramp = [min(max((i - low) / width, Decimal(0)), Decimal(1)) for i in range(rot // 2)]
        theta = [t * (1 - r) + t / f * r for t, r in zip(theta, ramp)]
    return [t / TWO_PI for t in theta]


def table(rot, base, factor=1.0, original=0, fast=32.0, slow=1.0):
    ds.build()
    t = np.zeros(rot // 2, np.uint64)
    assert ds.load().ds_rows_rope_turns(rot, base, factor, original, fast, slow, t.ctypes.data) == 0
    return t


@pytest.mark.parametrize("args", [
    (2, 10000.0), (64, 10000.0), (128, 10000.0), (6, 10000.0), (96, 10000.0), (510, 10000.0), (512, 10000.0),
    (128, 500000.0), (512, 5e6), (64, 1.0625), (64, 1.0 + 2.0 ** -52), (256, 1e12), (512, 1e300), (4, 1.7e308),
    (128, 10000.0, 4.0), (64, 10000.0, 40.0), (128, 10000.0, 1.3), (64, 10000.0, 1e9),
    (64, 10000.0, 16.0, 65536), (128, 10000.0, 4.0, 4096), (64, 10000.0, 40.0, 4096), (512, 500000.0, 8.0, 8192, 4.0, 1.0),
    (2, 10000.0, 40.0, 4096), (64, 10000.0, 3.7, 17), (64, 10000.0, 3.7, 4096, 1.0, 1.0),
])
def test_every_entry_is_the_nearest(args):
    """The nearest 64-bit fraction of a turn; 2^-20 of a step for what two doubles leave (2^-95 of the value)."""
    got, want = table(*args), exact_turns(*args)
    off = [abs(Decimal(int(g)) - w * 2 ** 64) for g, w in zip(got, want)]
    assert max(off) <= Decimal(0.5) + Decimal(2.0 ** -20), max(off)


def test_ramps_without_an_inside():
    """A context so short, or betas so far, that the ramp is a step or lies outside the pairs."""
    for fast, slow in ((1e308, 1e-308), (1e-300, 1e-308), (1e308, 1e300)):
        t = table(64, 10000.0, 8.0, 4096, fast, slow)
        plain, divided = table(64, 10000.0), table(64, 10000.0, 8.0)
        assert np.all((t <= plain) & (t >= divided))
