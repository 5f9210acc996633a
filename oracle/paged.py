"""Oracle of the rotary positions and of the paged cache's types (float64, plain numpy).

Test infrastructure, as the rest of this package. The rotation follows its formula
with 64-bit angles; the 4-bit type is spelled out value by value and byte by byte
(groups of 16 values n * s, s e4m3, n in -7..7 held as n + 8; value i of a word at
bits 4 (i // 2) + 16 (i mod 2)), and so is the 8-bit type (blocks of 128 values v * 2^e,
v e4m3, e in -100..7 held as e + 127).
"""

from __future__ import annotations

import numpy as np

GROUP = 16


def frequencies(rot_dim, base=10000.0, factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """theta_i of a rotation (float64)."""
    theta = np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    if factor == 1.0:
        return theta
    if not original_len:
        return theta / factor

    def pair_at(turns):  # the pair that makes `turns` turns over the original context
        return rot_dim * np.log(original_len / (2 * np.pi * turns)) / (2 * np.log(base))

    low, high = max(np.floor(pair_at(beta_fast)), 0.0), min(np.ceil(pair_at(beta_slow)), rot_dim - 1.0)
    mix = np.clip((np.arange(rot_dim // 2) - low) / max(high - low, 0.001), 0.0, 1.0)
    return theta * (1 - mix) + theta / factor * mix


def pairs(rot_dim, first, layout):
    """Element numbers (a, b) of the pairs of a row."""
    i = np.arange(rot_dim // 2)
    return (first + 2 * i, first + 2 * i + 1) if layout == "interleaved" else (first + i, first + rot_dim // 2 + i)


def rope(x, positions, theta, first, layout, magnitude=1.0, inverse=False):
    """x [tokens, ..., dim] rotated (float64). Rows of a negative position are returned as they are."""
    x = np.asarray(x, np.float64)
    a, b = pairs(2 * len(theta), first, layout)
    pos = np.asarray(positions, np.float64)
    angle = pos[:, None] * theta[None] * (-1.0 if inverse else 1.0)
    angle = angle.reshape(len(pos), *[1] * (x.ndim - 2), len(theta))
    y = x.copy()
    y[..., a] = magnitude * (x[..., a] * np.cos(angle) - x[..., b] * np.sin(angle))
    y[..., b] = magnitude * (x[..., a] * np.sin(angle) + x[..., b] * np.cos(angle))
    y[pos < 0] = x[pos < 0]
    return y


# ---------------------------------------------------------------------------
# e4m3 and the 4-bit groups
# ---------------------------------------------------------------------------

def e4m3_value(byte):
    b = np.asarray(byte, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where((b & 127) == 127, np.nan, np.where(b & 128, -v, v))


E4M3 = e4m3_value(np.arange(127))  # the nonnegative finite values, ascending


def e4m3_byte(x):
    """Nonnegative x to the nearest e4m3 (ties to the even code), saturating at 448."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(E4M3, x, side="left"), 1, len(E4M3) - 1)
    lo = hi - 1
    dl, dh = x - E4M3[lo], E4M3[hi] - x
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return pick.astype(np.uint8)


def int4_quantise(y):
    """float32 rows [rows, dim] -> (n int [rows, dim], scale bytes [rows, dim / 16]), divisions in float32."""
    y = np.asarray(y, np.float32)
    g = y.reshape(len(y), -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], np.float32(0), g)
    byte = e4m3_byte((np.abs(g).max(-1) / np.float32(7)).astype(np.float32))
    s = E4M3[byte].astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        n = np.where(s[..., None] > 0, np.rint(g / s[..., None]), 0)
    n = np.clip(n, -7, 7).astype(np.int64)
    return n.reshape(y.shape), np.where(bad, 0x7F, byte).astype(np.uint8)


def int4_values(n, scales):
    return (n.reshape(len(n), -1, GROUP) * e4m3_value(scales)[..., None]).reshape(n.shape)


def int4_bytes(n):
    """n [rows, dim] -> bytes [rows, dim / 2] in the word order."""
    out = np.zeros((n.shape[0], n.shape[1] // 2), np.uint8)
    for e in range(n.shape[1]):
        i = e % 8
        bit = 4 * (i // 2) + 16 * (i % 2)
        out[:, 4 * (e // 8) + bit // 8] |= ((n[:, e] + 8) << (bit % 8)).astype(np.uint8)
    return out


def int4_numbers(data):
    """The inverse of int4_bytes."""
    n = np.zeros((data.shape[0], 2 * data.shape[1]), np.int64)
    for e in range(n.shape[1]):
        i = e % 8
        bit = 4 * (i // 2) + 16 * (i % 2)
        n[:, e] = ((data[:, 4 * (e // 8) + bit // 8].astype(np.int64) >> (bit % 8)) & 15) - 8
    return n


# ---------------------------------------------------------------------------
# the 8-bit blocks
# ---------------------------------------------------------------------------

BLOCK = 128


def fp8_quantise(y):
    """Rows [rows, dim] -> (value bytes [rows, dim], exponent bytes [rows, dim / 128])."""
    g = np.asarray(y, np.float64).reshape(len(y), -1, BLOCK)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    top = np.abs(g).max(-1)
    e = np.full(top.shape, 7)
    for k in range(6, -101, -1):
        e = np.where(top <= 448 * 2.0 ** k, k, e)
    v = g / 2.0 ** e[..., None]
    byte = e4m3_byte(np.abs(v)) | np.where(np.signbit(v), 0x80, 0).astype(np.uint8)
    return byte.reshape(np.shape(y)), np.where(bad, 255, e + 127).astype(np.uint8)


def fp8_values(byte, exponents):
    """The numbers of value bytes [rows, dim]; the codes of e4m3's NaN stand for +-480."""
    b = np.asarray(byte, np.int64)
    v = np.where((b & 127) == 127, np.where(b & 128, -480.0, 480.0), e4m3_value(b))
    x = np.asarray(exponents, np.int64)
    scale = np.where((x >= 27) & (x <= 134), 2.0 ** (np.clip(x, 27, 134) - 127.0), np.nan)
    return (v.reshape(len(b), -1, BLOCK) * scale[..., None]).reshape(b.shape)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------

def fp8_places(dim, page_size):
    """Byte offsets inside an 8-bit page of each row's values [page_size, dim] and exponents [page_size, dim / 128]."""
    r = np.arange(page_size)[:, None]
    v, s = np.arange(dim)[None], np.arange(dim // BLOCK)[None]
    scales = dim * page_size + dim // BLOCK * r + s
    return (r * 512 + v if dim == 512 else v // 16 * (16 * page_size) + 16 * r + v % 16), scales


def row_places(dim, page_size):
    """Byte offsets inside a 4-bit page of each row's values [page_size, dim / 2] and scales [page_size, dim / 16]."""
    r = np.arange(page_size)[:, None]
    v, s = np.arange(dim // 2)[None], np.arange(dim // GROUP)[None]
    if dim == 512:
        return r * 288 + v, r * 288 + 256 + s
    return v // 16 * (16 * page_size) + 16 * r + v % 16, 64 * page_size + 8 * r + s


def write_int4_page(page, dim, page_size, n, scales):
    """Rows (n, scales) of one page into its bytes."""
    v, s = row_places(dim, page_size)
    page[v[: len(n)]] = int4_bytes(n)
    page[s[: len(n)]] = scales


def read_int4_page(page, dim, page_size):
    """(n, scales) of every row of a page."""
    v, s = row_places(dim, page_size)
    return int4_numbers(page[v]), page[s]
