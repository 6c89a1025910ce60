"""CPU oracle of the paged 4-bit cache and of rotary positions.  TEST INFRASTRUCTURE ONLY.

Plain float64 numpy restatements of the calls of include/idx_cache4.h and
include/idx_rope.h, one block, one page, one row at a time:

  e2m1_values, e2m1_encode   the 4-bit codes and their rounding (nearest, ties to even)
  block_scale, quantise      the scale byte and the codes of one block of 32 values
  cache_write, cache_read    new keys and values into their slots, and back
  request_tokens             a request's keys and values, for paged_cache.attend
  attend                     paged_cache.attend, with the largest weight times value scale
  turned                     rotary positions, angles from whole numbers
"""
from __future__ import annotations

import math

import numpy as np

from oracle import paged_cache as pc

__all__ = ["e2m1_values", "e2m1_encode", "block_scale", "quantise", "cache_write", "cache_read",
           "request_tokens", "attend", "turned", "pack", "unpack"]

BLOCK = 32
MIN_EXP, MAX_EXP = -60, 60


def e2m1_values() -> np.ndarray:
    """The 16 codes' values: sign, 2 exponent bits (bias 1), 1 fraction bit."""
    out = np.empty(16)
    for c in range(16):
        e, f = (c >> 1) & 3, c & 1
        v = f * 0.5 if e == 0 else (1 + f / 2) * 2.0 ** (e - 1)
        out[c] = -v if c & 8 else v
    return out


_VALUES = e2m1_values()
_POSITIVE = _VALUES[:8]


def e2m1_encode(x: np.ndarray) -> np.ndarray:
    """Codes nearest to x (ties to the even code), saturating at +-6; the sign stays."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=6.0, neginf=-6.0)), 6.0)
    hi = np.searchsorted(_POSITIVE, a, side="left")
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(dh == 0, hi, code)
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def block_scale(x: np.ndarray) -> int:
    """The scale byte of a block: 255 where it holds a NaN."""
    if np.isnan(x).any():
        return 255
    amax = float(np.abs(x).max())
    e = MIN_EXP
    while e < MAX_EXP and 6.0 * 2.0 ** e < amax:
        e += 1
    return e + 127


def quantise(row: np.ndarray):
    """Codes [D] and scale bytes [D / 32] of one row (codes of NaN blocks: 0)."""
    codes, scales = np.zeros(len(row), np.uint8), np.zeros(len(row) // BLOCK, np.uint8)
    for i in range(len(scales)):
        x = row[i * BLOCK:(i + 1) * BLOCK]
        scales[i] = block_scale(x)
        if scales[i] != 255:
            codes[i * BLOCK:(i + 1) * BLOCK] = e2m1_encode(x / 2.0 ** (int(scales[i]) - 127))
    return codes, scales


def pack(codes: np.ndarray) -> np.ndarray:
    """Codes [..., 2 n] two a byte, the first in the low bits."""
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(data: np.ndarray) -> np.ndarray:
    out = np.empty((*data.shape[:-1], 2 * data.shape[-1]), np.uint8)
    out[..., 0::2], out[..., 1::2] = data & 15, data >> 4
    return out


def power(byte) -> np.ndarray:
    b = np.asarray(byte, np.float64)
    return np.where(b == 255, np.nan, np.exp2(np.minimum(b, 254) - 127))


def cache_write(k, v, slots, kc, vc, ks, vs):
    """New rows k, v [n, H, D] into copies of a cache (codes unpacked: kc [pages, H, page,
    D], vc [pages, H, D, page]); returns them."""
    kc, vc, ks, vs = kc.copy(), vc.copy(), ks.copy(), vs.copy()
    n_pages, H, page, _ = kc.shape
    for t, slot in enumerate(slots):
        if not 0 <= slot < n_pages * page:
            continue
        p, o = divmod(int(slot), page)
        for h in range(H):
            kc[p, h, o], ks[p, h, o] = quantise(k[t, h])
            vc[p, h, :, o], vs[p, h, :, o] = quantise(v[t, h])
    return kc, vc, ks, vs


def cache_read(slots, kc, vc, ks, vs):
    n_pages, H, page, D = kc.shape
    k, v = np.zeros((len(slots), H, D)), np.zeros((len(slots), H, D))
    for t, slot in enumerate(slots):
        if 0 <= slot < n_pages * page:
            p, o = divmod(int(slot), page)
            k[t] = _VALUES[kc[p, :, o]] * np.repeat(power(ks[p, :, o]), BLOCK, -1)
            v[t] = _VALUES[vc[p, :, :, o]] * np.repeat(power(vs[p, :, :, o]), BLOCK, -1)
    return k, v


def request_tokens(pages, kc, vc, ks, vs, h, page):
    """Keys and values [len(pages) * page, D] of one request and head, which of them exist
    (a page outside the pool holds none), and each token's largest value scale."""
    D = kc.shape[-1]
    n = len(pages) * page
    k, v, top, there = np.zeros((n, D)), np.zeros((n, D)), np.zeros(n), np.zeros(n, bool)
    for i, p in enumerate(pages):
        if 0 <= p < len(kc):
            at = slice(i * page, (i + 1) * page)
            k[at] = _VALUES[kc[p, h]] * np.repeat(power(ks[p, h]), BLOCK, -1)
            v[at] = (_VALUES[vc[p, h]] * np.repeat(power(vs[p, h]), BLOCK, 0)).T
            top[at] = np.nan_to_num(power(vs[p, h])).max(0)
            there[at] = True
    return k, v, there, top


def attend(q, k, v, there, top, seen, slots, page, scale, softcap=0.0, slope=0.0):
    """paged_cache.attend; also a bound of the largest product of a weight and the largest
    value scale among its token's 16 (those that the row sees): the products' sum."""
    args = (there, seen, slots, page, scale, softcap, slope)
    visible = there & (np.arange(len(k)) < seen)
    unit = np.repeat(np.where(visible, top, 0).reshape(-1, 16).max(1), 16) if len(k) else top
    reach = pc.attend(q, k, np.repeat(unit[:, None], len(q), 1), *args)[0]
    return *pc.attend(q, k, v, *args), float(np.nan_to_num(reach).max())


def turned(x, positions, turns, first, adjacent, inverse, factor):
    """Rotary positions of rows x [n, heads, D] (float64): pair i of row t turns by
    positions[t] * turns[i] / 2^64 turns (whole numbers: the fraction is exact)."""
    y = x.copy()
    pairs = len(turns)
    for t, p in enumerate(positions):
        part = (int(p) * np.array([int(f) for f in turns], object)) % (1 << 64)
        angle = np.array([2 * math.pi * (a / 2.0 ** 64) for a in part])
        c, s = factor * np.cos(angle), factor * np.sin(angle)
        if inverse:
            s = -s
        i = np.arange(pairs)
        a, b = (first + 2 * i, first + 2 * i + 1) if adjacent else (first + i, first + pairs + i)
        y[t][:, a] = x[t][:, a] * c - x[t][:, b] * s
        y[t][:, b] = x[t][:, b] * c + x[t][:, a] * s
    return y
