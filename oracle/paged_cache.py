"""CPU oracle of the paged 8-bit cache.  TEST INFRASTRUCTURE ONLY.

Plain float64 numpy restatements of the calls of include/idx_cache.h, one request, one
page, one row at a time:

  e4m3_values, e4m3_encode   the 8-bit codes and their rounding (nearest, ties to even)
  page_tables   one step of the page allocator and the step's lists
  cache_write   quantisation of new keys and values into their slots
  attend        softmax attention of given rows over the tokens they see

A row of `attend` also gets the quantities its error bounds need: the weighted sum of
|value| and the largest score magnitude before cancellation.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["e4m3_values", "e4m3_encode", "page_tables", "page_scale", "cache_write", "attend",
           "request_tokens"]

SCALE_MIN_EXP = -120


def e4m3_values() -> np.ndarray:
    """The 256 codes' values: sign, 4 exponent bits (bias 7), 3 fraction bits; no
    infinities, 0x7F and 0xFF are NaN."""
    out = np.empty(256, np.float64)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        if e == 15 and f == 7:
            v = math.nan
        elif e == 0:
            v = f * 2.0 ** -9
        else:
            v = (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = -v if c & 0x80 else v
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # ascending


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Codes nearest to x (ties to the even code), saturating at +-448; NaN is 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.searchsorted(_POSITIVE, a, side="left")      # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(dh == 0, hi, code).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def page_tables(seq_len, n_new, table, ring, cursor, n_tokens, page):
    """One step; returns a dict of the outputs and the updated copies of table and ring
    (kv_indices as a list of exactly the pages held)."""
    table, ring = np.array(table), np.array(ring)
    B, max_pages = table.shape
    n_pages = len(ring)
    head, free = int(cursor[0]) % n_pages, min(max(int(cursor[1]), 0), n_pages)
    need_sum, taken, given = 0, 0, []
    out = {"seq_len": [], "kv_indptr": [0], "kv_indices": [], "tok_indptr": [0], "slots": [],
           "tok_req": [], "tok_len": [], "refused": 0}
    rows = 0
    old_ring = ring.copy()
    for b in range(B):
        have = min(max(int(seq_len[b]), 0), max_pages * page)
        fresh = max(int(n_new[b]), 0)
        after = max(have + int(n_new[b]), 0)
        rows += fresh
        old, wide = -(-have // page), -(-after // page)
        served = after <= max_pages * page and (fresh == 0 or rows <= n_tokens)
        if served:
            need = max(wide - old, 0)
            need_sum += need
            served = need == 0 or need_sum <= free
        if not served:
            out["refused"] += 1
            after, wide = have, old
        for i in range(old, wide):
            table[b, i] = old_ring[(head + taken) % n_pages]
            taken += 1
        given += [table[b, i] for i in range(wide, old)]
        out["seq_len"].append(after)
        out["kv_indices"] += [table[b, i] for i in range(wide)]
        out["kv_indptr"].append(len(out["kv_indices"]))
        for i in range(fresh):
            if len(out["slots"]) == n_tokens:
                break
            p = have + i
            ok = served and 0 <= table[b, p // page] < n_pages
            out["slots"].append(table[b, p // page] * page + p % page if ok else -1)
            out["tok_len"].append(p + 1 if ok else 0)
            out["tok_req"].append(b)
        out["tok_indptr"].append(len(out["slots"]))
    for j, p in enumerate(given):
        if free + j < n_pages:
            ring[(head + free + j) % n_pages] = p
    while len(out["slots"]) < n_tokens:
        out["slots"].append(-1)
        out["tok_len"].append(0)
        out["tok_req"].append(-1)
    out["cursor"] = [(head + taken) % n_pages, min(free - taken + len(given), n_pages),
                     out.pop("refused")]
    out = {k: np.array(v, np.int64) for k, v in out.items()}
    return out | {"table": table, "ring": ring}


def page_scale(amax: float) -> float:
    """The smallest power of two, at least 2^-120, with amax <= 448 s."""
    e = SCALE_MIN_EXP
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def cache_write(x, slots, codes, scale, page, columns):
    """New rows x [n, H, D] (float64) into codes [pages, H, page, D] (or with `columns`
    [pages, H, D, page]) and scale [pages, H]; returns updated copies. Divisions and the
    rescaling factor are rounded to float32, as the scales are."""
    codes, scale = codes.copy(), scale.copy()
    n_pages, H = scale.shape
    view = codes.transpose(0, 1, 3, 2) if columns else codes
    t = 0
    while t < len(slots):
        slot = int(slots[t])
        if slot < 0 or slot >= n_pages * page:
            t += 1
            continue
        p, first = divmod(slot, page)
        n = 1
        while first + n < page and t + n < len(slots) and slots[t + n] == slot + n:
            n += 1
        for h in range(H):
            rows = x[t:t + n, h]
            finite = np.abs(rows[np.isfinite(rows)])
            s = page_scale(finite.max() if finite.size else 0.0)
            if first:
                old = float(scale[p, h])
                s = max(s, old)
                if s != old:
                    f = float(np.float32(old) / np.float32(s))
                    view[p, h, :first] = e4m3_encode(_VALUES[view[p, h, :first]] * f)
            scale[p, h] = s
            with np.errstate(over="ignore", invalid="ignore"):
                view[p, h, first:first + n] = e4m3_encode(
                    rows.astype(np.float32) / np.float32(s))
        t += n
    return codes, scale


def request_tokens(pages, codes_k, codes_v, k_scale, v_scale, h, page, n_pages):
    """Keys and values [len(pages) * page, D] of one request and head in float64, and
    which of them exist (a page outside the pool holds none)."""
    D = codes_k.shape[-1]
    k = np.zeros((len(pages) * page, D))
    v = np.zeros_like(k)
    there = np.zeros(len(k), bool)
    for i, p in enumerate(pages):
        if 0 <= p < n_pages:
            k[i * page:(i + 1) * page] = _VALUES[codes_k[p, h]] * float(k_scale[p, h])
            v[i * page:(i + 1) * page] = _VALUES[codes_v[p, h]].T * float(v_scale[p, h])
            there[i * page:(i + 1) * page] = True
    return k, v, there


def attend(q, k, v, there, seen, slots, page, scale, softcap=0.0, slope=0.0):
    """One row and query head q [D] over a request's tokens: the first `seen`, all of
    them or those of the listed page `slots` (a slot listed twice counts twice).
    Returns out [D], sum of weights x |value| [D], and the largest sum |q k| scale."""
    n = len(k)
    if slots is None:
        at = np.arange(min(n, max(seen, 0)))
    else:
        at = [np.arange(s * page, (s + 1) * page) for s in slots if 0 <= s < n // page]
        at = np.concatenate(at) if at else np.zeros(0, int)
        at = at[at < seen]
    at = at[there[at]]
    D = len(q)
    if at.size == 0:
        return np.zeros(D), np.zeros(D), 0.0
    x = (k[at] @ q) * scale
    mag = (np.abs(k[at]) @ np.abs(q)).max() * abs(scale)
    if softcap:
        x = softcap * np.tanh(x / softcap)
    x = x - slope * (seen - 1 - at)
    p = np.exp(x - x.max())
    p /= p.sum()
    return p @ v[at], p @ np.abs(v[at]), float(mag)
