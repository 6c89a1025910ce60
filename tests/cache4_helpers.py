"""Inputs and bounds for the paged 4-bit cache's tests.

Attention bound, per output value (u = 2^-24, the oracle in float64 on the same codes,
scales and bf16 queries). Scores, weights and sums are off as tests/cache_helpers.py works
out (a key with its scale is exact in bf16, so a score is again a sum of 128 exact products
in fp32, times a rounded scale). Beside that:
  - a probability is rounded to fp16, 2^-11 of itself, or 2^-25 below the normal range; times a power of two of at most 1 that is exact, or 2^-25 again: 2^-24 in units
    where the row's largest weight times value scale is 2^9 or more, and a value is at most
    6 scales: 6 * 2^-33 < 2^-30 of `reach`, that largest product, for each token;
  - the output is rounded to bf16: 2^-8 |out|, and 2^-134 below its normal range.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache4 as c4
from tests.cache_helpers import U


def tolerance(out, absum, mag, reach, n, cap=0.0, bias=0.0):
    e = 160 * U * mag + 16 * U * (cap + bias) + 4 * U
    weights = 2 * np.expm1(e) + 2.0 ** -11 + (2 * n + 8) * U
    off = absum * weights + n * 2.0 ** -30 * reach
    return off + (np.abs(out) + off) * 2.0 ** -8 + 2.0 ** -130


class Cache4:
    """A pool of random codes and scales with page lists for requests of given lengths
    (all lists drawn from one permutation of the pool)."""

    def __init__(self, seed, lens, Hkv, page, spare=3, max_pages=None, spread=4):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.Hkv, self.page = rng, list(lens), Hkv, page
        blocks = [-(-n // page) for n in lens]
        self.n_pages = sum(blocks) + spare
        shape = (self.n_pages, Hkv)
        self.k = c4.e2m1_encode(rng.standard_normal((*shape, page, 128)) * 2)
        self.v = c4.e2m1_encode(rng.standard_normal((*shape, 128, page)) * 2)
        self.ks = (127 - 1 - rng.integers(0, spread, (*shape, page, 4))).astype(np.uint8)
        self.vs = (127 - 1 - rng.integers(0, spread, (*shape, 4, page))).astype(np.uint8)
        self.indptr = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int32)
        self.indices = rng.permutation(self.n_pages)[:sum(blocks)].astype(np.int32)
        self.max_pages = max_pages or max(1, max(blocks))
        self.poison_tails()

    def poison_tails(self):
        """NaN scales, or huge ones, behind every request's last token and in the pages of
        no request."""
        used = np.zeros(self.n_pages, bool)
        for b, n in enumerate(self.lens):
            pages = self.indices[self.indptr[b]:self.indptr[b + 1]]
            used[pages] = True
            if n % self.page:
                bad = 255 if b % 2 == 0 else 254
                self.ks[pages[-1], :, n % self.page:] = bad
                self.vs[pages[-1], :, :, n % self.page:] = bad
        self.ks[~used], self.vs[~used] = 255, 254

    def device(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return (t(c4.pack(self.k)), t(c4.pack(self.v)), t(self.ks), t(self.vs), t(self.indptr),
                t(self.indices))

    def pages(self, b):
        lo, hi = int(self.indptr[b]), int(self.indptr[b + 1])
        hi = min(hi, lo + self.max_pages)
        return [int(self.indices[i]) if 0 <= i < len(self.indices) else -1
                for i in range(lo, hi)]

    def tokens(self, b, h):
        return c4.request_tokens(self.pages(b), self.k, self.v, self.ks, self.vs, h, self.page)


def check_rows(out, c, q, req, seen, ids=None, scale=128 ** -0.5, cap=0.0, slopes=None,
               rows=None):
    """out [n, Hq, 128] (bf16, any device) against the oracle, row by row."""
    out = out.double().cpu().numpy()
    n, Hq, _ = out.shape
    G = Hq // c.Hkv
    cache = {}
    worst = 0.0
    for r in (range(n) if rows is None else rows):
        b = int(req[r])
        for hq in range(Hq):
            h = hq // G
            if not 0 <= b < len(c.indptr) - 1:
                assert not out[r, hq].any(), (r, hq)
                continue
            if (b, h) not in cache:
                cache[b, h] = c.tokens(b, h)
            k, v, there, top = cache[b, h]
            slope = 0.0 if slopes is None else float(slopes[hq])
            want, absum, mag, reach = c4.attend(
                q[r, hq], k, v, there, top, int(seen[r]), None if ids is None else ids[r], c.page,
                float(np.float32(scale)), float(np.float32(cap)), slope)
            nan = np.isnan(want)
            assert np.array_equal(np.isnan(out[r, hq]), nan), (r, hq)
            tol = tolerance(want, absum, mag, reach,
                            len(k) if ids is None else len(ids[r]) * c.page, cap,
                            slope * max(int(seen[r]), 0))
            err = np.abs(out[r, hq] - want)
            bad = np.argwhere((err > tol) & ~nan)
            assert bad.size == 0, (r, hq, bad[0], out[r, hq][bad[0]], want[bad[0]], tol[bad[0]])
            if not nan.any():
                worst = max(worst, float((err / tol).max()))
    return worst
