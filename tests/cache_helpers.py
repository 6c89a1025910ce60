"""Inputs and bounds for the paged-cache tests.

Attention bound, per output value, from the arithmetic that the header states
(u = 2^-24, the oracle in float64 on the same codes, scales and bf16 queries):
  - a score is a sum of 128 exact products in fp32 (128 additions in any order), times a
    rounded scale (3 roundings), capped and biased in fp32: its error is at most
    e = 140 u A + 8 u (|cap| + |bias|) in natural units, A the largest sum |q k| scale;
    the exponential's argument adds 4 u times its size (at most 2 A + cap + bias) and the
    instruction 2 u;
  - so a weight is off by a factor exp(e'), e' = 160 u A + 16 u (cap + bias) + 4 u; the
    weights' sum too, which doubles it;
  - a probability meets its value rounded to 11 bits: 2^-12 (half a step of fp16), plus
    2^-38 absolute for those below its normal range, relative to the largest;
  - n products and the sum of weights accumulate in fp32: 2 n u, and joining partial
    sums adds 8 roundings;
  - all of these act on sum weight |value|; the output is rounded to bf16: 2^-8 |out|
    (half a step), and 2^-134 below its normal range.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged_cache as pc

U = 2.0 ** -24


def tolerance(out, absum, mag, n, cap=0.0, bias=0.0):
    e = 160 * U * mag + 16 * U * (cap + bias) + 4 * U
    weights = 2 * np.expm1(e) + 2.0 ** -12 + n * 2.0 ** -38 + (2 * n + 8) * U
    return absum * weights + (np.abs(out) + absum * weights) * 2.0 ** -8 + 2.0 ** -130


class Cache:
    """A pool of random codes and scales with page lists for requests of given lengths
    (all lists drawn from one permutation of the pool)."""

    def __init__(self, seed, lens, Hkv, page, spare=3, nan_free=True, max_pages=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.Hkv, self.page = rng, list(lens), Hkv, page
        blocks = [-(-n // page) for n in lens]
        self.n_pages = sum(blocks) + spare
        self.k = pc.e4m3_encode(rng.standard_normal((self.n_pages, Hkv, page, 128)) * 60)
        self.v = pc.e4m3_encode(rng.standard_normal((self.n_pages, Hkv, 128, page)) * 60)
        self.ks = np.exp2(rng.integers(-7, -4, (self.n_pages, Hkv))).astype(np.float32)
        self.vs = (np.exp2(rng.integers(-7, -4, (self.n_pages, Hkv)))
                   * rng.uniform(0.6, 1, (self.n_pages, Hkv))).astype(np.float32)
        self.indptr = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int32)
        self.indices = rng.permutation(self.n_pages)[:sum(blocks)].astype(np.int32)
        self.max_pages = max_pages or max(1, max(blocks))
        self.poison_tails()

    def poison_tails(self):
        """NaN codes behind every request's last token and in the pages of no request."""
        used = np.zeros(self.n_pages, bool)
        for b, n in enumerate(self.lens):
            pages = self.indices[self.indptr[b]:self.indptr[b + 1]]
            used[pages] = True
            if n % self.page:
                self.k[pages[-1], :, n % self.page:] = 0x7F
                self.v[pages[-1], :, :, n % self.page:] = 0xFF
        self.k[~used], self.v[~used] = 0xFF, 0x7F
        self.ks[~used], self.vs[~used] = np.nan, np.inf

    def device(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return (t(self.k).view(torch.float8_e4m3fn), t(self.v).view(torch.float8_e4m3fn),
                t(self.ks), t(self.vs), t(self.indptr), t(self.indices))

    def tokens(self, b, h):
        lo, hi = int(self.indptr[b]), int(self.indptr[b + 1])
        hi = min(hi, lo + self.max_pages)
        pages = [int(self.indices[i]) if 0 <= i < len(self.indices) else -1
                 for i in range(lo, hi)]
        return pc.request_tokens(pages, self.k, self.v, self.ks, self.vs, h, self.page,
                                 self.n_pages)


def queries(rng, n, Hq, std=1.5):
    q = torch.from_numpy((rng.standard_normal((n, Hq, 128)) * std).astype(np.float32)).bfloat16()
    return q, q.double().numpy()


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
            k, v, there = cache[b, h]
            slope = 0.0 if slopes is None else float(slopes[hq])
            want, absum, mag = pc.attend(q[r, hq], k, v, there, int(seen[r]),
                                         None if ids is None else ids[r], c.page,
                                         float(np.float32(scale)), float(np.float32(cap)), slope)
            nan = np.isnan(want)
            assert np.array_equal(np.isnan(out[r, hq]), nan), (r, hq)
            tol = tolerance(want, absum, mag, len(k) if ids is None else len(ids[r]) * c.page,
                            cap, slope * max(int(seen[r]), 0))
            err = np.abs(out[r, hq] - want)
            bad = np.argwhere((err > tol) & ~nan)
            assert bad.size == 0, (r, hq, bad[0], out[r, hq][bad[0]], want[bad[0]], tol[bad[0]])
            if not nan.any():
                worst = max(worst, float((err / tol).max()))
    return worst
