"""Caps of scores far above the scores: a capped score keeps the precision of an uncapped
one. Bound: a capped score is off by 2^-20 of the cap where that is 64 or less, by 2^-19
of itself above; beside it the score's own error as in tests/cache_helpers.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged_cache as pc
from tests.cache_helpers import Cache, queries, tolerance

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("cap", [2.0, 50.0, 64.0, 65.0, 1000.0, 2.0 ** 14, 2.0 ** 16])
@pytest.mark.parametrize("Hq", [8, 24, 40])
def test_large_caps(Hq, cap, biased):
    lens, news = [500, 90], [70, 3]
    c = Cache(64, lens, 1, 16)
    # values of either sign and one size, so that the outputs are differences of weights
    c.v[:] = np.where(c.rng.random(c.v.shape) < 0.5, 0x38, 0xB8).astype(np.uint8)
    c.vs[:] = 1.0
    c.poison_tails()
    ptr = np.concatenate([[0], np.cumsum(news)])
    req = np.repeat([0, 1], news)
    seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
    seen[::2] = np.minimum(seen[::2], 3)                  # few tokens: large differences
    q, q64 = queries(c.rng, len(req), Hq)
    slopes = np.full(Hq, 0.01, np.float32) if biased else None
    kw = dict(softcap=cap, slopes=None if slopes is None else torch.from_numpy(slopes).cuda())
    d = c.device()
    outs = [idx.idx_attend_prefill(q.cuda(), *d, i32(ptr), i32(seen), c.max_pages, **kw),
            idx.idx_attend(q.cuda(), *d, i32(seen), c.max_pages, row_req=i32(req), **kw)]
    # a row of each: few rows a request
    outs.append(idx.idx_attend_prefill(q[[0, 71]].cuda(), *d, i32([0, 1, 2]), i32(seen[[0, 71]]),
                                       c.max_pages, **kw))
    where = [np.arange(len(req))] * 2 + [np.array([0, 71])]
    scale = float(np.float32(128 ** -0.5))
    k, v, there = zip(*(c.tokens(b, 0) for b in (0, 1)))
    for out, rows in zip(outs, where):
        out = out.double().cpu().numpy()
        for i, r in enumerate(rows):
            for hq in range(0, Hq, 7):
                b = req[r]
                want, absum, mag = pc.attend(q64[r, hq], k[b], v[b], there[b], int(seen[r]), None,
                                             16, scale, cap, 0.01 if biased else 0.0)
                # (that bound takes 2^-20 of what is given as the cap)
                off = cap if cap <= 64 else 2 * min(mag, cap)
                tol = tolerance(want, absum, mag, int(seen[r]), off,
                                0.01 * int(seen[r]) if biased else 0.0)
                err = np.abs(out[i, hq] - want)
                assert (err <= tol).all(), (cap, r, hq, (err / tol).max())
