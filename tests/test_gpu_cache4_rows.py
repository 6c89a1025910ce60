"""The paged 4-bit cache: rows of single tokens with a selection and a request each, NaN scales
under caps and biases, and workspaces of the prompt kernel, against the CPU oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.cache4_helpers import Cache4, check_rows
from tests.cache_helpers import queries

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("K", [1, 5, 130])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (40, 2)])
def test_several_rows_of_a_request_with_a_selection_each(Hq, Hkv, K, page):
    """Rows, requests and selections in orders of their own, unknown requests among them."""
    lens = [3 * page + 5, 140 * page - 9, page]
    c = Cache4(K + page, lens, Hkv, page)
    req = [1, 0, 2, 1, -1, 1, 0, 3, 2, 1, 0]
    R = len(req)
    ids, seen = np.full((R, K), -1, np.int32), np.zeros(R, int)
    for r, b in enumerate(req):
        if not 0 <= b < len(lens):
            ids[r], seen[r] = 0, 17
            continue
        seen[r] = lens[b] - c.rng.integers(0, min(lens[b], 40))
        pick = c.rng.permutation(-(-int(seen[r]) // page))[:K]
        ids[r, :len(pick)] = np.sort(pick) if r % 2 else pick
        if K > 1 and r % 3 == 0:
            ids[r, 0] = 2 ** 31 - 1 if r % 2 else -1
    cut = idx.idx_attend4_workspace_bytes(R, Hq, Hkv, c.max_pages, K, page) > 0
    assert cut == (K == 130)
    q, q64 = queries(c.rng, R, Hq)
    for kw in ({}, dict(softcap=20.0)):
        out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, row_req=i32(req),
                              ids=dev(ids), **kw)
        check_rows(out, c, q64, req, seen, ids, cap=kw.get("softcap", 0.0))


def test_many_rows_with_a_selection_each():
    """Rows that are not cut, several of each request."""
    lens, K = [700, 90, 1500, 333], 9
    c = Cache4(5, lens, 2, 16)
    R = 300
    req = c.rng.integers(0, 4, R)
    seen = np.array([c.rng.integers(1, lens[b] + 1) for b in req])
    ids = np.full((R, K), -1, np.int32)
    for r in range(R):
        pick = np.sort(c.rng.permutation(-(-int(seen[r]) // 16))[:K])
        ids[r, :len(pick)] = pick
    assert idx.idx_attend4_workspace_bytes(R, 8, 2, c.max_pages, K, 16) == 0
    q, q64 = queries(c.rng, R, 8)
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, row_req=i32(req),
                          ids=dev(ids))
    check_rows(out, c, q64, req, seen, ids, rows=range(0, R, 5))


KINDS = [dict(softcap=30.0), dict(softcap=500.0), dict(biased=True), dict(softcap=5.0, biased=True)]


def kind_of(kw, Hq):
    slopes = np.exp2(-8 * np.arange(1, Hq + 1) / Hq).astype(np.float32) if "biased" in kw else None
    cap = kw.get("softcap", 0.0)
    return cap, slopes, dict(softcap=cap, slopes=None if slopes is None else dev(slopes))


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("Hq", [4, 20])
def test_nan_scales_under_caps_and_biases(Hq, kw):
    lens = [100, 100, 100, 64]
    cap, slopes, call = kind_of(kw, Hq)
    c = Cache4(10, lens, 1, 16)
    q, q64 = queries(c.rng, 4, Hq)
    clean = idx.idx_attend4(q.cuda(), *c.device(), i32(lens), c.max_pages, **call)
    c.ks[c.pages(0)[3], 0, 5, 2] = 255
    c.vs[c.pages(1)[0], 0, 1, 9] = 255
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(lens), c.max_pages, **call)
    check_rows(out, c, q64, range(4), lens, cap=cap, slopes=slopes)
    assert torch.isnan(out[0]).all() and torch.isnan(out[1, :, 32:64]).all()
    rest = [i for i in range(128) if not 32 <= i < 64]
    assert torch.equal(out[1][:, rest], clean[1][:, rest])
    assert torch.equal(out[2:], clean[2:])
    seen = [53, 9, 100, 63]  # the tokens before the NaN
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, **call)
    check_rows(out, c, q64, range(4), seen, cap=cap, slopes=slopes)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("n,t", [(300, 5), (300, 130), (6000, 130)])
def test_nan_scales_under_caps_and_biases_in_prompts(n, t, kw):
    Hq = 4
    cap, slopes, call = kind_of(kw, Hq)
    c = Cache4(11, [n], 2, 16)
    q, q64 = queries(c.rng, t, Hq)
    seen = np.arange(n - t, n) + 1
    run = lambda: idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([0, t]), i32(seen),  # noqa: E731
                                          c.max_pages, **call)
    clean = run()
    at = n - 2  # two rows see it
    c.vs[c.pages(0)[at // 16], 0, 2, at % 16] = 255
    c.ks[c.pages(0)[at // 16], 1, at % 16, 1] = 255
    out = run()
    assert torch.isnan(out[-2:, :2, 64:96]).all() and torch.isnan(out[-2:, 2:]).all()
    rest = [i for i in range(128) if not 64 <= i < 96]
    assert torch.equal(out[-2:, :2][:, :, rest], clean[-2:, :2][:, :, rest])
    assert torch.equal(out[:-2], clean[:-2])
    check_rows(out, c, q64, np.zeros(t), seen, cap=cap, slopes=slopes,
               rows=sorted({0, t // 2, t - 3, t - 2, t - 1}))


@pytest.mark.parametrize("news,B", [([130], 1), ([300, 90], 2), ([500], 1)])
def test_prompt_workspaces_may_hold_anything(news, B):
    """The 256-row kernel, cut, with a bound above the lists: the later stretches hold nothing."""
    lens = [6000 - 700 * b for b in range(B)]
    c = Cache4(12, lens, 2, 16)
    n = sum(news)
    q, q64 = queries(c.rng, n, 8)
    bound = 2 * c.max_pages
    size = idx.idx_attend4_prefill_workspace_bytes(n, B, 8, 2, bound)
    assert size > 0 and n * 8 / 2 / B > 64
    seen = np.concatenate([np.arange(a - k, a) + 1 for a, k in zip(lens, news)])
    seen[::11] = 0
    ptr = np.concatenate([[0], np.cumsum(news)])
    outs = [idx.idx_attend4_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), bound,
                                    ws=torch.full((size,), fill, dtype=torch.uint8, device="cuda"))
            for fill in (0, 255, 127)]
    assert torch.isfinite(outs[0]).all() and not outs[0][::11].any()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check_rows(outs[0], c, q64, np.repeat(np.arange(B), news), seen, rows=range(0, n, 37))
