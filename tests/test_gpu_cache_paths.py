"""Paths of the cache calls that only some sizes take: rows without a slot among the
written ones, and prompt rows cut into stretches that the kernel lengthens."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402
from tests.cache_helpers import Cache, check_rows, queries  # noqa: E402
from tests.test_gpu_cache import i32, prefill, write_case, write_check  # noqa: E402

CUS, ROWS, TILE = 256, 256, 64


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("spans,refused", [
    ([(0, 1), (16, 17), (7, 8), (33, 34)], [1, 2]), ([(0, 40), (5, 90), (63, 65)], [1]),
    ([(3, 1500), (0, 700), (5, 900)], [1]), ([(0, 5)], [0])])
def test_rows_without_a_slot(spans, refused, page, dtype):
    """Refused requests' rows and rows behind the last token: slot -1, nothing written."""
    x, slots, c = write_case(21, spans, 8, page, dtype)
    first = 0
    for b, (start, stop) in enumerate(spans):
        if b in refused:
            slots[first:first + stop - start] = -1
        first += stop - start
    more = 9
    x = torch.cat([x, x[:1].expand(more, -1, -1, -1)])
    write_check(x, np.concatenate([slots, np.full(more, -1, np.int32)]), c)


def seen_rows(kind, lens, news):
    seen = [np.arange(n - k, n) + 1 for n, k in zip(lens, news)]
    for s, n in zip(seen, lens):
        if kind == "ends_see_all":          # the first and last row misjudge the rest
            s[1:-1] = np.minimum(s[1:-1], 70)
            s[0] = n
        elif kind == "ends_see_nothing":
            s[0] = s[-1] = 0
        elif kind == "unbounded":
            s[::3] = 2 ** 31 - 1
    return np.concatenate(seen).astype(np.int32)


@pytest.mark.parametrize("kind", ["causal", "ends_see_all", "ends_see_nothing", "unbounded"])
@pytest.mark.parametrize("lens,news", [([4608, 9000], [512, 512]), ([9000, 20, 4608],
                                                                   [512, 3, 500])])
def test_lengthened_stretches(lens, news, kind):
    Hq, Hkv, page = 32, 8, 16
    G, n = Hq // Hkv, sum(news)
    c = Cache(96, lens, Hkv, page)
    if kind == "unbounded":                 # what a last page holds is seen whole
        for b in range(len(lens)):
            tail = c.indices[c.indptr[b + 1] - 1]
            c.k[tail], c.v[tail] = 0x31, 0x32
    ptr = np.concatenate([[0], np.cumsum(news)])
    req = np.repeat(np.arange(len(lens)), news)
    seen = seen_rows(kind, lens, news)
    # the host's cut, from the partial results it asks for, and the share of a CU
    ws = idx.idx_attend_prefill_workspace_bytes(n, len(lens), Hq, Hkv, c.max_pages, page)
    splits = ws // (n * Hq * 130 * 4)
    tiles = -(-c.max_pages * page // TILE)
    chunk = -(-tiles // splits)
    work = 0
    for b in range(len(lens)):
        held = (c.indptr[b + 1] - c.indptr[b]) * page
        ends = min(held, seen[ptr[b]]) + min(held, seen[ptr[b + 1] - 1])
        work += -(-news[b] * G // ROWS) * -(-(int(ends) // 2) // TILE)
    share = -(-work * Hkv // CUS)
    assert splits > 1 and (share > chunk or kind == "ends_see_nothing"), (splits, chunk, share)
    if kind == "causal":
        assert (splits - 1) * share >= tiles  # the last stretch has no tile
    q, q64 = queries(c.rng, n, Hq)
    out = prefill(c, q, ptr, seen)
    rows = sorted({0, 1, 255, 256, news[0] - 1, news[0], n - 1, n // 2, 9, 300, n - 64})
    check_rows(out, c, q64, req, seen, rows=rows)
    assert torch.equal(out, prefill(c, q, ptr, seen))


FORMS = {"plain": {}, "biased": dict(slope=0.02), "capped": dict(cap=10.0),
         "capped_biased": dict(cap=10.0, slope=0.02), "far": dict(cap=500.0),
         "far_biased": dict(cap=500.0, slope=0.02)}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (17, 1), (33, 1), (64, 1), (40, 2)])
def test_places_without_tokens_in_every_kernel(Hq, Hkv, form):
    """Units without tokens read the pool's first page in their place, whose codes and
    scales are NaN here: kernels of one and two row tiles, two bands of heads, packed
    tokens and prompts, every form of the scores."""
    lens, page = [1, 16, 77, 500, 1300], 16
    c = Cache(97, lens, Hkv, page)
    if (c.indices == 0).any():              # the first page is nobody's
        c.indices[c.indices == 0] = np.setdiff1d(np.arange(1, c.n_pages), c.indices)[0]
        c.ks[c.indices], c.vs[c.indices] = 0.03, 0.05
        c.k[c.indices], c.v[c.indices] = c.k[c.indices] & 0x77, c.v[c.indices] & 0x77
    c.k[0], c.v[0], c.ks[0], c.vs[0] = 0xFF, 0x7F, np.nan, np.nan
    slope, cap = FORMS[form].get("slope"), FORMS[form].get("cap", 0.0)
    slopes = None if slope is None else np.full(Hq, slope, np.float32)
    kw = dict(softcap=cap, slopes=None if slope is None else torch.from_numpy(slopes).cuda())
    chk = dict(cap=cap, slopes=slopes)
    q, q64 = queries(c.rng, len(lens), Hq, 3.0)
    out = idx.idx_attend(q.cuda(), *c.device(), i32(lens), c.max_pages, **kw)
    check_rows(out, c, q64, range(len(lens)), lens, **chk)
    ptr = np.arange(len(lens) + 1)          # a row a request: the packed kernel
    check_rows(prefill(c, q, ptr, lens, **kw), c, q64, range(len(lens)), lens, **chk)
    news = [1, 16, 77, 300, 90]             # prompts
    ptr = np.concatenate([[0], np.cumsum(news)])
    req = np.repeat(np.arange(len(lens)), news)
    seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
    q, q64 = queries(c.rng, len(req), Hq, 3.0)
    out = prefill(c, q, ptr, seen, **kw)
    check_rows(out, c, q64, req, seen, rows=range(0, len(req), 29), **chk)
