"""A row's output comes from the tokens it sees alone: neither the codes nor the scales of
the others (the rest of its own prompt, say) change a bit of it, whatever rows share its
products."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged_cache as pc
from tests.cache_helpers import Cache, check_rows, queries

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402

# lengths, new tokens, Hq, Hkv: whole prompts (256 rows a tile); their keys cut into
# stretches; few rows a request (16 a tile, short and over several workgroups)
CALLS = {"whole": ([700, 300], [700, 300], 8, 2), "cut": ([6000], [130], 4, 1),
         "few": ([300, 77, 40], [7, 5, 3], 8, 2), "few_cut": ([5000, 900], [6, 6], 4, 1)}
KINDS = {"plain": {}, "capped": dict(softcap=20.0), "biased": dict(slopes=0.03)}


def say(*a):
    print(*a)
    sys.stdout.flush()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def case(name, page, seed, cut):
    """A cache and packed rows, every other one of which sees the first cut[b] tokens."""
    lens, news, Hq, Hkv = CALLS[name]
    c = Cache(seed, lens, Hkv, page)
    ptr = np.concatenate([[0], np.cumsum(news)])
    req = np.repeat(np.arange(len(lens)), news)
    seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
    at = np.arange(len(req))
    seen = np.where(at % 2 == 0, np.minimum(seen, np.array(cut)[req]), seen)
    q, q64 = queries(c.rng, len(req), Hq)
    return c, ptr, req, seen, q, q64


def prefill(c, ptr, seen, q, **kw):
    if "slopes" in kw:
        kw["slopes"] = torch.full((q.shape[1],), kw["slopes"], device="cuda")
    return idx.idx_attend_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), c.max_pages, **kw)


def change_from(c, cut, scales):
    """New codes for every token from cut[b] on, NaN among them, and (for whole pages)
    new scales."""
    for b, first in enumerate(cut):
        for i, p in enumerate(c.indices[c.indptr[b]:c.indptr[b + 1]]):
            o = max(first - i * c.page, 0)
            if o >= c.page:
                continue
            c.k[p, :, o:] = pc.e4m3_encode(c.rng.standard_normal(c.k[p, :, o:].shape) * 200)
            c.v[p, :, :, o:] = pc.e4m3_encode(c.rng.standard_normal(c.v[p, :, :, o:].shape) * 200)
            if i % 3 == 0:
                c.k[p, :, -1, 3], c.v[p, :, 5, -1] = 0x7F, 0xFF
            if o == 0 and scales:
                c.ks[p] *= 4
                c.vs[p] *= np.float32(2.0 ** c.rng.integers(-30, 31))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("name", list(CALLS))
def test_bits_do_not_depend_on_tokens_a_row_does_not_see(name, page, kind):
    lens = CALLS[name][0]
    for cut, scales in (([n // 2 // page * page for n in lens], True),
                        ([max(n // 2 - 5, 1) for n in lens], True)):
        say(f"[unseen] {name} page={page} {kind} cut={cut}")
        c, ptr, req, seen, q, _ = case(name, page, 61, cut)
        first = prefill(c, ptr, seen, q, **KINDS[kind])
        change_from(c, cut, scales)
        again = prefill(c, ptr, seen, q, **KINDS[kind])
        rows = torch.from_numpy(seen <= np.array(cut)[req])
        assert rows.sum() >= len(req) // 2
        assert not first[rows].isnan().any()
        assert torch.equal(first[rows].view(torch.int16), again[rows].view(torch.int16))


@pytest.mark.parametrize("name", list(CALLS))
def test_value_scales_a_row_does_not_see_cost_it_nothing(name):
    """The pages behind what half of the rows see hold values 2^30 times as large."""
    lens = CALLS[name][0]
    cut = [n // 2 // 16 * 16 for n in lens]
    c, ptr, req, seen, q, q64 = case(name, 16, 62, cut)
    for b, first in enumerate(cut):
        c.vs[c.indices[c.indptr[b] + first // 16:c.indptr[b + 1]]] *= np.float32(2.0 ** 30)
    out = prefill(c, ptr, seen, q)
    rows = np.flatnonzero(seen <= np.array(cut)[req])
    check_rows(out, c, q64, req, seen, rows=rows[:: max(1, len(rows) // 40)])


def test_value_scales_behind_the_first_phase_of_a_long_prompt():
    """Rows that end in the first, at the border and in the second 32768 tokens, on scales
    that grow with every page."""
    n = 34000
    c = Cache(63, [n], 1, 16)
    pages = c.indices
    c.vs[pages, 0] = np.exp2(np.linspace(-60, 0, len(pages))).astype(np.float32)
    seen = np.array([1, 16, 17, 5000, 32767, 32768, 32769, 33000, n] * 10)
    q, q64 = queries(c.rng, len(seen), 1)
    out = prefill(c, [0, len(seen)], seen, q)
    check_rows(out, c, q64, np.zeros(len(seen), int), seen)
