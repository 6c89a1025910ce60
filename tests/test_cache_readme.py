"""The serving step that README.md shows, run as it stands on steps in which the packed
token rows are not the requests one by one: some idle, one adds several tokens, and there
are more token rows than tokens."""
import os
import re
from types import SimpleNamespace

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged_cache as pc
from tests.cache_helpers import Cache, check_rows, queries

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
# (lengths before the step, new tokens, token rows); 64 tokens of room a request
STEPS = [([20, 33, 5, 47], [1, 0, 1, 1], 3), ([20, 33, 5, 47], [0, 1, -5, 1], 4),
         ([1, 40, 0, 16], [3, 0, 0, 1], 6)]
PAGES = 4  # of a request, at most


def serving_step():
    with open(README) as f:
        blocks = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S)
                  if "idx_page_tables" in b]
    assert len(blocks) == 1
    return blocks[0]


def lists(lens):
    """Page lists of `lens` tokens in pages of 16, and the free ones in a ring."""
    rng = np.random.default_rng(8)
    n_pages = len(lens) * PAGES
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), PAGES), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        held = -(-n // 16)
        table[b, :held] = order[at:at + held]
        at += held
    ring = np.concatenate([order[at:], np.full(at, -1, np.int32)])
    return table, ring, [0, n_pages - at]


def run(lens, new, n_tokens, calls, **names):
    table, ring, cursor = lists(lens)
    i32 = names.pop("i32")
    got = []

    def recorded(name):
        def call(*a, **kw):
            out = calls[name](*a, **kw)
            if name.startswith("idx_attend"):
                got.append((name, kw, out))
            return out
        return call

    scope = dict(idx=SimpleNamespace(**{n: recorded(n) for n in calls}), seq_len=i32(lens),
                 n_new=i32(new), table=i32(table), free_ring=i32(ring), cursor=i32(cursor),
                 n_tokens=n_tokens, max_pages=PAGES, **names)
    exec(serving_step(), scope)
    return scope, got


@pytest.mark.parametrize("lens,new,n_tokens", STEPS)
def test_readme_rows_read_their_own_request(lens, new, n_tokens):
    """Which request each attention row reads, with the calls' argument rules alone."""
    i32 = lambda a: torch.from_numpy(np.array(a, np.int32))  # noqa: E731
    B = len(lens)

    def tables(seq, n, table, ring, cursor, rows):
        want = pc.page_tables(seq, n, table, ring, cursor, rows, 16)
        return SimpleNamespace(**{k: i32(v) for k, v in want.items()})

    def attend(q, kc, vc, ks, vs, kv_indptr, kv_indices, kv_len, max_pages, row_req=None,
               ids=None, **kw):
        rows = q.shape[0]
        assert kv_len.numel() == rows
        assert row_req is not None or rows <= B
        return (torch.arange(rows) if row_req is None else row_req, ids)

    calls = dict(
        idx_page_tables=tables, idx_cache_write=lambda *a: None,
        idx_attend_prefill=lambda *a: None, idx_attend=attend,
        # a row for each request, of ids that name it
        idx_select_paged=lambda q, *a: (torch.arange(B, dtype=torch.int32)[:, None].repeat(1, 2),
                                        None, None))
    scope, got = run(lens, new, n_tokens, calls, i32=i32, q=torch.zeros(n_tokens, 4, 128),
                     q_idx=None, c_pool=None, k=None, v=None, k_cache=None, v_cache=None,
                     k_scale=None, v_scale=None)
    single = [out for name, _, out in got if name == "idx_attend"]
    assert len(single) == 2 and any(ids is not None for _, ids in single)
    want = scope["t"].tok_req
    real = want >= 0
    for req, ids in single:
        assert torch.equal(req[real].int(), want[real])
        assert not ((req[~real] >= 0) & (req[~real] < B)).any()
        if ids is not None:
            assert torch.equal(ids[real, 0].int(), want[real])


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("lens,new,n_tokens", STEPS)
def test_readme_step_against_the_oracle(lens, new, n_tokens):
    import block_scoring_top_amd as idx
    i32 = lambda a: torch.from_numpy(np.array(a, np.int32)).cuda()  # noqa: E731
    Hq, Hkv = 8, 2
    c = Cache(12, [PAGES * 16] * len(lens), Hkv, 16, spare=0)
    c.ks, c.vs = (np.exp2(np.round(np.log2(s))).astype(np.float32) for s in (c.ks, c.vs))
    kc, vc, ks, vs, _, _ = c.device()
    x = torch.from_numpy(c.rng.standard_normal((n_tokens, 2, Hkv, 128)).astype(np.float32))
    x = x.bfloat16().cuda()
    q, q64 = queries(c.rng, n_tokens, Hq)
    q_idx, _ = queries(c.rng, len(lens), 4)
    pool = torch.from_numpy(c.rng.standard_normal((c.n_pages, 128)).astype(np.float32))
    calls = {n: getattr(idx, n) for n in ("idx_page_tables", "idx_cache_write", "idx_select_paged",
                                          "idx_attend", "idx_attend_prefill")}
    scope, got = run(lens, new, n_tokens, calls, i32=i32, q=q.cuda(), k=x[:, 0], v=x[:, 1],
                     k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, q_idx=q_idx.cuda(),
                     c_pool=pool.bfloat16().cuda())
    t = scope["t"]
    c.k, c.v = kc.view(torch.uint8).cpu().numpy(), vc.view(torch.uint8).cpu().numpy()
    c.ks, c.vs = ks.cpu().numpy(), vs.cpu().numpy()
    c.indptr, c.indices = t.kv_indptr.cpu().numpy(), t.kv_indices.cpu().numpy()
    req, seen = t.tok_req.cpu().numpy(), t.tok_len.cpu().numpy()
    rows = int(t.tok_indptr[-1])
    assert len(got) == 3
    for name, kw, out in got:
        ids = kw.get("ids")
        check_rows(out, c, q64, req, seen, ids=None if ids is None else ids.cpu().numpy(),
                   cap=kw.get("softcap", 0.0),
                   rows=range(rows) if name == "idx_attend_prefill" else None)
