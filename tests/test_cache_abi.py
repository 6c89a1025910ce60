"""The paged-cache calls without a GPU: documented refusals before any HIP call (the
fake pointers are never dereferenced), workspace sizes, and the binding's own checks."""
import math
import os

import pytest

torch = pytest.importorskip("torch")

import block_scoring_top_amd as idx
from tests.test_abi import INVALID, OK, P, UNSUPPORTED, WORKSPACE, declared


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(idx.lib_path()):
        pytest.skip("libidx.so not built")
    return idx.load()


def test_header_declares_the_cache_calls():
    for n in ("idx_page_tables", "idx_cache_write", "idx_attend", "idx_attend_prefill",
              "idx_attend_workspace_bytes", "idx_attend_prefill_workspace_bytes"):
        assert n in declared()


TABLES = dict(seq_len=P, n_new=P + 64, cursor=P + 128, table=P, free_ring=P, seq_out=P + 4096,
              cursor_out=P + 8192, kv_indptr=P, kv_indices=P, tok_indptr=P, slots=P, tok_req=P,
              tok_len=P, B=4, max_pages=8, page_size=16, n_pages=100, n_indices=100, n_tokens=10)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, INVALID) for k in list(TABLES)[:13]],
    *[({k: P + 2}, INVALID) for k in list(TABLES)[:13]],
    (dict(B=0), INVALID), (dict(max_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_indices=-1), INVALID), (dict(n_tokens=-1), INVALID),
    (dict(B=16384, max_pages=1 << 18), INVALID), (dict(max_pages=1 << 27), INVALID),
    (dict(n_pages=1 << 27), INVALID), (dict(seq_out=P), INVALID),
    (dict(cursor_out=P + 128), INVALID), (dict(B=16385), UNSUPPORTED),
])
def test_page_tables_rejects(lib, kw, want):
    assert lib.idx_page_tables(*(TABLES | kw).values(), None) == want


WRITE = dict(k=P, v=P, k_stride=512, v_stride=512, slots=P, k_cache=P, v_cache=P, k_scale=P,
             v_scale=P, n_tok=3, Hkv=4, D=128, n_pages=10, page_size=16, dt=1)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, INVALID) for k in ("k", "v", "slots", "k_cache", "v_cache", "k_scale",
                                     "v_scale")],
    *[({k: P + 8}, INVALID) for k in ("k", "v", "k_cache", "v_cache")],
    *[({k: P + 2}, INVALID) for k in ("slots", "k_scale", "v_scale")],
    (dict(k_stride=511), INVALID), (dict(v_stride=504), INVALID), (dict(k_stride=516), INVALID),
    (dict(n_tok=-1), INVALID), (dict(Hkv=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(dt=2), INVALID), (dict(n_pages=1 << 30), INVALID),
    (dict(n_tok=(1 << 30) + 1, Hkv=1), INVALID),
    (dict(n_tok=1 << 26, Hkv=32, k_stride=4096, v_stride=4096), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=128), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(n_tok=0), OK), (dict(n_tok=0, k=None, slots=None), OK),
])
def test_cache_write_rejects(lib, kw, want):
    assert lib.idx_cache_write(*(WRITE | kw).values(), None) == want


ROWS = dict(q=P, q_stride=2048, k_cache=P, v_cache=P, k_scale=P, v_scale=P, kv_indptr=P,
            kv_indices=P, kv_len=P, row_req=None, ids=None, slopes=None, out=P, R=2, B=2, Hq=16,
            Hkv=4, D=128, n_pages=100, n_indices=64, max_pages=32, page_size=16, K=0, scale=0.1,
            softcap=0.0, dt=1, ws=None, ws_bytes=0)
SHARED = [
    *[({k: None}, INVALID) for k in ("q", "k_cache", "v_cache", "k_scale", "v_scale",
                                     "kv_indptr", "kv_indices", "kv_len", "out")],
    *[({k: P + 8}, INVALID) for k in ("q", "k_cache", "v_cache", "out")],
    *[({k: P + 2}, INVALID) for k in ("k_scale", "v_scale", "kv_indptr", "kv_indices", "kv_len",
                                      "slopes")],
    (dict(q_stride=2040), INVALID), (dict(q_stride=2052), INVALID), (dict(B=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(Hq=18), INVALID), (dict(Hq=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_indices=-1), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 28), INVALID), (dict(n_pages=1 << 30), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=math.nan), INVALID), (dict(dt=2), INVALID),
    (dict(softcap=1e-30), UNSUPPORTED), (dict(softcap=1e6), UNSUPPORTED),
    (dict(dt=0), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(Hq=65 * 4, q_stride=65 * 512), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(R=-1), INVALID), (dict(R=3), INVALID), (dict(row_req=P + 2), INVALID),
    (dict(ids=P, K=0), INVALID), (dict(K=4), INVALID), (dict(ids=P + 1, K=4), INVALID),
    (dict(ids=P, K=-1), INVALID), (dict(max_pages=4096), WORKSPACE),
    (dict(R=1 << 22, row_req=P), INVALID), (dict(R=1 << 26, Hq=1, Hkv=1, q_stride=128, row_req=P), INVALID),
    (dict(max_pages=4096, ws=P + 16, ws_bytes=1 << 30), WORKSPACE), (dict(R=0), OK),
    (dict(R=0, q=None, out=None), OK),
])
def test_attend_rejects(lib, kw, want):
    assert lib.idx_attend(*(ROWS | kw).values(), None) == want


PRE = {k: v for k, v in ROWS.items() if k not in ("row_req", "ids", "R", "K", "slopes", "out")}
PRE = (dict(list(PRE.items())[:8]) | dict(tok_indptr=P, kv_len=P, slopes=None, out=P, n_tok=3)
       | dict(list(PRE.items())[9:]))


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(n_tok=-1), INVALID), (dict(tok_indptr=None), INVALID), (dict(tok_indptr=P + 2), INVALID),
    (dict(n_tok=1 << 30), INVALID),
    (dict(B=16385), UNSUPPORTED), (dict(max_pages=4096), WORKSPACE),
    (dict(max_pages=4096, ws=P + 16, ws_bytes=1 << 30), WORKSPACE), (dict(n_tok=0), OK),
])
def test_attend_prefill_rejects(lib, kw, want):
    assert lib.idx_attend_prefill(*(PRE | kw).values(), None) == want


def test_workspace_sizes(lib):
    # none where a row is not cut; else, per row and head, the same count of partial
    # results: 128 sums and two statistics
    assert lib.idx_attend_workspace_bytes(2, 16, 4, 8, 0, 16) == 0
    assert lib.idx_attend_workspace_bytes(0, 16, 4, 4096, 0, 16) == 0
    assert lib.idx_attend_workspace_bytes(4, 17, 4, 4096, 0, 16) == 0   # not a legal shape
    n = lib.idx_attend_workspace_bytes(2, 16, 4, 4096, 0, 16)
    assert n > 0 and n % (32 * 130 * 4) == 0
    n = lib.idx_attend_prefill_workspace_bytes(3, 2, 16, 4, 4096, 16)
    assert n > 0
    assert lib.idx_attend_prefill_workspace_bytes(3, 2, 16, 4, 1, 16) == 0


def test_workspaces_do_not_grow_with_a_generous_bound(lib):
    for pages in (4096, 1 << 18, 1 << 24):
        assert lib.idx_attend_workspace_bytes(4, 16, 4, pages, 0, 16) <= 4 * 16 * 128 * 521
        assert lib.idx_attend_workspace_bytes(512, 16, 4, pages, 0, 16) == 0
        assert lib.idx_attend_prefill_workspace_bytes(8192, 2, 16, 4, pages, 16) == 0


def test_binding_refuses_tensors_off_the_gpu():
    t = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="same GPU"):
        idx.idx_page_tables(t, t, torch.zeros(1, 4, dtype=torch.int32), t, t, 1)
    c = torch.zeros(2, 1, 16, 128, dtype=torch.uint8)
    s = torch.zeros(2, 1)
    with pytest.raises(ValueError, match="same GPU"):
        idx.idx_cache_write(torch.zeros(1, 1, 128), torch.zeros(1, 1, 128), t, c, c, s, s)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    for call in (idx.idx_attend, idx.idx_attend_prefill):
        args = (q, c, c, s, s, t, t) + ((t,) if call is idx.idx_attend_prefill else ()) + (t, 4)
        with pytest.raises(ValueError, match="same GPU"):
            call(*args)
