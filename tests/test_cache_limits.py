"""How large the attention calls may be: the launch alone bounds them."""
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_scoring_top_amd as idx
from tests.cache_helpers import Cache, check_rows, queries
from tests.test_abi import HIPERR, INVALID, P
from tests.test_cache_abi import PRE, ROWS, WRITE

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would run")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(idx.lib_path()):
        pytest.skip("libidx.so not built")
    return idx.load()


def sized(n, Hq, Hkv, **kw):
    return dict(Hq=Hq, Hkv=Hkv, q_stride=128 * Hq, max_pages=2) | kw


# an accepted call gets as far as its launch, which fails without a GPU
@no_gpu
@pytest.mark.parametrize("R,Hq,Hkv,want", [
    (1 << 22, 16, 1, HIPERR), (1 << 20, 64, 1, HIPERR), ((1 << 24) - 1, 1, 1, HIPERR),
    ((1 << 24) - 1, 32, 1, HIPERR), (1 << 24, 1, 1, INVALID), ((1 << 23) - 1, 33, 1, HIPERR),
    (1 << 23, 33, 1, INVALID), ((1 << 21) - 1, 128, 8, HIPERR), (1 << 21, 128, 8, INVALID)])
def test_rows_up_to_the_launch(lib, R, Hq, Hkv, want):
    assert lib.idx_attend_workspace_bytes(R, Hq, Hkv, 2, 0, 16) == 0
    args = ROWS | sized(R, Hq, Hkv, R=R, row_req=P)
    assert lib.idx_attend(*args.values(), None) == want


@no_gpu
@pytest.mark.parametrize("n,Hq,Hkv,B,want", [
    (1 << 22, 16, 1, 2, HIPERR), (1 << 20, 64, 1, 2, HIPERR), ((1 << 23) - 2, 256, 8, 1, INVALID),
    ((1 << 23) - 256, 256, 8, 1, HIPERR), (1 << 16, 1 << 14, 1 << 14, 1, HIPERR),
    (1 << 17, 1 << 14, 1 << 14, 1, INVALID)])
def test_prompt_tokens_up_to_the_launch(lib, n, Hq, Hkv, B, want):
    assert lib.idx_attend_prefill_workspace_bytes(n, B, Hq, Hkv, 2, 16) == 0
    args = PRE | sized(n, Hq, Hkv, n_tok=n, B=B)
    assert lib.idx_attend_prefill(*args.values(), None) == want


# 256 threads for 16 rows and 2 KV heads: n_tok * ceil(Hkv / 2) below 2^28, as documented
@no_gpu
@pytest.mark.parametrize("n,Hkv,want", [
    ((1 << 28) - 17, 1, HIPERR), ((1 << 28) - 17, 2, HIPERR), (1 << 28, 1, INVALID),
    ((1 << 26) - 17, 8, HIPERR), (1 << 26, 8, INVALID), ((1 << 31) - 1, 1, INVALID)])
def test_written_tokens_up_to_the_launch(lib, n, Hkv, want):
    stride = 128 * Hkv
    args = WRITE | dict(n_tok=n, Hkv=Hkv, k_stride=stride, v_stride=stride)
    assert lib.idx_cache_write(*args.values(), None) == want


def test_the_header_states_the_bound_of_written_tokens():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "idx_cache.h")) as f:
        text = f.read()
    assert "n_tok <= 2^30" not in text and "n_tok * ceil(Hkv / 2)" in text


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
def test_calls_of_2_to_the_26_query_heads():
    """17 GB of queries: rows in a pattern of 1024, every repetition as the first, which is
    checked against the oracle."""
    lens, Hq, n, pattern = [20, 5], 16, 1 << 22, 1024
    c = Cache(95, lens, 1, 16)
    d = c.device()
    q, q64 = queries(c.rng, pattern, Hq)
    qd = q.cuda().repeat(n // pattern, 1, 1)
    req = np.arange(pattern) % 2
    seen = np.array([20, 4, 1, 5, 17, 0])[np.arange(pattern) % 6]

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()

    def check(out, req):
        check_rows(out[:pattern], c, q64, req, seen, rows=range(0, pattern, 37))
        for part in out.view(n // pattern, pattern, Hq, 128).split(256):
            assert torch.equal(part, out[:pattern].expand_as(part))

    many = i32(seen).repeat(n // pattern)
    out = idx.idx_attend(qd, *d, many, c.max_pages, row_req=i32(req).repeat(n // pattern))
    check(out, req)
    # request 0 has all the rows
    out = idx.idx_attend_prefill(qd, *d, i32([0, n, n]), many, c.max_pages, out=out)
    check(out, np.zeros(pattern, int))
