"""The 4-bit cache's and the rotary calls without a GPU: documented refusals before any HIP
call (the fake pointers are never dereferenced), workspace sizes, the rotary tables, and the
binding's own checks."""
import ctypes
import math
import os
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_scoring_top_amd as idx
from tests.test_abi import INVALID, OK, P, UNSUPPORTED, WORKSPACE, declared
from tests.test_cache_abi import PRE, ROWS, SHARED, WRITE

# 60 digits of pi, over 10^59
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(idx.lib_path()):
        pytest.skip("libidx.so not built")
    return idx.load()


def test_headers_declare_the_calls():
    for n in ("idx_cache4_write", "idx_cache4_read", "idx_attend4", "idx_attend4_prefill",
              "idx_attend4_workspace_bytes", "idx_attend4_prefill_workspace_bytes", "idx_rope",
              "idx_rope_table", "idx_rope_turns"):
        assert n in declared() and n in idx.__all__


ALIGNED = [({k: P + 8}, INVALID) for k in ("k_cache", "v_cache", "k_scale", "v_scale")]
ROWS_OF = [
    (dict(k_stride=511), INVALID), (dict(v_stride=504), INVALID), (dict(k_stride=516), INVALID),
    (dict(n_tok=-1), INVALID), (dict(Hkv=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(dt=2), INVALID), (dict(n_pages=1 << 30), INVALID),
    (dict(n_tok=(1 << 30) + 1, Hkv=1), INVALID),
    (dict(n_tok=1 << 26, Hkv=32, k_stride=4096, v_stride=4096), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=128), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    *[({k: P + 8}, INVALID) for k in ("k", "v")], (dict(slots=P + 2), INVALID),
    (dict(slots=None), INVALID), (dict(n_tok=0), OK), (dict(n_tok=0, k=None, slots=None), OK),
]


@pytest.mark.parametrize("kw,want", ALIGNED + ROWS_OF + [
    ({k: None}, INVALID) for k in ("k", "v", "k_cache", "v_cache", "k_scale", "v_scale")])
def test_write_rejects(lib, kw, want):
    assert lib.idx_cache4_write(*(WRITE | kw).values(), None) == want


READ = dict(slots=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P, k=P, v=P, k_stride=512,
            v_stride=512, n_tok=3, Hkv=4, D=128, n_pages=10, page_size=16, dt=1)


@pytest.mark.parametrize("kw,want", ALIGNED + ROWS_OF + [
    *[({k: None}, INVALID) for k in ("k_cache", "v_cache", "k_scale", "v_scale")],
    (dict(k=None, v=None), OK), (dict(k=None, v_stride=0), INVALID)])
def test_read_rejects(lib, kw, want):
    assert lib.idx_cache4_read(*(READ | kw).values(), None) == want


@pytest.mark.parametrize("kw,want", ALIGNED + SHARED + [
    (dict(R=-1), INVALID), (dict(R=3), INVALID), (dict(row_req=P + 2), INVALID),
    (dict(ids=P, K=0), INVALID), (dict(K=4), INVALID), (dict(ids=P + 1, K=4), INVALID),
    (dict(ids=P, K=-1), INVALID), (dict(max_pages=1 << 16), WORKSPACE),
    (dict(R=1 << 22, row_req=P), INVALID),
    (dict(R=1 << 26, Hq=1, Hkv=1, q_stride=128, row_req=P), INVALID),
    (dict(max_pages=1 << 16, ws=P + 16, ws_bytes=1 << 30), WORKSPACE), (dict(R=0), OK),
    (dict(R=0, q=None, out=None), OK)])
def test_attend_rejects(lib, kw, want):
    assert lib.idx_attend4(*(ROWS | kw).values(), None) == want


@pytest.mark.parametrize("kw,want", ALIGNED + SHARED + [
    (dict(n_tok=-1), INVALID), (dict(tok_indptr=None), INVALID), (dict(tok_indptr=P + 2), INVALID),
    (dict(n_tok=1 << 30), INVALID), (dict(B=16385), UNSUPPORTED),
    (dict(max_pages=1 << 16), WORKSPACE),
    (dict(max_pages=1 << 16, ws=P + 16, ws_bytes=1 << 30), WORKSPACE), (dict(n_tok=0), OK)])
def test_attend_prefill_rejects(lib, kw, want):
    assert lib.idx_attend4_prefill(*(PRE | kw).values(), None) == want


def test_workspace_sizes(lib):
    assert lib.idx_attend4_workspace_bytes(2, 16, 4, 8, 0, 16) == 0
    assert lib.idx_attend4_workspace_bytes(0, 16, 4, 4096, 0, 16) == 0
    assert lib.idx_attend4_workspace_bytes(4, 17, 4, 4096, 0, 16) == 0   # not a legal shape
    n = lib.idx_attend4_workspace_bytes(2, 16, 4, 4096, 0, 16)
    assert n > 0 and n % (32 * 130 * 4) == 0
    assert lib.idx_attend4_prefill_workspace_bytes(3, 2, 16, 4, 4096, 16) > 0
    assert lib.idx_attend4_prefill_workspace_bytes(3, 2, 16, 4, 1, 16) == 0
    for pages in (4096, 1 << 18, 1 << 24):  # they do not grow with a generous bound
        assert lib.idx_attend4_workspace_bytes(4, 16, 4, pages, 0, 16) <= 4 * 16 * 128 * 521
        assert lib.idx_attend4_workspace_bytes(512, 16, 4, pages, 0, 16) == 0


ROPE = dict(q=P, k=P, q_stride=2048, k_stride=512, tok_len=P, turns=P, q_out=P, k_out=P,
            q_out_stride=2048, k_out_stride=512, n_tok=3, Hq=16, Hkv=4, D=128, first=0, rot=128,
            factor=1.0, flags=0, dt=1)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, INVALID) for k in ("q", "k", "tok_len", "turns", "q_out", "k_out")],
    *[({k: P + 8}, INVALID) for k in ("q", "k", "q_out", "k_out")],
    (dict(tok_len=P + 2), INVALID), (dict(turns=P + 4), INVALID),
    (dict(q_stride=2040), INVALID), (dict(q_out_stride=2052), INVALID),
    (dict(k_stride=504), INVALID), (dict(k_out_stride=516), INVALID),
    (dict(q_out_stride=4096), INVALID),  # in place, other rows
    (dict(k_out_stride=1024), INVALID), (dict(n_tok=-1), INVALID), (dict(n_tok=1 << 24), INVALID),
    (dict(Hq=0), INVALID), (dict(Hkv=-1), INVALID), (dict(first=-8), INVALID),
    (dict(first=8), INVALID), (dict(rot=0), INVALID), (dict(rot=17), INVALID),
    (dict(rot=130), INVALID), (dict(factor=math.nan), INVALID), (dict(factor=math.inf), INVALID),
    (dict(flags=4), INVALID), (dict(dt=2), INVALID), (dict(D=64, rot=64), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(rot=64, first=4), UNSUPPORTED), (dict(n_tok=0), OK),
    (dict(n_tok=0, q=None, k=None), OK), (dict(Hkv=0, k=None, k_out=None, n_tok=0), OK),
])
def test_rope_rejects(lib, kw, want):
    assert lib.idx_rope(*(ROPE | kw).values(), None) == want


def turns_of(f):
    """f / 2 pi in units of 2^-64, modulo a turn (rational numbers)."""
    return Fraction(f) / (2 * PI) * 2 ** 64


def near(table, freq):
    for t, f in zip(table.tolist(), freq):
        off = (t - turns_of(f)) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, (t, f)


def test_rope_turns(lib):
    freq = [1.0, 1e-4, 0.3, 1e-9, 0.0, -0.5, 4.0, -1e-12, math.pi]
    near(idx.idx_rope_turns(freq, device="cpu"), freq)
    near(idx.idx_rope_turns(torch.tensor(freq, dtype=torch.float64), device="cpu"), freq)
    out = (ctypes.c_uint64 * 64)()
    one = (ctypes.c_double * 65)(*[0.5] * 65)
    assert lib.idx_rope_turns(one, 64, out) == OK
    assert lib.idx_rope_turns(one, 65, out) == UNSUPPORTED
    assert lib.idx_rope_turns(one, 0, out) == INVALID
    assert lib.idx_rope_turns(None, 4, out) == INVALID
    assert lib.idx_rope_turns(one, 4, None) == INVALID
    for bad in (math.nan, math.inf, 4.1, -1e3):
        with pytest.raises(idx.IdxError):
            idx.idx_rope_turns([0.5, bad], device="cpu")
    with pytest.raises(ValueError):
        idx.idx_rope_turns([[0.5]], device="cpu")


def keep_by_turns(f, original, lo, hi):
    return min(max((original * f / (2 * math.pi) - lo) / (hi - lo), 0), 1)


@pytest.mark.parametrize("rot", [16, 64, 128])
@pytest.mark.parametrize("base", [1e4, 5e5])
def test_rope_table(lib, rot, base):
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]

    def close(table, freq):  # a double's rounding of base^x apart
        for t, f in zip(table.tolist(), freq):
            assert abs(t - turns_of(f)) <= 1 + 2.0 ** -46 * turns_of(f), (t, f)

    made = lambda **kw: idx.idx_rope_table(rot, base, device="cpu", **kw)  # noqa: E731
    close(made(), plain)
    close(made(kind="linear", stretch=4.0), [f / 4 for f in plain])
    wide = base * 4.0 ** (rot / (rot - 2))
    close(made(kind="base", stretch=4.0), [wide ** (-2 * i / rot) for i in range(rot // 2)])
    keep = [keep_by_turns(f, 4096, 1, 4) for f in plain]
    assert 0 in keep and (1 in keep or rot == 16)
    close(made(kind="by_turns", stretch=8.0, original=4096.0, lo=1.0, hi=4.0),
          [f * (w + (1 - w) / 8) for f, w in zip(plain, keep)])
    index = lambda n: rot / 2 * math.log(4096 / (2 * math.pi * n)) / math.log(base)  # noqa: E731
    a, b = math.floor(index(32)), math.ceil(index(1))
    keep = [min(max(1 - (i - a) / (b - a), 0), 1) for i in range(rot // 2)]
    close(made(kind="by_index", stretch=8.0, original=4096.0, lo=1.0, hi=32.0),
          [f * (w + (1 - w) / 8) for f, w in zip(plain, keep)])


@pytest.mark.parametrize("kw,want", [
    (dict(base=1.0), INVALID), (dict(base=math.nan), INVALID), (dict(base=math.inf), INVALID),
    (dict(rot=15), INVALID), (dict(rot=0), INVALID), (dict(rot=130), UNSUPPORTED),
    (dict(kind=5), INVALID), (dict(kind=-1), INVALID), (dict(kind=1, stretch=0.5), INVALID),
    (dict(kind=1, stretch=math.nan), INVALID), (dict(kind=2, rot=2), INVALID),
    (dict(kind=2, base=1e300, stretch=1e300, rot=4), INVALID),
    (dict(kind=3, lo=0.0), INVALID), (dict(kind=3, lo=32.0), INVALID),
    (dict(kind=4, hi=math.inf), INVALID), (dict(kind=4, original=0.0), INVALID),
    (dict(kind=3, original=-5.0), INVALID), (dict(stretch=0.0, lo=9.0, hi=1.0), OK),
])
def test_rope_table_rejects(lib, kw, want):
    args = dict(base=1e4, rot=64, kind=0, stretch=2.0, original=8192.0, lo=1.0, hi=32.0) | kw
    out = (ctypes.c_uint64 * 64)(*[7] * 64)
    assert lib.idx_rope_table(*args.values(), out) == want
    assert want == OK or list(out) == [7] * 64
    assert lib.idx_rope_table(*args.values(), None) == INVALID


def test_binding_checks_without_a_gpu():
    t = torch.zeros(1, dtype=torch.int32)
    c, v = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 128, 8, dtype=torch.uint8)
    ks, vs = torch.zeros(2, 1, 16, 4, dtype=torch.uint8), torch.zeros(2, 1, 4, 16, dtype=torch.uint8)
    x = torch.zeros(1, 1, 128)
    q = x.bfloat16()
    for call in (lambda: idx.idx_cache4_write(x, x, t, c, v, ks, vs),
                 lambda: idx.idx_cache4_read(t, c, v, ks, vs),
                 lambda: idx.idx_attend4(q, c, v, ks, vs, t, t, t, 4),
                 lambda: idx.idx_attend4_prefill(q, c, v, ks, vs, t, t, t, t, 4),
                 lambda: idx.idx_rope(q, q, t, torch.zeros(64, dtype=torch.int64))):
        with pytest.raises(ValueError, match="same GPU"):
            call()
    with pytest.raises(ValueError, match="kind"):
        idx.idx_rope_table(64, kind="other", device="cpu")
    with pytest.raises(ValueError, match="even"):
        idx.idx_rope_table(63, device="cpu")
