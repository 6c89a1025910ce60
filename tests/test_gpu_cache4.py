"""The paged 4-bit cache on the GPU against its CPU oracle: writes and reads exactly,
attention within bounds derived from its arithmetic (tests/cache4_helpers.py)."""
import os
import re
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache4 as c4
from tests.cache4_helpers import Cache4, check_rows, tolerance
from tests.cache_helpers import queries

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


# ------------------------------------------------------------------- write and read

# tokens [start, stop) of each request
SPANS = {"one": [(0, 1)], "last of a page": [(15, 16), (31, 32), (63, 64)],
         "inside": [(3, 9), (17, 18), (0, 33)], "odd ends": [(5, 40), (64, 131), (1, 2), (30, 95)],
         "many": [(i % 37, i % 37 + 1 + i % 21) for i in range(60)],
         "long": [(7, 1500), (0, 901), (1023, 2100)]}


def write_case(seed, spans, Hkv, page, dtype):
    rng = np.random.default_rng(seed)
    c = Cache4(seed, [stop for _, stop in spans], Hkv, page)
    slots = []
    for b, (start, stop) in enumerate(spans):
        pages = c.pages(b)
        slots += [pages[t // page] * page + t % page for t in range(start, stop)]
    n = len(slots)
    x = rng.standard_normal((n, 2, Hkv, 128)) * np.exp2(rng.integers(-6, 7, (n, 2, Hkv, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return c, np.array(slots, np.int64), x


def state(c):
    return c.device()[:4]


def write_check(c, slots, x):
    """Writes rows x [n, 2, Hkv, 128]; the whole cache against the oracle's."""
    cache = state(c)
    y = x.cuda()
    idx.idx_cache4_write(y[:, 0], y[:, 1], i32(slots), *cache)
    k, v = x[:, 0].double().numpy(), x[:, 1].double().numpy()
    want = c4.cache_write(k, v, slots, c.k, c.v, c.ks, c.vs)
    got = [t.cpu().numpy() for t in cache]
    got[0], got[1] = c4.unpack(got[0]), c4.unpack(got[1])
    # (codes of blocks that hold a NaN say nothing)
    for i in (0, 1):
        nan = np.repeat(want[i + 2] == 255, 32, 3 - i)
        bad = (got[i] != want[i]) & ~nan
        assert not bad.any(), ("k", "v")[i] + str(np.argwhere(bad)[0])
        np.testing.assert_array_equal(got[i + 2], want[i + 2])
    return cache, want


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spans", list(SPANS))
def test_write_and_read_back(spans, dtype, page):
    say(f"[write4] {spans} {dtype} page={page}")
    for Hkv in ((1, 3) if spans != "long" else (2,)):
        c, slots, x = write_case(len(spans), SPANS[spans], Hkv, page, dtype)
        cache, want = write_check(c, slots, x)
        k, v = c4.cache_read(slots, *want)
        for out in (dtype, torch.float32):
            ko, vo = idx.idx_cache4_read(i32(slots), *cache, dtype=out)
            assert ko.dtype is vo.dtype is out
            np.testing.assert_array_equal(ko.double().cpu().numpy(), k)
            np.testing.assert_array_equal(vo.double().cpu().numpy(), v)


def test_write_many_rows_takes_the_long_calls_path():
    c, slots, x = write_case(8, [(3, 2500), (0, 1811), (77, 900)], 4, 16, torch.bfloat16)
    assert len(slots) * 2 > 8192
    write_check(c, slots, x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_special_values(dtype):
    """Infinities, NaN, zeros, the smallest and largest values; each block on its own."""
    c, slots, x = write_case(11, [(0, 20), (5, 9)], 2, 16, dtype)
    x[0, 0, 0, :32] = 0
    x[0, 0, 0, 40] = torch.inf
    x[0, 1, 0, 70] = -torch.inf
    x[1, 0, 1, 3] = torch.nan
    x[1, 1, 1, 127] = -torch.nan
    x[2, :, 0] = 2.0 ** -126
    x[2, :, 1] = 2.0 ** 127
    x[3, 0, 0, 5] = 2.0 ** -140
    x[4, 1, 0] = -0.0
    x[5, 0, 0, 64:96] = 6 * 2.0 ** 60
    x[5, 0, 0, 96:] = 6.25 * 2.0 ** 60
    x[6, 0, 1, :32] = 6 * 2.0 ** -60
    x[6, 0, 1, 32:64] = 0.25 * 2.0 ** -60
    write_check(c, slots, x)


def test_codes_round_to_the_nearest():
    """Every boundary between codes and its neighbours, at several scales."""
    edges = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    x = np.concatenate([edges, np.nextafter(edges, np.float32(0)),
                        np.nextafter(edges, np.float32(9)), [0, 0.1, 0.5, 1, 3, 4, 5.5, 4.5]])
    x = np.where(x > 6, 6, x).astype(np.float32)
    rows = np.stack([np.concatenate([x * s, -x * s, x[::-1] * s, x * s])
                     for s in np.exp2(np.arange(-59, 60, 7)).astype(np.float32)])
    n = len(rows)
    c = Cache4(3, [n], 1, 32)
    slots = np.array([c.pages(0)[t // 32] * 32 + t % 32 for t in range(n)])
    write_check(c, slots, torch.from_numpy(np.stack([rows, -rows], 1))[:, :, None])


def test_write_skips_and_no_tokens():
    c, slots, x = write_case(12, [(0, 30), (3, 8)], 2, 16, torch.bfloat16)
    slots[[0, 7, 8, 31]] = [-1, c.n_pages * 16, 2 ** 31 - 1, -5]
    # (a run that begins behind a skipped row, inside a byte)
    write_check(c, slots, x)
    write_check(c, slots[:0], x[:0])


@pytest.mark.parametrize("order", ["reversed", "shuffled", "odd first"])
def test_write_slots_in_any_order(order):
    """Tokens that share a byte, in rows far apart."""
    c, slots, x = write_case(21, [(3, 1700), (0, 900)], 2, 16, torch.bfloat16)
    n = len(slots)
    at = {"reversed": np.arange(n)[::-1], "shuffled": np.random.default_rng(1).permutation(n),
          "odd first": np.concatenate([np.arange(1, n, 2), np.arange(0, n, 2)])}[order]
    write_check(c, slots[at], x[torch.from_numpy(at.copy())])
    write_check(c, slots[at][:500], x[torch.from_numpy(at[:500].copy())])


def test_a_token_at_a_time_is_the_same_as_all_at_once():
    c, slots, x = write_case(13, [(0, 37)], 2, 32, torch.float32)
    cache, _ = write_check(c, slots, x)
    one = state(c)
    y = x.cuda()
    for t, s in enumerate(slots):
        idx.idx_cache4_write(y[t:t + 1, 0], y[t:t + 1, 1], i32([s]), *one)
    assert all(torch.equal(a, b) for a, b in zip(one, cache))


def test_read_any_order_repeats_and_unknown_slots():
    c = Cache4(14, [200, 31], 3, 32)
    rng = np.random.default_rng(1)
    slots = np.concatenate([rng.integers(0, c.n_pages * 32, 500), [-1, 5, 5, 6, 7, 5],
                            [c.n_pages * 32, 2 ** 31 - 1, -2 ** 31], np.arange(60)[::-1]])
    k, v = c4.cache_read(slots, c.k, c.v, c.ks, c.vs)
    for dtype in (torch.bfloat16, torch.float32):
        n = len(slots)
        y = torch.full((n, 2, 4, 128), 3.0, dtype=dtype, device="cuda")
        ko, vo = y[:, 0, :3], y[:, 1, :3]   # rows that lie apart
        idx.idx_cache4_read(i32(slots), *state(c), k_out=ko, v_out=vo)
        with np.errstate(over="ignore"):
            for got, want in ((ko, k), (vo, v)):
                got = got.double().cpu().numpy()
                big = np.abs(want) > 2.0 ** 126  # poisoned pages' scales: 2^127 and NaN
                np.testing.assert_array_equal(got[~big], want[~big])
        assert (y[:, :, 3] == 3.0).all()


def test_read_one_side():
    """Keys alone, or values alone: the other pointer is NULL."""
    c = Cache4(28, [100], 2, 16)
    slots = i32(np.concatenate([np.arange(100) % 60, [-1]]))
    kc, vc, ks, vs = state(c)
    k, v = idx.idx_cache4_read(slots, kc, vc, ks, vs, dtype=torch.float32)
    lib = idx.load()
    for side, want in ((0, k), (1, v)):
        out = torch.full_like(want, 5.0)
        ptr = [None, None]
        ptr[side] = out.data_ptr()
        assert lib.idx_cache4_read(slots.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks.data_ptr(),
                                   vs.data_ptr(), *ptr, 256, 256, slots.numel(), 2, 128,
                                   c.n_pages, 16, 0, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


def test_calls_past_4gib():
    """Pages behind the first 4 GiB of each cache: a small pool would hide an offset of 32
    bits."""
    Hkv, page = 8, 64
    n_pages = (1 << 32) // (Hkv * page * 64) + 40
    kc = torch.zeros(n_pages, Hkv, page, 64, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(n_pages, Hkv, 128, page // 2, dtype=torch.uint8, device="cuda")
    ks = torch.full((n_pages, Hkv, page, 4), 127, dtype=torch.uint8, device="cuda")
    vs = torch.full((n_pages, Hkv, 4, page), 127, dtype=torch.uint8, device="cuda")
    pages = np.array([n_pages - 1, 0, n_pages - 2, n_pages // 2])
    slots = (pages[:, None] * page + np.arange(page)).reshape(-1)[:230]
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((230, 2, Hkv, 128)).astype(np.float32)).cuda()
    idx.idx_cache4_write(x[:, 0], x[:, 1], i32(slots), kc, vc, ks, vs)
    ko, vo = idx.idx_cache4_read(i32(slots), kc, vc, ks, vs, dtype=torch.float32)
    small = Cache4(1, [230], Hkv, page, spare=0)
    small.indices = np.arange(4, dtype=np.int32)
    small.k, small.v, small.ks, small.vs = c4.cache_write(
        x[:, 0].double().cpu().numpy(), x[:, 1].double().cpu().numpy(), np.arange(230),
        small.k, small.v, small.ks, small.vs)
    k, v = c4.cache_read(np.arange(230), small.k, small.v, small.ks, small.vs)
    np.testing.assert_array_equal(ko.double().cpu().numpy(), k)
    np.testing.assert_array_equal(vo.double().cpu().numpy(), v)
    q, q64 = queries(rng, 1, Hkv)
    args = (kc, vc, ks, vs, i32([0, 4]), i32(pages))
    out = idx.idx_attend4(q.cuda(), *args, i32([230]), 4)
    check_rows(out, small, q64, [0], [230])
    out = idx.idx_attend4_prefill(q.cuda(), *args, i32([0, 1]), i32([230]), 4)
    check_rows(out, small, q64, [0], [230])


# ------------------------------------------------------------------- single tokens

HEADS = [(1, 1), (4, 1), (8, 8), (6, 2), (16, 1), (20, 1), (32, 1), (33, 1), (64, 1)]


def attend_case(seed, lens, Hq, Hkv, page, scale=128 ** -0.5, cap=0.0, biased=False, rows=None,
                **kw):
    c = Cache4(seed, lens, Hkv, page, **kw)
    q, q64 = queries(c.rng, len(lens), Hq)
    slopes = np.exp2(-8 * np.arange(1, Hq + 1) / Hq).astype(np.float32) if biased else None
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(lens), c.max_pages, scale=scale, softcap=cap,
                          slopes=None if slopes is None else dev(slopes))
    worst = check_rows(out, c, q64, range(len(lens)), lens, None, scale, cap, slopes, rows)
    say(f"[attend4] {Hq}/{Hkv} page={page} cap={cap} biased={biased}: {worst:.2f} of the bound")
    return c, out


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64])
def test_attend_lengths(Hq, Hkv, page):
    attend_case(Hq + page, [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 500], Hq, Hkv, page)


@pytest.mark.parametrize("cap,biased", [(30.0, False), (0.0, True), (5.0, True), (500.0, False)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (40, 2), (33, 1)])
def test_attend_softcap_and_slopes(Hq, Hkv, cap, biased):
    attend_case(3, [1, 40, 333, 64], Hq, Hkv, 16, cap=cap, biased=biased)


@pytest.mark.parametrize("scale,cap", [(-0.2, 0.0), (-0.2, 4.0), (0.0, 0.0), (3.0, 0.0)])
def test_attend_call_scales_of_any_sign_and_size(scale, cap):
    attend_case(4, [5, 77, 300], 8, 2, 16, scale=scale, cap=cap)


def test_attend_rows_that_see_nothing_or_less_than_they_hold():
    c = Cache4(5, [100, 64, 30, 7], 2, 16)
    q, q64 = queries(c.rng, 4, 8)
    for seen in ([0, 64, 3, -5], [99, 1, 0, 2 ** 31 - 1], [16, 48, 17, 7]):
        # lengths past the list end with it; what its last page holds behind is the row's own
        seen_of = np.minimum(seen, [112, 64, 32, 16])
        if seen_of[3] == 16:
            c.ks[c.pages(3)[0], :, 7:], c.vs[c.pages(3)[0], :, :, 7:] = 126, 126
        out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages)
        check_rows(out, c, q64, range(4), seen_of)


def test_attend_more_rows_than_requests_and_unknown_requests():
    c = Cache4(6, [40, 90], 2, 32)
    req = [0, 1, 1, -1, 2, 0, 2 ** 31 - 1, 1]
    q, q64 = queries(c.rng, len(req), 4)
    seen = [40, 90, 13, 5, 5, 1, 9, 64]
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, row_req=i32(req))
    check_rows(out, c, q64, req, seen)


def test_attend_bad_pages_and_short_lists():
    c = Cache4(7, [100, 100, 50], 2, 16)
    q, q64 = queries(c.rng, 3, 4)
    c.indices[2], c.indices[9] = -1, c.n_pages        # pages that are not there
    c.indices[4] = 2 ** 31 - 1
    out = idx.idx_attend4(q.cuda(), *c.device(), i32([100, 100, 50]), c.max_pages)
    check_rows(out, c, q64, range(3), [100, 100, 50])
    c.indices = c.indices[:-3]                        # a list that ends before its pointer
    out = idx.idx_attend4(q.cuda(), *c.device(), i32([100, 100, 50]), c.max_pages)
    check_rows(out, c, q64, range(3), [100, 100, 50])
    c.max_pages = 3                                   # no more pages than the bound
    out = idx.idx_attend4(q.cuda(), *c.device(), i32([100, 100, 50]), c.max_pages)
    check_rows(out, c, q64, range(3), [48, 48, 48])
    kc, vc, ks, vs, indptr, indices = c.device()
    for bad in ([0, -7, 2 ** 31 - 1, 5], [20, 10, 5, 0]):  # nothing is read out of range
        idx.idx_attend4(q.cuda(), kc, vc, ks, vs, i32(bad), indices, i32([100, 100, 50]), 8)
    torch.cuda.synchronize()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("K", [1, 3, 17, 130])
def test_attend_selected_pages(K, page):
    lens = [1, page, 5 * page + 3, 150 * page, 150 * page - 9]
    c = Cache4(K + page, lens, 2, page)
    q, q64 = queries(c.rng, len(lens), 12)
    ids = np.full((len(lens), K), -1, np.int32)
    for r, n in enumerate(lens):
        nb = -(-n // page)
        pick = np.sort(c.rng.permutation(nb)[:K])
        ids[r, :len(pick)] = pick
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(lens), c.max_pages, ids=dev(ids))
    check_rows(out, c, q64, range(len(lens)), lens, ids)


def test_attend_selected_pages_repeated_unknown_and_none():
    c = Cache4(9, [500, 500, 500], 1, 16)
    q, q64 = queries(c.rng, 3, 4)
    ids = np.array([[3, 3, 3, 7], [-1, 2 ** 31 - 1, 40, -9], [31, 0, 30, 31]], np.int32)
    seen = [500, 500, 487]
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, ids=dev(ids))
    check_rows(out, c, q64, range(3), seen, ids)
    assert not out[1].any()
    none = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages,
                           ids=torch.empty(3, 0, dtype=torch.int32, device="cuda"))
    assert not none.any()


@pytest.mark.parametrize("B,n", [(1, 40000), (2, 9001), (3, 131072)])
def test_attend_long_rows_over_several_workgroups(B, n):
    attend_case(B, [n - 777 * b for b in range(B)], 4, 1, 16, rows=[0] if n > 50000 else None)


def test_attend_uncut_rows_over_several_phases():
    """More tiles than a workgroup lists at once, in rows that are not cut."""
    c = Cache4(25, [20000], 1, 16)
    R = 512
    q, q64 = queries(c.rng, R, 2)
    seen = np.full(R, 20000)
    seen[1::2] = c.rng.integers(16000, 20001, R // 2)
    assert idx.idx_attend4_workspace_bytes(R, 2, 1, c.max_pages) == 0
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, row_req=i32(np.zeros(R)))
    check_rows(out, c, q64, np.zeros(R), seen, rows=[0, 1, 2, 3, 200, 511])


def test_prefill_uncut_prompts_over_several_phases():
    c = Cache4(26, [40000], 2, 16)
    n, Hq = 2048, 64
    q, q64 = queries(c.rng, n, Hq)
    seen = np.arange(40000 - n, 40000) + 1
    assert idx.idx_attend4_prefill_workspace_bytes(n, 1, Hq, 2, c.max_pages) == 0
    c.vs[c.pages(0)[2100], 1, 3, 7] = 255           # in the second phase
    out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([0, n]), i32(seen), c.max_pages)
    assert torch.isnan(out[:, 32:, 96:]).all() and torch.isfinite(out[:, :, :96]).all()
    assert torch.isfinite(out[:, :32]).all()
    keep = out[:, [0, 40]].clone()                  # two heads of the two groups
    check_rows(keep, c, q64[:, [0, 40]], np.zeros(n), seen, rows=[0, 1, 777, n - 1])


def test_attend_nan_scales_of_seen_tokens():
    """A key's NaN reaches the rows that see it; a value's its 32 dims of those rows, the
    others keep their bits."""
    for Hq in (4, 20):
        c = Cache4(10, [100, 100, 100, 64], 1, 16)
        q, q64 = queries(c.rng, 4, Hq)
        clean = idx.idx_attend4(q.cuda(), *c.device(), i32([100, 100, 100, 64]), c.max_pages)
        c.ks[c.pages(0)[3], 0, 5, 2] = 255
        c.vs[c.pages(1)[0], 0, 1, 9] = 255
        c.vs[c.pages(3)[3], 0, 3, 15] = 255
        out = idx.idx_attend4(q.cuda(), *c.device(), i32([100, 100, 100, 64]), c.max_pages)
        check_rows(out, c, q64, range(4), [100, 100, 100, 64])
        assert torch.isnan(out[0]).all() and torch.isnan(out[1, :, 32:64]).all()
        rest = [i for i in range(128) if not 32 <= i < 64]
        assert torch.equal(out[1][:, rest], clean[1][:, rest])
        assert torch.equal(out[2], clean[2])
        # not seen: 99 tokens of the first, and the token before
        out = idx.idx_attend4(q.cuda(), *c.device(), i32([53, 9, 100, 63]), c.max_pages)
        check_rows(out, c, q64, range(4), [53, 9, 100, 63])
        assert torch.isfinite(out).all()


def test_attend_value_scales_far_apart():
    """Token by token: large values without weight cost the others no bits. Within a unit,
    2^24 is kept."""
    c = Cache4(15, [900, 900], 1, 16)
    q, q64 = queries(c.rng, 2, 8)
    for b, grow in ((0, 1), (1, -1)):  # scales that grow, or fall, along the row
        for i, p in enumerate(c.pages(b)):
            c.vs[p] = np.clip(127 + grow * (2 * i - 56) + c.rng.integers(-7, 8, (1, 4, 16)), 67, 187)
    c.poison_tails()
    out = idx.idx_attend4(q.cuda(), *c.device(), i32([900, 900]), c.max_pages)
    check_rows(out, c, q64, range(2), [900, 900])
    # one token far above all others, whose score is far below theirs
    c = Cache4(16, [300], 1, 16)
    q = torch.ones(1, 4, 128).bfloat16()
    p, o = c.pages(0)[7], 3
    c.k[p, 0, o], c.ks[p, 0, o] = 15, 127   # key -6 everywhere
    c.vs[p, 0, :, o] = 127 + 9
    out = idx.idx_attend4(q.cuda(), *c.device(), i32([300]), c.max_pages)
    check_rows(out, c, q.double().numpy(), [0], [300])


def test_value_scales_far_apart_within_a_unit():
    """Blocks of dims, and tokens, whose scales lie up to 2^24 apart among 16 tokens."""
    for lens, news in (([900, 333], [1, 1]), ([900, 333], [9, 7]), ([900, 333], [200, 333])):
        c = Cache4(22, lens, 2, 16)
        c.vs[:] = 127 - c.rng.integers(0, 25, c.vs.shape)
        c.vs[:, :, 2] = 127 - 20 - c.rng.integers(0, 5, c.vs[:, :, 2].shape)  # a small block
        c.vs[:, :, 0, 0] = 127
        c.poison_tails()
        ptr, req = np.concatenate([[0], np.cumsum(news)]), np.repeat([0, 1], news)
        seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
        q, q64 = queries(c.rng, len(req), 8)
        out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), c.max_pages)
        check_rows(out, c, q64, req, seen, rows=range(0, len(req), 1 + len(req) // 40))
        out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, row_req=i32(req))
        check_rows(out, c, q64, req, seen, rows=range(0, len(req), 1 + len(req) // 40))


def test_attend_least_and_largest_scales():
    for e in (-60, 60):
        c = Cache4(17, [70, 33], 1, 16)
        c.vs[:] = 127 + e
        c.poison_tails()
        q, q64 = queries(c.rng, 2, 4)
        out = idx.idx_attend4(q.cuda(), *c.device(), i32([70, 33]), c.max_pages)
        check_rows(out, c, q64, range(2), [70, 33])
    c = Cache4(18, [70, 33], 1, 16)
    c.ks[:] = 127 - 60
    q = queries(c.rng, 2, 4)[0].double() * 2.0 ** 60
    out = idx.idx_attend4(q.bfloat16().cuda(), *c.device(), i32([70, 33]), c.max_pages)
    c.poison_tails()
    check_rows(out, c, q.numpy(), range(2), [70, 33])


def test_attend_strided_queries_given_output_and_none():
    c = Cache4(19, [50, 80], 2, 16)
    q, q64 = queries(c.rng, 2, 8)
    wide = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = q.cuda()
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    got = idx.idx_attend4(wide[:, 1], *c.device(), i32([50, 80]), c.max_pages, out=out)
    assert got is out
    check_rows(out, c, q64, range(2), [50, 80])
    empty = idx.idx_attend4(q.cuda()[:0], *c.device(), i32([]), c.max_pages)
    assert empty.shape == (0, 8, 128)


# ------------------------------------------------------------------- packed tokens

def prefill_case(seed, lens, news, Hq, Hkv, page, cap=0.0, biased=False, seen=None, rows=None,
                 scale=128 ** -0.5):
    c = Cache4(seed, lens, Hkv, page)
    req = np.repeat(np.arange(len(lens)), news)
    ptr = np.concatenate([[0], np.cumsum(news)])
    if seen is None:
        seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
    q, q64 = queries(c.rng, len(req), Hq)
    slopes = np.exp2(-8 * np.arange(1, Hq + 1) / Hq).astype(np.float32) if biased else None
    out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), c.max_pages,
                                  scale=scale, softcap=cap,
                                  slopes=None if slopes is None else dev(slopes))
    worst = check_rows(out, c, q64, req, seen, None, scale, cap, slopes, rows)
    say(f"[prefill4] {lens} {news} {Hq}/{Hkv} page={page}: {worst:.2f} of the bound")
    return c, out


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_prefill_ragged(Hq, Hkv, page):
    prefill_case(Hq + page, [3, 70, 200, 16, 129], [3, 1, 37, 16, 5], Hq, Hkv, page)


@pytest.mark.parametrize("n", [1, 2, 31, 33, 127, 129, 400])
def test_prefill_whole_prompts(n):
    prefill_case(n, [n, max(1, n // 3)], [n, max(1, n // 3)], 8, 2, 16)


@pytest.mark.parametrize("cap,biased", [(30.0, False), (0.0, True), (5.0, True), (500.0, False)])
@pytest.mark.parametrize("lens,news", [([90, 300], [4, 6]), ([90, 300], [90, 150])])
def test_prefill_softcap_and_slopes(lens, news, cap, biased):
    prefill_case(5, lens, news, 8, 2, 16, cap=cap, biased=biased)


@pytest.mark.parametrize("scale,cap", [(-0.2, 0.0), (-0.2, 4.0), (0.0, 0.0), (3.0, 0.0)])
def test_prefill_call_scales(scale, cap):
    prefill_case(6, [300], [130], 4, 2, 16, cap=cap, scale=scale)


def test_prefill_any_lengths_and_empty_rows():
    rng = np.random.default_rng(7)
    for lens, news in (([200, 90], [150, 80]), ([200, 90], [6, 9])):
        seen = np.concatenate([rng.integers(-2, n + 1, k) for n, k in zip(lens, news)])
        seen[:3] = [0, -5, 64]
        prefill_case(8, lens, news, 8, 2, 16, seen=seen)


@pytest.mark.parametrize("lens,news", [([300], [300]), ([6000], [130])])
def test_prefill_empty_rows_beside_nan_scales(lens, news):
    """Rows that see nothing are zero whatever the tiles of the others hold, cut or not."""
    c = Cache4(27, lens, 2, 16)
    n = news[0]
    seen = np.arange(lens[0] - n, lens[0]) + 1
    seen[::7], seen[3] = 0, -4
    c.vs[c.pages(0)[0], 1, 2, 3] = 255
    q, q64 = queries(c.rng, n, 8)
    out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([0, n]), i32(seen), c.max_pages)
    check_rows(out, c, q64, np.zeros(n), seen, rows=range(0, n, 3))
    assert not out[::7].any() and not out[3].any()
    assert torch.isnan(out[torch.from_numpy(seen > 3).cuda()][:, 4:, 64:96]).all()


def test_prefill_leaves_other_rows_as_they_were():
    c = Cache4(9, [40, 60], 2, 16)
    for n, ptr in ((20, [3, 8, 15]), (200, [3, 88, 150])):
        q, q64 = queries(c.rng, n, 4)
        out = torch.full((n, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        seen = c.rng.integers(1, 41, n)
        idx.idx_attend4_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), c.max_pages, out=out)
        req = np.where(np.arange(n) < ptr[1], 0, 1)
        check_rows(out, c, q64, req, seen, rows=range(ptr[0], ptr[2]))
        assert (out[:ptr[0]] == 5).all() and (out[ptr[2]:] == 5).all()


@pytest.mark.parametrize("lens,news", [([20000], [1]), ([9000, 30], [7, 2]), ([5000], [130])])
def test_prefill_long_contexts_over_several_workgroups(lens, news):
    prefill_case(10, lens, news, 4, 1, 16, rows=[0, 1, sum(news) - 1][:sum(news)])


def test_prefill_bad_pages_and_pointers():
    for news in ([5, 4], [70, 60]):
        c = Cache4(11, [100, 100], 2, 16)
        c.indices[2], c.indices[9] = -1, c.n_pages
        n = sum(news)
        q, q64 = queries(c.rng, n, 4)
        seen = np.concatenate([np.arange(100 - k, 100) + 1 for k in news])
        ptr = np.concatenate([[0], np.cumsum(news)])
        out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), c.max_pages)
        check_rows(out, c, q64, np.repeat([0, 1], news), seen)
        idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([-5, 2, 2 ** 31 - 1]), i32(seen),
                                c.max_pages)
        torch.cuda.synchronize()


def nan_cases():
    return [([300, 77], [7, 5]), ([300, 77], [300, 60]), ([6000], [130])]


@pytest.mark.parametrize("lens,news", nan_cases())
def test_prefill_nan_scales_reach_only_the_rows_that_see_them(lens, news):
    Hq, Hkv = 4, 2
    c = Cache4(12, lens, Hkv, 16)
    req = np.repeat(np.arange(len(lens)), news)
    ptr = np.concatenate([[0], np.cumsum(news)])
    seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
    q, q64 = queries(c.rng, len(req), Hq)
    call = lambda: idx.idx_attend4_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), c.max_pages)  # noqa: E731
    clean = call()
    b = 0
    at = lens[b] - 2                                 # all but one of its rows do not see it
    page, o = c.pages(b)[at // 16], at % 16
    c.vs[page, 0, 2, o] = 255
    c.ks[page, 1, o, 1] = 255
    out = call()
    sees = torch.from_numpy((req == b) & (seen > at)).cuda()
    assert int(sees.sum()) == min(2, news[0])
    assert torch.isnan(out[sees][:, :2, 64:96]).all() and torch.isnan(out[sees][:, 2:]).all()
    rest = [i for i in range(128) if not 64 <= i < 96]
    assert torch.equal(out[sees][:, :2][:, :, rest], clean[sees][:, :2][:, :, rest])
    assert torch.equal(out[~sees], clean[~sees])


@pytest.mark.parametrize("lens,news", nan_cases())
@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0)])
def test_no_bit_of_a_row_comes_from_tokens_that_it_does_not_see(lens, news, kw):
    Hq, Hkv = 8, 2
    c = Cache4(13, lens, Hkv, 16)
    ptr = np.concatenate([[0], np.cumsum(news)])
    req = np.repeat(np.arange(len(lens)), news)
    seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
    cut = np.array([n - k // 2 for n, k in zip(lens, news)])
    first = np.arange(len(req)) % 2 == 0
    seen = np.where(first, np.minimum(seen, cut[req]), seen)
    q, _ = queries(c.rng, len(req), Hq)
    call = lambda: idx.idx_attend4_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen),  # noqa: E731
                                           c.max_pages, **kw)
    before = call()
    for b in range(len(lens)):
        for i, p in enumerate(c.pages(b)):
            o = max(int(cut[b]) - 16 * i, 0)
            if o < 16:
                c.k[p, :, o:], c.v[p, :, :, o:] = 13, 6
                c.ks[p, :, o:] = c.rng.integers(100, 150, c.ks[p, :, o:].shape)
                c.vs[p, :, :, o:] = c.rng.integers(67, 188, c.vs[p, :, :, o:].shape)
    after = call()
    own = torch.from_numpy(seen <= cut[req]).cuda()
    assert torch.equal(before[own], after[own])
    assert not torch.equal(before[~own], after[~own])


def test_rows_and_prompt_tokens_agree():
    c = Cache4(20, [90, 700], 2, 16)
    q, q64 = queries(c.rng, 2, 16)
    seen = [90, 700]
    a = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages)
    b = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([0, 1, 2]), i32(seen), c.max_pages)
    check_rows(a, c, q64, range(2), seen)
    check_rows(b, c, q64, range(2), seen)


def test_bounds_far_above_the_lists():
    c = Cache4(21, [100, 5], 1, 16)
    q, q64 = queries(c.rng, 2, 4)
    for bound in (c.max_pages, 1000, 1 << 20):
        c.max_pages = bound
        out = idx.idx_attend4(q.cuda(), *c.device(), i32([100, 5]), bound)
        check_rows(out, c, q64, range(2), [100, 5])
        out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([0, 1, 2]), i32([100, 5]), bound)
        check_rows(out, c, q64, range(2), [100, 5])


# ------------------------------------------------------------------- as they are used

class Step:
    """A serving loop over the 4-bit cache: tables, rotary positions, write, attention."""

    def __init__(self, B=3, Hq=8, Hkv=2, page=16, max_pages=12, seed=30):
        self.rng = np.random.default_rng(seed)
        self.B, self.Hq, self.Hkv, self.page, self.max_pages = B, Hq, Hkv, page, max_pages
        n_pages = B * max_pages
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.cache = (torch.randint(0, 256, (n_pages, Hkv, page, 64), **u8),
                      torch.randint(0, 256, (n_pages, Hkv, 128, page // 2), **u8),
                      torch.full((n_pages, Hkv, page, 4), 255, **u8),
                      torch.full((n_pages, Hkv, 4, page), 255, **u8))
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.ring, self.cursor = i32(np.arange(n_pages)), i32([0, n_pages, 0])
        self.seq = i32(np.zeros(B))
        self.turns = idx.idx_rope_table(64)
        self.k = [np.zeros((0, Hkv, 128)) for _ in range(B)]  # what the requests hold
        self.v = [np.zeros((0, Hkv, 128)) for _ in range(B)]

    def rows(self, n):
        x = self.rng.standard_normal((n, self.Hq + 2 * self.Hkv, 128)).astype(np.float32)
        return torch.from_numpy(x).bfloat16()

    def calls(self, x, new, n_tokens, packed):
        """The step's device work on rows x; returns its tables and the attention."""
        t = idx.idx_page_tables(self.seq, new, self.table, self.ring, self.cursor, n_tokens,
                                page_size=self.page)
        q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
        q, k = idx.idx_rope(q, k, t.tok_len, self.turns, first=64, q_out=q, k_out=k)
        idx.idx_cache4_write(k, v, t.slots, *self.cache)
        args = (q, *self.cache, t.kv_indptr, t.kv_indices)
        if packed:
            out = idx.idx_attend4_prefill(*args, t.tok_indptr, t.tok_len, self.max_pages)
        else:
            out = idx.idx_attend4(*args, t.tok_len, self.max_pages, row_req=t.tok_req)
        return t, out


def quantised(rows):
    """Rows [..., 128] as the values that the cache keeps of them."""
    out = np.zeros_like(rows)
    for i in np.ndindex(rows.shape[:-1]):
        codes, scales = c4.quantise(rows[i])
        out[i] = c4.e2m1_values()[codes] * np.repeat(c4.power(scales), 32)
    return out


def attention64(q, k, v):
    x = k @ q * 128 ** -0.5
    p = np.exp(x - x.max())
    return p / p.sum() @ v, p / p.sum() @ np.abs(v), np.abs(k) @ np.abs(q) * 128 ** -0.5


def test_serving_steps():
    """Prompts, single tokens and drafts taken back: each step's attention against one over
    the requests' own rows, turned and quantised by the oracle."""
    s = Step()
    turns = [t % 2 ** 64 for t in s.turns.cpu().tolist()]
    for step, new in enumerate([[40, 3, 0], [1, 1, 17], [5, 5, 5], [-3, -5, 1], [1, 1, 1],
                                [0, 33, 1], [-38, 1, 2], [1, 1, 1]]):
        n = int(np.maximum(new, 0).sum())
        x = s.rows(n)
        y = x.cuda()
        packed = max(new) > 1
        t, out = s.calls(y, i32(new), n, packed)
        s.seq, s.cursor = t.seq_len, t.cursor
        at = 0
        for b, d in enumerate(new):
            if d < 0:
                s.k[b], s.v[b] = s.k[b][:d], s.v[b][:d]
            rows = slice(at, at + max(d, 0))
            have = len(s.k[b])
            # the rotation's own result is taken for the cache's input (it is rounded to bf16)
            turned = c4.turned(x[rows].double().numpy(), have + np.arange(max(d, 0)), turns, 64,
                               False, False, 1.0)
            got = y[rows].double().cpu().numpy()
            np.testing.assert_allclose(got[:, :s.Hq + s.Hkv], turned[:, :s.Hq + s.Hkv], atol=0.05)
            held = quantised(got[:, s.Hq:]).reshape(-1, 2, s.Hkv, 128)
            s.k[b] = np.concatenate([s.k[b], held[:, 0]])
            s.v[b] = np.concatenate([s.v[b], held[:, 1]])
            for i in range(max(d, 0)):
                for hq in range(s.Hq):
                    h = hq // (s.Hq // s.Hkv)
                    seen = have + i + 1
                    want, absum, mag = attention64(got[i, hq], s.k[b][:seen, h], s.v[b][:seen, h])
                    tol = tolerance(want, absum, mag.max(), 4.0, seen)
                    err = np.abs(out[at + i, hq].double().cpu().numpy() - want)
                    assert (err <= tol).all(), (step, b, i, hq, float((err / tol).max()))
            at += max(d, 0)
        assert s.seq.cpu().tolist() == [len(k) for k in s.k]


def test_a_window_moves_on():
    """Keys read back, turned on by a shift and written to other pages are the keys of the
    new positions, but for one more quantisation; values stay as they are."""
    s = Step(B=1)
    turns = [t % 2 ** 64 for t in s.turns.cpu().tolist()]
    x = s.rows(40)
    t, _ = s.calls(x.cuda(), i32([40]), 40, True)
    k, v = idx.idx_cache4_read(t.slots, *s.cache, dtype=torch.float32)
    shift = i32(np.full(40, 12 + 1))
    moved, _ = idx.idx_rope(k, None, shift, s.turns, first=64, inverse=True)
    want = c4.turned(k.double().cpu().numpy(), np.full(40, 12), turns, 64, False, True, 1.0)
    np.testing.assert_allclose(moved.double().cpu().numpy(), want, atol=1e-5)
    to = i32([s.max_pages * 16 - 1 - i // 16 * 16 - (15 - i % 16) for i in range(40)])
    before = [c.clone() for c in s.cache]
    idx.idx_cache4_write(moved, v, to, *s.cache)
    k2, v2 = idx.idx_cache4_read(to, *s.cache, dtype=torch.float32)
    assert torch.equal(v2, v)
    want = quantised(moved.double().cpu().numpy())
    np.testing.assert_array_equal(k2.double().cpu().numpy(), want)
    back = idx.idx_cache4_read(t.slots, *s.cache, dtype=torch.float32)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)
    assert not all(torch.equal(a, b) for a, b in zip(before, s.cache))


@pytest.mark.parametrize("packed", [False, True])
def test_captured_steps_replay_as_the_eager_ones(packed):
    """One captured step, replayed on changing inputs, with eager work in between."""
    s = Step(B=2)
    x = s.rows(6)
    t, _ = s.calls(x.cuda(), i32([3, 3]), 6, True)   # eager: something to read
    s.seq.copy_(t.seq_len)
    s.cursor.copy_(t.cursor)
    new, n = i32([1, 1]), 2
    rows = s.rows(n).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        tg, out = s.calls(rows, new, n, packed)
        s.seq.copy_(tg.seq_len)
        s.cursor.copy_(tg.cursor)
    for step in range(4):
        fresh = s.rows(n).cuda()
        keep = [c.clone() for c in (*s.cache, s.table, s.ring, s.seq, s.cursor)]
        te, want = s.calls(fresh.clone(), new, n, packed)
        after = [c.clone() for c in s.cache]
        for a, b in zip((*s.cache, s.table, s.ring, s.seq, s.cursor), keep):
            a.copy_(b)
        rows.copy_(fresh)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
        assert all(torch.equal(a, b) for a, b in zip(s.cache, after))
        assert s.seq.cpu().tolist() == [4 + step, 4 + step]


def test_calls_on_two_streams_at_once():
    cases = []
    for seed in (40, 41):
        c = Cache4(seed, [5000, 300], 2, 16)
        q, _ = queries(c.rng, 2, 8)
        args = (q.cuda(), *c.device())
        kw = (i32([5000, 300]), c.max_pages)
        cases.append((args, kw, idx.idx_attend4(*args, *kw)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(5):
        for i, ((args, kw, _), st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                outs[i].append(idx.idx_attend4(*args, *kw))
    torch.cuda.synchronize()
    for (_, _, want), got in zip(cases, outs):
        assert all(torch.equal(want, o) for o in got)


def test_results_do_not_depend_on_the_run():
    c = Cache4(42, [30000, 77], 2, 16)
    q, _ = queries(c.rng, 2, 16)
    args = (q.cuda(), *c.device())
    a = [idx.idx_attend4(*args, i32([30000, 77]), c.max_pages) for _ in range(4)]
    assert all(torch.equal(a[0], x) for x in a)
    b = [idx.idx_attend4_prefill(*args, i32([0, 1, 2]), i32([30000, 77]), c.max_pages)
         for _ in range(4)]
    assert all(torch.equal(b[0], x) for x in b)


def test_typed_caches_and_binding_checks():
    c = Cache4(43, [20, 30], 2, 16)
    q, q64 = queries(c.rng, 2, 4)
    kc, vc, ks, vs, indptr, indices = c.device()
    n = i32([20, 30])
    want = idx.idx_attend4(q.cuda(), kc, vc, ks, vs, indptr, indices, n, 2)
    typed = (kc.view(torch.float4_e2m1fn_x2), vc.view(torch.float4_e2m1fn_x2),
             ks.view(torch.float8_e8m0fnu), vs.view(torch.float8_e8m0fnu))
    assert torch.equal(want, idx.idx_attend4(q.cuda(), *typed, indptr, indices, n, 2))
    x = torch.zeros(2, 2, 128, device="cuda")
    for bad in (lambda: idx.idx_attend4(q.cuda(), kc, vc.view(-1, 2, 64, 16), ks, vs, indptr,
                                        indices, n, 2),
                lambda: idx.idx_attend4(q.cuda(), kc, vc, vs, ks, indptr, indices, n, 2),
                lambda: idx.idx_attend4(q.cuda(), kc, vc, ks, vs, indptr, indices, n[:1], 2),
                lambda: idx.idx_attend4(q.cuda(), kc.transpose(0, 1), vc, ks, vs, indptr, indices,
                                        n, 2),
                lambda: idx.idx_cache4_write(x, x[:1], n, kc, vc, ks, vs),
                lambda: idx.idx_cache4_read(n, kc, vc, ks, vs, k_out=x[:1]),
                lambda: idx.idx_cache4_read(n, kc, vc, ks, vs, k_out=x, v_out=x.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: idx.idx_attend4(q.cuda(), kc.float(), vc, ks, vs, indptr, indices, n, 2),
                lambda: idx.idx_attend4(q.cuda().float(), kc, vc, ks, vs, indptr, indices, n, 2),
                lambda: idx.idx_attend4(q.cuda(), kc, vc, ks.float(), vs, indptr, indices, n, 2),
                lambda: idx.idx_cache4_read(n, kc, vc, ks, vs, dtype=torch.float16),
                lambda: idx.idx_cache4_write(x.half(), x.half(), n, kc, vc, ks, vs)):
        with pytest.raises(TypeError):
            bad()


def test_readme_lines_run():
    """The lines that README.md shows, as they stand, after a step of page tables."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                           "README.md")) as f:
        blocks = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S)
                  if "idx_cache4_write" in b]
    assert len(blocks) == 1
    B, Hq, Hkv, page, max_pages = 3, 8, 2, 16, 4
    n_pages = 2 * B * max_pages
    u8 = dict(dtype=torch.uint8, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    t = idx.idx_page_tables(i32([0] * B), i32([20, 7, 33]), table, i32(np.arange(n_pages)),
                            i32([0, n_pages]), 60, page_size=page)
    rows = torch.randn(60, Hq + 2 * Hkv, 128, device="cuda").bfloat16()
    kept = t.slots[:60] >= 0
    scope = dict(
        idx=idx, torch=torch, t=t, max_pages=max_pages, q=rows[:, :Hq], k=rows[:, Hq:Hq + Hkv],
        v=rows[:, Hq + Hkv:], gq=torch.randn(60, Hq, 128, device="cuda"),
        gk=torch.randn(60, Hkv, 128, device="cuda"),
        k_cache=torch.zeros(n_pages, Hkv, page, 64, **u8),
        v_cache=torch.zeros(n_pages, Hkv, 128, page // 2, **u8),
        k_scale=torch.zeros(n_pages, Hkv, page, 4, **u8),
        v_scale=torch.zeros(n_pages, Hkv, 4, page, **u8),
        slots=t.slots, shift_plus_1=i32(np.full(60, 6)),
        new_slots=torch.where(kept, t.slots + B * max_pages * page, -1))
    turned = idx.idx_rope(rows[:, :Hq].contiguous(), None, t.tok_len,
                          idx.idx_rope_table(128, base=5e5, kind="by_turns", stretch=8.0,
                                             original=8192.0, lo=1.0, hi=4.0))[0]
    exec(blocks[0], scope)
    assert torch.equal(rows[:, :Hq], torch.where(kept[:, None, None], turned, rows[:, :Hq]))
    back = idx.idx_cache4_read(scope["new_slots"], *scope["cache4"], dtype=torch.float32)
    first = idx.idx_cache4_read(t.slots, *scope["cache4"], dtype=torch.float32)
    assert torch.equal(back[1], first[1]) and not torch.equal(back[0], first[0])
    one = idx.idx_attend4(scope["q"], *scope["cache4"], t.kv_indptr, t.kv_indices, t.tok_len,
                          max_pages, row_req=t.tok_req)
    # (each side is within 2^-8 of its value, and what its sums add is far below 2^-8)
    off = (one[kept].float() - scope["out"][kept].float()).abs()
    assert float((off / (one[kept].float().abs() + 1)).max()) < 2.0 ** -6


def test_workspaces_may_hold_anything():
    """Chunks behind a row's end leave no sums: what the workspace held there does not reach
    the output, in either join (few items, many)."""
    for B, Hq in ((3, 8), (40, 64)):
        lens = [(500 + 997 * b) % 9000 for b in range(B)]
        c = Cache4(50, lens, 2, 16)
        q, _ = queries(c.rng, B, Hq)
        args = (q.cuda(), *c.device())
        bound = 3 * c.max_pages
        ptr, n = i32(np.arange(B + 1)), i32(lens)
        for call, size, rest in (
                (idx.idx_attend4, idx.idx_attend4_workspace_bytes(B, Hq, 2, bound), (n,)),
                (idx.idx_attend4_prefill,
                 idx.idx_attend4_prefill_workspace_bytes(B, B, Hq, 2, bound), (ptr, n))):
            assert size > 0
            outs = [call(*args, *rest, bound,
                         ws=torch.full((size,), fill, dtype=torch.uint8, device="cuda"))
                    for fill in (0, 255, 127)]
            assert torch.isfinite(outs[0]).all()
            assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
