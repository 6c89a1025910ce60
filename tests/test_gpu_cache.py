"""The paged 8-bit cache on the GPU against its CPU oracle: page tables and cache writes
exactly, attention within bounds derived from its arithmetic (tests/cache_helpers.py)."""
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

F8 = torch.float8_e4m3fn


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


# ------------------------------------------------------------------- page tables

def pool(rng, held, free, max_pages):
    """A table with held[b] pages per request and a ring with `free` free pages."""
    n_pages = sum(held) + free
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(held), max_pages), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    head = int(rng.integers(0, n_pages))
    ring = np.full(n_pages, -1, np.int32)
    ring[(head + np.arange(free)) % n_pages] = order[at:]
    return table, ring, [head, free]


def tables_check(seq, new, table, ring, cursor, n_tokens, page, n_indices=None):
    want = pc.page_tables(seq, new, table, ring, cursor, n_tokens, page)
    td, rd, cd, sd, nd = i32(table), i32(ring), i32(cursor), i32(seq), i32(new)
    n_indices = len(ring) if n_indices is None else n_indices
    for again in range(2):  # the inputs are left as they were: the step can be repeated
        kv = torch.full((n_indices,), -7, dtype=torch.int32, device="cuda")
        t = idx.idx_page_tables(sd, nd, td, rd, cd, n_tokens, page_size=page, kv_indices=kv)
        torch.cuda.synchronize()
        for name in ("seq_len", "cursor", "kv_indptr", "tok_indptr", "slots", "tok_req",
                     "tok_len"):
            np.testing.assert_array_equal(getattr(t, name).cpu().numpy(), want[name], name)
        np.testing.assert_array_equal(td.cpu().numpy(), want["table"])
        np.testing.assert_array_equal(rd.cpu().numpy(), want["ring"])
        kv = kv.cpu().numpy()
        n = min(len(want["kv_indices"]), n_indices)
        np.testing.assert_array_equal(kv[:n], want["kv_indices"][:n])
        assert (kv[n:] == -7).all()
    np.testing.assert_array_equal(cd.cpu().numpy(), cursor)
    np.testing.assert_array_equal(sd.cpu().numpy(), seq)
    return want


@pytest.mark.parametrize("B,page,longest", [(1, 16, 5), (1, 16, 100000), (3, 1, 7), (4, 16, 3000),
                                            (70, 32, 900), (256, 16, 60), (257, 64, 60),
                                            (1500, 16, 40), (16384, 16, 40)])
@pytest.mark.parametrize("room", ["plenty", "short"])
def test_page_tables(B, page, longest, room):
    rng = np.random.default_rng(B * 31 + page)
    seq = rng.integers(0, longest + 1, B)
    new = np.where(rng.random(B) < 0.3, -rng.integers(0, longest + 5, B),
                   rng.integers(0, min(longest, 50) + 1, B))
    new[rng.random(B) < 0.2] = 0
    held = [-(-int(n) // page) for n in seq]
    grow = sum(max(0, -(-int(max(s + d, 0)) // page) - h) for s, d, h in zip(seq, new, held))
    free = grow + 5 if room == "plenty" else grow // 2
    max_pages = max(held) + (60 if room == "plenty" else 1)
    table, ring, cursor = pool(rng, held, free if sum(held) + free else 1, max_pages)
    tokens = int(np.maximum(new, 0).sum())
    want = tables_check(seq, new, table, ring, cursor, tokens + 3, page)
    say(f"[tables] B={B} page={page} {room}: refused {want['cursor'][2]}")
    if room == "plenty":
        assert want["cursor"][2] == 0


def test_page_tables_token_rows_list_room_and_clamps():
    rng = np.random.default_rng(5)
    seq, new = np.array([20, 0, 35, 16, 7]), np.array([3, 30, 4, -16, 2])
    table, ring, cursor = pool(rng, [2, 0, 3, 1, 1], 10, 4)
    for tokens in (0, 1, 3, 32, 33, 37, 39, 50):   # rows for some of the requests' tokens
        tables_check(seq, new, table, ring, cursor, tokens, 16)
    for n_indices in (0, 1, 4, 9):                 # the packed list is cut
        tables_check(seq, new, table, ring, cursor, 39, 16, n_indices)
    # lengths past the table, more given back than held, cursors out of range
    for seq2, new2 in (([100, -3, 64, 16, 7], [1, 2, 1, -100, 0]),
                       ([20, 0, 35, 16, 7], [2 ** 31 - 1, 5, -2 ** 31, 2 ** 31 - 1, 1])):
        tables_check(seq2, new2, np.abs(table), ring, cursor, 39, 16)
    for cur in ([-3, 10], [10 ** 6, 10], [4, -1], [4, 10 ** 6]):
        tables_check(seq, new, table, np.abs(ring), cur, 39, 16)


def test_page_tables_pages_return_and_serve_later_steps():
    """Many steps over a small pool: every page is held once or free, never both."""
    rng = np.random.default_rng(6)
    B, page, n_pages, max_pages = 9, 16, 40, 12
    table = i32(np.full((B, max_pages), -1))
    ring, cursor, seq = i32(np.arange(n_pages)), i32([0, n_pages, 0]), i32(np.zeros(B))
    held = np.zeros(B, np.int64)
    for step in range(60):
        new = np.where(rng.random(B) < 0.25, -held, rng.integers(-3, 30, B)).astype(np.int32)
        new = np.maximum(new, -held).astype(np.int32)
        t = idx.idx_page_tables(seq, i32(new), table, ring, cursor, int(np.maximum(new, 0).sum()),
                                page_size=page)
        seq, cursor = t.seq_len, t.cursor
        held = seq.cpu().numpy().astype(np.int64)
        head, count, _ = cursor.cpu().tolist()
        mine = t.kv_indices.cpu().numpy()[:int(t.kv_indptr[-1])]
        free = ring.cpu().numpy()[(head + np.arange(count)) % n_pages]
        assert sorted(mine.tolist() + free.tolist()) == list(range(n_pages)), step
        assert len(mine) == (-(-held // page)).sum()


# ------------------------------------------------------------------- cache write

def write_case(seed, spans, Hkv, page, dtype, values=None, spare=2):
    """Requests whose tokens [start, stop) are written: (rows, slots, cache)."""
    rng = np.random.default_rng(seed)
    c = Cache(seed, [max(stop, 1) for _, stop in spans], Hkv, page, spare)
    c.k = pc.e4m3_encode(rng.standard_normal(c.k.shape) * 100)
    c.v = pc.e4m3_encode(rng.standard_normal(c.v.shape) * 100)
    c.ks, c.vs = (np.exp2(rng.integers(-9, -3, c.ks.shape)).astype(np.float32) for _ in "kv")
    slots = []
    for b, (start, stop) in enumerate(spans):
        pages = c.indices[c.indptr[b]:c.indptr[b + 1]]
        slots += [int(pages[p // page]) * page + p % page for p in range(start, stop)]
    n = len(slots)
    x = rng.standard_normal((n, 2, Hkv, 128)) * np.exp2(rng.integers(-3, 4, (n, 2, 1, 1)))
    if values is not None:
        values(x)
    x = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return x, np.array(slots, np.int32), c


def write_check(x, slots, c):
    xd = x.cuda()                       # k and v lie in one row of a fused projection
    kd, vd, ks, vs, _, _ = c.device()
    idx.idx_cache_write(xd[:, 0], xd[:, 1], i32(slots), kd, vd, ks, vs)
    torch.cuda.synchronize()
    rows = x.double().numpy()
    k2, ks2 = pc.cache_write(rows[:, 0], slots, c.k, c.ks, c.page, False)
    v2, vs2 = pc.cache_write(rows[:, 1], slots, c.v, c.vs, c.page, True)
    np.testing.assert_array_equal(ks.cpu().numpy(), ks2)
    np.testing.assert_array_equal(vs.cpu().numpy(), vs2)
    for got, want in ((kd, k2), (vd, v2)):
        got = got.view(torch.uint8).cpu().numpy()
        nan = (want & 0x7F) == 0x7F
        np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan)
        np.testing.assert_array_equal(got[~nan], want[~nan])


SPANS = {
    "one": [(0, 1)], "last_of_page": [(15, 16)], "decode": [(n - 1, n) for n in
                                                            (1, 2, 16, 17, 33, 48, 64, 100)],
    "prompts": [(0, 16), (0, 100), (5, 90), (63, 65), (31, 32)], "long": [(3, 1500), (0, 700)],
}


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spans", list(SPANS))
def test_cache_write(spans, dtype, page):
    for Hkv in (1, 3, 8):
        say(f"[write] {spans} {dtype} page={page} Hkv={Hkv}")
        write_check(*write_case(11 + Hkv, SPANS[spans], Hkv, page, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cache_write_special_values(dtype):
    def values(x):
        x[0, 0, 0, :8] = [np.inf, -np.inf, np.nan, 448, -448, 0, 1e-30, -1e-30]
        x[1, :, 1] = 0.0                                # a head of zeros: the least scale
        x[2, 0, 0] = np.nan                             # nothing finite
        x[3, 1] = 1e38
        x[4, 1] = 1e-38
        x[5, 0, 0, 3] = 449
        x[6, 0, 1] = np.inf
    spans = [(0, 1)] * 4 + [(4, 5), (7, 8), (2, 9)]
    write_check(*write_case(17, spans, 2, 16, dtype, values))


def test_cache_write_keeps_a_larger_or_calibrated_scale():
    x, slots, c = write_case(18, [(4, 5), (9, 12)], 2, 16, torch.bfloat16)
    c.ks[:] = 0.7                                       # not a power of two, and kept
    c.vs[:] = 1e-3                                      # not a power of two, and outgrown
    write_check(x, slots, c)


def test_cache_write_skips_and_no_tokens():
    x, slots, c = write_case(19, [(0, 20), (3, 5)], 2, 16, torch.bfloat16)
    slots = slots.copy()
    slots[4:7] = -1                                     # three runs in a page are one call's
    slots[20] = c.n_pages * 16                          # past the pool
    slots[21] = -5
    write_check(x[:0], slots[:0], c)
    keep = np.r_[0:4, 16:22]                            # page 0's first run, page 1, skipped
    write_check(x[keep], slots[keep], c)


def test_cache_write_past_4gib():
    """Pages whose bytes start past 2^32."""
    n_pages, page = 1 << 21, 16
    k = torch.zeros(n_pages + 9, 1, page, 128, dtype=torch.uint8, device="cuda")
    v = torch.zeros(n_pages + 9, 1, 128, page, dtype=torch.uint8, device="cuda")
    ks = torch.ones(n_pages + 9, 1, device="cuda")
    vs = torch.ones(n_pages + 9, 1, device="cuda")
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 2, 1, 128, generator=g).bfloat16()
    first = (n_pages + 3) * page
    xd = x.cuda()
    idx.idx_cache_write(xd[:, 0], xd[:, 1], i32(np.arange(first, first + 40)), k, v, ks, vs)
    sub = Cache(1, [16], 1, 16, 8)
    z = np.zeros((9, 1, page, 128), np.uint8)
    rows = x.double().numpy()
    slots = np.arange(3 * page, 3 * page + 40)
    k2, s2 = pc.cache_write(rows[:, 0], slots, z, np.ones((9, 1), np.float32), page, False)
    v2, _ = pc.cache_write(rows[:, 1], slots, z.transpose(0, 1, 3, 2).copy(),
                           np.ones((9, 1), np.float32), page, True)
    np.testing.assert_array_equal(k[n_pages:].cpu().numpy(), k2)
    np.testing.assert_array_equal(v[n_pages:].cpu().numpy(), v2)
    np.testing.assert_array_equal(ks[n_pages:].cpu().numpy(), s2)
    assert not k[:n_pages].any()
    # and attention reads them there
    q, q64 = queries(np.random.default_rng(4), 1, 4)
    out = idx.idx_attend(q.cuda(), k, v, ks, vs, i32([0, 3]),
                         i32(np.arange(n_pages + 3, n_pages + 6)), i32([40]), 3)
    sub.k, sub.v, sub.ks, sub.vs = k2, v2, s2, vs[n_pages:].cpu().numpy()
    sub.indptr, sub.indices, sub.n_pages, sub.max_pages = (
        np.array([0, 3]), np.array([3, 4, 5]), 9, 3)
    check_rows(out, sub, q64, [0], [40])


# ------------------------------------------------------------------- single tokens

def attend(c, q, seen, max_pages=None, **kw):
    return idx.idx_attend(q.cuda(), *c.device(), i32(seen), max_pages or c.max_pages, **kw)


HEADS = [(1, 1), (8, 8), (8, 2), (6, 2), (16, 1), (20, 1), (64, 2), (64, 1)]


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64])
def test_attend_lengths(Hq, Hkv, page):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 300, 700]
    c = Cache(Hq * 7 + page, lens, Hkv, page)
    q, q64 = queries(c.rng, len(lens), Hq)
    w = check_rows(attend(c, q, lens), c, q64, range(len(lens)), lens)
    say(f"[attend] Hq={Hq} Hkv={Hkv} page={page}: {w:.3f} of the bound")


@pytest.mark.parametrize("cap,biased", [(30.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (40, 2), (33, 1)])
def test_attend_softcap_and_slopes(Hq, Hkv, cap, biased):
    lens = [1, 16, 77, 500, 1300]
    c = Cache(23, lens, Hkv, 16)
    q, q64 = queries(c.rng, len(lens), Hq, 4.0)
    slopes = np.exp2(-8 * (np.arange(Hq) + 1) / Hq).astype(np.float32) if biased else None
    out = attend(c, q, lens, softcap=cap, slopes=None if slopes is None else dev(slopes),
                 scale=0.125)
    check_rows(out, c, q64, range(len(lens)), lens, cap=cap, slopes=slopes, scale=0.125)


def test_attend_rows_that_see_nothing_or_less_than_they_hold():
    lens = [40, 100, 64, 0, 33]
    c = Cache(24, lens, 2, 16)
    q, q64 = queries(c.rng, 5, 8)
    seen = [0, 50, -3, 0, 2 ** 31 - 1]            # the last sees all it holds...
    c.k[c.indices[c.indptr[4] + 2]] = 0x30        # ...whole pages
    c.v[c.indices[c.indptr[4] + 2]] = 0x30
    out = attend(c, q, seen)
    check_rows(out, c, q64, range(5), seen)
    out = out.cpu()
    assert not out[0].any() and not out[2].any() and not out[3].any()


def test_attend_more_rows_than_requests_and_unknown_requests():
    lens = [100, 3, 250]
    c = Cache(25, lens, 2, 32)
    req = [2, 0, 0, 1, 2, -1, 3, 2, 1 << 30]
    seen = [250, 7, 100, 3, 1, 9, 9, 130, 5]
    q, q64 = queries(c.rng, 9, 4)
    out = attend(c, q, seen, row_req=i32(req))
    check_rows(out, c, q64, req, seen)


def test_attend_bad_pages_and_short_lists():
    lens = [160, 160, 160, 160]
    c = Cache(26, lens, 2, 16)
    c.indices = c.indices.copy()
    c.indices[3], c.indices[12], c.indices[14] = -1, c.n_pages, 1 << 30
    c.indices = c.indices[:35]                     # request 3's list runs past the array
    c.indptr = np.array([0, 10, 20, 30, 40], np.int32)
    q, q64 = queries(c.rng, 4, 8)
    check_rows(attend(c, q, lens), c, q64, range(4), lens)
    c.max_pages = 4                                # clamped lists
    check_rows(attend(c, q, lens), c, q64, range(4), lens)
    c.max_pages = 10
    c.indptr = np.array([5, 3, 20, 20, -2], np.int32)   # backwards, empty, negative
    check_rows(attend(c, q, lens), c, q64, range(4), lens)


def random_ids(rng, n_rows, lists, K):
    ids = np.full((n_rows, K), -1, np.int32)
    for r in range(n_rows):
        m = min(K, lists[r])
        ids[r, :m] = np.sort(rng.permutation(lists[r])[:m])
    return ids


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("K", [1, 3, 17, 130])
def test_attend_selected_pages(K, page):
    lens = [page * 40 - 3, 5, 900, page, 1]
    c = Cache(27 + K, lens, 2, page)
    q, q64 = queries(c.rng, 5, 8)
    ids = random_ids(c.rng, 5, [-(-n // page) for n in lens], K)
    out = attend(c, q, lens, ids=i32(ids))
    check_rows(out, c, q64, range(5), lens, ids)
    ids = ids[:, ::-1].copy()                     # any order, -1 first
    check_rows(attend(c, q, lens, ids=i32(ids)), c, q64, range(5), lens, ids)


def test_attend_selected_pages_repeated_unknown_and_none():
    lens = [200, 77, 500]
    c = Cache(28, lens, 1, 16)
    q, q64 = queries(c.rng, 3, 4)
    ids = np.array([[3, 3, 7, -1, -5, 12], [4, 99, 1 << 30, 4, 4, 5],
                    [-1, -1, -1, -1, -1, -1]], np.int32)
    out = attend(c, q, lens, ids=i32(ids))
    check_rows(out, c, q64, range(3), lens, ids)
    assert not out[2].any()
    assert not attend(c, q, lens, ids=torch.empty(3, 0, dtype=torch.int32, device="cuda")).any()


@pytest.mark.parametrize("B,n", [(1, 40000), (2, 9001), (3, 131072)])
def test_attend_long_rows_over_several_workgroups(B, n):
    lens = [n] + [max(1, n // 7 - 3)] * (B - 1)
    c = Cache(29, lens, 1, 16)
    assert idx.idx_attend_workspace_bytes(B, 4, 1, c.max_pages) > 0
    q, q64 = queries(c.rng, B, 4)
    check_rows(attend(c, q, lens), c, q64, range(B), lens)
    check_rows(attend(c, q, [5] * B), c, q64, range(B), [5] * B)   # empty splits
    check_rows(attend(c, q, [0] * B), c, q64, range(B), [0] * B)


def test_attend_nan_and_extreme_values_of_seen_tokens():
    """NaN codes reach the rows that see them; scales far apart, large scores."""
    lens = [90, 90, 90, 90]
    c = Cache(30, lens, 1, 16)
    c.v[c.indices[c.indptr[0]], 0, 5, 3] = 0x7F
    c.k[c.indices[c.indptr[1] + 5], 0, 9] = 0x7F          # token 89 of request 1
    c.vs[c.indices[c.indptr[2]:c.indptr[3]], 0] = np.exp2([-20., -4., 5., -9., 0., -13.])
    c.ks[c.indices[c.indptr[3]:c.indptr[4]], 0] = 30.0
    q, q64 = queries(c.rng, 4, 4)
    out = attend(c, q, lens)
    check_rows(out, c, q64, range(4), lens)
    assert out[1].isnan().all() and out[0, :, 5].isnan().all()
    seen = [3, 89, 90, 90]                                # neither NaN token is seen
    out = attend(c, q, seen)
    check_rows(out, c, q64, range(4), seen)
    assert not out.isnan().any()


def test_attend_strided_queries_given_output_and_none():
    lens = [100, 30, 7]
    c = Cache(31, lens, 2, 16)
    wide = torch.zeros(3, 3, 8, 128, dtype=torch.bfloat16)
    q, q64 = queries(c.rng, 3, 8)
    wide[:, 1] = q
    wide = wide.cuda()
    out = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = idx.idx_attend(wide[:, 1], *c.device(), i32(lens), c.max_pages, out=out)
    assert got.data_ptr() == out.data_ptr()
    check_rows(out, c, q64, range(3), lens)
    none = idx.idx_attend(wide[:0, 1], *c.device(), i32([]), c.max_pages)
    assert none.shape == (0, 8, 128)


# ------------------------------------------------------------------- prompt tokens

def prefill(c, q, ptr, seen, **kw):
    return idx.idx_attend_prefill(q.cuda(), *c.device(), i32(ptr), i32(seen), c.max_pages, **kw)


def causal(lens, news):
    """Packed rows of each request's last tokens: (indptr, request, visible length)."""
    ptr = np.concatenate([[0], np.cumsum(news)])
    req = np.repeat(np.arange(len(lens)), news)
    seen = np.concatenate([np.arange(n - k, n) + 1 for n, k in zip(lens, news)])
    return ptr.astype(np.int32), req, seen.astype(np.int32)


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_prefill_ragged(Hq, Hkv, page):
    lens, news = [1, 70, 200, 64, 333, 5], [1, 3, 65, 64, 17, 0]
    c = Cache(Hq + page, lens, Hkv, page)
    ptr, req, seen = causal(lens, news)
    q, q64 = queries(c.rng, len(req), Hq)
    w = check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)
    say(f"[prefill] Hq={Hq} Hkv={Hkv} page={page}: {w:.3f} of the bound")


@pytest.mark.parametrize("n", [1, 2, 31, 33, 127, 129, 400])
def test_prefill_whole_prompts(n):
    lens = [n, max(1, n // 2)]
    c = Cache(n, lens, 2, 16)
    ptr, req, seen = causal(lens, lens)
    q, q64 = queries(c.rng, len(req), 4)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)


@pytest.mark.parametrize("cap,biased", [(30.0, False), (0.0, True), (5.0, True)])
def test_prefill_softcap_and_slopes(cap, biased):
    lens, news = [150, 400], [20, 90]
    c = Cache(43, lens, 2, 16)
    ptr, req, seen = causal(lens, news)
    q, q64 = queries(c.rng, len(req), 8, 4.0)
    slopes = np.exp2(-(np.arange(8) + 1.0)).astype(np.float32) if biased else None
    out = prefill(c, q, ptr, seen, softcap=cap, scale=0.125,
                  slopes=None if slopes is None else dev(slopes))
    check_rows(out, c, q64, req, seen, cap=cap, slopes=slopes, scale=0.125)


def test_prefill_prefix_mask_any_lengths_and_empty_rows():
    lens = [300, 120]
    c = Cache(44, lens, 2, 16)
    ptr, req, seen = causal(lens, [300, 120])
    seen = np.maximum(seen, np.where(req == 0, 90, 0))    # 90 tokens of prefix
    seen[5], seen[100], seen[310] = 0, -4, 120            # nothing, or out of order
    seen[200] = 2 ** 31 - 1
    tail = c.indices[c.indptr[1] - 1]                     # sees what the page holds
    c.k[tail], c.v[tail] = 0x31, 0x32
    q, q64 = queries(c.rng, len(req), 4)
    out = prefill(c, q, ptr, seen)
    check_rows(out, c, q64, req, seen)
    assert not out[5].any() and not out[100].any()


def test_prefill_leaves_other_rows_as_they_were():
    for lens, news, cut in (([70, 200], [3, 65], 1), ([9000, 5], [2, 3], 2)):
        c = Cache(45, lens, 2, 16)
        ptr, req, seen = causal(lens, news)
        n = len(req)
        q, q64 = queries(c.rng, n + 7, 4)
        out = torch.full((n + 7, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        prefill(c, q, ptr, np.concatenate([seen, [50] * 7]), out=out)
        check_rows(out[:n], c, q64, req, seen)
        assert (out[n:] == 7.0).all()
        # rows in front of the first request, and lists outside the rows
        out.fill_(7.0)
        ptr2 = ptr + 4
        seen2 = np.concatenate([[50] * 4, seen, [50] * 3])
        prefill(c, q, ptr2, seen2, out=out)
        check_rows(out[4:n + 4], c, q64[4:], req, seen)
        assert (out[:4] == 7.0).all() and (out[n + 4:] == 7.0).all()
    out.fill_(7.0)
    prefill(c, q, [-5, 2, 10 ** 6], np.full(n + 7, 5), out=out)   # clamped to [0, n]
    check_rows(out, c, q64, [0] * 2 + [1] * (n + 5), [5] * (n + 7))


def test_prefill_few_rows_with_nan_values_prefixes_and_empty_rows():
    """The same in calls of few rows a request: drafted tokens on longer contexts."""
    lens, news = [200, 77, 1000, 5, 64, 300], [6, 5, 7, 5, 1, 0]
    c = Cache(54, lens, 2, 16)
    for b, pos, dim in ((0, 197, 3), (0, 10, 100), (2, 995, 127), (3, 2, 64), (4, 63, 0)):
        page = c.indices[c.indptr[b] + pos // 16]
        c.v[page, 1, dim, pos % 16] = 0x7F if dim % 2 else 0xFF
    c.k[c.indices[c.indptr[1] + 74 // 16], 0, 74 % 16, 5] = 0x7F
    ptr, req, seen = causal(lens, news)
    seen[7], seen[12], seen[19] = 77, 0, -3       # a prefix's row, rows that see nothing
    for Hq in (2, 6, 16, 32):
        q, q64 = queries(c.rng, len(req), Hq)
        assert len(req) * (Hq // 2) <= 64 * len(lens)
        for kw in ({}, dict(softcap=20.0), dict(slopes=dev(np.full(Hq, 0.05, np.float32)))):
            out = prefill(c, q, ptr, seen, **kw)
            check_rows(out, c, q64, req, seen, cap=kw.get("softcap", 0.0),
                       slopes=np.full(Hq, np.float32(0.05)) if "slopes" in kw else None)
            nan = out.isnan().cpu().numpy()
            assert nan[:6, Hq // 2:, 100].all() and not nan[:3, :, 3].any()
            assert nan[3:6, Hq // 2:, 3].all() and not nan[12].any() and not nan[19].any()


def test_prefill_nan_values_reach_only_the_rows_that_see_them():
    lens = [140, 140]
    c = Cache(46, lens, 2, 16)
    ptr, req, seen = causal(lens, lens)
    for pos, dim in ((0, 3), (70, 64), (139, 127), (100, 15)):
        page = c.indices[c.indptr[1] + pos // 16]
        c.v[page, 1, dim, pos % 16] = 0x7F if dim % 2 else 0xFF
    page = c.indices[c.indptr[0] + 6]                     # and a NaN key at 100
    c.k[page, 0, 4, 77] = 0x7F
    q, q64 = queries(c.rng, len(req), 4)
    out = prefill(c, q, ptr, seen)
    check_rows(out, c, q64, req, seen)
    nan = out.isnan().cpu().numpy()
    assert not nan[:100].any() and nan[100:140, :2].all() and not nan[:140, 2:].any()
    assert nan[140:, 2:, 3].all() and not nan[140:, 2:, 4].any()
    assert not nan[140:210, 2:, 64].any() and nan[210:, 2:, 64].all()


@pytest.mark.parametrize("lens,news", [([20000], [1]), ([9000, 30], [7, 2]), ([5000], [130])])
def test_prefill_long_contexts_over_several_workgroups(lens, news):
    c = Cache(47, lens, 1, 16)
    assert idx.idx_attend_prefill_workspace_bytes(sum(news), len(lens), 4, 1, c.max_pages) > 0
    ptr, req, seen = causal(lens, news)
    q, q64 = queries(c.rng, len(req), 4)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)


def test_bounds_far_above_the_lists():
    """max_pages far above the longest list, and rows longer than one phase of page data
    (16384 tokens of single tokens' rows, 32768 of prompt rows)."""
    lens, news = [300, 45], [60, 5]
    c = Cache(52, lens, 1, 16, max_pages=1 << 18)
    ptr, req, seen = causal(lens, news)
    q, q64 = queries(c.rng, len(req), 4)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)
    check_rows(attend(c, q, seen, row_req=i32(req)), c, q64, req, seen)
    lens = [70001]
    c = Cache(53, lens, 1, 16, max_pages=1 << 22)
    c.vs[c.indices, 0] = np.exp2(np.linspace(-9, -3, len(c.indices))).astype(np.float32)
    ptr, req, seen = causal(lens, [30])
    q, q64 = queries(c.rng, 30, 4)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen, rows=[0, 7, 29])
    check_rows(attend(c, q, seen, row_req=i32(req)), c, q64, req, seen, rows=[0, 7, 29])


def test_prefill_bad_pages():
    lens = [160, 160]
    c = Cache(48, lens, 2, 16)
    c.indices = c.indices.copy()
    c.indices[3], c.indices[12] = -1, c.n_pages
    c.indices = c.indices[:17]
    ptr, req, seen = causal(lens, [40, 160])
    q, q64 = queries(c.rng, len(req), 4)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("scale,cap", [(-0.2, 0.0), (-0.2, 4.0), (0.0, 0.0), (3.0, 0.0)])
def test_call_scales_of_any_sign_and_size(scale, cap):
    lens, news = [300, 77], [40, 77]
    c = Cache(49, lens, 2, 16)
    ptr, req, seen = causal(lens, news)
    q, q64 = queries(c.rng, len(req), 6)
    kw = dict(scale=scale, softcap=cap)
    check_rows(prefill(c, q, ptr, seen, **kw), c, q64, req, seen, scale=scale, cap=cap)
    check_rows(attend(c, q, seen, row_req=i32(req), **kw), c, q64, req, seen, scale=scale,
               cap=cap)


def test_value_scales_that_grow_along_the_row():
    """Each page's value scale above the ones before it, the last tiles' by far."""
    lens = [6000]
    c = Cache(51, lens, 1, 16)
    n = len(c.indices)
    c.vs[c.indices, 0] = np.exp2(np.linspace(-14, 0, n)).astype(np.float32)
    c.ks[c.indices, 0] = np.exp2(np.linspace(-9, -5, n)).astype(np.float32)
    c.k[c.indices[7]], c.v[c.indices[7]] = 0, 0           # a page of zeros: the least scale
    c.ks[c.indices[7]] = c.vs[c.indices[7]] = 2.0 ** -120
    ptr, req, seen = causal(lens, [40])
    q, q64 = queries(c.rng, 40, 4)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)
    check_rows(attend(c, q, seen, row_req=i32(req)), c, q64, req, seen)


def test_least_key_scales_under_large_queries():
    """Keys of very small scale with queries that make ordinary scores of them, in tiles
    that are masked in part."""
    lens, news = [300, 77, 20], [40, 77, 1]
    c = Cache(53, lens, 2, 16)
    used = c.indices
    c.ks[used] *= np.float32(2.0 ** -100)
    ptr, req, seen = causal(lens, news)
    q, _ = queries(c.rng, len(req), 6)
    q = (q.float() * 2.0 ** 100).bfloat16()
    q64 = q.double().numpy()
    check_rows(attend(c, q, seen, row_req=i32(req)), c, q64, req, seen)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)
    few = ptr[:3]                                         # a row of each request
    check_rows(prefill(c, q[few], [0, 1, 2, 3], seen[few]), c, q64[few], req[few], seen[few])


def test_least_value_scales_in_long_uncut_prompts():
    """Values of the least scale under a large sum of weights: 64 tokens of score 0, the
    others below the step at which the reference moves (5.5 in base 2)."""
    n, Hkv = 2000, 8
    c = Cache(54, [n], Hkv, 16)
    c.k[c.indices] = 0x38                                 # 1.0
    c.k[c.indices[:4]] = 0
    c.ks[c.indices] = 2.0 ** -7
    c.vs[c.indices] = 2.0 ** -120
    c.poison_tails()
    q = torch.ones(1000, 64, 128, dtype=torch.bfloat16)
    ptr, req, seen = causal([n], [1000])
    # enough row tiles that no row is cut: there are no partial results
    assert idx.idx_attend_prefill_workspace_bytes(1000, 1, 64, Hkv, c.max_pages, 16) == 0
    scale = 5.5 * np.log(2.0)                             # times the product, 128 * 2^-7
    rows = [0, 500, 999]
    out = prefill(c, q, ptr, seen, scale=scale)
    check_rows(out, c, q.double().numpy(), req, seen, scale=scale, rows=rows)


def test_rows_and_prompt_tokens_agree():
    """The same rows through both calls: equal within both bounds of the oracle."""
    lens, news = [700, 90, 1300], [5, 1, 3]
    c = Cache(50, lens, 2, 16)
    ptr, req, seen = causal(lens, news)
    q, q64 = queries(c.rng, len(req), 8)
    check_rows(prefill(c, q, ptr, seen), c, q64, req, seen)
    check_rows(attend(c, q, seen, row_req=i32(req)), c, q64, req, seen)


def test_serving_steps():
    """Prompts, then decode steps, one request ending and another starting: tables,
    writes, the indexer's selection over the pages' centroids, attention."""
    rng = np.random.default_rng(60)
    B, Hq, Hkv, page, n_pages, max_pages = 3, 8, 2, 16, 64, 24
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    kc, vc = z(n_pages, Hkv, page, 128, dtype=torch.uint8), z(n_pages, Hkv, 128, page,
                                                               dtype=torch.uint8)
    ks, vs = torch.ones(n_pages, Hkv, device="cuda"), torch.ones(n_pages, Hkv, device="cuda")
    table, ring = i32(np.full((B, max_pages), -1)), i32(np.arange(n_pages))
    cursor, seq = i32([0, n_pages, 0]), i32(np.zeros(B))
    ref = [kc.cpu().numpy(), vc.cpu().numpy(), ks.cpu().numpy(), vs.cpu().numpy()]
    steps = [[50, 200, 0], [1, 1, 33], [1, -201, 1], [1, 120, 1], [1, 1, -2], [1, 1, 1]]
    for step, new in enumerate(steps):
        n = sum(max(0, d) for d in new)
        t = idx.idx_page_tables(seq, i32(new), table, ring, cursor, n, page_size=page)
        x = torch.from_numpy(rng.standard_normal((n, 2, Hkv, 128)).astype(np.float32)).bfloat16()
        q, q64 = queries(rng, n, Hq)
        xd, qd = x.cuda(), q.cuda()
        idx.idx_cache_write(xd[:, 0], xd[:, 1], t.slots, kc, vc, ks, vs)
        out = idx.idx_attend_prefill(qd, kc, vc, ks, vs, t.kv_indptr, t.kv_indices, t.tok_indptr,
                                     t.tok_len, max_pages)
        slots = t.slots.cpu().numpy()
        assert (slots >= 0).all() and int(t.cursor[2]) == 0
        rows = x.double().numpy()
        ref[0], ref[2] = pc.cache_write(rows[:, 0], slots, ref[0], ref[2], page, False)
        ref[1], ref[3] = pc.cache_write(rows[:, 1], slots, ref[1], ref[3], page, True)
        for got, want in zip((kc, vc, ks, vs), ref):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        c = Cache.__new__(Cache)
        c.k, c.v, c.ks, c.vs = ref
        c.indptr, c.indices = t.kv_indptr.cpu().numpy(), t.kv_indices.cpu().numpy()
        c.Hkv, c.page, c.n_pages, c.max_pages = Hkv, page, n_pages, max_pages
        req, seen = t.tok_req.cpu().numpy(), t.tok_len.cpu().numpy()
        check_rows(out, c, q64, req, seen)

        # each token's 4 best pages by the mean key of head 0, and attention over them
        cent = z(n_pages, 128)
        means = (pc.e4m3_values()[ref[0][:, 0]] * ref[2][:, 0, None, None]).mean(1)
        cent.copy_(torch.from_numpy(means.astype(np.float32)))
        dec = [r for r in range(n) if r == n - 1 or req[r + 1] != req[r]]   # last tokens
        if len(dec) == B:
            ids, counts, _ = idx.idx_select_paged(qd[dec].float().contiguous(), cent, t.kv_indptr,
                                                  t.kv_indices, 4, max_pages)
            got = idx.idx_attend(qd[dec], kc, vc, ks, vs, t.kv_indptr, t.kv_indices,
                                 t.tok_len[dec], max_pages, row_req=t.tok_req[dec], ids=ids)
            check_rows(got, c, q64[dec], req[dec], seen[dec], ids.cpu().numpy())
        seq, cursor = t.seq_len, t.cursor
    assert seq.cpu().tolist() == [55, 122, 34]


def test_captured_steps_replay_as_the_eager_ones():
    """One decode step (tables, write, attention over all and over selected pages, prompt
    form) in a graph, replayed with other inputs and eager work in between."""
    lens = [100, 15, 3000, 47]
    B, Hq, Hkv, page = 4, 8, 2, 16
    c = Cache(70, [n + 1 for n in lens], Hkv, page, spare=20)
    kc, vc, ks, vs, _, _ = c.device()
    start = [t.clone() for t in (kc, vc, ks, vs)]
    max_pages = c.max_pages + 2
    table = np.full((B, max_pages), -1, np.int32)
    for b, n in enumerate(lens):
        h = -(-n // page)
        table[b, :h] = c.indices[c.indptr[b]:c.indptr[b] + h]
    free = np.setdiff1d(np.arange(c.n_pages), table[table >= 0])
    ring = np.full(c.n_pages, -1, np.int32)
    ring[:len(free)] = free
    td, rd, seq, cur = i32(table), i32(ring), i32(lens), i32([0, len(free), 0])
    new = i32([1] * B)
    kv = torch.full((c.n_pages,), -1, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, 2, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, Hq, 128, dtype=torch.bfloat16, device="cuda")
    ids = i32(random_ids(c.rng, B, [-(-(n + 1) // page) for n in lens], 5))

    def step():
        t = idx.idx_page_tables(seq, new, td, rd, cur, B, page_size=page, kv_indices=kv)
        idx.idx_cache_write(x[:, 0], x[:, 1], t.slots, kc, vc, ks, vs)
        args = (q, kc, vc, ks, vs, t.kv_indptr, t.kv_indices)
        return (t.slots, t.tok_len, t.cursor, idx.idx_attend(*args, t.tok_len, max_pages),
                idx.idx_attend(*args, t.tok_len, max_pages, ids=ids),
                idx.idx_attend_prefill(*args, t.tok_indptr, t.tok_len, max_pages))

    def restore():
        for a, b in zip((kc, vc, ks, vs), start):
            a.copy_(b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    outs = []
    for g in (g1, g2):
        with torch.cuda.graph(g):
            outs.append(step())
    rng = np.random.default_rng(71)
    for rep in range(4):
        say(f"[graph] replay {rep}")
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape).astype(np.float32)))
        q.copy_(torch.from_numpy(rng.standard_normal(q.shape).astype(np.float32)))
        restore()
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for g, out in zip((g1, g2), outs):
            restore()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    cs = [Cache(80 + i, [9000, 400, 40], 2, 16) for i in range(2)]
    ins = []
    for c in cs:
        q, q64 = queries(c.rng, 3, 8)
        ins.append((q.cuda(), q64, c.device(), i32([9000, 400, 40])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for rep in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                q, _, d, seen = ins[i]
                outs[i].append(idx.idx_attend(q, *d, seen, cs[i].max_pages))
    torch.cuda.synchronize()
    for i, c in enumerate(cs):
        check_rows(outs[i][0], c, ins[i][1], range(3), [9000, 400, 40])
        for o in outs[i][1:]:
            assert torch.equal(o, outs[i][0])


def test_results_do_not_depend_on_the_run():
    """Fixed orders of summation: the same call gives the same bits."""
    c = Cache(90, [20000, 700], 2, 16)
    q, _ = queries(c.rng, 2, 8)
    first = attend(c, q, [20000, 700])
    for _ in range(5):
        assert torch.equal(attend(c, q, [20000, 700]), first)


# ------------------------------------------------------------------- refusals

def test_binding_checks():
    c = Cache(91, [30, 40], 2, 16)
    d = c.device()
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    seen, ptr = i32([30, 40]), i32([0, 1, 2])
    bad = [
        (TypeError, dict(q=q.float())), (ValueError, dict(q=q[:, :, :64])),
        (ValueError, dict(q=q.transpose(0, 1))), (TypeError, dict(kc=d[0].view(torch.int8))),
        (ValueError, dict(vc=d[1].transpose(2, 3).contiguous())),
        (TypeError, dict(ks=d[2].double())), (ValueError, dict(vs=d[3][:, :1].contiguous())),
        (TypeError, dict(ptr=d[4].long())), (TypeError, dict(ind=d[5].long())),
        (TypeError, dict(seen=seen.long())), (ValueError, dict(seen=seen[:1])),
        (ValueError, dict(slopes=torch.zeros(3, device="cuda"))),
        (ValueError, dict(slopes=torch.zeros(4, device="cuda").double())),
        (ValueError, dict(out=torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16))),
        (ValueError, dict(ws=torch.zeros(8, dtype=torch.uint8))),
    ]
    for err, kw in bad:
        a = dict(q=q, kc=d[0], vc=d[1], ks=d[2], vs=d[3], ptr=d[4], ind=d[5], seen=seen) | kw
        more = {k: a[k] for k in ("slopes", "out", "ws") if k in a}
        base = [a[k] for k in ("q", "kc", "vc", "ks", "vs", "ptr", "ind")]
        with pytest.raises(err):
            idx.idx_attend(*base, a["seen"], 8, **more)
        with pytest.raises(err):
            idx.idx_attend_prefill(*base, ptr, a["seen"], 8, **more)
    with pytest.raises(TypeError):
        idx.idx_attend(q, *d, seen, 8, ids=torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        idx.idx_attend(q, *d, seen, 8, ids=i32(np.zeros((3, 2))))
    with pytest.raises(ValueError):
        idx.idx_attend_prefill(q, *d, i32([0, 2]), seen, 8)
    for kw in (dict(softcap=-1.0), dict(scale=float("nan")), dict(max_pages=0)):
        with pytest.raises(idx.IdxError) as e:
            idx.idx_attend(q, *d, seen, kw.pop("max_pages", 8), **kw)
        assert e.value.status == -1
    x = torch.zeros(2, 2, 128, device="cuda")
    for err, k, v, slots in ((ValueError, x[:1], x, seen), (TypeError, x.half(), x.half(), seen),
                             (ValueError, x, x.bfloat16(), seen), (TypeError, x, x, seen.long()),
                             (ValueError, x.transpose(0, 1), x, seen)):
        with pytest.raises(err):
            idx.idx_cache_write(k, v, slots, *d[:4])
    with pytest.raises(TypeError):
        idx.idx_page_tables(seen.long(), seen, i32(np.zeros((2, 3))), seen, seen, 4)
    with pytest.raises(ValueError):
        idx.idx_page_tables(seen, seen, i32(np.zeros((3, 3))), seen, seen, 4)
