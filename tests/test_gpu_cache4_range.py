"""Attention over the 4-bit cache at the ends of the value scales' range, against the float64
oracle. The bound is the one of tests/cache4_helpers.py with the largest product of a weight
and its unit's largest scale where that one has their sum:
  - a weight is rounded to fp16, 2^-11 of itself or 2^-25 where it is small, and its product
    with a scale by 2^-25 again, in units where the row's largest such product is 2^9 or more;
    a code is at most 6: 6 * 2^-33 of the largest product for each token;
  - the sum of weights loses no more than 2^-35 of the largest weight for each token, far
    below its 2^-24 a token of rounding.
"""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache4 as c4
from oracle import paged_cache as pc
from tests.cache4_helpers import Cache4
from tests.cache_helpers import U

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def expected(c, q, b, seen, scale, h=0, cap=0.0, slope=0.0):
    """One row and query head q [128]: its output and how far off it may be."""
    k, v, there, top = c.tokens(b, h)
    out, absum, mag = pc.attend(q, k, v, there, seen, None, c.page, scale, cap, slope)
    n = min(seen, len(k))
    x = k[:n] @ q * scale
    if cap:
        x = cap * np.tanh(x / cap)
    x -= slope * (seen - 1 - np.arange(n))
    w = np.exp(x - x.max())
    w /= w.sum()
    unit = np.pad(top[:n], (0, -n % 16)).reshape(-1, 16).max(1).repeat(16)[:n]
    e = 160 * U * mag + 16 * U * (cap + slope * n) + 4 * U
    weights = 2 * np.expm1(e) + 2.0 ** -11 + (2 * n + 8) * U
    off = absum * weights + n * 6 * 2.0 ** -33 * float((w * unit).max())
    return out, off + (np.abs(out) + off) * 2.0 ** -8 + 2.0 ** -130


def check(name, out, c, q, seen, scale):
    """out [rows, Hq, 128], all rows and heads of request 0 with the query q [128] and the
    visible length seen."""
    want, tol = expected(c, q.double().numpy(), 0, seen, float(np.float32(scale)))
    err = (out.double().cpu().numpy() - want) / tol
    print(f"[range4] {name}: {np.abs(err).max():.2f} of the bound", flush=True)
    sys.stdout.flush()
    bad = np.argwhere(~(np.abs(err) <= 1))
    assert bad.size == 0, (name, bad[0], float(out[tuple(bad[0])]), want[bad[0][-1]], tol[bad[0][-1]])


def forms(c, q, n, scale):
    """The outputs of each kernel and cut for rows that see the first n tokens: single rows,
    cut and whole, few packed rows, and prompts whose rows see all tiles whole, or, with a
    shorter row in each workgroup, in part."""
    args, bound = c.device(), c.max_pages
    rows = lambda r, h: q.bfloat16().cuda().expand(r, h, 128).contiguous()  # noqa: E731
    kw = dict(scale=scale)
    for r, h in ((1, 4), (1, 20), (512, 1)):
        cut = idx.idx_attend4_workspace_bytes(r, h, 1, bound) > 0
        out = idx.idx_attend4(rows(r, h), *args, i32([n] * r), bound, row_req=i32([0] * r), **kw)
        yield f"{r} rows of {h} heads{', cut' if cut else ''}", out
    for t, h in ((3, 4), (130, 2), (512, 64)):
        cut = idx.idx_attend4_prefill_workspace_bytes(t, 1, h, 1, bound) > 0
        seen = np.full(t, n)
        name = f"{t} tokens of {h} heads{', cut' if cut else ''}"
        out = idx.idx_attend4_prefill(rows(t, h), *args, i32([0, t]), i32(seen), bound, **kw)
        yield name, out
        seen[1::4] = 1
        out = idx.idx_attend4_prefill(rows(t, h), *args, i32([0, t]), i32(seen), bound, **kw)
        yield name + " among short ones", out[torch.from_numpy(seen == n).cuda()]


def plain_cache(n):
    """Keys of zeros, values of ones."""
    c = Cache4(1, [n], 1, 16)
    c.k[:], c.ks[:] = 0, 127
    c.v[:], c.vs[:] = 2, 127
    return c


def put(c, t, name, codes, scale):
    """Token t of request 0: codes [128] and scale bytes [4]."""
    page, o = c.pages(0)[t // 16], t % 16
    if name == "k":
        c.k[page, 0, o], c.ks[page, 0, o] = codes, scale
    else:
        c.v[page, 0, :, o], c.vs[page, 0, :, o] = codes, scale


@pytest.mark.parametrize("gap", [7.0, 12.0, 16.5, 40.0])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("n", [200, 1100, 9000])
def test_many_least_scales_beside_one_largest(n, at, gap):
    """Tokens of the least value scale, and one of the largest whose weight is 2^gap times
    theirs: the largest product of weight and scale moves by 2^(120 + gap), the weights' sum
    does not lose what it held, whichever comes first."""
    c = plain_cache(n)
    c.vs[:] = 67
    key = np.zeros(128, np.uint8)
    key[0] = 2
    t = {"first": 0, "middle": n // 2, "last": n - 1}[at]
    put(c, t, "k", key, 127)
    put(c, t, "v", 2, 187)
    c.poison_tails()
    q = torch.zeros(128)
    q[0] = gap
    for name, out in forms(c, q, n, np.log(2)):
        check(f"{n} tokens, {at}, 2^{gap}: {name}", out, c, q, n, np.log(2))


@pytest.mark.parametrize("code", [1, 3, 7, 9])
@pytest.mark.parametrize("below", [20, 22, 23, 24])
def test_blocks_far_below_their_units_largest_scale(below, code):
    """A block of dims whose scales lie 2^below under those of another block of the same
    tokens, codes of one sign."""
    n = 400
    c = plain_cache(n)
    c.v[:, :, 64:96] = code
    c.vs[:, :, 2] = 127 - below
    c.poison_tails()
    q = torch.zeros(128)
    for name, out in forms(c, q, n, 1.0):
        check(f"2^-{below} of code {code}: {name}", out, c, q, n, 1.0)
        want = c4.e2m1_values()[code] * 2.0 ** -below
        assert float((out[..., 64:96].double() / want - 1).abs().max()) < 2.0 ** -6


@pytest.mark.parametrize("below", [10, 17, 24])
def test_tokens_far_below_their_units_largest_scale(below):
    """All tokens of a unit but one have scales 2^below under it, and the weight."""
    n = 400
    c = plain_cache(n)
    key = np.zeros(128, np.uint8)
    key[0] = 2
    for t in range(n):
        if t % 16 != 5:
            put(c, t, "k", key, 127)
            put(c, t, "v", 3, 127 - below)
    c.poison_tails()
    q = torch.zeros(128)
    q[0] = float(below)
    for name, out in forms(c, q, n, np.log(2)):
        check(f"2^-{below}: {name}", out, c, q, n, np.log(2))


def test_largest_queries_and_keys():
    """|q| times the largest key scale up to 2^117, key scales from 2^-125 to 2^125: the
    products and their sums stay within fp32."""
    n = 150
    rng = np.random.default_rng(6)
    for exp, low, high in ((57, 0, 60), (117, -125, 0), (-8, 100, 125), (117, 0, 0)):
        c = plain_cache(n)
        c.k[:] = rng.integers(0, 16, c.k.shape)
        c.k[c.pages(0)[1]] = 7                 # keys of 6 everywhere, in the largest scale
        c.ks[:] = 127 + rng.integers(low, high + 1, c.ks.shape)
        c.ks[c.pages(0)[1]] = 127 + high
        c.v[:] = rng.integers(0, 16, c.v.shape)
        c.poison_tails()
        for sign in (np.ones(128), rng.choice([-1.0, 1.0], 128)):
            q = torch.from_numpy(sign * 2.0 ** exp).float()
            scale = 2.0 ** -(exp + high) / 256
            for name, out in forms(c, q, n, scale):
                check(f"q 2^{exp}, keys 2^{low}..2^{high}: {name}", out, c, q, n, scale)


def far_apart(seed, n):
    """Scales 2^0 to 2^-24 of their unit's largest, a block 2^-20 or less of it; its codes are of
    one sign, so that its outputs are as large as they can be."""
    c = Cache4(seed, [n], 2, 16)
    c.vs[:] = 127 - c.rng.integers(0, 25, c.vs.shape)
    c.vs[:, :, 2] = 127 - c.rng.integers(20, 25, c.vs[:, :, 2].shape)
    c.vs[:, :, 0, 0] = 127
    c.v[:, :, 64:96] &= 7
    c.v[:, :, 64:96] |= 1
    c.poison_tails()
    return c


def rows_within(name, c, q, out, seen):
    """Rows out [n, Hq, 128] of request 0, each with its own query and length. The bound sees
    the small block: zeros in its place would be outside."""
    out, q = out.double().cpu().numpy(), q.double().numpy()
    worst, blind, count = 0.0, 0, 0
    for r in range(len(out)):
        for hq in range(out.shape[1]):
            want, tol = expected(c, q[r, hq], 0, int(seen[r]), float(np.float32(128 ** -0.5)),
                                 hq * 2 // out.shape[1])
            err = np.abs(out[r, hq] - want) / tol
            assert (err <= 1).all(), (name, r, hq, int(err.argmax()), float(err.max()))
            worst = max(worst, float(err.max()))
            blind += int((np.abs(want[64:96]) <= tol[64:96]).sum())
            count += 32
    print(f"[range4] {name}: {worst:.2f} of the bound, {blind} of {count} unseen", flush=True)
    assert blind < count / 50


@pytest.mark.parametrize("Hq", [2, 8, 40])
@pytest.mark.parametrize("n", [16, 47, 64, 90])
def test_scales_far_apart_single_rows(n, Hq):
    c = far_apart(n, n)
    q = torch.from_numpy(c.rng.standard_normal((4, Hq, 128))).bfloat16()
    seen = np.array([n, n, max(1, n - 9), n - n % 16])
    out = idx.idx_attend4(q.cuda(), *c.device(), i32(seen), c.max_pages, row_req=i32([0] * 4))
    rows_within(f"{n} tokens, {Hq} heads", c, q, out, seen)


@pytest.mark.parametrize("shape", ["few", "whole", "mixed", "causal"])
def test_scales_far_apart_packed_rows(shape):
    """Few packed rows; a prompt whose rows see all of it, whose workgroups hold shorter rows
    too, or whose rows each see one token more."""
    n = 128
    t = 5 if shape == "few" else 110
    c = far_apart(t, n)
    q = torch.from_numpy(c.rng.standard_normal((t, 4, 128))).bfloat16()
    seen = np.full(t, n)
    if shape == "mixed":
        seen[::3] = c.rng.integers(1, n, len(seen[::3]))
    if shape in ("causal", "few"):
        seen = np.arange(n - t, n) + 1
    out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([0, t]), i32(seen), c.max_pages)
    step = slice(None, None, 1 + t // 30)
    rows_within(shape, c, q[step], out[step], seen[step])


def test_other_rows_lengths_leave_a_row_within_its_bound():
    """A prompt's row that keeps its own length while the others' change: the kernel may take
    another way through its tiles; both results are within the bound."""
    n, t = 128, 120
    c = far_apart(3, n)
    q = torch.from_numpy(c.rng.standard_normal((t, 4, 128))).bfloat16()
    keep = np.arange(0, t, 4)
    for other in (n, n - 1, 70, 1, 0):
        seen = np.full(t, other)
        seen[keep] = n
        out = idx.idx_attend4_prefill(q.cuda(), *c.device(), i32([0, t]), i32(seen), c.max_pages)
        rows_within(f"others see {other}", c, q[keep], out[torch.from_numpy(keep).cuda()],
                    seen[keep])


@pytest.mark.parametrize("cap,biased", [(0.0, False), (60.0, False), (300.0, False), (0.0, True)])
@pytest.mark.parametrize("n,t,Hq", [(90, 4, 8), (700, 6, 40), (700, 140, 4), (3000, 130, 8)])
def test_pages_of_any_scales(n, t, Hq, cap, biased):
    """Each page with value scales of its own anywhere in the range, and scores far apart: rows
    one by one, and packed, each seeing a token more than the one before."""
    c = Cache4(n + t, [n], 2, 16)
    c.vs[:] = 127 + c.rng.integers(-57, 58, (c.n_pages, 2, 1, 1)) + c.rng.integers(-3, 4, c.vs.shape)
    c.poison_tails()
    q = torch.from_numpy(c.rng.standard_normal((t, Hq, 128)) * 8).bfloat16()
    slopes = np.exp2(-8 * np.arange(1, Hq + 1) / Hq).astype(np.float32) if biased else None
    kw = dict(softcap=cap, slopes=None if slopes is None else torch.from_numpy(slopes).cuda())
    seen = np.arange(n - t, n) + 1
    args = (q.cuda(), *c.device())
    outs = {"rows": idx.idx_attend4(*args, i32(seen), c.max_pages, row_req=i32([0] * t), **kw),
            "packed": idx.idx_attend4_prefill(*args, i32([0, t]), i32(seen), c.max_pages, **kw)}
    for name, out in outs.items():
        out = out.double().cpu().numpy()
        for r in sorted({0, 1, t // 2, t - 1}):
            for hq in range(0, Hq, 1 + Hq // 8):
                want, tol = expected(c, q[r, hq].double().numpy(), 0, int(seen[r]),
                                     float(np.float32(128 ** -0.5)), hq * 2 // Hq, cap,
                                     0.0 if slopes is None else float(slopes[hq]))
                err = np.abs(out[r, hq] - want) / tol
                assert (err <= 1).all(), (name, r, hq, int(err.argmax()), float(err.max()))
