"""Rotary positions on the GPU against the CPU oracle (angles from whole numbers), within
the bound of the header: 2^-21 |factor| (|a| + |b|), and one rounding to the dtype."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache4 as c4

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def rows(rng, n, heads, dtype):
    return torch.from_numpy(rng.standard_normal((n, heads, 128)).astype(np.float32)).to(dtype)


def unsigned(turns):
    return [t % 2 ** 64 for t in turns.cpu().tolist()]


def check(got, x, tok_len, turns, first, adjacent, inverse, factor, dtype, kept=None):
    """got (on the GPU) against x (on the CPU); rows without a token are `kept`."""
    tok_len = np.asarray(tok_len)
    live = tok_len > 0
    x64 = x.double().numpy()
    want = x64.copy()
    want[live] = c4.turned(x64[live], tok_len[live].astype(np.int64) - 1, unsigned(turns), first,
                           adjacent, inverse, float(np.float32(factor)))
    got = got.double().cpu().numpy()
    pairs = len(turns)
    i = np.arange(pairs)
    a, b = (first + 2 * i, first + 2 * i + 1) if adjacent else (first + i, first + pairs + i)
    room = np.zeros_like(x64)
    room[..., a] = room[..., b] = (np.abs(x64[..., a]) + np.abs(x64[..., b])) * abs(factor) * 2.0 ** -21
    tol = room + HALF_STEP[dtype] * (np.abs(want) + room)
    rest = np.setdiff1d(np.arange(128), np.concatenate([a, b]))
    tol[..., rest] = 0
    err = np.abs(got - want)
    bad = np.argwhere(~(err <= tol) & live[:, None, None])
    assert bad.size == 0, (bad[0], got[tuple(bad[0])], want[tuple(bad[0])])
    if kept is not None:
        assert (got[~live] == kept).all()
    return float((err[live] / np.maximum(tol[live], 1e-300)).max()) if live.any() else 0.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("rot,first", [(128, 0), (64, 0), (64, 64), (16, 8), (96, 24), (112, 16),
                                       (48, 0)])
def test_rope_parts_and_layouts(rot, first, adjacent, dtype):
    rng = np.random.default_rng(rot + first)
    turns = idx.idx_rope_table(rot)
    for n, Hq, Hkv in ((1, 1, 1), (5, 7, 3), (33, 16, 4)):
        q, k = rows(rng, n, Hq, dtype), rows(rng, n, Hkv, dtype)
        tok_len = rng.integers(1, 70000, n)
        for inverse, factor in ((False, 1.0), (True, 1.2)):
            say(f"[rope] {rot}@{first} adjacent={adjacent} {dtype} n={n} inverse={inverse}")
            qo, ko = idx.idx_rope(q.cuda(), k.cuda(), i32(tok_len), turns, first=first,
                                  interleaved=adjacent, inverse=inverse, factor=factor)
            for got, x in ((qo, q), (ko, k)):
                check(got, x, tok_len, turns, first, adjacent, inverse, factor, dtype)


@pytest.mark.parametrize("n", [1, 2, 3, 2047, 2048, 2049, 4099, 5002])
def test_rope_many_tokens(n):
    rng = np.random.default_rng(n)
    q, k = rows(rng, n, 3, torch.bfloat16), rows(rng, n, 1, torch.bfloat16)
    tok_len = rng.integers(-3, 200000, n)
    turns = idx.idx_rope_table(128, base=5e5, kind="by_index", stretch=8.0)
    qo, ko = torch.full(q.shape, 7.0, dtype=q.dtype).cuda(), torch.full(k.shape, 7.0, dtype=k.dtype).cuda()
    idx.idx_rope(q.cuda(), k.cuda(), i32(tok_len), turns, q_out=qo, k_out=ko)
    check(qo, q, tok_len, turns, 0, False, False, 1.0, q.dtype, kept=7.0)
    check(ko, k, tok_len, turns, 0, False, False, 1.0, q.dtype, kept=7.0)


def test_rope_far_positions_and_any_frequency():
    """Angles lose nothing however far the position is; frequencies of any sign."""
    rng = np.random.default_rng(3)
    tok_len = np.array([1, 2, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31 - 7, 123456789, 0])
    freq = np.concatenate([rng.uniform(-4, 4, 60), [0.0, 1e-12, 4.0, -1e-6]])
    turns = idx.idx_rope_turns(freq)
    q = rows(rng, len(tok_len), 2, torch.float32)
    out = q.cuda()
    idx.idx_rope(out, None, i32(tok_len), turns, q_out=out)
    worst = check(out, q, tok_len, turns, 0, False, False, 1.0, q.dtype)
    say(f"[rope] far positions: {worst:.2f} of the bound")
    assert (out[-1].cpu() == q[-1]).all()  # no token: as it was


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_in_place_rows_of_a_projection(adjacent):
    """Queries and keys as views of one row; the values beside them, and the dims outside
    the turned part, are not touched."""
    rng = np.random.default_rng(4)
    n, Hq, Hkv = 21, 6, 2
    x = rows(rng, n, Hq + 2 * Hkv, torch.bfloat16)
    tok_len = rng.integers(0, 3000, n)
    turns = idx.idx_rope_table(32)
    want_q, want_k = idx.idx_rope(x[:, :Hq].cuda().contiguous(),
                                  x[:, Hq:Hq + Hkv].cuda().contiguous(), i32(tok_len), turns,
                                  first=40, interleaved=adjacent)
    y = x.cuda()
    q, k = y[:, :Hq], y[:, Hq:Hq + Hkv]
    out = idx.idx_rope(q, k, i32(tok_len), turns, first=40, interleaved=adjacent, q_out=q, k_out=k)
    assert out[0] is q and out[1] is k
    live = torch.from_numpy(tok_len > 0).cuda()
    assert (q[live] == want_q[live]).all() and (k[live] == want_k[live]).all()
    assert (y[~live] == x.cuda()[~live]).all()
    assert (y[:, Hq + Hkv:] == x.cuda()[:, Hq + Hkv:]).all()


def test_rope_inverse_is_the_gradient_and_undoes_a_turn():
    rng = np.random.default_rng(5)
    n = 9
    q, g = rows(rng, n, 2, torch.float32), rows(rng, n, 2, torch.float32)
    tok_len = i32(rng.integers(1, 5000, n))
    turns = idx.idx_rope_table(64)
    kw = dict(first=32, factor=1.5)
    turn = lambda x, **more: idx.idx_rope(x.cuda(), None, tok_len, turns, **kw, **more)[0]  # noqa: E731
    # sum(turn(x) * g) is linear in x: its gradient in any direction d, from a difference
    d = rows(rng, n, 2, torch.float32)
    diff = ((turn(q + d) - turn(q)).double() * g.cuda()).sum()
    grad = (turn(g, inverse=True).double() * d.cuda()).sum()
    # 2304 products of values around 1, each side off by a few 2^-22 of them
    assert abs(float(diff - grad)) < 2304 * 2.0 ** -17
    back = idx.idx_rope(turn(q), None, tok_len, turns, first=32, inverse=True, factor=1 / 1.5)[0]
    assert float((back - q.cuda()).abs().max()) < 2.0 ** -17


def test_rope_without_rows_special_values_and_refusals():
    turns = idx.idx_rope_table(128)
    q = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    assert idx.idx_rope(q, None, i32([]), turns)[0].shape == q.shape
    q = torch.ones(2, 4, 128, device="cuda")
    q[0, 1, 5] = torch.nan
    q[0, 2, 69] = torch.inf
    out = idx.idx_rope(q, None, i32([3, 3]), turns)[0]
    nan = torch.isnan(out[0])
    assert nan[1, 5] and nan[1, 69] and int(nan.sum()) == 2
    assert torch.isinf(out[0, 2, [5, 69]]).all() and torch.isfinite(out[1]).all()
    k, t = torch.ones(2, 1, 128, device="cuda"), i32([1, 1])
    for bad in (lambda: idx.idx_rope(q, k[:1], t, turns), lambda: idx.idx_rope(q, k, t[:1], turns),
                lambda: idx.idx_rope(q, k, t, turns.cpu()),
                lambda: idx.idx_rope(q, k, t, turns.view(2, -1)),
                lambda: idx.idx_rope(q, k, t, turns, q_out=q[:1]),
                lambda: idx.idx_rope(q, None, t, turns, k_out=k),
                lambda: idx.idx_rope(q.transpose(0, 1), None, i32([1] * 4), turns)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: idx.idx_rope(q, k.bfloat16(), t, turns),
                lambda: idx.idx_rope(q.half(), None, t, turns)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(idx.IdxError):
        idx.idx_rope(q, k, t, turns, first=8)
    with pytest.raises(idx.IdxError):
        idx.idx_rope(q, k, t, turns[:10])
