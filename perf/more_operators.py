"""Cases of the paged 4-bit cache operators and of rotary positions: rotation of queries
and keys (and of their gradients, back), the quantising write of a 4-bit cache, reading
it back, attention of single tokens over all or the selected pages of it, and attention
of packed prompt tokens.

`listed()` names the cases, `draw(rng)` gives another one of the same ranges,
`prepare(case, seed)` makes what a serving loop holds before the call, `run(state)`
is one pass: in elementary torch operations (float32 inside, rounded once at the end),
or through the library's entry points when `own` is true. `exact(case, seed)` is the
definition in float64. `work(case)` counts the bytes and operations that a pass cannot
do without.

Layouts (page = `page` tokens of one request, D = 128; a code is e2m1: sign, 2 exponent
bits, 1 fraction bit; a scale is e8m0, 2^(byte - 127), byte 255 NaN, one for each token,
head and 32 dims):
  k_cache [pages, Hkv, page, D/2]   byte j of a token: dims 2j (low four bits), 2j + 1
  v_cache [pages, Hkv, D, page/2]   byte j of a dim: tokens 2j (low four bits), 2j + 1
  k_scale [pages, Hkv, page, 4]     v_scale [pages, Hkv, 4, page]
  request b's pages: kv_indices[kv_indptr[b] : kv_indptr[b+1]]
Rotary positions: pair i of a row at position p turns by the angle p * inv_freq[i]; the
call's table holds inv_freq / 2 pi in units of 2^-64 of a turn.
"""
import math

import torch

own = False

D = 128
BLOCK = 32                     # dims of one scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIN_EXP, MAX_EXP = -60, 60     # of the scales that the write gives


# ------------------------------------------------------------------- cases

def listed():
    return [
        # rotation in one decode step: a few microseconds of work
        {"name": "rope_decode", "op": "rope", "B": 128, "Hq": 16, "Hkv": 4, "lo": 8192,
         "hi": 32768, "new": 1, "rot": 128, "first": 0, "interleaved": False, "inverse": False,
         "stretch": 1.0, "dtype": "bf16"},
        # two whole prompts, positions stretched for long contexts
        {"name": "rope_prompt", "op": "rope", "B": 2, "Hq": 32, "Hkv": 8, "lo": 8009, "hi": 8192,
         "new": 8192, "rot": 128, "first": 0, "interleaved": False, "inverse": False,
         "stretch": 8.0, "dtype": "bf16"},
        # gradients turned back, far positions, adjacent pairs in the heads' second half
        {"name": "rope_back", "op": "rope", "B": 3, "Hq": 16, "Hkv": 2, "lo": 30512,
         "hi": 131072, "new": 1367, "rot": 64, "first": 64, "interleaved": True, "inverse": True,
         "stretch": 1.0, "dtype": "f32"},
        # one decode step's keys and values, each into a part-filled page (what a write leaves
        # in 4 bits is returned as the values it stands for: read back, within the pass)
        {"name": "write4_decode", "op": "write", "B": 128, "Hkv": 4, "lo": 2048, "hi": 8192,
         "new": 1, "page": 16, "dtype": "bf16"},
        # chunks of prompts that start and end inside pages
        {"name": "write4_prompt", "op": "write", "B": 4, "Hkv": 8, "lo": 5, "hi": 16999,
         "new": 4099, "page": 16, "dtype": "bf16"},
        # the last tokens of some requests, read back (a window that moves on)
        {"name": "read4_window", "op": "read", "B": 7, "Hkv": 4, "lo": 300, "hi": 2777,
         "new": 129, "page": 16, "dtype": "bf16"},
        # a long prefix, read back whole
        {"name": "read4_prefix", "op": "read", "B": 2, "Hkv": 8, "lo": 30512, "hi": 32768,
         "new": 32768, "page": 16, "dtype": "bf16"},
        # the smallest decode call: one request, a short context
        {"name": "attend4_one", "op": "attend", "B": 1, "T": 1, "Hq": 16, "Hkv": 4, "lo": 3999,
         "hi": 3999, "K": 0, "page": 16, "softcap": 0.0, "slopes": False},
        # dense decode of four ragged requests up to 131072 tokens
        {"name": "attend4_dense_ragged", "op": "attend", "B": 4, "T": 1, "Hq": 32, "Hkv": 8,
         "lo": 4096, "hi": 131072, "K": 0, "page": 16, "softcap": 0.0, "slopes": False},
        # the indexer's GQA decode batch: each request attends its 256 selected pages
        {"name": "attend4_selected", "op": "attend", "B": 128, "T": 1, "Hq": 16, "Hkv": 4,
         "lo": 8192, "hi": 32768, "K": 256, "page": 16, "softcap": 0.0, "slopes": False},
        # a few tokens for each of some requests (drafted tokens), capped scores
        {"name": "prefill4_few", "op": "prefill", "B": 4, "Hq": 16, "Hkv": 4, "lo": 900,
         "hi": 2777, "new": 5, "page": 16, "softcap": 30.0, "slopes": False},
        # whole long prompts
        {"name": "prefill4_long", "op": "prefill", "B": 2, "Hq": 32, "Hkv": 8, "lo": 8009,
         "hi": 8192, "new": 8192, "page": 16, "softcap": 0.0, "slopes": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend", "prefill", "prefill"])
    page = rng.choice([16, 16, 32, 64])
    lo = _log(rng, 1, 30000)
    c = {"op": op, "lo": lo, "hi": _log(rng, lo, 131072)}
    heads = rng.choice([(4, 1), (8, 8), (16, 1), (16, 2), (16, 4), (32, 4), (32, 8), (20, 4),
                        (64, 2), (7, 7), (6, 2)])
    if op == "rope":
        rot = rng.choice([16, 32, 64, 96, 112, 128, 128, 128])
        c |= {"B": _log(rng, 1, 256), "Hq": heads[0], "Hkv": heads[1], "new": _log(rng, 1, 8192),
              "rot": rot, "first": rng.choice([0, 128 - rot]),
              "interleaved": rng.random() < 0.4, "inverse": rng.random() < 0.3,
              "stretch": rng.choice([1.0, 1.0, 2.5, 8.0]),
              "dtype": rng.choice(["bf16", "bf16", "f32"])}
        return c
    c["page"] = page
    if op in ("write", "read"):
        c |= {"B": _log(rng, 1, 512), "Hkv": heads[1], "new": _log(rng, 1, 32768),
              "dtype": rng.choice(["bf16", "bf16", "f32"])}
        return c
    c |= {"Hq": heads[0], "Hkv": heads[1], "softcap": rng.choice([0.0, 0.0, 30.0]),
          "slopes": rng.random() < 0.25}
    if op == "attend":
        c |= {"B": _log(rng, 1, 256), "T": rng.choice([1, 1, 1, _log(rng, 2, 512)])}
        c["K"] = _log(rng, 1, 512) if c["T"] > 1 else rng.choice([0, _log(rng, 1, 512)])
    else:
        c |= {"B": _log(rng, 1, 64), "new": _log(rng, 1, 8192)}
    return c


def _cost(c):
    """Values that the elementary form makes for the case (its time and memory)."""
    if c["op"] == "rope":
        return sum(_news(c)) * (c["Hq"] + c["Hkv"]) * (2 if c["dtype"] == "f32" else 1)
    if c["op"] in ("write", "read"):
        return (sum(_lengths(c)) + 8 * sum(_news(c))) * c["Hkv"] * D
    if c["op"] == "attend":
        blocks = c["K"] or -(-c["hi"] // c["page"])
        return c["B"] * c["T"] * blocks * c["page"] * (2 * c["Hkv"] * D + 4 * c["Hq"])
    new = min(c["new"], c["hi"])
    return c["B"] * c["hi"] * (2 * c["Hkv"] * D + c["Hq"] * new)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        c = _draw(rng)
        if _cost(c) <= most[c["op"]]:
            return c


def _lengths(c):
    """The requests' lengths (after the step): spread over [lo, hi], in mixed order."""
    lo, hi, n = c["lo"], c["hi"], c["B"]
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 7919) % n) // (n - 1) if n % 7919 else lo for i in range(n)]


def _news(c):
    """Tokens of each request that the step is about: its last ones."""
    return [max(1, min(length, c["new"] - (i % 3))) for i, length in enumerate(_lengths(c))]


def _pages(n, page):
    return -(-n // page)


def work(case):
    c = case
    lens = _lengths(c)
    if c["op"] == "rope":
        n, heads = sum(_news(c)), c["Hq"] + c["Hkv"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * (2 * heads * D * size + 4) + 4 * c["rot"],
                "flops": 3 * n * heads * c["rot"]}
    if c["op"] in ("write", "read"):
        n = sum(_news(c))
        size = 4 if c["dtype"] == "f32" else 2
        held = n * 2 * c["Hkv"] * (D // 2 + D // BLOCK)
        rows = n * 2 * c["Hkv"] * D * size
        # the write's values come back as the read call gives them
        return {"bytes": (held + rows + 4 * n) * (2 if c["op"] == "write" else 1), "flops": 0}
    if c["op"] == "attend":
        seen, once = 0, 0
        for a in lens:
            rows = [a - c["T"] + 1 + t for t in range(c["T"])]
            rows = [max(0, min(r, c["K"] * c["page"] - c["page"] + ((r - 1) % c["page"]) + 1))
                    if c["K"] else max(0, r) for r in rows]
            seen += sum(rows)
            once += min(sum(rows), a)
        n = c["B"] * c["T"]
    else:
        seen = sum(sum(range(a - k + 1, a + 1)) for a, k in zip(lens, _news(c)))
        once = sum(lens)
        n = sum(_news(c))
    return {"bytes": once * c["Hkv"] * 2 * (D // 2 + D // BLOCK) + 4 * n * c["Hq"] * D
            + (4 * n * c["K"] if c["op"] == "attend" else 0),
            "flops": 4 * D * c["Hq"] * seen}


# ------------------------------------------------------------------- inputs

def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _codes(shape, gen, dev):
    """Two codes a byte, of normal values with a deviation of 2 scales."""
    x = torch.randn(*shape, 2, generator=gen, device=dev) * 2
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    c = torch.bucketize(x.abs(), edges, out_int32=True).to(torch.uint8)
    c |= (x < 0).to(torch.uint8) << 3
    return c[..., 0] | c[..., 1] << 4


def _inv_freq(c, dev):
    """The frequencies of the rotated pairs; with a stretch, those of long wavelengths
    (under one turn in 8192 tokens) are divided by it, those of short ones (32 turns or
    more) kept, the others blended."""
    f = 10000.0 ** (-2.0 * torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev) / c["rot"])
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return f * (keep + (1 - keep) / c["stretch"])


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens = _lengths(c)
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    if c["op"] == "rope":
        news = _news(c)
        n, Hq, H = sum(news), c["Hq"], c["Hkv"]
        # rows of a fused projection: a token's queries, keys and values lie in one row
        x = torch.randn(n, Hq + 2 * H, D, generator=gen, device=dev)
        x *= torch.exp2(torch.randn(n, 1, 1, generator=gen, device=dev))
        x = x.to(dt)
        f = _inv_freq(c, dev)
        return {"case": c, "q": x[:, :Hq], "k": x[:, Hq:Hq + H], "inv_freq": f,
                "turns": torch.round(f / (2 * math.pi) * 2.0 ** 64).to(torch.int64),
                "factor": 1.0 if c["stretch"] == 1.0 else 0.1 * math.log(c["stretch"]) + 1.0,
                "tok_len": torch.cat([torch.arange(a - k + 1, a + 1, device=dev)
                                      for a, k in zip(lens, news)]).int()}
    page = c["page"]
    blocks = [_pages(a, page) for a in lens]
    n_pages = sum(blocks) + 7
    pool = torch.randperm(n_pages, generator=gen, device=dev).int()
    kv_indices = pool[:sum(blocks)].contiguous()
    indptr = _offsets(blocks)
    H = c["Hkv"]
    s = {"case": c, "kc": _codes((n_pages, H, page, D // 2), gen, dev),
         "vc": _codes((n_pages, H, D, page // 2), gen, dev)}
    for name, shape in (("ks", (page, D // BLOCK)), ("vs", (D // BLOCK, page))):
        e = torch.randint(-4, 0, (n_pages, H, *shape), generator=gen, device=dev)
        s[name] = (e + 127).to(torch.uint8)
    s |= {"kv_indices": kv_indices, "kv_indptr": _ints(indptr, dev), "max_pages": max(blocks)}
    if c["op"] in ("write", "read"):
        news = _news(c)
        pos = torch.cat([torch.arange(a - k, a, device=dev) for a, k in zip(lens, news)])
        req = torch.repeat_interleave(torch.arange(c["B"], device=dev),
                                      torch.tensor(news, device=dev))
        first = torch.tensor(indptr[:-1], device=dev)
        pages = kv_indices[first[req] + pos // page].long()
        s["slots"] = (pages * page + pos % page).int()
        s["dtype"] = dt
        if c["op"] == "write":
            # rows of a fused projection, some channels larger than the others
            x = torch.randn(len(pos), 2, H, D, generator=gen, device=dev)
            x *= torch.exp2(torch.randn(len(pos), 2, 1, 1, generator=gen, device=dev))
            x *= torch.exp2(torch.randn(2, H, D, generator=gen, device=dev))
            x = x.to(dt)
            s["k"], s["v"] = x[:, 0], x[:, 1]
        return s
    Hq = c["Hq"]
    s["scale"] = D ** -0.5
    s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq).float()
                   if c["slopes"] else None)
    if c["op"] == "attend":
        T = c["T"]
        n = c["B"] * T
        seen = [max(0, a - T + 1 + t) for a in lens for t in range(T)]
        s["kv_len"] = _ints(seen, dev)
        s["row_req"] = _ints([b for b in range(c["B"]) for _ in range(T)], dev) if T > 1 else None
        s["ids"] = None
        if c["K"]:
            keys = torch.rand(n, max(max(blocks), c["K"]), generator=gen, device=dev)
            nb = ((s["kv_len"] + page - 1) // page).long()[:, None]
            at = torch.arange(keys.shape[1], device=dev)[None]
            keys = torch.where(at < nb, keys, -1.0)
            keys = torch.where(at == nb - 1, 2.0, keys)  # the token's own page among them
            top = torch.topk(keys, c["K"], dim=1)
            ids = torch.where(top.values < 0, 1 << 30, top.indices)
            ids = ids.sort(dim=1).values  # ascending, then -1, as the selects give them
            s["ids"] = torch.where(ids == 1 << 30, -1, ids).int().contiguous()
    else:
        news = _news(c)
        n = sum(news)
        s["tok_indptr"] = _ints(_offsets(news), dev)
        s["kv_len"] = torch.cat([torch.arange(a - k + 1, a + 1, device=dev)
                                 for a, k in zip(lens, news)]).int()
        s["max_new"] = max(news)
    s["q"] = (1.5 * torch.randn(n, Hq, D, generator=gen, device=dev)).bfloat16()
    return s


# ------------------------------------------------------------------- plain form

def _turned(s, x, cos, sin):
    c = s["case"]
    y = x.float()
    part = y[..., c["first"]:c["first"] + c["rot"]]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    y = torch.cat([y[..., :c["first"]], part, y[..., c["first"] + c["rot"]:]], -1)
    return y.to(x.dtype)


def _plain_rope(s):
    angle = (s["tok_len"].double() - 1)[:, None, None] * s["inv_freq"]  # far positions: 64 bits
    if s["case"]["inverse"]:
        angle = -angle
    cos, sin = (s["factor"] * torch.cos(angle)).float(), (s["factor"] * torch.sin(angle)).float()
    return {"q": _turned(s, s["q"], cos, sin), "k": _turned(s, s["k"], cos, sin)}


def _two_to(e):
    """2^e in float32, e a tensor of whole numbers within the normal range."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _scale_of(amax):
    """Exponent of the smallest power of two s with amax <= 6 s, within the range."""
    m, e = torch.frexp(amax)
    e = e - torch.where(m <= 0.75, 3, 2)  # 6 = 0.75 * 2^3
    return torch.where(amax > 0, e, MIN_EXP).clamp(MIN_EXP, MAX_EXP)


def _code_of(y):
    """The code nearest to y, ties to the even one."""
    a = y.abs()
    c = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
         + (a > 5.0))
    return (c + 8 * (y < 0)).to(torch.uint8)


def _values(byte):
    """The two values of each byte [..., 2], in float32."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=byte.device)
    return t[torch.stack([byte & 15, byte >> 4], -1).int()]


def _put_values(vc, pages, byte, code, keep):
    """Half of each of those bytes of the value cache: the other half is kept."""
    vc[pages, :, :, byte] = vc[pages, :, :, byte] & keep | code


def _plain_write(s):
    page = s["case"]["page"]
    slots = s["slots"].long()
    pages, offs = slots // page, slots % page
    n, H = s["k"].shape[:2]
    k, v = s["k"].float().view(n, H, -1, BLOCK), s["v"].float().view(n, H, -1, BLOCK)
    ke, ve = _scale_of(k.abs().amax(-1)), _scale_of(v.abs().amax(-1))
    kn = _code_of(k / _two_to(ke)[..., None]).view(n, H, D // 2, 2)
    s["kc"][pages, :, offs] = kn[..., 0] | kn[..., 1] << 4
    s["ks"][pages, :, offs] = (ke + 127).to(torch.uint8)
    s["vs"][pages, :, :, offs] = (ve + 127).to(torch.uint8)
    vn = _code_of(v / _two_to(ve)[..., None]).view(n, H, D)
    odd = offs % 2 == 1
    _put_values(s["vc"], pages[~odd], offs[~odd] // 2, vn[~odd], 0xF0)
    _put_values(s["vc"], pages[odd], offs[odd] // 2, vn[odd] << 4, 0x0F)
    return _plain_read(s)


def _plain_read(s):
    page = s["case"]["page"]
    slots = s["slots"].long()
    pages, offs = slots // page, slots % page
    n, H = len(slots), s["case"]["Hkv"]
    k = _values(s["kc"][pages, :, offs]).view(n, H, -1, BLOCK)
    k = k * _two_to(s["ks"][pages, :, offs].int() - 127)[..., None]
    byte = s["vc"][pages, :, :, offs // 2]
    v = _values(byte >> (4 * (offs % 2)).to(torch.uint8)[:, None, None])[..., 0]
    v = v.reshape(n, H, -1, BLOCK) * _two_to(s["vs"][pages, :, :, offs].int() - 127)[..., None]
    return {"k": k.reshape(n, H, D).to(s["dtype"]), "v": v.reshape(n, H, D).to(s["dtype"])}


def _gathered(s, slots, first):
    """Keys, values [rows, Hkv, tokens, D] in float32 of the page slots [rows, n] of
    the page lists that start at `first` [rows]."""
    live = slots >= 0
    last = s["kv_indices"].numel() - 1
    pages = s["kv_indices"][(first[:, None] + slots.clamp(min=0)).clamp(max=last).long()].long()
    R, n = pages.shape
    H, page = s["kc"].shape[1:3]
    k = _values(s["kc"][pages]).view(R, n, H, page, -1, BLOCK)
    k = k * _two_to(s["ks"][pages].int() - 127)[..., None]
    k = k.view(R, n, H, page, D).permute(0, 2, 1, 3, 4).reshape(R, H, n * page, D)
    v = _values(s["vc"][pages]).view(R, n, H, -1, BLOCK, page)
    v = v * _two_to(s["vs"][pages].int() - 127)[:, :, :, :, None]
    v = v.view(R, n, H, D, page).permute(0, 2, 1, 4, 3).reshape(R, H, n * page, D)
    at = slots[:, :, None] * page + torch.arange(page, device=slots.device)
    at = torch.where(live[:, :, None], at, 1 << 30).reshape(R, n * page)
    return k, v, at


def _attention(s, q, k, v, at, seen):
    """q [rows, T, Hq, D], k and v [rows, Hkv, L, D], key positions [rows, L], visible
    lengths [rows, T]; a token that sees nothing gets zeros."""
    c = s["case"]
    R, T, Hq, _ = q.shape
    H = c["Hkv"]
    q = q.float().view(R, T, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(R, H, -1, D)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    x = x.view(R, H, Hq // H, T, -1)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if s["slopes"] is not None:
        far = (seen[:, :, None] - 1 - at[:, None, :]).float()
        x = x - s["slopes"].view(1, H, Hq // H, 1, 1) * far[:, None, None]
    mask = (at[:, None, :] < seen[:, :, None])[:, None, None]
    x = torch.where(mask, x, -torch.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -torch.inf, 0.0, m))
    o = torch.matmul(p.view(R, H, -1, p.shape[-1]), v).view(R, H, Hq // H, T, D)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(R, T, Hq, D).bfloat16()


def _plain_attend(s):
    dev = s["q"].device
    seen = s["kv_len"].long()
    req = (s["row_req"].long() if s["row_req"] is not None
           else torch.arange(seen.numel(), device=dev))
    slots = s["ids"]
    if slots is None:
        slots = torch.arange(s["max_pages"], device=dev)[None]
        slots = torch.where(slots * s["case"]["page"] < seen[:, None], slots, -1)
    k, v, at = _gathered(s, slots.long(), s["kv_indptr"].long()[req])
    return {"out": _attention(s, s["q"][:, None], k, v, at, seen[:, None])[:, 0]}


def _plain_prefill(s):
    dev, B = s["q"].device, s["case"]["B"]
    ptr = s["tok_indptr"].long()
    t = torch.arange(s["max_new"], device=dev)
    there = t[None] < (ptr[1:] - ptr[:-1])[:, None]
    row = torch.where(there, ptr[:-1, None] + t, 0)      # padded to [B, max_new]
    seen = torch.where(there, s["kv_len"][row].long(), 0)
    slots = torch.arange(s["max_pages"], device=dev)[None].expand(B, -1)
    slots = torch.where(slots * s["case"]["page"] < seen.amax(1, keepdim=True), slots, -1)
    k, v, at = _gathered(s, slots, s["kv_indptr"].long()[:-1])
    o = _attention(s, s["q"][row], k, v, at, seen)
    out = torch.empty_like(s["q"])
    out[row[there]] = o[there]
    return {"out": out}


# ------------------------------------------------------------------- the calls

def _own_rope(s):
    import block_scoring_top_amd as idx
    c = s["case"]
    q, k = idx.idx_rope(s["q"], s["k"], s["tok_len"], s["turns"], first=c["first"],
                        interleaved=c["interleaved"], inverse=c["inverse"], factor=s["factor"])
    return {"q": q, "k": k}


def _own_write(s):
    import block_scoring_top_amd as idx
    idx.idx_cache4_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
    return _own_read(s)


def _own_read(s):
    import block_scoring_top_amd as idx
    k, v = idx.idx_cache4_read(s["slots"], s["kc"], s["vc"], s["ks"], s["vs"], dtype=s["dtype"])
    return {"k": k, "v": v}


def _own_attend(s):
    import block_scoring_top_amd as idx
    return {"out": idx.idx_attend4(
        s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["kv_indptr"], s["kv_indices"],
        s["kv_len"], s["max_pages"], row_req=s["row_req"], ids=s["ids"], scale=s["scale"],
        softcap=s["case"]["softcap"], slopes=s["slopes"])}


def _own_prefill(s):
    import block_scoring_top_amd as idx
    return {"out": idx.idx_attend4_prefill(
        s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["kv_indptr"], s["kv_indices"],
        s["tok_indptr"], s["kv_len"], s["max_pages"], scale=s["scale"],
        softcap=s["case"]["softcap"], slopes=s["slopes"])}


_PLAIN = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read,
          "attend": _plain_attend, "prefill": _plain_prefill}
_OWN = {"rope": _own_rope, "write": _own_write, "read": _own_read, "attend": _own_attend,
        "prefill": _own_prefill}


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- float64

def _nibble(code):
    """The value of codes 0..15 from their bits, in float64."""
    e, f = (code >> 1 & 3).double(), (code & 1).double()
    a = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.exp2(e - 1))
    return torch.where(code >= 8, -a, a)


def _power(byte):
    """The value of e8m0 scales, in float64."""
    return ((byte.long() + 1023 - 127) << 52).view(torch.float64)


def _dequantised(s, pages):
    """Keys and values [Hkv, tokens, D] of the pages' tokens, in float64."""
    kc, vc = s["kc"][pages], s["vc"][pages]
    P, H, page, _ = kc.shape
    k = torch.empty(P, H, page, D, dtype=torch.float64, device=kc.device)
    k[..., 0::2], k[..., 1::2] = _nibble(kc & 15), _nibble(kc >> 4)
    v = torch.empty(P, H, D, page, dtype=torch.float64, device=kc.device)
    v[..., 0::2], v[..., 1::2] = _nibble(vc & 15), _nibble(vc >> 4)
    for d in range(0, D, BLOCK):
        k[..., d:d + BLOCK] *= _power(s["ks"][pages][..., d // BLOCK, None])
        v[:, :, d:d + BLOCK] *= _power(s["vs"][pages][:, :, d // BLOCK, None])
    return (k.transpose(0, 1).reshape(H, -1, D),
            v.permute(1, 0, 3, 2).reshape(H, -1, D))


def _softmax_rows(s, q, k, v, head, pos, seen):
    """One query head's rows q [n, D] over keys [L, D] at `pos`, visible below `seen`
    [n], in float64."""
    cap = s["case"]["softcap"]
    x = (q @ k.T.contiguous()) * s["scale"]
    if cap:
        x = cap * (1 - 2 / (torch.exp(2 * x / cap) + 1))
    if s["slopes"] is not None:
        x -= s["slopes"][head].double() * (seen[:, None] - 1 - pos[None]).double()
    x.masked_fill_(pos[None] >= seen[:, None], -torch.inf)
    x = torch.softmax(x, dim=1)
    return torch.nan_to_num(x) @ v if (seen <= 0).any() else x @ v


def _nearest(x):
    """x [..., 32] as the value that its block keeps of it, in float64: a search over the
    scales and the codes' values."""
    s = _power(torch.arange(MIN_EXP, MAX_EXP + 1, device=x.device) + 127)
    top = x.abs().amax(-1)
    s = s[torch.searchsorted(6 * s, top).clamp(max=len(s) - 1)][..., None]
    y = x / s
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    up = torch.searchsorted(grid, y.abs().contiguous()).clamp(max=7)
    down = (up - 1).clamp(min=0)
    below, above = y.abs() - grid[down], grid[up] - y.abs()
    even = torch.where(down % 2 == 0, down, up)
    pick = torch.where(below < above, down, torch.where(above < below, up, even))
    return grid[pick] * torch.sign(y) * s


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        z = torch.polar(torch.full_like(s["inv_freq"], s["factor"])[None],
                        (s["tok_len"].double() - 1)[:, None] * s["inv_freq"])[:, None]
        z = z.conj() if c["inverse"] else z
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            part = x[..., c["first"]:c["first"] + c["rot"]]
            shape = (*part.shape[:2], -1, 2) if c["interleaved"] else (*part.shape[:2], 2, -1)
            pair = 3 if c["interleaved"] else 2
            p = part.reshape(shape)
            w = torch.complex(p.select(pair, 0), p.select(pair, 1)) * z
            x[..., c["first"]:c["first"] + c["rot"]] = torch.stack(
                [w.real, w.imag], pair).reshape(part.shape)
            out[name] = x
        return out
    page = c["page"]
    if c["op"] == "write":
        n, H = s["k"].shape[:2]
        return {x: _nearest(s[x].double().reshape(n, H, -1, BLOCK)).reshape(n, H, D)
                for x in ("k", "v")}
    if c["op"] == "read":
        pages, where = torch.unique(s["slots"].long() // page, return_inverse=True)
        k, v = _dequantised(s, pages)
        at = where * page + s["slots"].long() % page
        return {"k": k[:, at].transpose(0, 1), "v": v[:, at].transpose(0, 1)}
    Hq, G = c["Hq"], c["Hq"] // c["Hkv"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    first = s["kv_indptr"].tolist()

    def tokens(b, n):
        return _dequantised(s, s["kv_indices"][first[b]:first[b] + _pages(n, page)].long())

    if c["op"] == "prefill":
        ptr = s["tok_indptr"].tolist()
        for b in range(c["B"]):
            seen = s["kv_len"][ptr[b]:ptr[b + 1]].long()
            n = int(seen.max())
            k, v = tokens(b, n)
            pos = torch.arange(n, device=q.device)
            for h in range(Hq):
                out[ptr[b]:ptr[b + 1], h] = _softmax_rows(
                    s, q[ptr[b]:ptr[b + 1], h], k[h // G, :n], v[h // G, :n], h, pos, seen)
        return {"out": out}
    if q.shape[0] > 1100:
        return None
    at = torch.arange(page, device=q.device)
    lens = s["kv_len"].tolist()
    last = None
    for r in range(q.shape[0]):
        b = r if s["row_req"] is None else int(r // c["T"])
        if lens[r] <= 0:
            continue
        if last is None or last[0] != b:
            last = (b, *tokens(b, max(lens[r:r + c["T"]])))
        _, k, v = last
        pos = torch.arange(lens[r], device=q.device)
        if s["ids"] is not None:
            ids = s["ids"][r].long()
            pos = (ids[ids >= 0][:, None] * page + at).reshape(-1)
            pos = pos[pos < lens[r]]
        kk, vv = k[:, pos], v[:, pos]
        qq = q[r].view(c["Hkv"], G, D)
        x = torch.matmul(qq, kk.transpose(1, 2).contiguous()) * s["scale"]
        if c["softcap"]:
            x = c["softcap"] * (1 - 2 / (torch.exp(2 * x / c["softcap"]) + 1))
        if s["slopes"] is not None:
            x = x - (s["slopes"].double().view(c["Hkv"], G, 1)
                     * (lens[r] - 1 - pos).double())
        out[r] = torch.matmul(torch.softmax(x, -1), vv).view(Hq, D)
    return {"out": out}
