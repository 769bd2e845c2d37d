"""The measured cases of what a check round needs around its attention, and of that attention over a
cache in 4 bits: page tables and slot maps from the requests' lengths, norms and rotation of query and
key heads on their way into the cache, rows written to a 4-bit cache and read back, and drafted rows
attending over it.

`own` false: the operators in plain torch operations, in 32 bits (angles and quantisation in 64).
`own` true: the calls of `serial_draft_head_gb300`.  Both take what `prepare` returns.

A 4-bit row is e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign; two a byte, the even element low) and
a byte for every 16 elements, the upper bits of its scale as a 16-bit float: a block's scale is the
smallest with three mantissa bits that brings its largest magnitude to 6 or below.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one round's tables: 16 users with 8 drafted tokens each
        dict(name="tables draft", op="tables", B=16, T_lo=8, T_hi=8, L_lo=300, L_hi=6000, page=16, tree=False, shape=21),
        # tables of a full house: 1,024 requests, trees and prompts of up to 260 tokens, positions by depth
        dict(name="tables 1024 requests", op="tables", B=1024, T_lo=1, T_hi=260, L_lo=0, L_hi=2000, page=16, tree=True,
             shape=22),
        # one round's heads on their way in: 16 users with 8 tokens each, norms and rotation
        dict(name="place draft", op="rotate", B=16, T_lo=8, T_hi=8, L_lo=300, L_hi=6000, Hq=32, Hkv=8, D=128, R=128,
             page=16, dtype="bf16", norm=True, pairs=False, place=True, shape=23),
        # new prompts of about 27,000 tokens, far positions among them
        dict(name="place prompts", op="rotate", B=7, T_lo=1001, T_hi=8191, L_lo=0, L_hi=131071, Hq=32, Hkv=8, D=128,
             R=128, page=64, dtype="bf16", norm=True, pairs=False, place=True, shape=24),
        # heads of 96 of which 64 elements turn, neighbours in pairs, no norms, no cache
        dict(name="rotate odd f16", op="rotate", B=13, T_lo=5, T_hi=161, L_lo=1, L_hi=3001, Hq=14, Hkv=2, D=96, R=64,
             page=24, dtype="f16", norm=False, pairs=True, place=False, shape=25),
        # the cache write of one round, and the rows back as they stand in 4 bits
        dict(name="write draft", op="write", B=16, T_lo=8, T_hi=8, L_lo=300, L_hi=6000, Hkv=8, D=128, page=16,
             dtype="bf16", shape=26),
        # the same for new prompts of about 40,000 tokens
        dict(name="write prompts", op="write", B=9, T_lo=901, T_hi=8191, L_lo=0, L_hi=63, Hkv=8, D=128, page=64,
             dtype="bf16", shape=27),
        # one chat user, one new token, a short history: latency only
        dict(name="attend 1 token short", op="attend", B=1, T_lo=1, T_hi=1, L_lo=517, L_hi=517, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", tree=False, softcap=0.0, shape=28),
        # a round of a gamma = 7 draft: 16 users, the anchor and 7 drafted tokens in a chain
        dict(name="attend chain 8 x 16", op="attend", B=16, T_lo=8, T_hi=8, L_lo=300, L_hi=6000, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", tree=False, softcap=0.0, shape=29),
        # trees of odd sizes, 7 query heads a cached head of 96, capped scores
        dict(name="attend tree odd f16", op="attend", B=13, T_lo=5, T_hi=61, L_lo=1, L_hi=3001, Hq=14, Hkv=2, D=96,
             page=24, dtype="f16", tree=True, softcap=30.0, shape=30),
        # many users without a draft, long histories: what a 4-bit cache is there for
        dict(name="attend 1 token x 128", op="attend", B=128, T_lo=1, T_hi=1, L_lo=500, L_hi=9000, Hq=64, Hkv=8, D=128,
             page=64, dtype="bf16", tree=False, softcap=0.0, shape=31),
        # serving at its densest: 64 users, trees of 64 nodes, long contexts
        dict(name="attend tree 64 x 64", op="attend", B=64, T_lo=64, T_hi=64, L_lo=4096, L_hi=8192, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16", tree=True, softcap=0.0, shape=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    top = [work(c) for c in listed()]
    most = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(("tables", "rotate", "write", "attend", "attend", "attend"))
        page = rng.choice((16, 16, 24, 32, 64, 100, 128))
        if op == "tables":
            c = dict(op=op, B=_log(rng, 1, 1024), page=page, tree=rng.random() < 0.5)
            T = _log(rng, 1, 256 if c["tree"] else 4000)
            c.update(T_lo=rng.randint(0, T), T_hi=T, L_lo=0, L_hi=_log(rng, 1, 20000))
            # pages of every request and rows: a few hundred MB in the plain form at most
            if c["B"] * T > 1 << 19 or c["B"] * (c["L_hi"] + T) // page > 1 << 22:
                continue
        else:
            c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16")), page=page, D=rng.choice((32, 64, 96, 128, 128)),
                     Hkv=rng.choice((1, 2, 4, 5, 8, 8, 16)), B=_log(rng, 1, 128))
            if op == "attend":
                T, L = _log(rng, 1, 96), _log(rng, 8, 131072)
                c.update(Hq=c["Hkv"] * rng.choice((1, 2, 3, 4, 4, 5, 7, 8)), T_lo=rng.randint(1, T), T_hi=T,
                         L_lo=rng.randint(L // 4, L), L_hi=L, tree=rng.random() < 0.5,
                         softcap=rng.choice((0.0, 0.0, 50.0)))
                # padded scores and 32-bit copies of the cache are what the plain form holds
                if c["B"] * (L + T) * max(c["Hq"] * T, 4 * c["Hkv"] * c["D"]) * 4 > 10 << 30:
                    continue
            else:
                T = _log(rng, 1, 8192)
                c.update(T_lo=rng.randint(1, T), T_hi=T, L_lo=0, L_hi=rng.randint(0, 200))
                if op == "rotate":
                    c.update(Hq=c["Hkv"] * rng.choice((1, 2, 4, 4, 7, 8)), L_hi=_log(rng, 1, 131072),
                             R=rng.choice((c["D"], c["D"], c["D"] // 2)), norm=rng.random() < 0.7,
                             pairs=rng.random() < 0.3, place=rng.random() < 0.7)
                    if c["place"]:
                        c["L_hi"] = min(c["L_hi"], 20000)
                if c["B"] * T * (c["Hkv"] * 2 + c.get("Hq", 0)) * c["D"] > 1 << 28 or \
                        c["B"] * (T + c["L_hi"]) * c["Hkv"] * c["D"] > 1 << 29:
                    continue
        c["shape"] = rng.randrange(1 << 20)
        w = work(c)
        if w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"] and (w["bytes"] > 0 or w["flops"] > 0):
            return c


def _lengths(case):
    """Tokens each request brings, and tokens it holds before them."""
    rng = random.Random(case["shape"])
    T = [rng.randint(case["T_lo"], case["T_hi"]) for _ in range(case["B"])]
    L = [rng.randint(case["L_lo"], case["L_hi"]) for _ in range(case["B"])]
    return T, L


def work(case):
    T, L = _lengths(case)
    N = sum(T)
    if case["op"] == "tables":
        # lengths, counts and pages held in, offsets and held out, a slot and a position a row, a page
        # number in and out and its place in the table for every page that comes and goes; mask words
        new = sum(-(-(t + n) // case["page"]) - -(-n // case["page"]) for t, n in zip(T, L))
        words = (max(T) + 31) // 32 if case["tree"] else 0
        return {"bytes": 20 * case["B"] + N * (8 + 4 * words) + 24 * new, "flops": 0}
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "rotate":
        heads = case["Hq"] + Hkv * (2 if case["place"] else 1)
        return {"bytes": N * (4 * heads * D + 4 + (4 if case["place"] else 0)), "flops": N * 8 * (case["Hq"] + Hkv) * D}
    row = 2 * Hkv * (D // 2 + D // 16)                                  # K and V of one cached token
    if case["op"] == "attend":
        keys = sum(t + n for t, n in zip(T, L))
        pairs = sum(t * n + t * (t + 1) // 2 for t, n in zip(T, L))     # a chain's; a tree has fewer
        return {"bytes": keys * row + N * case["Hq"] * (4 * D + 4), "flops": 4 * pairs * case["Hq"] * D}
    # written and read again
    return {"bytes": N * 2 * (row + 4 * Hkv * D), "flops": N * 8 * Hkv * D}


def _tree_bits(T, g, dev):
    """Mask words of random trees, int32 [N, words]: a node sees itself and its ancestors."""
    B, Tm = len(T), max(T)
    back = 1 + (torch.rand(B, Tm, generator=g, device=dev) ** 2 * 12).long()
    parent = (torch.arange(Tm, device=dev) - back).clamp(min=0)
    see = torch.eye(Tm, dtype=torch.bool, device=dev).expand(B, Tm, Tm).clone()
    at = torch.arange(B, device=dev)
    for i in range(1, Tm):
        see[:, i] |= see[at, parent[:, i]]
    words = (Tm + 31) // 32
    bits = torch.zeros(B, Tm, words * 32, dtype=torch.bool, device=dev)
    bits[:, :, :Tm] = see
    w = torch.zeros(B, Tm, words, dtype=torch.int64, device=dev)
    for i in range(32):
        w |= bits.view(B, Tm, words, 32)[..., i].long() << i
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).int()
    here = torch.arange(Tm, device=dev) < torch.tensor(T, device=dev)[:, None]
    return w[here].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + case["shape"])
    T, L = _lengths(case)
    B, page, N, Tm, Lm = case["B"], case["page"], sum(T), max(T), max(L)
    P = max(max(-(-(t + n) // page) for t, n in zip(T, L)), 1)
    first = torch.tensor([sum(T[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    s = dict(case=case, B=B, N=N, Tm=Tm, Lm=Lm, P=P, page=page, first=first,
             length=torch.tensor(L, dtype=torch.int32, device=dev), count=torch.tensor(T, dtype=torch.int32, device=dev))
    if case["op"] == "tables":
        held = [-(-n // page) for n in L]
        n_pages = sum(-(-(t + n) // page) for t, n in zip(T, L)) + 7
        order = torch.randperm(n_pages, generator=g, device=dev).int()     # a pool that has been in use
        table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
        used = sum(held)
        table[torch.arange(P, device=dev) < torch.tensor(held, device=dev)[:, None]] = order[:used]
        free = torch.cat([order[used:], order[:used]])                     # behind the free ones: anything
        held = torch.tensor(held, dtype=torch.int32, device=dev)
        n_free = torch.tensor([n_pages - used], dtype=torch.int32, device=dev)
        s["mask"] = _tree_bits(T, g, dev) if case["tree"] and N > 0 else None
        if own:
            from serial_draft_head_gb300 import Pages
            s["pool"] = Pages(n_pages, page, B, P)
            for mine, x in ((s["pool"].table, table), (s["pool"].held, held), (s["pool"].free, free),
                            (s["pool"].n_free, n_free)):
                mine.copy_(x)
        else:
            s.update(table=table, held=held, free=free, n_free=n_free)
        return s
    Hkv, D = case["Hkv"], case["D"]
    dt = DTYPES[case["dtype"]]
    n_pages = B * P + 1
    s.update(Hkv=Hkv, D=D, dtype=dt)
    s["pages"] = torch.randperm(n_pages, generator=g, device=dev)[:B * P].int().view(B, P).contiguous()
    chan = 0.5 + torch.rand(Hkv, D, generator=g, device=dev)   # channels of unlike sizes, as projections have

    def rows(*shape):
        y = torch.randn(*shape, Hkv, D, generator=g, device=dev) * chan
        return torch.where(torch.rand(*shape, Hkv, 1, generator=g, device=dev) < 0.02, 8 * y, y)

    if case["op"] == "rotate":
        Hq = case["Hq"]
        # one projection's output: query, key and value heads of a token next to each other
        qkv = torch.empty(N, Hq + 2 * Hkv, D, dtype=dt, device=dev)
        for a in range(0, N, 1 << 13):
            x = torch.randn(qkv[a:a + (1 << 13)].shape, generator=g, device=dev)
            x[:, Hq:Hq + Hkv] *= chan
            qkv[a:a + (1 << 13)] = x.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        b, i = _rows(s)
        at = s["length"][b].long() + i
        s["position"] = at.int()
        s["freq"] = 10000.0 ** (-torch.arange(case["R"] // 2, dtype=torch.float64, device=dev) / (case["R"] // 2))
        s["norms"] = [0.5 + torch.rand(D, generator=g, device=dev) for _ in range(2)] if case["norm"] else [None, None]
        if case["place"]:
            # the requests' new rows alone: a pool of just their pages, places as a table gives them
            used = -(-(s["count"] + s["length"] % page) // page)
            place = i + s["length"][b] % page
            pool = int(used.sum()) + 1
            to = torch.randperm(pool, generator=g, device=dev)[(used.cumsum(0) - used)[b].long() + place // page]
            s["slot"] = (to * page + place % page).int()
            s["cache_k"], s["cache_v"] = (torch.zeros(pool, page, Hkv, D, dtype=dt, device=dev) for _ in range(2))
        if own:
            from serial_draft_head_gb300 import KVCache, Rotation, Tree
            s["tree"] = Tree(q_heads=Hq, kv_heads=Hkv, head_dim=D, dtype=dt)
            s["rotation"] = Rotation(D, s["freq"], *s["norms"], interleaved=case["pairs"])
            if case["place"]:
                s["cache"] = KVCache(s["cache_k"], s["cache_v"])
        return s
    # a 4-bit cache, the slots of one head in a page next to each other
    codes = [torch.zeros(n_pages, Hkv, page, D // 2, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.zeros(n_pages, Hkv, page, D // 16, dtype=torch.uint8, device=dev) for _ in range(2)]
    if case["op"] == "attend":
        step = max(1, (1 << 25) // (page * Hkv * D))
        for x, e in zip(codes, scales):
            for a in range(0, n_pages, step):
                y, z = _quantise(rows(len(x[a:a + step]), page))
                x[a:a + step], e[a:a + step] = y.transpose(1, 2), z.transpose(1, 2)
        s["Hq"], s["G"] = case["Hq"], case["Hq"] // Hkv
        s["scale"], s["softcap"] = D ** -0.5, case["softcap"]
        s["q"] = (1.5 * torch.randn(N, case["Hq"], D, generator=g, device=dev)).to(dt)
        s["mask"] = _tree_bits(T, g, dev) if case["tree"] else None
    else:
        s["new_k"], s["new_v"] = rows(N).to(dt), rows(N).to(dt)
    s["k"], s["v"], s["k_scale"], s["v_scale"] = (x.transpose(1, 2) for x in codes + scales)
    if own:
        from serial_draft_head_gb300 import KVCache, Tree
        s["cache"] = KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["tree"] = Tree(q_heads=case.get("Hq", Hkv), kv_heads=Hkv, head_dim=D, dtype=dt, max_requests=B,
                         max_nodes=Tm if case["op"] == "attend" else 1)
    return s


# ------------------------------------------------------------------ plain forms --


def _rows(s):
    """Request and place within it of every packed row."""
    n = torch.arange(s["N"], device=s["first"].device)
    b = torch.searchsorted(s["first"], n, right=True) - 1
    return b, n - s["first"][b]


def _plain_tables(s):
    page, B, P, dev = s["page"], s["B"], s["P"], s["length"].device
    length, count, held = s["length"].long(), s["count"].long(), s["held"].long()
    first = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    first[1:] = count.cumsum(0)
    need = ((length + count + page - 1) // page - held).clamp(min=0)
    before = need.cumsum(0) - need
    # new pages from the end of the free ones, request by request
    p = torch.arange(P, device=dev)
    new = (p >= held[:, None]) & (p < (held + need)[:, None])
    take = s["n_free"].long() - 1 - (before[:, None] + p - held[:, None])
    grown = torch.where(new, s["free"][take.clamp(0, len(s["free"]) - 1)], s["table"])
    n = torch.arange(s["N"], device=dev)
    b = torch.searchsorted(first, n, right=True) - 1
    i = n - first[b]
    at = length[b] + i
    slot = grown[b, at // page].long() * page + at % page
    position = at
    if s["mask"] is not None:
        bits = torch.zeros_like(at)
        for k in range(32):
            bits += ((s["mask"] >> k) & 1).sum(1)
        position = length[b] + bits - 1
    # and back: the pages past the lengths, onto the places that they came from
    held = held + need
    keep = torch.minimum(held, (length + page - 1) // page)
    gone = held - keep
    past = (p >= keep[:, None]) & (p < held[:, None])
    total = need.sum()
    back = s["n_free"].long() - total + gone.sum() - 1 - ((gone.cumsum(0) - gone)[:, None] + p - keep[:, None])
    s["free"][back[past]] = grown[past]
    s["table"].copy_(torch.where(past, torch.full_like(grown, -1), grown))
    s["held"].copy_(keep)
    s["n_free"].add_((gone.sum() - total).int())
    return {"first": first.int(), "slot": slot.int(), "position": position.int(), "table": s["table"], "held": s["held"],
            "free": s["free"], "n_free": s["n_free"]}


def _plain_rotate(s):
    R, pairs = s["case"]["R"], s["case"]["pairs"]
    angle = s["position"].double()[:, None] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    got = []
    for x, w in zip((s["q"], s["k"]), s["norms"]):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if pairs else (y[..., :R // 2], y[..., R // 2:R])
        c, d = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([c, d], -1).flatten(-2) if pairs else torch.cat([c, d], -1)
        got.append(torch.cat([turned, y[..., R:]], -1).to(s["dtype"]))
    if not s["case"]["place"]:
        return tuple(got)
    page, slot = s["slot"].long() // s["page"], s["slot"].long() % s["page"]
    s["cache_k"][page, slot], s["cache_v"][page, slot] = got[1], s["v"]
    return got[0], s["cache_k"], s["cache_v"]


_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)     # between neighbouring codes; ties to the even one


def _quantise(x):
    """Codes, two a byte, and scale bytes of rows [..., D]."""
    y = x.unflatten(-1, (-1, 16)).double()
    a = y.abs().amax(-1) / 6
    m, e = torch.frexp(a)                              # a = m 2^e, m in [0.5, 1)
    e = e.clamp(min=-13)                               # scales are multiples of 2^-17 at least
    unit = torch.exp2((e - 4).double())
    scale = (torch.ceil(a / unit) * unit).clamp(max=10240.0)
    y = y / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    code = (y < 0).to(torch.uint8) * 8
    y = y.abs()
    for i, border in enumerate(_BORDERS):
        code += (y >= border) if i % 2 else (y > border)
    code = code.flatten(-2)
    byte = (scale.half().view(torch.int16) >> 7).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, byte


def _slot(s, b, pos):
    """Page and slot of positions `pos` of requests `b`."""
    return s["pages"][b, pos // s["page"]].long(), pos % s["page"]


def _values(s, name, page, slot):
    x, e = s[name][page, slot], s[name + "_scale"][page, slot]
    code = torch.stack([x & 15, x >> 4], -1).flatten(-2)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    y = torch.cat([grid, -grid])[code.int()]
    scale = (e.to(torch.int16) << 7).view(torch.float16).float()
    return (y.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2)


def _plain_write(s):
    b, i = _rows(s)
    page, slot = _slot(s, b, s["length"][b].long() + i)
    for name in ("k", "v"):
        s[name][page, slot], s[name + "_scale"][page, slot] = _quantise(s["new_" + name].float())
    return tuple(_values(s, name, page, slot).to(s["dtype"]) for name in ("k", "v"))


def _plain_attend(s):
    B, N, Tm, Hkv, G, D, dev = s["B"], s["N"], s["Tm"], s["Hkv"], s["G"], s["D"], s["q"].device
    first, length = s["first"].long(), s["length"].long()
    count = first[1:] - first[:-1]
    i = torch.arange(Tm, device=dev)
    row = (first[:-1, None] + i).clamp(max=N - 1)
    q = s["q"][row].float().view(B, Tm, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Tm * G, D)
    pos = torch.arange(min(s["Lm"] + Tm, s["P"] * s["page"]), device=dev)
    page, slot = _slot(s, slice(None), pos)
    beyond = (pos >= (length + count)[:, None])[:, :, None, None]
    k = _values(s, "k", page, slot)                                        # [B, L, Hkv, D]
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                # [B, Hkv, Tm G, L]
    del k
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    j = pos - length[:, None]                                              # place in the draft
    if s["mask"] is None:
        see = (j[:, None] <= i[:, None]) & (j < count[:, None])[:, None]
    else:
        jj = j.clamp(0, s["mask"].shape[1] * 32 - 1)
        word = torch.gather(s["mask"][row], 2, (jj // 32)[:, None].expand(B, Tm, len(pos)))
        see = (word >> (jj % 32)[:, None].int()) & 1 != 0
        see = (j < 0)[:, None] | (see & (j < count[:, None])[:, None])
    x = x.view(B, Hkv, Tm, G, -1).masked_fill(~see[:, None, :, None], -math.inf).view(B, Hkv, Tm * G, -1)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    del x
    z = p.sum(-1, keepdim=True)
    v = _values(s, "v", page, slot).masked_fill(beyond, 0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + torch.log(z)).view(B, Hkv, Tm, G)
    b, i = _rows(s)
    out = o.view(B, Hkv, Tm, G, D)[b, :, i].reshape(N, Hkv * G, D).to(s["dtype"])
    return out, lse[b, :, i].reshape(N, Hkv * G)


# ------------------------------------------------------------------------- runs --


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"tables": _plain_tables, "rotate": _plain_rotate, "write": _plain_write, "attend": _plain_attend}[op](s)
    if op == "tables":
        pool = s["pool"]
        first, slot, position = pool.grow(s["length"], s["count"], s["N"], mask=s["mask"])
        pool.trim(s["length"])
        return {"first": first, "slot": slot, "position": position, "table": pool.table, "held": pool.held,
                "free": pool.free, "n_free": pool.n_free}
    if op == "rotate":
        if not s["case"]["place"]:
            return s["tree"].rotate(s["q"], s["k"], s["position"], s["rotation"])
        q = s["tree"].place(s["cache"], s["slot"], s["q"], s["k"], s["v"], s["position"], s["rotation"])
        return q, s["cache_k"], s["cache_v"]
    if op == "write":
        s["tree"].write(s["cache"], s["pages"], s["length"], s["first"], s["new_k"], s["new_v"])
        return s["tree"].read(s["cache"], s["pages"], s["length"], s["first"], s["N"])
    return s["tree"].attend(s["q"], s["cache"], s["pages"], s["length"], s["first"], mask=s["mask"], scale=s["scale"],
                            softcap=s["softcap"])


# ------------------------------------------------------- definitions in 64 bits --


def _exact_tables(s, T, L):
    """Request by request, in lists."""
    page, B, P = s["page"], s["B"], s["P"]
    pool = s["pool"] if "pool" in s else None
    table, held, free, n_free = (x.tolist() for x in ((pool.table, pool.held, pool.free, pool.n_free) if pool else
                                                      (s["table"], s["held"], s["free"], s["n_free"])))
    top, first, slot, position = n_free[0], [0], [], []
    words = None if s["mask"] is None else s["mask"].tolist()
    popped = []
    for b in range(B):
        while held[b] * page < L[b] + T[b]:
            top -= 1
            table[b][held[b]] = free[top]
            popped.append((b, held[b], top))
            held[b] += 1
        for i in range(T[b]):
            at = L[b] + i
            slot.append(table[b][at // page] * page + at % page)
            if words is not None:
                at = L[b] + sum(bin(w & 0xffffffff).count("1") for w in words[first[b] + i]) - 1
            position.append(at)
        first.append(first[b] + T[b])
    for b, p, t in reversed(popped):
        free[t] = table[b][p]
        table[b][p] = -1
        held[b] -= 1
        top += 1
    assert top == n_free[0] and all(len(r) == P for r in table)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    return {"first": ints(first), "slot": ints(slot), "position": ints(position), "table": ints(table).view(B, P),
            "held": ints(held), "free": ints(free), "n_free": ints([top])}


def _exact_rotate(s):
    R, D = s["case"]["R"], s["D"]
    half = R // 2
    got = []
    turn = torch.remainder(s["position"].to(torch.float64)[:, None] * s["freq"], 2 * math.pi)[:, None]
    for x, w in ((s["q"], s["norms"][0]), (s["k"], s["norms"][1])):
        y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for lo in range(0, len(x), 4096):
            z = x[lo:lo + 4096].to(torch.float64)
            if w is not None:
                z = z / torch.sqrt(z.square().sum(-1, keepdim=True) / D + 1e-6) * w.to(torch.float64)
            t = turn[lo:lo + 4096]
            out = z.clone()
            for i in range(half):
                p, r = (2 * i, 2 * i + 1) if s["case"]["pairs"] else (i, i + half)
                c, d = torch.cos(t[..., i]), torch.sin(t[..., i])
                out[..., p] = z[..., p] * c - z[..., r] * d
                out[..., r] = z[..., r] * c + z[..., p] * d
            y[lo:lo + 4096] = out
        got.append(y)
    if not s["case"]["place"]:
        return tuple(got)
    k, v = (s[n].to(torch.float64).flatten(0, 1) for n in ("cache_k", "cache_v"))
    k[s["slot"].long()] = got[1]
    v[s["slot"].long()] = s["v"].to(torch.float64)
    return got[0], k.view(s["cache_k"].shape), v.view(s["cache_k"].shape)


def _exact_codes(x):
    """What rows are worth in 4 bits: scales and codes by search over all that there are."""
    scales = torch.arange(227, dtype=torch.int32, device=x.device)
    scales = torch.where(scales < 8, scales.double() * 2.0 ** -17,
                         (8 + scales % 8).double() * torch.exp2((scales // 8).double() - 18))
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    flat, to = x.reshape(-1, 16), out.view(-1, 16)
    for lo in range(0, len(flat), 1 << 20):
        y = flat[lo:lo + (1 << 20)].to(torch.float64)
        s = scales[torch.searchsorted(6 * scales, y.abs().amax(1)).clamp(max=226)][:, None]
        z = torch.where(s > 0, y.abs() / s, torch.zeros_like(y))
        hi = torch.searchsorted(grid, z.contiguous()).clamp(1, 7)
        up, down = grid[hi] - z, z - grid[hi - 1]
        pick = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)
        to[lo:lo + (1 << 20)] = torch.copysign(grid[pick] * s, y)
    return out


def _exact_kept(s, name, b, n):
    """Positions 0 .. n-1 of request b, float64 [n, Hkv, D]."""
    at = torch.arange(n, device="cuda")
    p, t = s["pages"][b][at // s["page"]].long(), at % s["page"]
    x, e = s[name][p, t].int(), s[name + "_scale"][p, t].int()
    code = torch.empty(*x.shape[:-1], s["D"], dtype=torch.int32, device="cuda")
    code[..., 0::2], code[..., 1::2] = x % 16, x // 16
    low, field = code % 2, code // 2 % 4
    mag = torch.where(field == 0, low * 0.5, (1 + low * 0.5).double() * torch.exp2((field - 1).double()))
    scale = torch.where(e < 8, e.double() * 2.0 ** -17, (8 + e % 8).double() * torch.exp2((e // 8).double() - 18))
    return torch.where(code >= 8, -mag, mag) * scale.repeat_interleave(16, -1)


def exact(case, seed):
    s = prepare(case, seed)
    T, L = _lengths(case)
    if case["op"] == "tables":
        return _exact_tables(s, T, L)
    if case["op"] == "rotate":
        return _exact_rotate(s)
    if case["op"] == "write":
        return _exact_codes(s["new_k"]), _exact_codes(s["new_v"])
    starts = [sum(T[:b]) for b in range(case["B"])]
    out = torch.empty(s["N"], s["Hq"], s["D"], dtype=torch.float64, device="cuda")
    lse = torch.empty(s["N"], s["Hq"], dtype=torch.float64, device="cuda")
    for b, (t, n) in enumerate(zip(T, L)):
        k, v = _exact_kept(s, "k", b, n + t), _exact_kept(s, "v", b, n + t)
        see = torch.ones(t, n + t, dtype=torch.bool, device="cuda")
        for i in range(t):
            if s["mask"] is None:
                see[i, n + i + 1:] = False
            else:
                w = [int(x) & 0xffffffff for x in s["mask"][starts[b] + i].tolist()]
                see[i, n:] = torch.tensor([w[j // 32] >> j % 32 & 1 for j in range(t)], device="cuda") != 0
        for h in range(s["Hq"]):
            q = s["q"][starts[b]:starts[b] + t, h].to(torch.float64)
            x = q @ k[:, h // s["G"]].T * s["scale"]
            if s["softcap"]:
                x = s["softcap"] * torch.tanh(x / s["softcap"])
            x[~see] = -math.inf
            lse[starts[b]:starts[b] + t, h] = torch.logsumexp(x, 1)
            out[starts[b]:starts[b] + t, h] = torch.softmax(x, 1) @ v[:, h // s["G"]]
    return out, lse
