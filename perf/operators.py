"""The measured cases of the draft-check operators: writing drafted tokens' keys and values into
a paged cache (16-bit or quantised), attention of a tree of drafted tokens over that cache,
keeping the accepted path's rows, and reading the cache back.

`own` false: the operators in plain torch operations, in 32 bits.  `own` true: the calls of
`serial_draft_head_gb300.tree`.  Both take what `prepare` returns.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one chat user, one new token, a short history: the smallest call, latency only
        dict(name="attend 1 token short", op="attend", B=1, T_lo=1, T_hi=1, L_lo=517, L_hi=517, Hq=32,
             Hkv=8, D=128, page=16, dtype="bf16", cache="bf16", tree=False, softcap=0.0, shape=1),
        # an ordinary round of a gamma = 7 draft: 16 users, the anchor and 7 drafted tokens in a chain
        dict(name="attend chain 8 x 16", op="attend", B=16, T_lo=8, T_hi=8, L_lo=300, L_hi=6000, Hq=32,
             Hkv=8, D=128, page=16, dtype="bf16", cache="bf16", tree=False, softcap=0.0, shape=2),
        # trees of odd sizes over a quantised cache, 7 query heads a cached head of 80, capped scores
        dict(name="attend tree odd f16", op="attend", B=13, T_lo=5, T_hi=61, L_lo=1, L_hi=3001, Hq=14,
             Hkv=2, D=80, page=24, dtype="f16", cache="e4m3", tree=True, softcap=30.0, shape=3),
        # a gamma = 16 draft of one user with a long document: the whole device on one request
        dict(name="attend chain 17 long", op="attend", B=1, T_lo=17, T_hi=17, L_lo=131071, L_hi=131071,
             Hq=32, Hkv=8, D=128, page=64, dtype="bf16", cache="bf16", tree=False, softcap=0.0, shape=4),
        # serving at its densest: 64 users, trees of 64 nodes, long contexts
        dict(name="attend tree 64 x 64", op="attend", B=64, T_lo=64, T_hi=64, L_lo=4096, L_hi=8192,
             Hq=32, Hkv=8, D=128, page=64, dtype="bf16", cache="bf16", tree=True, softcap=0.0, shape=5),
        # many users without a draft (single tokens) over a quantised cache, wide grouping
        dict(name="attend 1 token x 128 e4m3", op="attend", B=128, T_lo=1, T_hi=1, L_lo=500, L_hi=9000,
             Hq=64, Hkv=8, D=128, page=64, dtype="bf16", cache="e4m3", tree=False, softcap=0.0, shape=6),
        # the cache write of one round: 16 users, 8 tokens each
        dict(name="write draft e4m3", op="write", B=16, T_lo=8, T_hi=8, L_lo=300, L_hi=6000, Hkv=8, D=128,
             page=16, dtype="bf16", cache="e4m3", shape=7),
        # the cache write of new prompts: about 40,000 tokens
        dict(name="write prompts e4m3", op="write", B=9, T_lo=901, T_hi=8191, L_lo=0, L_hi=63, Hkv=8, D=128,
             page=64, dtype="bf16", cache="e4m3", shape=8),
        # a few short histories back in 16 bits (for a drafter that reads them)
        dict(name="read short e4m3", op="read", B=5, T_lo=33, T_hi=400, L_lo=0, L_hi=0, Hkv=2, D=80, page=24,
             dtype="f16", cache="e4m3", shape=9),
        # long histories back in 16 bits
        dict(name="read long e4m3", op="read", B=8, T_lo=3001, T_hi=8192, L_lo=0, L_hi=0, Hkv=8, D=128,
             page=64, dtype="bf16", cache="e4m3", shape=10),
        # after acceptance: 16 users keep up to 6 rows of a small tree
        dict(name="keep paths of small trees", op="keep", B=16, T_lo=15, T_hi=31, L_lo=300, L_hi=6000, Hkv=8,
             D=128, page=16, dtype="bf16", cache="e4m3", keep=6, shape=11),
        # the same for 128 users with trees of 64 nodes and paths of up to 17, 16-bit cache
        dict(name="keep paths of large trees", op="keep", B=128, T_lo=64, T_hi=64, L_lo=300, L_hi=900, Hkv=8,
             D=128, page=64, dtype="bf16", cache="bf16", keep=17, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = max(listed(), key=lambda c: work(c)["flops"])
    top = work(most)
    while True:
        op = rng.choice(("attend", "attend", "attend", "write", "read", "keep"))
        dtype = rng.choice(("bf16", "bf16", "f16"))
        c = dict(op=op, dtype=dtype, cache=rng.choice((dtype, "e4m3")), page=rng.choice((16, 16, 24, 32, 64, 100, 128)),
                 D=rng.choice((64, 80, 96, 112, 128, 128)), Hkv=rng.choice((1, 2, 4, 5, 8, 8, 16)), B=_log(rng, 1, 128))
        if op == "attend":
            G = rng.choice((1, 2, 3, 4, 4, 5, 7, 8))
            T = _log(rng, 1, 96)
            L = _log(rng, 8, 131072)
            c.update(Hq=c["Hkv"] * G, T_lo=rng.randint(1, T), T_hi=T, L_lo=rng.randint(L // 4, L), L_hi=L,
                     tree=rng.random() < 0.5, softcap=rng.choice((0.0, 0.0, 50.0)))
        elif op == "keep":
            T = _log(rng, 2, 64)
            c.update(T_lo=rng.randint(1, T), T_hi=T, L_lo=rng.randint(0, 300), L_hi=rng.randint(300, 2000),
                     keep=rng.randint(1, T))
        else:
            T = _log(rng, 1, 8192)
            c.update(T_lo=rng.randint(1, T), T_hi=T, L_lo=0, L_hi=rng.randint(0, 200) if op == "write" else 0)
        c["shape"] = rng.randrange(1 << 20)
        w = work(c)
        if op == "attend":   # padded scores and 32-bit copies of the cache are what the plain form holds
            if c["B"] * (c["L_hi"] + c["T_hi"]) * max(c["Hq"] * c["T_hi"], 4 * c["Hkv"] * c["D"]) * 4 > 10 << 30:
                continue
        elif c["B"] * (c["T_hi"] + c["L_hi"]) * c["Hkv"] * c["D"] > 1 << 26:
            continue
        if w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"]:
            return c


def _lengths(case):
    """Tokens each request brings, and tokens its cache holds before them."""
    rng = random.Random(case["shape"])
    T = [rng.randint(case["T_lo"], case["T_hi"]) for _ in range(case["B"])]
    L = [rng.randint(case["L_lo"], case["L_hi"]) for _ in range(case["B"])]
    keep = [rng.randint(1, min(t, case["keep"])) for t in T] if case["op"] == "keep" else [0] * case["B"]
    return T, L, keep


def work(case):
    T, L, keep = _lengths(case)
    Hkv, D = case["Hkv"], case["D"]
    row = 2 * Hkv * (D + 1 if case["cache"] == "e4m3" else 2 * D)     # K and V of one cached token
    if case["op"] == "attend":
        keys = sum(t + n for t, n in zip(T, L))
        pairs = sum(t * n + t * (t + 1) // 2 for t, n in zip(T, L))   # a chain's; a tree has fewer
        return {"bytes": keys * row + sum(T) * case["Hq"] * (4 * D + 4), "flops": 4 * pairs * case["Hq"] * D}
    if case["op"] == "keep":
        return {"bytes": 2 * sum(keep) * row, "flops": 0}
    return {"bytes": sum(T) * (row + 4 * Hkv * D), "flops": sum(T) * 4 * Hkv * D}


def _trees(T, tree, g, dev):
    """Visibility of each request's nodes, [B, Tm, Tm]: a node sees itself and its ancestors."""
    B, Tm = len(T), max(T)
    parent = torch.arange(Tm, device=dev)[None].expand(B, Tm) - 1
    if tree:   # a parent among the nodes up to 12 before: branches of several lengths
        back = 1 + (torch.rand(B, Tm, generator=g, device=dev) ** 2 * 12).long()
        parent = (torch.arange(Tm, device=dev) - back).clamp(min=0)
        parent[:, 0] = -1
    see = torch.eye(Tm, dtype=torch.bool, device=dev).expand(B, Tm, Tm).clone()
    at = torch.arange(B, device=dev)
    for i in range(1, Tm):
        see[:, i] |= see[at, parent[:, i]]
    return see


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + case["shape"])
    T, L, keep = _lengths(case)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    dt = DTYPES[case["dtype"]]
    N, Tm, Lm = sum(T), max(T), max(L)
    P = max((t + n + page - 1) // page for t, n in zip(T, L))
    n_pages = B * P + 1
    first = torch.tensor([sum(T[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    s = dict(case=case, B=B, N=N, Tm=Tm, Lm=Lm, first=first, length=torch.tensor(L, dtype=torch.int32, device=dev),
             pages=torch.randperm(n_pages, generator=g, device=dev)[:B * P].int().view(B, P).contiguous(),
             k_scale=None, v_scale=None, Hkv=Hkv, D=D, page=page, dtype=dt, e4m3=case["cache"] == "e4m3")

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    # channels of unlike sizes, as projected keys and values have
    chan = 0.5 + torch.rand(Hkv, D, generator=g, device=dev)
    for name in ("k", "v"):
        if s["e4m3"]:
            # codes and scales as a quantised cache holds them: the row's largest code near the top of e4m3
            x = torch.empty(n_pages, page, Hkv, D, dtype=torch.float8_e4m3fn, device=dev)
            e = torch.empty(n_pages, page, Hkv, dtype=torch.uint8, device=dev)
            step = max(1, (1 << 27) // (page * Hkv * D))
            for a in range(0, n_pages, step):
                y = torch.randn(x[a:a + step].shape, generator=g, device=dev) * chan
                y = torch.where(torch.rand(e[a:a + step].shape, generator=g, device=dev)[..., None] < 0.02, 8 * y, y)
                y, z = _quantise(y)
                x[a:a + step], e[a:a + step] = y, z
            s[name], s[name + "_scale"] = x, e
        else:
            s[name] = torch.empty(n_pages, page, Hkv, D, dtype=dt, device=dev)
            step = max(1, (1 << 27) // (page * Hkv * D))
            for a in range(0, n_pages, step):
                s[name][a:a + step] = (torch.randn(s[name][a:a + step].shape, generator=g, device=dev) * chan).to(dt)
    if case["op"] == "attend":
        s["Hq"], s["G"] = case["Hq"], case["Hq"] // Hkv
        s["scale"], s["softcap"] = D ** -0.5, case["softcap"]
        s["q"] = (1.5 * torch.randn(N, case["Hq"], D, generator=g, device=dev)).to(dt)
        s["mask"] = None
        if case["tree"]:
            see = _trees(T, True, g, dev)
            words = (Tm + 31) // 32
            bits = torch.zeros(B, Tm, words * 32, dtype=torch.int64, device=dev)
            bits[:, :, :Tm] = see
            w = (bits.view(B, Tm, words, 32) << torch.arange(32, device=dev)).sum(-1)
            w = torch.where(w >= 1 << 31, w - (1 << 32), w).int()
            s["mask"] = torch.cat([w[b, :T[b]] for b in range(B)]).contiguous()
    elif case["op"] == "write":
        for name in ("new_k", "new_v"):
            y = randn(N, Hkv, D, dtype=torch.float32) * chan
            s[name] = torch.where(torch.rand(N, Hkv, 1, generator=g, device=dev) < 0.02, 8 * y, y).to(dt)
    elif case["op"] == "keep":
        path = torch.zeros(B, max(keep), dtype=torch.int32, device=dev)
        for b in range(B):
            path[b, :keep[b]] = torch.randperm(T[b], generator=g, device=dev)[:keep[b]].sort().values.int()
        s["path"], s["count"] = path, torch.tensor(keep, dtype=torch.int32, device=dev)
    if own:
        from serial_draft_head_gb300 import tree
        s["cache"] = tree.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["tree"] = tree.Tree(q_heads=case.get("Hq", Hkv), kv_heads=Hkv, head_dim=D, dtype=dt, max_requests=B,
                              max_nodes=Tm if case["op"] in ("attend", "keep") else 1)
    return s


# ------------------------------------------------------------------ plain forms --


def _two_to(e):
    """2^e in float32, exactly, for -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 codes of float32 rows and the rows' power-of-two scales as biased exponents."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a / 448)                 # a / 448 = m 2^e, m in [0.5, 1): 2^e holds it, 2^(e-1) if m = 0.5
    e = torch.where(448 * _two_to((e - 1).clamp(-126, 100)) >= a, e - 1, e)
    e = torch.where(a > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    half = e // 2                               # two factors: 2^-e can pass what 32 bits hold
    y = x * _two_to(-half)[..., None] * _two_to(half - e)[..., None]
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _rows(s):
    """Request and place within it of every packed row."""
    n = torch.arange(s["N"], device=s["first"].device)
    b = torch.searchsorted(s["first"], n, right=True) - 1
    return b, n - s["first"][b]


def _slot(s, b, pos):
    """Page and slot of positions `pos` of requests `b`."""
    return s["pages"][b, pos // s["page"]].long(), pos % s["page"]


def _values(s, name, page, slot):
    x = s[name][page, slot].float()
    if s["e4m3"]:
        x = x * _two_to(s[name + "_scale"][page, slot].int() - 127)[..., None]
    return x


def _plain_attend(s):
    B, N, Tm, Hkv, G, D, dev = s["B"], s["N"], s["Tm"], s["Hkv"], s["G"], s["D"], s["q"].device
    first, length = s["first"].long(), s["length"].long()
    count = first[1:] - first[:-1]
    i = torch.arange(Tm, device=dev)
    row = (first[:-1, None] + i).clamp(max=N - 1)
    q = s["q"][row].float().view(B, Tm, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Tm * G, D)
    pos = torch.arange(min(s["Lm"] + Tm, s["pages"].shape[1] * s["page"]), device=dev)
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


def _plain_write(s):
    b, i = _rows(s)
    page, slot = _slot(s, b, s["length"][b].long() + i)
    for name in ("k", "v"):
        x = s["new_" + name]
        if s["e4m3"]:
            x, e = _quantise(x.float())
            s[name + "_scale"][page, slot] = e
            s[name].view(torch.uint8)[page, slot] = x.view(torch.uint8)
        else:
            s[name][page, slot] = x


def _plain_read(s):
    b, i = _rows(s)
    page, slot = _slot(s, b, s["length"][b].long() + i)
    return tuple(_values(s, name, page, slot).to(s["dtype"]) for name in ("k", "v"))


def _plain_keep(s):
    i = torch.arange(s["path"].shape[1], device=s["path"].device)
    here = i < s["count"][:, None]
    b = torch.arange(s["B"], device=i.device)[:, None]
    to = s["length"][:, None].long() + i
    # rows past a request's count move onto themselves
    src = _slot(s, b, torch.where(here, s["length"][:, None].long() + s["path"], to).clamp(max=s["pages"].shape[1] * s["page"] - 1))
    dst = _slot(s, b, to.clamp(max=s["pages"].shape[1] * s["page"] - 1))
    for name in ("k", "v", "k_scale", "v_scale"):
        x = s[name]
        if x is not None:
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[dst] = x[src]


# ------------------------------------------------------------------------- runs --


def _state(s):
    """The cache as it stands: the state's own buffers."""
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None}


def run(state):
    s, op = state, state["case"]["op"]
    if op == "attend":
        if own:
            return s["tree"].attend(s["q"], s["cache"], s["pages"], s["length"], s["first"], mask=s["mask"],
                                    scale=s["scale"], softcap=s["softcap"])
        return _plain_attend(s)
    if op == "read":
        if own:
            return s["tree"].read(s["cache"], s["pages"], s["length"], s["first"], s["N"])
        return _plain_read(s)
    if op == "write":
        if own:
            s["tree"].write(s["cache"], s["pages"], s["length"], s["first"], s["new_k"], s["new_v"])
        else:
            _plain_write(s)
    else:
        if own:
            s["tree"].keep(s["cache"], s["pages"], s["length"], s["path"], s["count"])
        else:
            _plain_keep(s)
    return _state(s)


# ------------------------------------------------------- definitions in 64 bits --


def _exact_rows(x, e, pages, page, lo, hi):
    """Rows lo..hi-1 of one request's cache, float64 [n, Hkv, D]."""
    at = torch.arange(lo, hi, device=x.device)
    p, t = pages[at // page].long(), at % page
    y = x[p, t].to(torch.float64)
    return y if e is None else y * torch.exp2(e[p, t].to(torch.float64) - 127)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    T, L, keep = _lengths(case)
    page, starts = s["page"], [sum(T[:b]) for b in range(case["B"])]
    if case["op"] == "attend":
        out = torch.empty(s["N"], s["Hq"], s["D"], dtype=torch.float64, device="cuda")
        lse = torch.empty(s["N"], s["Hq"], dtype=torch.float64, device="cuda")
        for b, (t, n) in enumerate(zip(T, L)):
            k = _exact_rows(s["k"], s["k_scale"], s["pages"][b], page, 0, n + t)
            v = _exact_rows(s["v"], s["v_scale"], s["pages"][b], page, 0, n + t)
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
    if case["op"] == "read":
        both = [torch.cat([_exact_rows(s[m], s[m + "_scale"], s["pages"][b], page, L[b], L[b] + T[b])
                           for b in range(case["B"])]) for m in ("k", "v")]
        return tuple(both)
    got = {m: s[m].to(torch.float64) for m in ("k", "v")}
    got.update({m: s[m].clone() for m in ("k_scale", "v_scale") if s[m] is not None})
    if case["op"] == "write":
        grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).to(torch.float64)
        for m in ("k", "v"):
            x = s["new_" + m].to(torch.float64)
            e = None
            if s["e4m3"]:
                a = x.abs().amax(-1)
                e = torch.full_like(a, -127)
                for c in range(-40, 41):      # the smallest power of two that holds the row
                    e = torch.where((a > 448 * 2.0 ** (c - 1)) & (a <= 448 * 2.0 ** c), torch.full_like(e, c), e)
                y = (x * torch.exp2(-e)[..., None])
                flat, near = y.abs().view(-1), torch.empty(y.numel(), dtype=torch.float64, device="cuda")
                for c in range(0, flat.numel(), 1 << 24):     # nearest of the non-negative codes, ties to the even one
                    z = flat[c:c + (1 << 24)]
                    hi = torch.searchsorted(grid, z).clamp(1, 126)
                    up, down = grid[hi] - z, z - grid[hi - 1]
                    hi = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)
                    near[c:c + (1 << 24)] = grid[hi]
                x = torch.copysign(near.view_as(y), y)
            for b in range(case["B"]):
                at = torch.arange(L[b], L[b] + T[b], device="cuda")
                p, t = s["pages"][b][at // page].long(), at % page
                got[m][p, t] = x[starts[b]:starts[b] + T[b]]
                if e is not None:
                    got[m + "_scale"][p, t] = (e[starts[b]:starts[b] + T[b]] + 127).to(torch.uint8)
        return got
    for b in range(case["B"]):
        to = torch.arange(L[b], L[b] + keep[b], device="cuda")
        fr = L[b] + s["path"][b, :keep[b]].long()
        for x in got.values():
            x[s["pages"][b][to // page].long(), to % page] = x[s["pages"][b][fr // page].long(), fr % page]
    return got
