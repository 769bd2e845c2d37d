"""Norms and rotation of heads, alone and on the way into the cache, against their formulas in 64 bits."""
import math

import pytest
import torch

import e2m1_reference as e2m1
from test_gpu_tree import BF16, E4M3, F16, same, tree  # noqa: F401

pytestmark = pytest.mark.gpu
F64 = torch.float64


def formula(x, position, freq, norm, eps, pairs):
    """(result, what its two terms are in size, at most)."""
    y = x.to(F64)
    if norm is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * norm.to(F64)
    size = y.abs()
    if freq is None:
        return y, size
    R = 2 * len(freq)
    t = (position.to(F64)[:, None] * freq.to(F64)).remainder(2 * math.pi)[:, None]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if pairs else (slice(0, R // 2), slice(R // 2, R))
    u, w = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * torch.cos(t) - w * torch.sin(t), w * torch.cos(t) + u * torch.sin(t)
    both = size[..., a] + size[..., b]
    size[..., a], size[..., b] = both, both
    return y, size


def near(got, want, size, dtype):
    """One rounding of the result, and before it, of either term: 2^-20 for the norm (a sum of D squares,
    two products), 2^-22 for the angle's sine or cosine (an angle to 2^-25 turns), 2^-22 for the rest."""
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -24 if dtype == F16 else 2.0 ** -120
    off = (got.double() - want).abs() - (half * want.abs() + 2.0 ** -18 * size + tiny)
    assert not torch.isnan(got).any() and (off <= 0).all(), "%g past its bound" % off.max()


def frequencies(R, base=10000.0):
    return base ** (-torch.arange(R // 2, dtype=F64) / max(R // 2, 1)) if R else None


class Case:
    def __init__(self, tree, N, Hq, Hkv, D, R, dtype, pairs=False, norm=True, far=False, seed=0, eps=1e-6):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + N + D)
        self.g, self.N, self.Hq, self.Hkv, self.D, self.dtype, self.eps, self.pairs = g, N, Hq, Hkv, D, dtype, eps, pairs
        fused = torch.randn(N, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dtype)
        self.q, self.k, self.v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        self.position = torch.randint(0, 2 ** 31 - 1 if far else 5000, (N,), generator=g, device="cuda").int()
        if N > 3:
            self.position[:3] = torch.tensor([0, 2 ** 31 - 1 if far else 131071, -7])
        self.freq = frequencies(R)
        self.norms = [0.5 + torch.rand(D, generator=g, device="cuda") for _ in range(2)] if norm else [None, None]
        self.rotation = tree.Rotation(D, self.freq, *self.norms, eps=eps, interleaved=pairs)
        self.tree = tree.Tree(Hq, Hkv, D, dtype)

    def want(self, which):
        return formula(getattr(self, which), self.position, None if self.freq is None else self.freq.cuda(),
                       self.norms[which == "k"], self.eps, self.pairs)


SHAPES = [
    # N, Hq, Hkv, D, R
    (1, 32, 8, 128, 128),
    (2, 4, 4, 16, 16),
    (7, 14, 2, 96, 64),
    (128, 32, 8, 128, 128),
    (333, 5, 1, 64, 32),
    (600, 40, 8, 128, 64),
    (1217, 3, 3, 80, 48),
    (50, 64, 8, 112, 112),
    (21, 6, 2, 48, 0),
    (5000, 16, 2, 32, 32),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pairs,norm,far", [(False, True, False), (True, True, True), (False, False, True), (True, False, False)])
@pytest.mark.parametrize("N,Hq,Hkv,D,R", SHAPES)
def test_rotate(tree, N, Hq, Hkv, D, R, dtype, pairs, norm, far):
    c = Case(tree, N, Hq, Hkv, D, R, dtype, pairs, norm, far)
    q, k = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    assert q.shape == (N, Hq, D) and k.shape == (N, Hkv, D)
    near(q, *c.want("q"), dtype)
    near(k, *c.want("k"), dtype)
    assert c.tree.status() == 0


def cache_of(tree, held, n_pages, page, Hkv, D, dtype, fill=0x11):
    c = tree.KVCache.zeros(n_pages, page, Hkv, D, {"16": dtype, "e4m3": E4M3, "e2m1": torch.uint8}[held])
    for x in (c.k, c.v):
        x.view(torch.uint8).fill_(fill)
    for x in (c.k_scale, c.v_scale):
        if x is not None:
            x.fill_(fill)
    return c


def bits(cache):
    return [x.view(torch.uint8).clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale) if x is not None]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pairs,norm", [(False, True), (True, True), (False, False)])
@pytest.mark.parametrize("held", ["16", "e4m3", "e2m1"])
@pytest.mark.parametrize("N,Hq,Hkv,D,R", [s for s in SHAPES if s[3] % 32 == 0])
def test_place_is_rotate_and_write(tree, N, Hq, Hkv, D, R, dtype, pairs, norm, held):
    """The same bits in q and in the cache, slots in any order, rows left out, nothing else touched."""
    c = Case(tree, N, Hq, Hkv, D, R, dtype, pairs, norm)
    page = 24
    n_pages = N // page + 3
    slot = torch.randperm(n_pages * page, generator=c.g, device="cuda")[:N].int()
    left_out = torch.rand(N, generator=c.g, device="cuda") < 0.2
    left_out[0] = False
    a, b = (cache_of(tree, held, n_pages, page, Hkv, D, dtype) for _ in range(2))
    q, k = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    out = torch.full_like(q, 7.0)
    got = c.tree.place(a, torch.where(left_out, torch.full_like(slot, -1), slot), c.q, c.k, c.v, c.position, c.rotation,
                       out=out)
    # write puts single rows at a position of requests of one row each
    keep = torch.nonzero(~left_out)[:, 0]
    pages = (slot[keep] // page)[:, None].contiguous()
    first = torch.arange(len(keep) + 1, dtype=torch.int32, device="cuda")
    c.tree.write(b, pages, (slot[keep] % page).contiguous(), first, k[keep], c.v[keep])
    assert c.tree.status() == 0
    assert torch.equal(got[keep], q[keep]) and (got[left_out] == 7).all()
    assert all(torch.equal(x, y) for x, y in zip(bits(a), bits(b)))


@pytest.mark.parametrize("held", ["16", "e4m3", "e2m1"])
def test_rows_that_are_not_finite_stay_their_own(tree, held):
    """NaN and infinities of a row reach that row's head; of the part that is not turned, their element."""
    c = Case(tree, 40, 8, 2, 64, 32, BF16, norm=False)
    clean = [x.clone() for x in (c.q, c.k, c.v)]
    q, k = c.tree.rotate(*clean[:2], c.position, c.rotation)
    c.q[5, 3, 2], c.q[6, 1, 40], c.k[7, 1, 63] = math.nan, math.inf, -math.inf
    q2, k2 = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    assert torch.isnan(q2[5, 3, [2, 18]]).all() and q2[6, 1, 40] == math.inf and k2[7, 1, 63] == -math.inf
    q2[5, 3, [2, 18]], q2[6, 1, 40], k2[7, 1, 63] = q[5, 3, [2, 18]], q[6, 1, 40], k[7, 1, 63]
    assert torch.equal(q, q2) and torch.equal(k, k2)
    slot = torch.arange(40, dtype=torch.int32, device="cuda")
    a, b = (cache_of(tree, held, 3, 16, 2, 64, BF16) for _ in range(2))
    c.tree.place(a, slot, *clean, c.position, c.rotation)
    c.tree.place(b, slot, c.q, c.k, c.v, c.position, c.rotation)
    pages, z = torch.arange(3, dtype=torch.int32, device="cuda")[None], torch.zeros(1, dtype=torch.int32, device="cuda")
    first = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    x, y = (c.tree.read(m, pages, z, first, 40) for m in (a, b))
    assert torch.equal(x[1], y[1])
    hit = torch.zeros(40, 2, 64, dtype=torch.bool, device="cuda")
    hit[7, 1, slice(None) if held == "e4m3" else slice(48, 64) if held == "e2m1" else slice(63, 64)] = True
    assert torch.equal(x[0][~hit], y[0][~hit]) and not torch.isfinite(y[0][hit]).any()


def test_norm_of_zero_and_large_rows(tree):
    c = Case(tree, 30, 4, 2, 64, 64, F16, seed=3)
    c.q[3], c.q[4], c.k[5] = 0.0, 60000.0, 6e-8
    q, k = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    near(q, *c.want("q"), F16)
    near(k, *c.want("k"), F16)


def test_norms_of_one_side_and_refusals(tree):
    from serial_draft_head_gb300 import walk
    c = Case(tree, 9, 4, 2, 64, 64, BF16)
    for norms in ((c.norms[0], None), (None, c.norms[1])):
        rotation = tree.Rotation(64, c.freq, *norms)
        got = c.tree.rotate(c.q, c.k, c.position, rotation)
        for x, y, w in zip(got, (c.q, c.k), norms):
            near(x, *formula(y, c.position, c.freq.cuda(), w, 1e-6, False), BF16)
    for bad in (lambda: tree.Rotation(72, c.freq), lambda: tree.Rotation(64, frequencies(80)), lambda: tree.Rotation(64, frequencies(8)),
                lambda: tree.Rotation(64, c.freq, c.norms[0][:32]), lambda: tree.Rotation(64, c.freq, eps=-1.0),
                lambda: tree.Rotation(64, torch.full((32,), math.inf)),
                lambda: c.tree.rotate(c.q, c.k[:8], c.position, c.rotation),
                lambda: c.tree.rotate(c.q, c.k, c.position[:8], c.rotation),
                lambda: c.tree.rotate(c.q, c.k, c.position.long(), c.rotation),
                lambda: c.tree.rotate(c.q, c.k, c.position, tree.Rotation(128, frequencies(64))),
                lambda: c.tree.rotate(c.q.to(F16), c.k, c.position, c.rotation)):
        with pytest.raises(ValueError):
            bad()
    cache = cache_of(tree, "e2m1", 2, 16, 2, 64, BF16)
    slot = torch.arange(9, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        c.tree.place(cache, slot.long(), c.q, c.k, c.v, c.position, c.rotation)
    with pytest.raises(ValueError):
        c.tree.place(cache, slot, c.q, c.k, c.v[:8], c.position, c.rotation)
    # a slot past the cache is left out and reported
    before = bits(cache)
    slot[4] = 32
    out = torch.full((9, 4, 64), 7.0, dtype=BF16, device="cuda")
    c.tree.place(cache, slot, c.q, c.k, c.v, c.position, c.rotation, out=out)
    assert c.tree.status() == walk.EPAGES and (out[4] == 7).all() and not (out[5] == 7).all()
    assert all(torch.equal(x[:, 9:], y[:, 9:]) and torch.equal(x[:, 4], y[:, 4]) for x, y in zip(before, bits(cache))
               if x.shape[0] == 2) and c.tree.status() == 0
    # no rows
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    q, k = c.tree.rotate(c.q[:0], c.k[:0], e, c.rotation)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    c.tree.place(cache, e, c.q[:0], c.k[:0], c.v[:0], e, c.rotation)


def test_stream_and_graph(tree):
    """On another stream, and replayed from a graph with positions and slots that have changed."""
    c = Case(tree, 70, 8, 2, 128, 128, BF16)
    cache = cache_of(tree, "e2m1", 8, 16, 2, 128, BF16)
    slot = torch.randperm(128, generator=c.g, device="cuda")[:70].int()
    want = c.tree.place(cache, slot, c.q, c.k, c.v, c.position, c.rotation)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = cache_of(tree, "e2m1", 8, 16, 2, 128, BF16)
    side.wait_stream(torch.cuda.current_stream())
    q = c.tree.place(other, slot, c.q, c.k, c.v, c.position, c.rotation, stream=side)
    side.synchronize()
    assert torch.equal(q, want) and all(torch.equal(x, y) for x, y in zip(bits(cache), bits(other)))
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tree.place(other, slot, c.q, c.k, c.v, c.position, c.rotation, out=out)
    slot.copy_(slot.flip(0))
    c.position += 11
    graph.replay()
    fresh = cache_of(tree, "e2m1", 8, 16, 2, 128, BF16)
    want = c.tree.place(fresh, slot, c.q, c.k, c.v, c.position, c.rotation)
    assert torch.equal(out, want)
    at = slot.long()
    assert all(torch.equal(x[at // 16, at % 16], y[at // 16, at % 16]) for x, y in zip(bits(other), bits(fresh)))
