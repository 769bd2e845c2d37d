"""The draft-check operators over a cache in 4 bits, against their definitions in 64 bits."""
import math

import pytest
import torch

import e2m1_reference as e2m1
import tree_reference as ref
from test_gpu_tree import BF16, F16, same, special_rows, tree  # noqa: F401

pytestmark = pytest.mark.gpu


class Case:
    """A 4-bit cache with random rows, its page tables, and the packed rows of some requests.  Slots
    that no request owns hold blocks that are no numbers."""

    def __init__(self, tree, Hq, Hkv, D, page, dtype, T, L, seed, spare=3, mask="tree", spread=1.0,
                 max_nodes=None, garbage=True, head_major=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lib, self.g, self.Hq, self.Hkv, self.D, self.page, self.dtype = tree, g, Hq, Hkv, D, page, dtype
        self.T, self.L, self.B, self.N = T, L, len(T), sum(T)
        P = max([-(-(t + n) // page) for t, n in zip(T, L)] + [1])
        self.n_pages = self.B * P + spare
        self.pages = torch.randperm(self.n_pages, generator=g, device="cuda")[:self.B * P].int().view(self.B, P)
        owned = torch.zeros(self.n_pages, page, dtype=torch.bool, device="cuda")
        for b in range(self.B):
            at = torch.arange(L[b] + T[b], device="cuda")
            owned[self.pages[b][at // page].long(), at % page] = True
        data = []
        for _ in range(2):
            x = torch.randn(self.n_pages, page, Hkv, D, generator=g, device="cuda") * spread
            value, byte = e2m1.quantise(x)
            codes = e2m1.pack(value)
            if garbage:
                byte[~owned], codes[~owned] = 255, 0x5a
            for y in (codes, byte):
                data.append(y.transpose(1, 2).contiguous().transpose(1, 2) if head_major else y)
        self.k, self.ks, self.v, self.vs = data
        self.length = torch.tensor(L, dtype=torch.int32, device="cuda")
        self.first = torch.tensor([sum(T[:b]) for b in range(self.B + 1)], dtype=torch.int32, device="cuda")
        self.q = torch.randn(self.N, Hq, D, generator=g, device="cuda").to(dtype)
        self.mask = None
        if mask == "tree":
            parent = [-1 if i == 0 else max(0, i - 1 - (i * 7 + t) % 5) for t in T for i in range(t)]
            self.mask = tree.ancestor_bits(torch.tensor(parent, dtype=torch.int32, device="cuda"), self.first)
        elif mask == "random":
            w = (max(T) + 31) // 32
            self.mask = torch.randint(-2 ** 31, 2 ** 31, (self.N, w), generator=g, device="cuda").int()
        self.cache = tree.KVCache(self.k, self.v, self.ks, self.vs)
        self.tree = tree.Tree(Hq, Hkv, D, dtype, max_requests=self.B, max_nodes=max_nodes or max(T + [1]))

    def attend(self, **kw):
        r = self.tree.attend(self.q, self.cache, self.pages, self.length, self.first, mask=self.mask, **kw)
        assert self.tree.status(stream=kw.get("stream")) == 0      # a call of the handle as any other: in order
        return r

    def check(self, out, lse, scale=None, softcap=0.0, rows=slice(None)):
        scale = self.D ** -0.5 if scale is None else scale
        k, v = e2m1.values(self.k, self.ks), e2m1.values(self.v, self.vs)
        want, want_lse, weight, sums = ref.attend(self.q, k, v, None, None, self.pages, self.page, self.length,
                                                  self.first, self.mask, scale, softcap)
        tol, tol_lse = e2m1.bounds(want, weight, sums, self.D, self.dtype, softcap, max(self.T) + max(self.L),
                                   self.q.abs().max().item() * abs(scale), torch.nan_to_num(k).abs().max().item(),
                                   torch.nan_to_num(v).abs().max().item(),
                                   self.N * self.Hq // self.Hkv > 32 * self.B)
        out, lse, want, want_lse, tol, tol_lse = (x[rows] for x in (out, lse, want, want_lse, tol, tol_lse))
        assert not torch.isnan(out).any() and not torch.isnan(lse).any()
        off = (out.double() - want).abs() - tol
        assert (off <= 0).all(), "out is %g past its bound" % off.max()
        empty = torch.isinf(want_lse)
        assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
        far = (lse.double() - want_lse)[~empty].abs() - tol_lse[~empty]
        assert (far <= 0).all(), "lse is %g past its bound" % far.max()


# ---------------------------------------------------------------- the cache --

ROWS = [
    # Hkv, D, page, T, L
    (8, 128, 16, [8] * 16, [11 * i for i in range(16)]),
    (1, 32, 1, [1], [0]),
    (2, 96, 24, [33, 0, 400], [5, 7, 23]),
    (5, 64, 7, [1] * 40, list(range(40))),
    (16, 64, 64, [700, 1500], [63, 64]),
    (3, 32, 32, [5000], [31]),
]


@pytest.mark.parametrize("head_major", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hkv,D,page,T,L", ROWS)
def test_write_and_read(tree, Hkv, D, page, T, L, dtype, head_major):
    c = Case(tree, Hkv, Hkv, D, page, dtype, T, L, seed=D, mask=None, max_nodes=1, head_major=head_major)
    k = special_rows(torch.randn(c.N, Hkv, D, generator=c.g, device="cuda").to(dtype))
    v = (torch.randn(c.N, Hkv, D, generator=c.g, device="cuda") * 100).to(dtype)
    before = [x.clone() for x in (c.k, c.ks, c.v, c.vs)]
    c.tree.write(c.cache, c.pages, c.length, c.first, k, v)
    got = c.tree.read(c.cache, c.pages, c.length, c.first, c.N)
    assert c.tree.status() == 0
    touched = torch.zeros(c.n_pages, page, dtype=torch.bool, device="cuda")
    for b in range(c.B):
        at = torch.arange(L[b], L[b] + T[b], device="cuda")
        touched[c.pages[b][at // page].long(), at % page] = True
    for x, codes, byte, old, old_byte, back in ((k, c.k, c.ks, *before[:2], got[0]), (v, c.v, c.vs, *before[2:], got[1])):
        value, want_byte = e2m1.quantise(x)
        assert torch.equal(codes[~touched], old[~touched]) and torch.equal(byte[~touched], old_byte[~touched])
        for b in range(c.B):
            at = torch.arange(L[b], L[b] + T[b], device="cuda")
            where = c.pages[b][at // page].long(), at % page
            rows = slice(int(c.first[b]), int(c.first[b + 1]))
            assert torch.equal(byte[where], want_byte[rows])
            assert torch.equal(e2m1.unpack(codes[where]), value[rows])             # a zero's sign is free
        want = value * e2m1.scale_of(want_byte).repeat_interleave(16, -1)
        assert same(back.double(), want)                                           # exact in the handle's type


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_write_every_16_bit_value(tree, dtype):
    """Every value as a block's only one, and below others: all borders of scales and codes."""
    bits = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(dtype)
    x = torch.zeros(65536, 1, 32, dtype=dtype, device="cuda")
    x[:, 0, 3] = bits
    x[:, 0, 16:] = torch.stack([bits] + [bits.roll(1237 * i) for i in range(1, 16)], 1)
    y = torch.zeros_like(x)
    # ties: every border between codes times every scale, beside six times that scale
    scales = e2m1.scale_of(torch.arange(227, device="cuda"))[1:]
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=torch.float64, device="cuda")
    ties = scales[:, None] * border
    fits = (ties.to(dtype).double() == ties).all(1)
    ties = torch.cat([ties, -ties], 1)[fits].to(dtype)
    assert len(ties) > 100
    y[:len(ties), 0, :16] = ties
    # and their neighbours among the type's values, the six left as it is
    near = ties.view(torch.int16).clone()
    near[:, [i for i in range(16) if i % 8 != 7]] += 1
    y[:len(ties), 0, 16:] = near.view(dtype)
    t = tree.Tree(1, 1, 32, dtype)
    cache = tree.KVCache.zeros(1024, 64, 1, 32, torch.uint8)
    pages = torch.arange(1024, dtype=torch.int32, device="cuda")[None]
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = torch.tensor([0, 65536], dtype=torch.int32, device="cuda")
    t.write(cache, pages, z, first, x, y)
    back = t.read(cache, pages, z, first, 65536)
    assert t.status() == 0
    for src, codes, byte, got in ((x, cache.k, cache.k_scale, back[0]), (y, cache.v, cache.v_scale, back[1])):
        value, want_byte = e2m1.quantise(src[:, 0])
        assert torch.equal(byte.transpose(1, 2).reshape(65536, 2), want_byte)
        assert torch.equal(e2m1.unpack(codes.transpose(1, 2).reshape(65536, 16)), value)
        assert same(got[:, 0].double(), value * e2m1.scale_of(want_byte).repeat_interleave(16, -1))


@pytest.mark.parametrize("D,page", [(128, 16), (96, 5), (32, 64)])
def test_keep(tree, D, page):
    T, L = [9, 40, 1, 0, 17], [3, 63, 130, 7, 0]
    c = Case(tree, 4, 2, D, page, BF16, T, L, seed=30 + D, mask=None)
    keep = [5, 17, 1, 0, 17]
    path = torch.zeros(5, 20, dtype=torch.int32, device="cuda")
    for b, n in enumerate(keep):
        path[b, :n] = torch.randperm(max(T[b], 1), generator=c.g, device="cuda")[:n].sort().values.int()
    want = [x.clone() for x in (c.k, c.ks, c.v, c.vs)]
    for b, n in enumerate(keep):
        to, fr = torch.arange(n, device="cuda") + L[b], path[b, :n].long() + L[b]
        for x in want:
            x[c.pages[b][to // page].long(), to % page] = x[c.pages[b][fr // page].long(), fr % page]
    c.tree.keep(c.cache, c.pages, c.length, path, torch.tensor(keep, dtype=torch.int32, device="cuda"))
    assert c.tree.status() == 0
    assert all(torch.equal(x, y) for x, y in zip((c.k, c.ks, c.v, c.vs), want))


# ---------------------------------------------------------------- attention --

SHAPES = [
    # Hq, Hkv, D, page, T, L
    (1, 1, 64, 16, [1], [0]),                          # one key: itself
    (8, 2, 128, 16, [1], [37]),
    (4, 4, 128, 16, [1, 1, 1, 1, 1], [31, 32, 33, 63, 64]),    # around a block's end
    (32, 8, 128, 16, [8] * 4, [300, 1, 0, 777]),
    (32, 8, 128, 64, [17], [5000]),                    # one request over many SMs
    (16, 2, 64, 1, [3, 5], [130, 64]),                 # pages of one slot
    (14, 2, 96, 24, [5, 33, 1, 61], [10, 200, 511, 3]),
    (6, 1, 96, 7, [64], [250]),
    (24, 8, 32, 100, [9, 0, 2], [99, 50, 101]),        # a request without rows
    (5, 5, 32, 32, [2, 40], [64, 65]),
    (40, 8, 128, 16, [26, 51], [384, 385]),            # 130 and 255 rows a head
    (8, 1, 128, 128, [256], [1000]),                   # the largest tree: 2,048 rows a head
    (16, 1, 32, 48, [16, 17, 8, 9], [0, 0, 0, 0]),     # no context
    (2, 1, 128, 16, [1] * 300, [i % 67 for i in range(300)]),
    (64, 8, 128, 64, [1] * 20, [100 + 211 * i for i in range(20)]),
    (16, 2, 64, 64, [1, 2, 1], [70, 4000, 129]),       # nine to sixteen rows a head
    (3, 1, 64, 16, [43, 86], [0, 2000]),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D,page,T,L", SHAPES)
def test_attend_shapes(tree, Hq, Hkv, D, page, T, L, dtype):
    c = Case(tree, Hq, Hkv, D, page, dtype, T, L, seed=Hq * 1000 + D)
    c.check(*c.attend())


@pytest.mark.parametrize("mask", [None, "tree", "random"])
@pytest.mark.parametrize("softcap", [0.0, 0.5, 30.0])
@pytest.mark.parametrize("T,L", [([70, 1, 26, 130], [129, 7, 0, 1000]), ([1, 3, 2], [129, 7, 2000])])
def test_attend_masks_and_cap(tree, mask, softcap, T, L):
    c = Case(tree, 10, 2, 64, 20, BF16, T, L, seed=5, mask=mask)
    c.check(*c.attend(softcap=softcap), softcap=softcap)


@pytest.mark.parametrize("T,L", [([9, 40], [600, 33]), ([1, 2], [600, 33]), ([3, 4], [100, 1200])])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale,spread", [(1.0, 4.0), (-0.3, 1.0), (0.0, 1.0), (0.01, 0.01)])
def test_attend_large_and_small_scores(tree, scale, spread, dtype, T, L):
    """Sharp softmax (scores of hundreds), negative, equal and tiny scores."""
    c = Case(tree, 8, 2, 128, 16, dtype, T, L, seed=6, spread=spread)
    c.check(*c.attend(scale=scale), scale=scale)


@pytest.mark.parametrize("order", ["up", "down"])
@pytest.mark.parametrize("T", [4, 40])
def test_attend_rising_maximum(tree, order, T):
    """Scores that rise (or fall) along the cache, fast enough to move the running maximum often."""
    c = Case(tree, 4, 1, 64, 16, BF16, [T], [2000], seed=7, mask=None)
    total = 2000 + T
    at = torch.arange(total, device="cuda")
    ramp = (at if order == "up" else total - at).float() * 0.05
    c.q[:] = 1.0
    value, byte = e2m1.quantise(ramp[:, None, None].expand(total, 1, 64))
    c.k[c.pages[0][at // 16].long(), at % 16] = e2m1.pack(value)
    c.ks[c.pages[0][at // 16].long(), at % 16] = byte
    c.check(*c.attend())


@pytest.mark.parametrize("T,L", [([40, 3, 200], [0, 0, 5]), ([2, 1, 1], [0, 0, 5])])
def test_attend_rows_that_see_nothing(tree, T, L):
    """An empty mask row without context: out 0, lse -inf; its neighbours are unaffected."""
    c = Case(tree, 8, 2, 128, 16, BF16, T, L, seed=8)
    c.mask[::3] = 0
    out, lse = c.attend()
    c.check(out, lse)
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()


@pytest.mark.parametrize("T,L", [([9, 150], [130, 20]), ([3, 2], [130, 20])])
@pytest.mark.parametrize("byte", [255, 227, 248])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attend_invisible_rows_hold_anything(tree, T, L, byte, where):
    """Blocks that are no numbers of a node reach the nodes that see it and no other."""
    c = Case(tree, 4, 2, 64, 16, BF16, T, L, seed=9, mask=None)
    parent = torch.tensor([i for t in T for i in [-1] + [0] * (t - 1)], dtype=torch.int32, device="cuda")
    c.mask = tree.ancestor_bits(parent, c.first)       # all nodes are children of node 0
    node = {0: T[0] - 1, 1: T[1] - 1}
    clean_out, clean_lse = c.attend()
    for b, j in node.items():
        p = L[b] + j
        (c.ks if where == "k" else c.vs)[c.pages[b][p // 16].long(), p % 16, :, 1] = byte
    out, lse = c.attend()
    hit = torch.tensor([T[0] - 1, c.N - 1], device="cuda")
    rest = torch.ones(c.N, dtype=torch.bool, device="cuda")
    rest[hit] = False
    assert torch.equal(out[rest], clean_out[rest]) and torch.equal(lse[rest], clean_lse[rest])
    if where == "v":
        assert torch.equal(lse[hit], clean_lse[hit])
        assert torch.isnan(out[hit][..., 16:32]).all()
        other = [i for i in range(64) if i not in range(16, 32)]
        assert torch.equal(out[hit][..., other], clean_out[hit][..., other])
    elif byte == 255:
        assert torch.isnan(out[hit]).all()


@pytest.mark.parametrize("T,L", [([5, 6], [130, 20]), ([1, 2], [130, 20])])
def test_attend_nan_reaches_its_rows(tree, T, L):
    """A NaN in a row of q is that row's alone; one in the context is all rows' of its request and head."""
    c = Case(tree, 4, 2, 64, 16, BF16, T, L, seed=10)
    clean, _ = c.attend()
    c.q[0, 1, 7] = math.nan
    out, lse = c.attend()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    rest = torch.ones(c.N, 4, dtype=torch.bool, device="cuda")
    rest[0, 1] = False
    assert torch.equal(out[rest], clean[rest])
    c.q[0, 1, 7] = 1.0
    c.vs[c.pages[0][3].long(), 5, 1, 2] = 255
    out, lse = c.attend()
    assert not torch.isnan(lse).any()
    hit = torch.zeros(c.N, 4, 64, dtype=torch.bool, device="cuda")
    hit[:T[0], 2:, 32:48] = True
    assert torch.equal(torch.isnan(out), hit)


@pytest.mark.parametrize("T", [[7, 30], [1, 3]])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_attend_strides(tree, T, D):
    """Heads after slots, K and V in one tensor, scales beside codes, q inside a fused projection."""
    c = Case(tree, 12, 4, D, 16, BF16, T, [100, 257], seed=11)
    out, lse = c.attend()
    wide = torch.zeros(c.n_pages, 16, 4, 2, D // 2 + 16, dtype=torch.uint8, device="cuda")
    wide[..., 0, :D // 2], wide[..., 1, :D // 2] = c.k, c.v
    wide[..., 0, D // 2:D // 2 + D // 16], wide[..., 1, D // 2:D // 2 + D // 16] = c.ks, c.vs
    k, v = wide[..., 0, :D // 2], wide[..., 1, :D // 2]
    ks, vs = (wide[..., i, D // 2:D // 2 + D // 16] for i in range(2))
    fused = torch.randn(c.N, 20, D, device="cuda").to(BF16)
    fused[:, 4:16] = c.q
    pages = torch.full((c.B, c.pages.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    pages[:, :c.pages.shape[1]] = c.pages
    mask = torch.cat([c.mask, c.mask + 1], 1)[:, :c.mask.shape[1]]
    o2, l2 = c.tree.attend(fused[:, 4:16], tree.KVCache(k, v, ks, vs), pages, c.length, c.first, mask=mask)
    assert c.tree.status() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("T", [[8] * 5, [1] * 5])
def test_attend_repeats_and_graph(tree, T):
    """The same bits every time, on another stream, and replayed from a graph after the lengths have
    changed."""
    c = Case(tree, 32, 8, 128, 16, BF16, T, [3000, 10, 0, 900, 4000], seed=12)
    out, lse = c.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = c.attend(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask, out=o3, lse=l3)
    for L in ([3000, 10, 0, 900, 4000], [17, 10, 0, 900, 2]):
        c.L = L
        c.length.copy_(torch.tensor(L, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check(o3, l3)


@pytest.mark.parametrize("T,page", [([17], 64), ([17], 24), ([1], 64), ([2], 16)])
def test_attend_back_to_back(tree, T, page):
    """Long shares of every CTA, calls over several caches in a row without a wait between."""
    cases = [Case(tree, 32, 8, 128, page, BF16, T, [40000 + 511 * i], seed=40 + i, spare=1, mask=None)
             for i in range(3)]
    want = [c.attend() for c in cases]
    cases[1].check(*want[1])
    for _ in range(20):
        got = [c.tree.attend(c.q, c.cache, c.pages, c.length, c.first) for c in cases * 4]
        for i, (o, l) in enumerate(got):
            assert torch.equal(o, want[i % 3][0]) and torch.equal(l, want[i % 3][1])
    assert all(c.tree.status() == 0 for c in cases)


@pytest.mark.parametrize("T", [1, 20])
def test_attend_one_item_over_all_workers(tree, T):
    """A single cached head: every SM has a part of the one item."""
    c = Case(tree, 4, 1, 64, 16, F16, [T], [60000], seed=50, mask=None)
    c.check(*c.attend())


@pytest.mark.parametrize("T", [[4] * 6, [4] * 5 + [5], [1] * 11 + [33], [0, 0, 0, 12], [17, 1, 64, 65, 3], [2] * 4])
def test_attend_rows_of_all_kernels(tree, T):
    """Averages of rows around which the kernels change, with requests above and below them."""
    L = [(311 * i + 95) % 1500 for i in range(len(T))]
    c = Case(tree, 16, 4, 128, 16, BF16, T, L, seed=60 + len(T))
    c.check(*c.attend())


@pytest.mark.parametrize("T", [[1, 3], [30, 2]])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attend_scales_of_any_size(tree, T, dtype):
    """Blocks under every scale that there is, the smallest and the largest, one by one among others."""
    c = Case(tree, 8, 2, 64, 20, dtype, T, [700, 300], seed=71)
    for scale, top in ((c.vs, 226 if dtype == BF16 else 200), (c.ks, 150)):
        keep = scale == 255
        some = torch.rand(scale.shape, generator=c.g, device="cuda") < 0.3
        any_ = torch.randint(0, top + 1, scale.shape, generator=c.g, device="cuda").to(torch.uint8)
        scale[some & ~keep] = any_[some & ~keep]
    c.check(*c.attend(scale=0.002), scale=0.002)


@pytest.mark.parametrize("T", [1, 30])
def test_attend_slots_past_the_end_change_no_bit(tree, T):
    """What stands behind a request's rows in its last page is not gone by."""
    c = Case(tree, 8, 2, 128, 64, BF16, [T], [70], seed=72)
    out, lse = c.attend()
    clean = Case(tree, 8, 2, 128, 64, BF16, [T], [70], seed=72, garbage=False)
    o2, l2 = clean.attend()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("T", [1, 30])
def test_attend_far_offsets(tree, T):
    """A cache of more than 2^32 bytes: pages at its far end."""
    page, Hkv, D = 64, 8, 128
    n_pages = (1 << 32) // (page * Hkv * D // 2) + 40
    c = Case(tree, 16, Hkv, D, page, BF16, [T, 3], [300, 20], seed=14)
    shift = n_pages - c.n_pages
    big = torch.zeros(n_pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda").transpose(1, 2)
    small = torch.zeros(n_pages, Hkv, page, D // 16, dtype=torch.uint8, device="cuda").transpose(1, 2)
    big[shift:], small[shift:] = c.v, c.vs
    c.v, c.vs = big, small
    big2, small2 = big.clone(), small.clone()          # clone keeps the strides
    big2[shift:], small2[shift:] = c.k, c.ks
    c.k, c.ks = big2, small2
    c.pages += shift
    c.cache = tree.KVCache(c.k, c.v, c.ks, c.vs)
    out, lse = c.attend()
    c.k, c.v, c.ks, c.vs = (x[shift:] for x in (c.k, c.v, c.ks, c.vs))
    c.pages -= shift
    c.check(out, lse)
    c.pages += shift
    new = torch.randn(T + 3, Hkv, D, device="cuda").to(BF16)
    c.tree.write(c.cache, c.pages, c.length, c.first, new, new)
    got, _ = c.tree.read(c.cache, c.pages, c.length, c.first, T + 3)
    value, byte = e2m1.quantise(new)
    assert torch.equal(got.double(), value * e2m1.scale_of(byte).repeat_interleave(16, -1))
    assert c.tree.status() == 0


@pytest.mark.parametrize("T", [[2, 3, 1], [20, 30, 9]])
def test_device_checks_leave_the_others_alone(tree, T):
    """A bad page, and lengths that do not fit: reported, and the other requests' rows are right."""
    from serial_draft_head_gb300 import walk
    c = Case(tree, 8, 2, 128, 16, BF16, T, [100, 40, 70], seed=80)
    out, lse = c.attend()
    bad = c.pages.clone()
    bad[1, 1] = c.n_pages
    mine, mine_lse = torch.empty_like(out), torch.empty_like(lse)
    for pages, length in ((bad, c.length), (c.pages, torch.tensor([100, -1, 70], dtype=torch.int32, device="cuda")),
                          (c.pages, torch.tensor([100, 1 << 30, 70], dtype=torch.int32, device="cuda"))):
        mine[:], mine_lse[:] = 7.0, 7.0
        c.tree.attend(c.q, c.cache, pages, length, c.first, mask=c.mask, out=mine, lse=mine_lse)
        assert c.tree.status() == walk.EPAGES and c.tree.status() == 0
        for rows in (slice(0, T[0]), slice(T[0] + T[1], c.N)):
            c.check(mine, mine_lse, rows=rows)
        if pages is c.pages:
            assert (mine[T[0]:T[0] + T[1]] == 7).all()


def test_refusals(tree):
    from serial_draft_head_gb300 import walk
    t = tree.Tree(4, 2, 64, BF16, max_requests=2, max_nodes=4)
    good = tree.KVCache.zeros(2, 16, 2, 64, torch.uint8)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pages = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    q = torch.ones(1, 4, 64, dtype=BF16, device="cuda")
    t.attend(q, good, pages, z, first)
    with pytest.raises(ValueError):
        tree.KVCache(good.k, good.v)                                       # no scales
    with pytest.raises(ValueError):
        tree.KVCache(good.k, good.v, good.k_scale[..., :2], good.v_scale)
    with pytest.raises(ValueError):
        tree.KVCache(good.k, good.v, good.k_scale.float(), good.v_scale)
    odd = torch.zeros(2, 16, 2, 6, dtype=torch.uint8, device="cuda")[..., 1:5]
    with pytest.raises(walk.WalkError):                                    # scales not on their step
        t.attend(q, tree.KVCache(good.k, good.v, odd, good.v_scale), pages, z, first)
    narrow = torch.zeros(2, 16, 2, 40, dtype=torch.uint8, device="cuda")[..., :32]
    with pytest.raises(walk.WalkError):                                    # rows not on 16 bytes
        t.attend(q, tree.KVCache(narrow, good.v, good.k_scale, good.v_scale), pages, z, first)
    with pytest.raises(ValueError):                                        # another head size
        t.attend(q, tree.KVCache.zeros(2, 16, 2, 32, torch.uint8), pages, z, first)
    u = tree.Tree(4, 2, 80, BF16)
    wide = torch.zeros(2, 16, 2, 48, dtype=torch.uint8, device="cuda")[..., :40]
    five = torch.zeros(2, 16, 2, 5, dtype=torch.uint8, device="cuda")
    with pytest.raises(walk.WalkError):                                    # heads of 80
        u.write(tree.KVCache(wide, wide.clone(), five, five), pages, z, first,
                torch.zeros(1, 2, 80, dtype=BF16, device="cuda"), torch.zeros(1, 2, 80, dtype=BF16, device="cuda"))
    assert t.status() == 0
