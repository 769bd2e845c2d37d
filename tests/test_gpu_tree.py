"""The draft-check operators on the GPU against their definitions in 64 bits."""
import math

import pytest
import torch

import tree_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="session")
def tree():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    from serial_draft_head_gb300 import tree as t
    t.load()
    return t


class Case:
    """A cache with random rows, its page tables, and the packed rows of some requests."""

    def __init__(self, tree, Hq, Hkv, D, page, dtype, cache, T, L, seed, spare=3, garbage=math.nan,
                 mask="tree", spread=1.0, max_nodes=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.Hq, self.Hkv, self.D, self.page, self.dtype = g, Hq, Hkv, D, page, dtype
        self.T, self.L, self.B, self.N = T, L, len(T), sum(T)
        P = max([-(-(t + n) // page) for t, n in zip(T, L)] + [1])
        self.n_pages = self.B * P + spare
        self.pages = torch.randperm(self.n_pages, generator=g, device="cuda")[:self.B * P] \
            .int().view(self.B, P)
        e4m3 = cache == "e4m3"
        shape = (self.n_pages, page, Hkv, D)
        self.k, self.v, self.ks, self.vs = [], [], None, None
        data = []
        for _ in range(2):
            x = torch.randn(shape, generator=g, device="cuda") * spread
            if e4m3:
                code, byte = ref.quantise(x)
                data.append((code.to(torch.float32).to(E4M3), byte))
            else:
                data.append((x.to(dtype), None))
        # slots that no request owns hold garbage
        owned = torch.zeros(self.n_pages, page, dtype=torch.bool, device="cuda")
        for b in range(self.B):
            at = torch.arange(L[b] + T[b], device="cuda")
            owned[self.pages[b][at // page].long(), at % page] = True
        for x, byte in data:
            if garbage is not None:
                y = x.view(torch.uint8) if e4m3 else x
                y[~owned] = 0x7f if e4m3 else garbage
                if e4m3:
                    byte[~owned] = 255
        (self.k, self.ks), (self.v, self.vs) = data
        self.length = torch.tensor(L, dtype=torch.int32, device="cuda")
        self.first = torch.tensor([sum(T[:b]) for b in range(self.B + 1)], dtype=torch.int32,
                                  device="cuda")
        self.q = torch.randn(self.N, Hq, D, generator=g, device="cuda").to(dtype)
        self.mask = None
        if mask == "tree":
            parent = [-1 if i == 0 else max(0, i - 1 - (i * 7 + t) % 5) for t in T for i in range(t)]
            self.mask = tree.ancestor_bits(torch.tensor(parent, dtype=torch.int32,
                                                        device="cuda"), self.first)
        elif mask == "random":
            w = (max(T) + 31) // 32
            self.mask = torch.randint(-2 ** 31, 2 ** 31, (self.N, w), generator=g,
                                      device="cuda").int()
        self.cache = tree.KVCache(self.k, self.v, self.ks, self.vs)
        self.tree = tree.Tree(Hq, Hkv, D, dtype, max_requests=self.B,
                              max_nodes=max_nodes or max(T + [1]))

    def attend(self, **kw):
        r = self.tree.attend(self.q, self.cache, self.pages, self.length, self.first,
                             mask=self.mask, **kw)
        assert self.tree.status() == 0
        return r

    def check(self, out, lse, scale=None, softcap=0.0):
        scale = self.D ** -0.5 if scale is None else scale
        want, want_lse, weight, sums = ref.attend(
            self.q, self.k, self.v, self.ks, self.vs, self.pages, self.page, self.length,
            self.first, self.mask, scale, softcap)
        tol, tol_lse = ref.bounds(want, weight, sums, self.D, self.dtype, softcap)
        assert not torch.isnan(out).any() and not torch.isnan(lse).any()
        off = (out.double() - want).abs() - tol
        assert (off <= 0).all(), "out is %g past its bound" % off.max()
        empty = torch.isinf(want_lse)
        assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
        far = (lse.double() - want_lse)[~empty].abs() - tol_lse[~empty]
        assert (far <= 0).all(), "lse is %g past its bound" % far.max()


SHAPES = [
    # Hq, Hkv, D, page, T, L
    (1, 1, 64, 16, [1], [0]),                          # one key: itself
    (8, 2, 128, 16, [1], [37]),
    (4, 4, 128, 16, [1, 1, 1], [127, 128, 129]),       # around a tile's end
    (32, 8, 128, 16, [8] * 4, [300, 1, 0, 777]),
    (32, 8, 128, 64, [17], [5000]),                    # one request over many SMs
    (16, 2, 64, 1, [3, 5], [130, 64]),                 # pages of one slot
    (14, 2, 80, 24, [5, 33, 1, 61], [10, 200, 511, 3]),
    (6, 1, 96, 7, [64], [250]),                        # rows past three tiles of 128
    (24, 8, 112, 100, [9, 0, 2], [99, 50, 101]),       # a request without rows
    (5, 5, 8, 32, [2, 40], [64, 65]),
    (40, 8, 128, 16, [26, 51], [384, 385]),            # 130 and 255 rows a head
    (8, 1, 128, 128, [256], [1000]),                   # the largest tree: 2,048 rows a head
    (16, 1, 32, 48, [16, 17, 8, 9], [0, 0, 0, 0]),     # no context
    (2, 1, 128, 16, [1] * 300, [i % 67 for i in range(300)]),
    (64, 8, 128, 64, [1] * 20, [100 + 211 * i for i in range(20)]),
    (3, 1, 40, 16, [43, 86], [0, 2000]),
]


@pytest.mark.parametrize("dtype,cache", [(BF16, "16"), (F16, "16"), (BF16, "e4m3"), (F16, "e4m3")])
@pytest.mark.parametrize("Hq,Hkv,D,page,T,L", SHAPES)
def test_attend_shapes(tree, Hq, Hkv, D, page, T, L, dtype, cache):
    if cache == "e4m3" and D % 16:
        pytest.skip("an e4m3 cache has head_dim a multiple of 16")
    c = Case(tree, Hq, Hkv, D, page, dtype, cache, T, L, seed=Hq * 1000 + D)
    c.check(*c.attend())


@pytest.mark.parametrize("mask", [None, "tree", "random"])
@pytest.mark.parametrize("softcap", [0.0, 0.5, 30.0])
@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_attend_masks_and_cap(tree, mask, softcap, cache):
    c = Case(tree, 10, 2, 64, 20, BF16, cache, [70, 1, 26, 130], [129, 7, 0, 1000], seed=5, mask=mask)
    c.check(*c.attend(softcap=softcap), softcap=softcap)


@pytest.mark.parametrize("scale,spread", [(1.0, 4.0), (-0.3, 1.0), (0.0, 1.0), (0.01, 0.01)])
def test_attend_large_and_small_scores(tree, scale, spread):
    """Sharp softmax (scores of hundreds), negative, equal and tiny scores."""
    c = Case(tree, 8, 2, 128, 16, BF16, "16", [9, 40], [600, 33], seed=6, spread=spread)
    c.check(*c.attend(scale=scale), scale=scale)


@pytest.mark.parametrize("order", ["up", "down"])
def test_attend_rising_maximum(tree, order):
    """Scores that rise (or fall) along the cache: the running maximum moves in every tile."""
    c = Case(tree, 4, 1, 64, 16, BF16, "16", [4], [2000], seed=7, mask=None)
    total = 2004
    at = torch.arange(total, device="cuda")
    ramp = at if order == "up" else total - at
    c.q[:] = 1.0
    c.k[c.pages[0][at // 16].long(), at % 16] = (ramp.float() * 0.05)[:, None, None].to(BF16)
    c.check(*c.attend())


def test_attend_rows_that_see_nothing(tree):
    """An empty mask row without context: out 0, lse -inf; its neighbours are unaffected."""
    c = Case(tree, 8, 2, 128, 16, BF16, "16", [40, 3, 200], [0, 0, 5], seed=8)
    c.mask[::3] = 0
    out, lse = c.attend()
    c.check(out, lse)
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attend_invisible_rows_hold_anything(tree, bad, where):
    """NaN and infinities of a node reach the nodes that see it and no other."""
    T, L = [9, 150], [130, 20]
    c = Case(tree, 4, 2, 64, 16, BF16, "16", T, L, seed=9, mask=None)
    parent = torch.tensor([-1] + [0] * 8 + [-1] + [0] * 149, dtype=torch.int32, device="cuda")
    c.mask = tree.ancestor_bits(parent, c.first)       # all nodes are children of node 0
    node = {0: 4, 1: 140}
    clean_out, clean_lse = c.attend()
    for b, j in node.items():
        p = L[b] + j
        getattr(c, where)[c.pages[b][p // 16].long(), p % 16, :, 3] = bad
    out, lse = c.attend()
    hit = torch.tensor([4, 9 + 140], device="cuda")
    rest = torch.ones(c.N, dtype=torch.bool, device="cuda")
    rest[hit] = False
    assert torch.equal(out[rest], clean_out[rest]) and torch.equal(lse[rest], clean_lse[rest])
    if where == "v":
        assert torch.equal(lse[hit], clean_lse[hit])
        got = out[hit][..., 3].float()
        assert torch.isnan(got).all() if math.isnan(bad) else (got == bad).all()
        other = [i for i in range(64) if i != 3]
        # finite elements are the same sums; the tile goes another way through the registers
        assert torch.equal(out[hit][..., other], clean_out[hit][..., other])
    elif not (bad == -math.inf or bad == math.inf):
        assert torch.isnan(out[hit]).all()


def test_attend_nan_query_and_context_reach_their_rows(tree):
    c = Case(tree, 4, 2, 64, 16, BF16, "16", [5, 6], [130, 20], seed=10)
    clean, _ = c.attend()
    c.q[2, 1, 7] = math.nan
    out, lse = c.attend()
    assert torch.isnan(out[2, 1]).all() and torch.isnan(lse[2, 1])
    keep = torch.ones(c.N, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_attend_strides(tree, cache):
    """Heads before slots, K and V in one tensor, q inside a fused projection, wide tables."""
    c = Case(tree, 12, 4, 64, 16, BF16, cache, [7, 30], [100, 257], seed=11)
    out, lse = c.attend()
    both = torch.stack([c.k.view(torch.uint8) if cache == "e4m3" else c.k,
                        c.v.view(torch.uint8) if cache == "e4m3" else c.v], 1) \
        .permute(0, 1, 3, 2, 4).contiguous()            # [pages, 2, heads, slots, dim]
    if cache == "e4m3":
        both = both.view(E4M3)
    k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    ks = vs = None
    if cache == "e4m3":
        ks = c.ks.transpose(1, 2).contiguous().transpose(1, 2)
        vs = torch.cat([c.vs, c.vs], 1)[:, :c.page]
    fused = torch.randn(c.N, 20, 64, device="cuda").to(BF16)
    fused[:, 4:16] = c.q
    wide = torch.full((c.B, c.pages.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.pages.shape[1]] = c.pages
    mask = torch.cat([c.mask, c.mask + 1], 1)[:, :c.mask.shape[1]]
    o2, l2 = c.tree.attend(fused[:, 4:16], tree.KVCache(k, v, ks, vs), wide, c.length, c.first,
                           mask=mask)
    assert c.tree.status() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_attend_repeats_and_graph(tree):
    """The same bits every time, on another stream, and replayed from a graph after the
    lengths have changed; the handle's workspace serves calls of other shapes in between."""
    c = Case(tree, 32, 8, 128, 16, BF16, "16", [8] * 5, [3000, 10, 0, 900, 4000], seed=12)
    out, lse = c.attend()
    d = Case(tree, 32, 8, 128, 16, BF16, "16", [30], [2500], seed=13)
    d.tree.close()
    d.tree = tree.Tree(32, 8, 128, BF16, max_requests=5, max_nodes=64)
    d.check(*d.attend())
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


@pytest.mark.parametrize("page,cache", [(64, "16"), (16, "16"), (24, "16"), (64, "e4m3")])
def test_attend_many_tiles_back_to_back(tree, page, cache):
    """Long shares of every CTA, calls over several caches in a row without a wait between:
    copies land late and out of order.  The same bits every time."""
    cases = [Case(tree, 32, 8, 128, page, BF16, cache, [17], [40000 + 511 * i], seed=40 + i, spare=1,
                  mask=None) for i in range(3)]
    want = [c.attend() for c in cases]
    cases[1].check(*want[1])
    for _ in range(30):
        got = [c.tree.attend(c.q, c.cache, c.pages, c.length, c.first) for c in cases * 4]
        for i, (o, l) in enumerate(got):
            assert torch.equal(o, want[i % 3][0]) and torch.equal(l, want[i % 3][1])
    assert all(c.tree.status() == 0 for c in cases)


def test_attend_empty_calls(tree):
    t = tree.Tree(4, 2, 64, BF16, max_requests=3, max_nodes=4)
    k = torch.zeros(2, 16, 2, 64, dtype=BF16, device="cuda")
    cache = tree.KVCache(k, k.clone())
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = t.attend(torch.zeros(0, 4, 64, dtype=BF16, device="cuda"), cache,
                        torch.zeros(3, 1, dtype=torch.int32, device="cuda"), z,
                        torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = t.attend(torch.zeros(0, 4, 64, dtype=BF16, device="cuda"), cache,
                        torch.zeros(0, 1, dtype=torch.int32, device="cuda"), z[:0], z[:1])
    # rows that belong to no request are not written
    q = torch.ones(5, 4, 64, dtype=BF16, device="cuda")
    mine = torch.full((5, 4, 64), 7.0, dtype=BF16, device="cuda")
    first = torch.tensor([1, 2, 2, 3], dtype=torch.int32, device="cuda")
    pages = torch.tensor([[0], [1], [1]], dtype=torch.int32, device="cuda")
    t.attend(q, cache, pages, z, first, out=mine)
    assert t.status() == 0
    assert (mine[[0, 3, 4]] == 7).all() and (mine[[1, 2]] == 0).all()


def test_attend_far_offsets(tree):
    """A cache of more than 2^32 bytes: pages at its far end."""
    page, Hkv, D = 64, 8, 128
    n_pages = (1 << 32) // (page * Hkv * D) + 40          # e4m3: a byte an element
    k = torch.zeros(n_pages, page, Hkv, D, dtype=torch.uint8, device="cuda").view(E4M3)
    ks = torch.zeros(n_pages, page, Hkv, dtype=torch.uint8, device="cuda")
    c = Case(tree, 16, Hkv, D, page, BF16, "e4m3", [5, 3], [300, 20], seed=14)
    shift = n_pages - c.n_pages
    for name in ("k", "v"):
        x = getattr(c, name)
        k.view(torch.uint8)[shift:] = x.view(torch.uint8)
        ks[shift:] = getattr(c, name + "s")
        setattr(c, name, k.clone() if name == "k" else k)
        setattr(c, name + "s", ks.clone() if name == "k" else ks)
    c.pages += shift
    c.cache = tree.KVCache(c.k, c.v, c.ks, c.vs)
    c.check(*c.attend())
    new = torch.randn(8, Hkv, D, device="cuda").to(BF16)
    c.tree.write(c.cache, c.pages, c.length, c.first, new, new)
    got, _ = c.tree.read(c.cache, c.pages, c.length, c.first, 8)
    code, byte = ref.quantise(new)
    assert torch.equal(got.double(), code * ref.scale_of(byte)[..., None])
    assert c.tree.status() == 0


# ---------------------------------------------------------------- the cache --

ROWS = [
    # Hkv, D, page, T, L
    (8, 128, 16, [8] * 16, [11 * i for i in range(16)]),
    (1, 16, 1, [1], [0]),
    (2, 80, 24, [33, 0, 400], [5, 7, 23]),
    (5, 112, 7, [1] * 40, list(range(40))),
    (16, 64, 64, [700, 1500], [63, 64]),
    (3, 32, 32, [5000], [31]),
]


def special_rows(x):
    """Rows that are zero, tiny, huge, of one value, ties of the grid, or not finite."""
    flat = x.view(-1, x.shape[-1])
    n = flat.shape[0]
    big = torch.finfo(x.dtype).max
    for i, value in enumerate([0.0, big, -big, torch.finfo(x.dtype).smallest_normal,
                               torch.finfo(x.dtype).smallest_normal / 16, 448.0, 449.0, 896.0]):
        if i < n:
            flat[i] = value
    if n > 12:
        flat[8, 1] = math.inf
        flat[9, 0] = -math.inf
        flat[10, -1] = math.nan
        flat[11] = torch.linspace(-448, 448, x.shape[-1], device=x.device).to(x.dtype)
        flat[12] = (torch.arange(x.shape[-1], device=x.device) % 32 + 16).to(x.dtype) * 14
    return x


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0))


@pytest.mark.parametrize("dtype,cache", [(BF16, "16"), (F16, "16"), (BF16, "e4m3"), (F16, "e4m3")])
@pytest.mark.parametrize("Hkv,D,page,T,L", ROWS)
def test_write_and_read(tree, Hkv, D, page, T, L, dtype, cache):
    c = Case(tree, Hkv, Hkv, D, page, dtype, cache, T, L, seed=D, garbage=None, mask=None,
             max_nodes=1)
    k = special_rows(torch.randn(c.N, Hkv, D, generator=c.g, device="cuda").to(dtype))
    v = (torch.randn(c.N, Hkv, D, generator=c.g, device="cuda") * 100).to(dtype)
    before = [x.clone() for x in (c.k, c.v)]
    scales = [x.clone() if x is not None else None for x in (c.ks, c.vs)]
    c.tree.write(c.cache, c.pages, c.length, c.first, k, v)
    got = c.tree.read(c.cache, c.pages, c.length, c.first, c.N)
    assert c.tree.status() == 0
    touched = torch.zeros(c.n_pages, page, dtype=torch.bool, device="cuda")
    for b in range(c.B):
        at = torch.arange(L[b], L[b] + T[b], device="cuda")
        touched[c.pages[b][at // page].long(), at % page] = True
    for x, pool, old, scale, old_scale, back in zip((k, v), (c.k, c.v), before, (c.ks, c.vs),
                                                    scales, got):
        if cache == "e4m3":
            code, byte = ref.quantise(x)
            want = code * ref.scale_of(byte)[..., None]
            top = torch.finfo(dtype).max
            want = want.clamp(-top, top)
            assert same(back.double(), want.to(dtype).double())
            assert torch.equal(scale[~touched], old_scale[~touched])
            pool, old = pool.view(torch.uint8), old.view(torch.uint8)
            for b in range(c.B):
                at = torch.arange(L[b], L[b] + T[b], device="cuda")
                rows = slice(int(c.first[b]), int(c.first[b + 1]))
                assert torch.equal(scale[c.pages[b][at // page].long(), at % page], byte[rows])
        else:
            assert same(back, x)
        assert torch.equal(pool[~touched], old[~touched])


def test_write_every_16_bit_value(tree):
    """Every finite bf16 and f16 value as a row's only one, and below a larger one."""
    for dtype in (BF16, F16):
        bits = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(dtype)
        x = torch.zeros(65536, 1, 16, dtype=dtype, device="cuda")
        x[:, 0, 3] = bits
        y = x.clone()
        y[:, 0, 7] = bits.roll(1237)
        t = tree.Tree(1, 1, 16, dtype)
        k = torch.zeros(1024, 64, 1, 16, dtype=torch.uint8, device="cuda").view(E4M3)
        ks = torch.zeros(1024, 64, 1, dtype=torch.uint8, device="cuda")
        cache = tree.KVCache(k, k.clone(), ks, ks.clone())
        pages = torch.arange(1024, dtype=torch.int32, device="cuda")[None]
        z = torch.zeros(1, dtype=torch.int32, device="cuda")
        first = torch.tensor([0, 65536], dtype=torch.int32, device="cuda")
        t.write(cache, pages, z, first, x, y)
        for src, pool, scale in ((x, cache.k, cache.k_scale), (y, cache.v, cache.v_scale)):
            code, byte = ref.quantise(src[:, 0])
            assert torch.equal(scale.view(-1), byte)
            got = pool.view(-1, 16).to(torch.float64)
            assert same(got, code)
        back, _ = t.read(cache, pages, z, first, 65536)
        code, byte = ref.quantise(x[:, 0])
        want = code * ref.scale_of(byte)[:, None]
        want = want.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max)
        assert same(back[:, 0].double(), want.to(dtype).double())


def test_write_strided_rows(tree):
    """k and v as parts of one fused projection."""
    c = Case(tree, 8, 4, 64, 16, BF16, "e4m3", [20, 13], [5, 100], seed=20, garbage=None)
    fused = torch.randn(33, 16, 64, device="cuda").to(BF16)
    k, v = fused[:, 8:12], fused[:, 12:16]
    c.tree.write(c.cache, c.pages, c.length, c.first, k, v)
    got = c.tree.read(c.cache, c.pages, c.length, c.first, 33)
    for x, y in zip((k, v), got):
        code, byte = ref.quantise(x)
        assert torch.equal(y.double(), code * ref.scale_of(byte)[..., None])


@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("page", [1, 7, 16])
def test_keep(tree, cache, page):
    T, L = [40, 1, 17, 256, 64], [3, 0, 30, 100, 16]
    paths = [[0, 2, 5, 6, 7, 20, 39], [0], [], list(range(0, 256, 2)), list(range(1, 64))]
    c = Case(tree, 4, 2, 48, page, BF16, cache, T, L, seed=21, garbage=None)
    path = torch.full((5, 200), -9, dtype=torch.int32, device="cuda")
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    pools = [x.view(torch.uint8) if x.dtype == E4M3 else x for x in (c.k, c.v, c.ks, c.vs)
             if x is not None]
    want = [x.clone() for x in pools]
    for x, src in zip(want, [x.clone() for x in pools]):
        for b, p in enumerate(paths):
            for i, j in enumerate(p):
                a, z = L[b] + i, L[b] + j
                x[c.pages[b, a // page].long(), a % page] = \
                    src[c.pages[b, z // page].long(), z % page]
    c.tree.keep(c.cache, c.pages, c.length, path, count)
    assert c.tree.status() == 0
    for x, y in zip(pools, want):
        assert torch.equal(x, y)
    none = torch.zeros(5, dtype=torch.int32, device="cuda")
    c.tree.keep(c.cache, c.pages, c.length, path, none)
    c.tree.keep(c.cache, c.pages, c.length, path[:, :0], none)
    assert c.tree.status() == 0
    for x, y in zip(pools, want):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ refusals --


def test_device_checks_leave_the_others_alone(tree):
    """A request whose numbers do not fit is left out and reported; the others run."""
    from serial_draft_head_gb300 import walk
    base = dict(T=[4, 5, 6], L=[40, 50, 60])
    bad = walk.EPAGES

    def fresh(**kw):
        c = Case(tree, 4, 2, 64, 16, BF16, "16", base["T"], base["L"], seed=30, **kw)
        return c, c.attend()[0]

    def rows(c, skip):
        return [r for b in range(3) if b != skip
                for r in range(sum(c.T[:b]), sum(c.T[:b + 1]))]

    def run(c, out, **kw):
        args = dict(pages=c.pages, length=c.length, first=c.first, mask=c.mask)
        args.update(kw)
        c.tree.attend(c.q, c.cache, args["pages"], args["length"], args["first"],
                      mask=args["mask"], out=out)
        return c.tree.status()

    c, good = fresh()
    for length in (-1, 1 << 20, 2 ** 31 - 1):
        bad_len = c.length.clone()
        bad_len[1] = length
        out = torch.full_like(good, 3.0)
        assert run(c, out, length=bad_len) == bad
        assert torch.equal(out[rows(c, 1)], good[rows(c, 1)])
        assert (out[4:9] == 3).all()
        assert c.tree.status() == 0                       # cleared by the last call
    for first in ([0, 4, 9, 16], [-1, 4, 9, 15], [5, 4, 9, 15], [0, 4, 9, 2 ** 31 - 1]):
        f = torch.tensor(first, dtype=torch.int32, device="cuda")
        out = torch.full_like(good, 3.0)
        assert run(c, out, first=f) == bad
        assert torch.equal(out[4:9], good[4:9])
    for page in (-1, c.n_pages, 2 ** 31 - 1):
        p = c.pages.clone()
        p[2, 0] = page
        out = torch.full_like(good, 3.0)
        assert run(c, out, pages=p) == bad
        assert torch.equal(out[:9], good[:9])
    small = tree.Tree(4, 2, 64, BF16, max_requests=3, max_nodes=5)
    big, c.tree = c.tree, small
    out = torch.full_like(good, 3.0)
    assert run(c, out) == bad                             # six nodes in a handle for five
    assert torch.equal(out[:9], good[:9]) and (out[9:] == 3).all()
    c.tree = big


def test_device_checks_of_cache_calls(tree):
    from serial_draft_head_gb300 import walk
    c = Case(tree, 2, 2, 64, 16, BF16, "e4m3", [4, 5], [40, 50], seed=31, garbage=None)
    pools = [x.view(torch.uint8) for x in (c.k, c.v, c.ks, c.vs)]
    old = [x.clone() for x in pools]
    new = torch.randn(9, 2, 64, device="cuda").to(BF16)
    for page in (-1, c.n_pages):
        p = c.pages.clone()
        p[:] = page
        c.tree.write(c.cache, p, c.length, c.first, new, new)
        assert c.tree.status() == walk.EPAGES
        out = tuple(torch.full((9, 2, 64), 5.0, dtype=BF16, device="cuda") for _ in range(2))
        c.tree.read(c.cache, p, c.length, c.first, 9, out=out)
        assert c.tree.status() == walk.EPAGES
        assert (out[0] == 5).all() and (out[1] == 5).all()
    c.tree.write(c.cache, c.pages, torch.full_like(c.length, 1 << 30), c.first, new, new)
    assert c.tree.status() == walk.EPAGES
    count = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    for path in ([[1, 1], [3, 2]], [[-1, 0], [0, -5]], [[0, 1 << 30], [5, 2 ** 31 - 1]]):
        c.tree.keep(c.cache, c.pages, c.length,
                    torch.tensor(path, dtype=torch.int32, device="cuda"), count)
        assert c.tree.status() == walk.EPAGES
    good = torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device="cuda")
    for n in (-1, 3):
        c.tree.keep(c.cache, c.pages, c.length, good, torch.full_like(count, n))
        assert c.tree.status() == walk.EPAGES
    for x, y in zip(pools, old):
        assert torch.equal(x, y)


def test_host_refusals(tree):
    from serial_draft_head_gb300 import walk
    for bad in (dict(q_heads=3), dict(kv_heads=0), dict(head_dim=12), dict(head_dim=136),
                dict(max_requests=0), dict(max_requests=1025), dict(max_nodes=257)):
        args = dict(q_heads=4, kv_heads=2, head_dim=64)
        args.update(bad)
        with pytest.raises(walk.WalkError):
            tree.Tree(**args)
    with pytest.raises(ValueError):
        tree.Tree(4, 2, 64, torch.float32)
    c = Case(tree, 4, 2, 64, 16, BF16, "16", [4], [40], seed=32)
    call = lambda **kw: c.tree.attend(**{**dict(  # noqa: E731
        q=c.q, cache=c.cache, pages=c.pages, length=c.length, first=c.first, mask=c.mask), **kw})
    call()
    other = torch.zeros(4, 16, 2, 64, device="cuda")
    for kw in (dict(q=c.q.float()), dict(q=c.q[:, :2]), dict(q=c.q.cpu()), dict(pages=c.pages.long()),
               dict(pages=c.pages[0]), dict(length=c.length[:0]), dict(first=c.first[:1]),
               dict(mask=c.mask[:2]), dict(mask=c.mask.long()), dict(out=c.q[:2]),
               dict(lse=torch.zeros(4, 4, dtype=F16, device="cuda")),
               dict(cache=tree.KVCache(other.half(), other.half()))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(scale=math.nan), dict(softcap=-1.0), dict(softcap=math.inf),
               dict(q=torch.zeros(4, 4, 65, dtype=BF16, device="cuda")[:, :, 1:])):
        with pytest.raises(walk.WalkError) as e:
            call(**kw)
        assert e.value.code == walk.EINVAL
    with pytest.raises(ValueError):
        tree.KVCache(other, other)
    with pytest.raises(ValueError):
        tree.KVCache(other.half(), other.half(), torch.zeros(4, 16, 2, dtype=torch.uint8,
                                                             device="cuda"))
    with pytest.raises(ValueError):
        tree.KVCache(c.k, c.v[:, :, :, :32])
    with pytest.raises(walk.WalkError):                   # an e4m3 cache of heads of 24
        x = torch.zeros(2, 16, 1, 24, dtype=torch.uint8, device="cuda").view(E4M3)
        s = torch.zeros(2, 16, 1, dtype=torch.uint8, device="cuda")
        t = tree.Tree(1, 1, 24)
        t.read(tree.KVCache(x, x, s, s), c.pages[:, :1], c.length, c.first, 4)
    with pytest.raises(walk.WalkError):                   # more requests than the handle takes
        call(pages=c.pages.repeat(2, 1), length=c.length.repeat(2),
             first=torch.tensor([0, 4, 4], dtype=torch.int32, device="cuda"))
    assert c.tree.status() == 0
