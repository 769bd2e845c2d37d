"""Where the attention kernels meet and what each does in its own way: the choice between
them, scales of the cache that are not easy, capped scores near and far from the cap, maxima
that move inside a tile, parts joined by the last to arrive, and the example that runs the
draft and its check together."""
import math
import os
import sys

import pytest
import torch

import tree_reference as ref
from test_gpu_tree import BF16, E4M3, F16, Case, tree  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("T", [
    [4] * 6,                        # 16 rows a cached head: the most that few-row tiles take
    [4] * 5 + [5],                  # one more on average
    [1] * 11 + [33],                # few on average, with a request of nine few-row tiles
    [0, 0, 0, 12],                  # the same by requests without rows
    [17, 1, 64, 65, 3],             # row tiles alone and in pairs, in turn, in one call
])
def test_attend_rows_of_both_kernels(tree, T, cache):
    L = [(311 * i + 95) % 1500 for i in range(len(T))]
    c = Case(tree, 16, 4, 128, 16, BF16, cache, T, L, seed=60 + len(T))
    c.check(*c.attend())


@pytest.mark.parametrize("T,L", [([3, 1], [700, 45]), ([40, 2], [300, 130])])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 20)])
def test_attend_scales_of_any_size(tree, T, L, dtype, D, page):
    """Rows of the cache whose power of two is not exact in f16, or outside what a code's
    product with it can be: one by one, among rows of usual size, and rows of zeros."""
    c = Case(tree, 8, 2, D, page, dtype, "e4m3", T, L, seed=71)
    bytes_ = [0, 1, 60, 100, 111, 112, 113, 120, 127, 133, 134] + ([135, 150] if dtype == BF16 else [])
    for scale, lowest in ((c.vs, 0), (c.ks, 100)):
        keep = scale == 255
        pick = torch.tensor([b for b in bytes_ if lowest <= b <= 134] if scale is c.ks else bytes_,
                            dtype=torch.uint8, device="cuda")
        at = torch.randint(0, len(pick), scale.shape, generator=c.g, device="cuda")
        some = torch.rand(scale.shape, generator=c.g, device="cuda") < 0.3
        scale[some & ~keep] = pick[at][some & ~keep]
    zero = torch.rand(c.vs.shape, generator=c.g, device="cuda") < 0.1
    c.v.view(torch.uint8)[zero & (c.vs != 255)] = 0
    c.check(*c.attend(scale=0.002), scale=0.002)


@pytest.mark.parametrize("T", [[1, 3], [30], [70]])
@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("softcap,scale", [(50.0, 0.1), (3.0, 0.1), (1.5, -0.2), (0.01, 1.0)])
def test_attend_cap_near_and_far(tree, T, cache, softcap, scale):
    """Scores well below the cap, around it and far above, for single rows, a row tile alone
    and a pair of them, with and without masked tiles."""
    c = Case(tree, 8, 2, 64, 32, BF16, cache, T, [400] * len(T), seed=80 + len(T))
    c.check(*c.attend(softcap=softcap, scale=scale), softcap=softcap, scale=scale)


@pytest.mark.parametrize("order", ["up", "down", "saw"])
@pytest.mark.parametrize("T", [3, 20, 64])
def test_attend_maximum_moves_within_tiles(tree, order, T):
    """Ramps with steps of 64 keys: O is rescaled between the two halves of a tile, while the
    products of the other half may still be running."""
    c = Case(tree, 4, 1, 128, 16, BF16, "16", [T], [3000], seed=90, mask=None)
    total = 3000 + T
    at = torch.arange(total, device="cuda")
    ramp = {"up": at // 64, "down": (total - at) // 64, "saw": at // 64 % 3 * 20}[order]
    c.q[:] = 1.0
    c.k[c.pages[0][at // 16].long(), at % 16] = (ramp.float() * 0.25)[:, None, None].to(BF16)
    c.check(*c.attend())


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_attend_pairs_back_to_back(tree, cache):
    """Pairs of row tiles over long shares, calls in a row without a wait: the same bits."""
    cases = [Case(tree, 8, 2, 128, 64 if i else 24, BF16, cache, [64, 50], [9000 + 511 * i, 300],
                  seed=100 + i, spare=1, mask="tree") for i in range(2)]
    want = [c.attend() for c in cases]
    cases[1].check(*want[1])
    for _ in range(20):
        got = [c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask)
               for c in cases * 4]
        for i, (o, l) in enumerate(got):
            assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    assert all(c.tree.status() == 0 for c in cases)


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_attend_few_rows_joined_by_the_last(tree, cache):
    """Items of many parts, whose last CTA joins them: the same bits every time, between calls
    of other shapes on the handle, and replayed from a graph with other lengths."""
    c = Case(tree, 8, 2, 128, 16, BF16, cache, [1, 2, 1], [20000, 37, 900], seed=110)
    d = Case(tree, 8, 2, 128, 16, BF16, cache, [1, 1, 1], [1, 5000, 64], seed=111)
    out, lse = c.attend()
    c.check(out, lse)
    want = d.attend()
    for _ in range(30):
        for e, (o, l) in ((c, (out, lse)), (d, want)):
            o2, l2 = c.tree.attend(e.q, e.cache, e.pages, e.length, e.first, mask=e.mask)
            assert torch.equal(o, o2) and torch.equal(l, l2)
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask, out=o3, lse=l3)
    for L in ([20000, 37, 900], [3, 0, 900], [12345, 37, 1]):
        c.L = L
        c.length.copy_(torch.tensor(L, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check(o3, l3)
    assert c.tree.status() == 0


def test_attend_on_every_worker(tree):
    """As many short items as there are SMs and a few more or less: shares that begin and end
    inside an item, at its first tile and in the units before it."""
    for n in (151, 152, 153, 304, 305):
        c = Case(tree, 4, 1, 64, 16, BF16, "16", [1] * n, [(37 * i) % 90 for i in range(n)], seed=n)
        c.check(*c.attend())


def test_write_rows_of_any_stride_and_size(tree):
    """Codes and scales against the definition for head sizes whose lanes do not fill a warp,
    tokens that do not fill a block, rows of every magnitude."""
    for Hkv, D, T, dtype in ((3, 16, [5, 0, 41], BF16), (1, 48, [33], F16), (5, 80, [17, 16], BF16),
                             (2, 112, [64, 1], F16)):
        c = Case(tree, Hkv, Hkv, D, 24, dtype, "e4m3", T, [7] * len(T), seed=D)
        x = [torch.randn(c.N, Hkv, D, generator=c.g, device="cuda") for _ in range(2)]
        span = 40 if dtype == BF16 else 10
        x = [(y * torch.exp2(torch.randint(-span, span - 4, y.shape[:2], generator=c.g, device="cuda")
                             .float())[..., None]).to(dtype) for y in x]
        c.tree.write(c.cache, c.pages, c.length, c.first, *x)
        assert c.tree.status() == 0
        for y, data, scale in ((x[0], c.k, c.ks), (x[1], c.v, c.vs)):
            code, byte = ref.quantise(y)
            for b in range(c.B):
                at = c.L[b] + torch.arange(T[b], device="cuda")
                p, s = c.pages[b][at // 24].long(), at % 24
                r = slice(int(c.first[b]), int(c.first[b]) + T[b])
                assert torch.equal(scale[p, s], byte[r])
                assert torch.equal(data[p, s].to(torch.float64), code[r])


@pytest.mark.parametrize("cache", ["e4m3", "16"])
def test_example_drafts_and_checks(tree, cache):
    """The example's texts: every token is what the target says after the ones before it, up to
    the rounding of the attended rows, and the cache holds the rows of the text."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import draft_and_check as ex
    finally:
        sys.path.pop(0)
    target = ex.Target(vocab=2048)
    texts, cached, pages, length = ex.decode(target, [5, 9, 77], rounds=5, gamma=5, cache=cache)
    assert [len(t) - 1 for t in texts] == length.tolist()
    assert max(len(t) for t in texts) > 6                        # some drafts were right
    t = tree.Tree(8, 2, 64, max_requests=3)
    n = int(length.sum())
    first = torch.tensor([0] + length.cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    k, v = t.read(cached, pages, torch.zeros_like(length), first, n)
    assert t.status() == 0
    D = 64
    for b, text in enumerate(texts):
        tok = torch.tensor(text, device="cuda")
        rows = slice(int(first[b]), int(first[b + 1]))
        want = []
        for x, got in ((target.k, k), (target.v, v)):
            y = x[tok[:-1]].double()
            if cache == "e4m3":
                code, byte = ref.quantise(y)
                y = code * ref.scale_of(byte)[..., None]
            assert torch.equal(got[rows].double(), y)
            want.append(y)
        kk, vv = want
        q = target.q[tok[:-1]].double()
        heads = torch.arange(8, device="cuda") // 4
        s = torch.einsum("ihd,jhd->hij", q, kk[:, heads]) * D ** -0.5
        m = len(text) - 1
        s = s.masked_fill(torch.ones(m, m, device="cuda").triu(1).bool(), -math.inf)
        p = torch.softmax(s, -1)
        o = torch.einsum("hij,jhd->ihd", p, vv[:, heads]).reshape(m, -1)
        weight = torch.einsum("hij,jhd->ihd", p, vv[:, heads].abs()).reshape(m, -1)
        w1, w2, out = target.W1[tok[:-1]].double(), target.W2.double(), target.out.double()
        logits = w1 @ w2.T + o @ out.T
        # the attended rows: their rounding and the weights' (two half units); sums in 32 bits
        tol = 2.0 ** -7 * weight @ out.abs().T + 2.0 ** -13 * (w1.abs() @ w2.abs().T + weight @ out.abs().T)
        says = logits.gather(1, tok[1:, None])
        t_said = tol.gather(1, tok[1:, None])
        assert (logits - tol <= says + t_said).all()
