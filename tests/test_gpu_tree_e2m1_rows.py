"""Attention over a 4-bit cache where the rows of q are of extreme size, and its tcgen05 kernel on other
streams and in graphs."""
import math

import pytest
import torch

import e2m1_reference as e2m1
from test_gpu_tree import BF16, F16, tree  # noqa: F401
from test_gpu_tree_e2m1 import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 4, 40])       # items of 8, 16 and 32 rows, and tcgen05
@pytest.mark.parametrize("size,scale", [(2.0 ** 120, 2.0 ** 30), (-2.0 ** 110, 2.0 ** 127), (2.0 ** 127, 1.0), (2.0 ** -126, 1.0)])
def test_scores_of_zero_under_any_scale(tree, T, size, scale):  # noqa: F811
    """Keys of zeros: every score is zero, whatever the rows and the scale, and every visible key weighs the
    same."""
    c = Case(tree, 8, 1, 64, 16, BF16, [T], [50], seed=400 + T, mask=None)
    c.k.zero_()
    c.ks[c.ks != 255] = 0
    c.q.fill_(size)
    out, lse = c.attend(scale=scale)
    v = e2m1.values(c.v, c.vs)
    for i in range(T):
        at = torch.arange(51 + i, device="cuda")
        rows = v[c.pages[0][at // 16].long(), at % 16, 0]
        # a weight of 1 is exact in both types, fp32 sums of up to 90 numbers, one rounding
        want, size_of = rows.mean(0), rows.abs().mean(0)
        assert ((out[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 90 * 2.0 ** -23 * size_of).all()
        assert (lse[i].double() - math.log(51 + i)).abs().max() < 1e-5


@pytest.mark.parametrize("T", [1, 2, 40])          # few rows, and tcgen05
@pytest.mark.parametrize("size,scale", [(2.0 ** 120, 2.0 ** 30), (-2.0 ** 110, 2.0 ** 127)])
def test_scores_of_zero_over_e4m3(tree, T, size, scale):  # noqa: F811
    """The same over a cache of e4m3, whose few-row kernel brings rows of q to f16 as well."""
    from test_gpu_tree import Case as Wide
    c = Wide(tree, 8, 1, 64, 16, BF16, "e4m3", [T], [50], seed=410 + T, mask=None, garbage=None)
    c.k.view(torch.uint8).zero_()
    c.ks.fill_(127)
    c.q.fill_(size)
    t = tree.Tree(8, 1, 64, BF16, max_nodes=T)
    out, lse = t.attend(c.q, tree.KVCache(c.k, c.v, c.ks, c.vs), c.pages, c.length, c.first, scale=scale)
    assert t.status() == 0
    v = c.v.double() * torch.exp2(c.vs.double() - 127)[..., None]
    for i in range(T):
        at = torch.arange(51 + i, device="cuda")
        rows = v[c.pages[0][at // 16].long(), at % 16, 0]
        want, size_of = rows.mean(0), rows.abs().mean(0)
        assert ((out[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 90 * 2.0 ** -23 * size_of).all()
        assert (lse[i].double() - math.log(51 + i)).abs().max() < 1e-5


@pytest.mark.parametrize("held", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T", [1, 2, 4, 40])
def test_an_infinity_beside_large_elements_of_a_row(tree, held, T):  # noqa: F811
    """A row with an infinity and elements past f16's range, capped scores: those are infinite, the cap or
    its negative by the sign that the infinity meets, however large the others' part is."""
    from test_gpu_tree import Case as Wide
    cap = 2.0
    if held == "e2m1":
        c = Case(tree, 8, 1, 64, 16, BF16, [T], [50], seed=420 + T, mask=None)
        k = torch.ones(c.n_pages, 16, 1, 64, dtype=torch.float64, device="cuda")
    else:
        c = Wide(tree, 8, 1, 64, 16, BF16, "e4m3", [T], [50], seed=420 + T, mask=None, garbage=None)
        k = torch.ones(c.n_pages, 16, 1, 64, dtype=torch.float64, device="cuda")
    sign = torch.where(torch.rand(c.n_pages, 16, 1, generator=c.g, device="cuda") < 0.5, -1.0, 1.0).double()
    k[..., 7] = sign
    if held == "e2m1":
        value, byte = e2m1.quantise(k)
        cache = tree.KVCache(e2m1.pack(value), c.v, byte, c.vs)
        v = e2m1.values(c.v, c.vs)
    else:
        import tree_reference as ref
        value, byte = ref.quantise(k)
        cache = tree.KVCache(value.float().to(torch.float8_e4m3fn), c.v, byte, c.vs)
        v = c.v.double() * torch.exp2(c.vs.double() - 127)[..., None]
    c.q[..., :] = -2.0 ** 20                           # against the infinity where it meets 1
    c.q[..., 7] = math.inf
    t = tree.Tree(8, 1, 64, BF16, max_nodes=T)
    out, lse = t.attend(c.q, cache, c.pages, c.length, c.first, softcap=cap)
    assert t.status() == 0
    for i in range(T):
        at = torch.arange(51 + i, device="cuda")
        where = c.pages[0][at // 16].long(), at % 16, 0
        w = torch.exp(cap * sign[where])
        want = (w[:, None] * v[where]).sum(0) / w.sum()
        size_of = (w[:, None] * v[where].abs()).sum(0) / w.sum()
        # a weight: one rounding to either type, 2^-8 at most, and 2^-19 of the exponential; the result's own
        assert ((out[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -15) * size_of).all()
        assert (lse[i].double() - w.sum().log()).abs().max() < 2.0 ** -15


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("step", [-1, 1, -2, 2])
def test_codes_beside_every_border(tree, dtype, step):  # noqa: F811
    """The values one and two of the type's steps below and above every border of codes, times every scale
    that the type holds it with, beside six times that scale."""
    scales = e2m1.scale_of(torch.arange(227, device="cuda"))[1:]
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=torch.float64, device="cuda")
    ties = scales[:, None] * border
    ties = torch.cat([ties, -ties], 1)[(ties.to(dtype).double() == ties).all(1)].to(dtype)
    near = ties.view(torch.int16).clone()
    near[:, [i for i in range(16) if i % 8 != 7]] += step          # magnitudes: the sign is a bit apart
    x = near.view(dtype)
    # the smallest steps below a border under the smallest scales must not pass zero
    assert len(x) > 100 and (x.sign() * ties.sign() >= 0).all()
    rows = torch.zeros(len(x), 1, 32, dtype=dtype, device="cuda")
    rows[:, 0, :16] = x
    rows[:, 0, 16:] = x.flip(0)
    n = -(-len(x) // 16)
    t = tree.Tree(1, 1, 32, dtype)
    cache = tree.KVCache.zeros(n, 16, 1, 32, torch.uint8)
    pages = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.write(cache, pages, z, torch.tensor([0, len(x)], dtype=torch.int32, device="cuda"), rows, rows)
    assert t.status() == 0
    value, byte = e2m1.quantise(rows[:, 0])
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert torch.equal(scale.transpose(1, 2).reshape(n * 16, 2)[:len(x)], byte)
        assert torch.equal(e2m1.unpack(codes.transpose(1, 2).reshape(n * 16, 16)[:len(x)]), value)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T", [[20] * 5, [40, 9, 1, 33, 64]])
def test_many_rows_on_streams_and_in_graphs(tree, T, dtype):  # noqa: F811
    """The tcgen05 kernel and its join: the same bits on another stream and from a graph, also after the
    lengths have changed, with calls of the handle in between."""
    L = [3000, 10, 0, 900, 4000]
    c = Case(tree, 32, 8, 128, 16, dtype, T, L, seed=430)
    out, lse = c.attend()
    c.check(out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = c.attend(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask, out=o3, lse=l3)
    for n in (L, [17, 10, 0, 900, 2], L):
        c.L = n
        c.length.copy_(torch.tensor(n, dtype=torch.int32))
        o3.fill_(7.0)
        graph.replay()
        c.attend()
        graph.replay()
        torch.cuda.synchronize()
        c.check(o3, l3)
    assert torch.equal(out, o3) and torch.equal(lse, l3)
