"""Norms and rotation at their edges: rows whose squares leave 32 bits, errors against the sum of their
terms, heads of every size on their way into the cache."""
import math
from fractions import Fraction

import pytest
import torch

from test_gpu_rotate import Case, bits, cache_of, formula, frequencies
from test_gpu_tree import BF16, F16, tree  # noqa: F401

pytestmark = pytest.mark.gpu
F64 = torch.float64


def size_rows(c, rows):
    """The case's rows of q and k as they are, some of them times numbers."""
    for x in (c.q, c.k):
        for i, by in rows.items():
            x[i] = (x[i].double() * by).to(c.dtype)


@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-37, 1e-25])
@pytest.mark.parametrize("D,Hq,Hkv,pairs", [(128, 32, 8, False), (64, 6, 2, True), (80, 3, 3, False)])
def test_norm_of_rows_whose_squares_leave_32_bits(tree, eps, D, Hq, Hkv, pairs):  # noqa: F811
    """bf16 rows of 2^64 and more, and without an eps that covers them of 2^-60 and less: normed as the
    formula says; the rows beside them in the same warp keep their bits."""
    plain = Case(tree, 40, Hq, Hkv, D, D // 32 * 32, BF16, pairs, eps=eps, seed=1)
    c = Case(tree, 40, Hq, Hkv, D, D // 32 * 32, BF16, pairs, eps=eps, seed=1)
    rows = {3: 2.0 ** 62, 4: 2.0 ** 80, 5: 2.0 ** 120, 9: 2.0 ** -50, 10: 2.0 ** -62, 11: 2.0 ** -75, 12: 2.0 ** -120}
    size_rows(c, rows)
    c.q[6, 0] = 0.0
    c.q[6, 0, 1] = 2.0 ** 127                          # alone in its row
    got = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    for x, which in zip(got, "qk"):
        want, size = c.want(which)
        # one rounding: bf16 has eight significant bits, so a step is 2^-7 of 1 and half of one 2^-8 of
        # the value at most; below its normal numbers a step is 2^-133
        off = (x.double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -18 * size + 2.0 ** -133)
        assert not torch.isnan(x).any() and (off <= 0).all(), off.flatten(1).amax(1)
    rest = [i for i in range(40) if i not in rows and i != 6]
    for x, y in zip(got, plain.tree.rotate(plain.q, plain.k, plain.position, plain.rotation)):
        assert torch.equal(x[rest], y[rest])
    assert torch.equal(got[0][6, 1:], plain.tree.rotate(plain.q, plain.k, plain.position, plain.rotation)[0][6, 1:])


def test_norm_of_rows_without_a_finite_size(tree):  # noqa: F811
    """A zero row without eps is 0 / 0; one with an infinity is NaN there and 0 elsewhere; NaN is all of it."""
    c = Case(tree, 8, 4, 2, 64, 0, BF16, eps=0.0)
    c.q[1, 2], c.q[2, 1, 5], c.q[3, 0, 7] = 0.0, math.inf, math.nan
    q, _ = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    assert torch.isnan(q[1, 2]).all() and torch.isnan(q[3, 0]).all() and torch.isnan(q[2, 1, 5])
    assert (q[2, 1, [i for i in range(64) if i != 5]] == 0).all()
    hit = torch.zeros(8, 4, dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[2, 1] = hit[3, 0] = True
    assert torch.isfinite(q[~hit]).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pairs,norm,far", [(False, True, False), (True, True, True), (False, False, True), (True, False, False)])
@pytest.mark.parametrize("N,Hq,Hkv,D,R", [(7, 14, 2, 96, 64), (128, 32, 8, 128, 128), (300, 5, 1, 64, 32), (50, 64, 8, 112, 112),
                                          (21, 6, 2, 48, 0), (700, 16, 2, 32, 32), (2, 4, 4, 16, 16)])
def test_rotate_within_the_sum_of_its_terms(tree, N, Hq, Hkv, D, R, dtype, pairs, norm, far):  # noqa: F811
    """Each term in units of 2^-24 of the two elements' size.  The norm: a sum of 128 squares in 12 steps
    and three operations on it, 15, of which the root leaves half, 7.5; the reciprocal root 4 (two units in
    the last place, 2^-23 each); the product with it 1.  Sine and cosine: 4 (two units in the last place);
    the angle, rounded to 24 bits of half a turn at most, 2^-25 pi, and cut at 2^-32 turns, 1.7; their product
    with the weights 1; the two products and their sum 2.  21.2 in all.  Angles of far positions are taken
    exactly here: in float64 their product alone is off by 2^-22."""
    c = Case(tree, N, Hq, Hkv, D, R, dtype, pairs, norm, far, seed=2)
    got = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -24 if dtype == F16 else 2.0 ** -120
    if R:
        from test_rotation_host import half_turn
        turn = 1 / (2 * half_turn(60))
        freq = [Fraction(f) * turn for f in c.freq.tolist()]
        angle = torch.tensor([[float(f * p % 1) for f in freq] for p in c.position.tolist()], dtype=F64).cuda() * 2 * math.pi
        cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        a, b = (slice(0, R, 2), slice(1, R, 2)) if pairs else (slice(0, R // 2), slice(R // 2, R))
    for x, src, w in zip(got, (c.q, c.k), c.norms):
        want, size = formula(src, c.position, None, w, c.eps, pairs)
        if R:
            u, z = want[..., a].clone(), want[..., b].clone()
            want[..., a], want[..., b] = u * cos - z * sin, z * cos + u * sin
            both = u.abs() + z.abs()
            size[..., a], size[..., b] = both, both
        off = (x.double() - want).abs() - (half * want.abs() + 21.2 * 2.0 ** -24 * (1 + half) * size + tiny)
        assert (off <= 0).all(), "%g past its bound" % off.max()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("held", ["16", "e4m3"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv,D,R", [(9, 4, 4, 16, 16), (70, 6, 2, 48, 0), (70, 6, 2, 48, 32), (200, 3, 3, 80, 48),
                                          (200, 10, 5, 80, 80), (50, 64, 8, 112, 112), (50, 16, 8, 112, 96)])
def test_place_of_heads_that_32_does_not_divide(tree, N, Hq, Hkv, D, R, dtype, pairs, held):  # noqa: F811
    """The bits of rotate and then write, in q and in the cache; rows left out; nothing else touched."""
    c = Case(tree, N, Hq, Hkv, D, R, dtype, pairs, seed=3)
    page = 16
    n_pages = N // page + 3
    slot = torch.randperm(n_pages * page, generator=c.g, device="cuda")[:N].int()
    slot[1::5] = -1
    a, b = (cache_of(tree, held, n_pages, page, Hkv, D, dtype) for _ in range(2))
    q, k = c.tree.rotate(c.q, c.k, c.position, c.rotation)
    out = torch.full_like(q, 7.0)
    c.tree.place(a, slot, c.q, c.k, c.v, c.position, c.rotation, out=out)
    keep = torch.nonzero(slot >= 0)[:, 0]
    pages = (slot[keep] // page)[:, None].contiguous()
    first = torch.arange(len(keep) + 1, dtype=torch.int32, device="cuda")
    c.tree.write(b, pages, (slot[keep] % page).contiguous(), first, k[keep], c.v[keep])
    assert c.tree.status() == 0
    assert torch.equal(out[keep], q[keep]) and (out[slot < 0] == 7).all()
    assert all(torch.equal(x, y) for x, y in zip(bits(a), bits(b)))
