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
