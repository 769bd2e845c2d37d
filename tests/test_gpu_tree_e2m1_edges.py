"""Attention over a 4-bit cache at its edges: each form of the kernels, parts of an item joined by
different workers, sizes near what indexes hold, capped scores, masks and rows of all kinds."""
import math

import pytest
import torch

import e2m1_reference as e2m1
from test_gpu_tree import BF16, F16, tree  # noqa: F401
from test_gpu_tree_e2m1 import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 4])           # items of 8, 16 and 32 rows
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 64), (64, 48), (96, 16), (128, 24)])
@pytest.mark.parametrize("B", [9, 41])             # workers of a CTA, and of four warps
def test_attend_forms(tree, T, D, page, B):
    """Runs of slots in pages of 16 and more, pages that cut blocks, heads that are no runs."""
    L = [(i * 137) % 700 for i in range(B)]
    c = Case(tree, 64, 8, D, page, BF16 if D != 64 else F16, [T if i % 5 else max(T - 1, 0) for i in range(B)], L,
             seed=300 + T + D)
    out, lse = c.attend()
    c.check(out, lse)
    slots = Case(tree, 64, 8, D, page, c.dtype, c.T, L, seed=300 + T + D, head_major=False)
    o2, l2 = slots.attend()
    slots.check(o2, l2)


@pytest.mark.parametrize("T", [1, 2, 4, 8])
def test_attend_repeats_with_shared_items(tree, T):
    """Few long requests: every item is shared by workers that arrive in any order.  The same bits always,
    with other calls of the handle in between."""
    c = Case(tree, 32, 8, 128, 64, BF16, [T] * 5, [3000, 700, 9000, 10, 5000], seed=310)
    d = Case(tree, 32, 8, 128, 64, BF16, [T], [50], seed=311)
    out, lse = c.attend()
    c.check(out, lse)
    for _ in range(10):
        c.tree.attend(d.q, d.cache, d.pages, d.length, d.first, mask=d.mask)
        got = [c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask) for _ in range(3)]
        assert all(torch.equal(out, o) and torch.equal(lse, l) for o, l in got)
    assert c.tree.status() == 0


@pytest.mark.parametrize("T", [1, 9, 40])
def test_attend_positions_near_what_an_index_holds(tree, T):
    """All positions are one slot (strides of zero), so that a cache of 2^31 - 1 rows fits: a request that
    would end past the longest length is left out and reported, its neighbour runs."""
    from serial_draft_head_gb300 import walk
    g = torch.Generator(device="cuda")
    g.manual_seed(320)
    slots, most = 2 ** 31 - 1, tree.TREE_MAX_LENGTH
    x = torch.randn(2, 1, 64, generator=g, device="cuda")
    value, byte = e2m1.quantise(x)
    k, v = e2m1.pack(value)
    ks, vs = byte
    cache = tree.KVCache(*(y.expand(1, slots, 1, y.shape[-1]) for y in (k, v, ks, vs)))
    q = torch.randn(2 * T, 1, 64, generator=g, device="cuda").to(BF16)
    t = tree.Tree(1, 1, 64, BF16, max_requests=2, max_nodes=T)
    pages = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    first = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
    kept = value * e2m1.scale_of(byte).repeat_interleave(16, -1)
    s = (q.double() @ kept[0, 0] / 8)[:, 0]
    for past in (slots - T, most - T + 1):
        length = torch.tensor([past, 77], dtype=torch.int32, device="cuda")
        out = torch.full((2 * T, 1, 64), 5.0, dtype=BF16, device="cuda")
        _, lse = t.attend(q, cache, pages, length, first, out=out)
        assert t.status() == walk.EPAGES
        assert (out[:T] == 5).all()
        # every weight of a row is the same: its sum's error is that of an addition a key
        assert ((out[T:].double() - kept[1]).abs() <= 2.0 ** -8 * kept[1].abs() * 1.01).all()
        n = 78 + torch.arange(T, device="cuda")
        assert (lse[T:, 0].double() - s[T:] - n.double().log()).abs().max() < 1e-4


@pytest.mark.parametrize("T", [[1, 3], [9, 8], [30], [70]])
@pytest.mark.parametrize("softcap,scale", [(50.0, 0.1), (3.0, 0.1), (1.5, -0.2), (0.01, 1.0)])
def test_attend_cap_near_and_far(tree, T, softcap, scale):
    """Scores well below the cap, around it and far above."""
    c = Case(tree, 8, 2, 64, 32, BF16, T, [400] * len(T), seed=330 + len(T))
    c.check(*c.attend(scale=scale, softcap=softcap), scale=scale, softcap=softcap)


@pytest.mark.parametrize("T", [[1, 2, 1], [12, 9, 11], [30, 80, 25]])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attend_keys_far_above_the_others(tree, T, dtype):
    """One key in fifty scores eight times the others': a row's maximum moves far and often, and a few keys
    have all its weight."""
    c = Case(tree, 8, 2, 128, 64, dtype, T, [3000, 500, 1200], seed=340, mask=None)
    for byte in (c.ks, c.vs):
        loud = torch.rand(byte.shape[:3], generator=c.g, device="cuda") < 0.02
        byte[loud] = torch.where(byte[loud] <= 226, (byte[loud] + 24).clamp(max=200), byte[loud])
    c.q *= 1.5
    c.check(*c.attend())


@pytest.mark.parametrize("T", [2, 12, 40])
def test_attend_where_no_request_has_rows(tree, T):
    """All requests fail, or none has a row: nothing is written."""
    from serial_draft_head_gb300 import walk
    c = Case(tree, 4, 2, 64, 16, BF16, [T, T], [40, 9], seed=350)
    for length, first, code in ((-1, c.first, walk.EPAGES), (3, torch.zeros_like(c.first), 0)):
        out = torch.full_like(c.q, 3.0)
        c.tree.attend(c.q, c.cache, c.pages, torch.full_like(c.length, length), first, mask=c.mask, out=out)
        assert c.tree.status() == code and (out == 3).all()
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, lse = c.tree.attend(c.q[:0], c.cache, c.pages[:0], e, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert out.shape[0] == lse.shape[0] == 0 and c.tree.status() == 0


@pytest.mark.parametrize("first", [[0, 2 ** 31 - 1, 9, 15], [0, -1, 9, 15], [3, 1, 9, 15], [0, 12, 9, 15], [0, 4, 2, 15]])
def test_a_bad_row_range_leaves_the_other_requests_alone(tree, first):
    """Requests behind one whose rows are out of range are attended to, written and read."""
    from serial_draft_head_gb300 import walk
    T, L = [9, 9, 6], [40, 50, 60]
    c = Case(tree, 4, 2, 64, 16, BF16, T, L, seed=360, mask=None)
    good = [b for b in range(3) if 0 <= first[b] <= first[b + 1] <= 15]
    rows = [first[b + 1] - first[b] for b in range(3)]
    f = torch.tensor(first, dtype=torch.int32, device="cuda")
    t = tree.Tree(4, 2, 64, BF16, max_requests=3, max_nodes=16)
    q = torch.randn(15, 4, 64, device="cuda").to(BF16)
    out = torch.full((15, 4, 64), 7.0, dtype=BF16, device="cuda")
    t.attend(q, c.cache, c.pages, c.length, f, out=out)
    assert t.status() == walk.EPAGES
    k, v = e2m1.values(c.k, c.ks), e2m1.values(c.v, c.vs)
    seen = torch.zeros(15, dtype=torch.bool, device="cuda")
    owners = torch.zeros(15, dtype=torch.int32, device="cuda")
    for b in good:
        owners[first[b]:first[b + 1]] += 1
    for b in good:
        if rows[b] == 0 or L[b] + rows[b] > c.pages.shape[1] * 16:
            continue
        seen[first[b]:first[b + 1]] = True
        at = torch.arange(L[b] + rows[b], device="cuda")
        p, s = c.pages[b][at // 16].long(), at % 16
        kk, vv = k[p, s].repeat_interleave(2, 1), v[p, s].repeat_interleave(2, 1)
        x = torch.einsum("ihd,jhd->ihj", q[first[b]:first[b + 1]].double(), kk) / 8
        i = torch.arange(rows[b], device="cuda")
        x.masked_fill_((at > L[b] + i[:, None])[:, None], -math.inf)
        want = torch.einsum("ihj,jhd->ihd", torch.softmax(x, -1), vv)
        if not torch.isfinite(want).all():           # slots that no request owns
            continue
        alone = owners[first[b]:first[b + 1]] == 1   # a row of two requests is either's
        assert ((out[first[b]:first[b + 1]].double() - want)[alone].abs() <= 2.0 ** -7 * (want[alone].abs() + 1)).all()
    assert (out[~seen] == 7).all()


def test_write_rows_of_any_stride(tree):
    """k and v inside a fused projection; a request whose rows do not fit hides no other."""
    from serial_draft_head_gb300 import walk
    c = Case(tree, 8, 4, 64, 16, BF16, [20, 13, 5], [5, 100, 40], seed=370)
    fused = torch.randn(38, 16, 64, device="cuda").to(BF16)
    k, v = fused[:, 8:12], fused[:, 12:16]
    c.tree.write(c.cache, c.pages, c.length, c.first, k, v)
    got = c.tree.read(c.cache, c.pages, c.length, c.first, 38)
    assert c.tree.status() == 0
    for x, y in zip((k, v), got):
        value, byte = e2m1.quantise(x)
        assert torch.equal(y.double(), value * e2m1.scale_of(byte).repeat_interleave(16, -1))
    c.tree.write(c.cache, c.pages, torch.tensor([5, -1, 40], dtype=torch.int32, device="cuda"), c.first, v, k)
    assert c.tree.status() == walk.EPAGES
    got = c.tree.read(c.cache, c.pages, c.length, c.first, 38)
    for x, y, z in zip((v, k), (k, v), got):
        value, byte = e2m1.quantise(torch.cat([x[:20], y[20:33], x[33:]]))
        assert torch.equal(z.double(), value * e2m1.scale_of(byte).repeat_interleave(16, -1))
