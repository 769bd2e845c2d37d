"""The draft-check operators at their edges: barriers' phases under load, streams, sizes near what
indexes hold, masked and visible values that are not finite, scales and caps of any size."""
import math

import pytest
import torch

import tree_reference as ref
from test_gpu_tree import BF16, E4M3, F16, Case, tree  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,cache", [(128, 64, "16"), (128, 16, "16"), (64, 64, "16"), (64, 24, "16"),
                                          (128, 64, "e4m3"), (64, 24, "e4m3")])
def test_attend_alternate_tiles_back_to_back(tree, D, page, cache):
    """One row tile (two streams in turn over the same ring): segments of one tile to many, so that a
    stream passes slots quickly while the other works; calls in a row without a wait.  The same bits
    every time, and no wait runs out."""
    T = [9, 14, 30, 9, 11, 25]
    cases = [Case(tree, 8, 2, D, page, BF16, cache, T, L, seed=200 + i, spare=1)
             for i, L in enumerate([[0, 100, 129, 20000, 5, 640], [7000, 1, 260, 130, 131, 9000],
                                    [120, 119, 118, 117, 116, 115]])]
    want = []
    for c in cases:
        want.append(c.attend())
        c.check(*want[-1])
    for _ in range(40):
        got = [c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask) for c in cases * 3]
        for i, (o, l) in enumerate(got):
            assert torch.equal(o, want[i % 3][0]) and torch.equal(l, want[i % 3][1])
    assert all(c.tree.status() == 0 for c in cases)


def test_attend_at_once_on_a_side_stream_of_a_new_handle(tree):
    """A handle made while the default stream is busy, and used on another stream at once: items of
    many parts go by counts that the making of the handle has cleared."""
    c = Case(tree, 8, 2, 128, 16, BF16, "16", [1, 2, 1], [20000, 37, 900], seed=210)
    out, lse = c.attend()
    c.check(out, lse)
    x = torch.randn(8192, 8192, device="cuda").to(BF16)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(40):                        # some 20 ms of queue
            torch.matmul(x, x, out=y)
        t = tree.Tree(8, 2, 128, BF16, max_requests=3, max_nodes=2)
        o2, l2 = t.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask, stream=side)
        side.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert t.status(stream=side) == 0
        t.close()


@pytest.mark.parametrize("T", [1, 40])
def test_attend_positions_near_what_an_index_holds(tree, T):
    """All positions are one slot (strides of zero), so that a cache of 2^31 - 1 rows fits: a request
    that would end past the longest length is left out and reported, its neighbour runs."""
    from serial_draft_head_gb300 import walk
    g = torch.Generator(device="cuda")
    g.manual_seed(220)
    slots, most = 2 ** 31 - 1, tree.TREE_MAX_LENGTH
    k, v, q = (torch.randn(n, 1, 64, generator=g, device="cuda").to(BF16) for n in (1, 1, 2 * T))
    cache = tree.KVCache(k[:, None].expand(1, slots, 1, 64), v[:, None].expand(1, slots, 1, 64))
    t = tree.Tree(1, 1, 64, BF16, max_requests=2, max_nodes=T)
    pages = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    first = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
    s = (q.double() @ k[0, 0].double() / 8)[:, 0]
    for past in (slots - T, most - T + 1):
        length = torch.tensor([past, 77], dtype=torch.int32, device="cuda")
        out = torch.full((2 * T, 1, 64), 5.0, dtype=BF16, device="cuda")
        _, lse = t.attend(q, cache, pages, length, first, out=out)
        assert t.status() == walk.EPAGES
        assert (out[:T] == 5).all() and torch.equal(out[T:], v.expand(T, 1, 64))
        n = 78 + torch.arange(T, device="cuda")
        assert (lse[T:, 0].double() - s[T:] - n.double().log()).abs().max() < 1e-4


# ---------------------------------------------------------------- scores --

FEW = [1, 3, 2]                     # 2 to 6 rows a cached head of 2 query heads
TILES = [30, 100]


@pytest.mark.parametrize("T", [FEW, [4] * 3, TILES])
@pytest.mark.parametrize("dtype,cache", [(BF16, "16"), (F16, "16"), (BF16, "e4m3"), (F16, "e4m3")])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attend_scale_of_any_sign_and_zero(tree, T, dtype, cache, scale):
    """Totals that end inside a block, in both kernels; a scale of zero weighs all visible keys alike."""
    c = Case(tree, 4, 2, 64, 20, dtype, cache, T, [200, 45, 0][:len(T)], seed=230)
    c.check(*c.attend(scale=scale), scale=scale)


def check_capped(c, out, lse, scale, softcap, sums=None, mask=None):
    """Against the definition, by bounds that do not grow with the cap: `ref.bounds` of uncapped scores, and
    2^-20 of a score for the cap itself (tanh(y) / y or 1 - 2 / (e^2y + 1), each a few roundings), which
    counts like a score's other error: twice in a weight, once more in lse."""
    keep, c.mask = c.mask, c.mask if mask is None else mask
    want, want_lse, weight, own = ref.attend(c.q, c.k, c.v, c.ks, c.vs, c.pages, c.page, c.length, c.first,
                                             c.mask, scale, softcap)
    c.mask = keep
    sums = own if sums is None else sums
    tol, tol_lse = ref.bounds(want, weight, sums, c.D, c.dtype, 0.0)
    extra = 2.0 ** -20 * sums.clamp(max=softcap)
    tol, tol_lse = tol + 2 * extra[..., None] * weight, tol_lse + 3 * extra
    off, far = (out.double() - want).abs() - tol, (lse.double() - want_lse).abs() - tol_lse
    assert (off <= 0).all(), "out is %g past its bound" % off.max()
    assert (far <= 0).all(), "lse is %g past its bound" % far.max()


@pytest.mark.parametrize("T", [FEW, TILES])
@pytest.mark.parametrize("dtype,cache", [(BF16, "16"), (F16, "16"), (BF16, "e4m3"), (F16, "e4m3")])
@pytest.mark.parametrize("softcap", [8.0, 50.0, 1e4, 1e6, 1e8, 1e20, 3e38, 1e-3, 1e-38])
def test_attend_cap_of_any_size(tree, T, dtype, cache, softcap):
    """Scores of about 10 keep their precision under any cap."""
    c = Case(tree, 4, 2, 64, 20, dtype, cache, T, [200, 45, 0][:len(T)], seed=231)
    out, lse = c.attend(scale=1.25, softcap=softcap)
    check_capped(c, out, lse, 1.25, softcap)


@pytest.mark.parametrize("T", [FEW, TILES])
@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_attend_scores_near_the_cap_beside_small_ones(tree, T, cache):
    """One key far below the others, near the cap: its weight is nothing, the others keep theirs."""
    c = Case(tree, 4, 2, 64, 20, BF16, cache, T, [200, 45, 0][:len(T)], seed=232, mask=None)
    c.q[:, :, 0] = 1.0
    for b, n in enumerate(c.L):                    # the last node of each request
        p = n + T[b] - 1
        page, slot = c.pages[b, p // 20].long(), p % 20
        row = torch.zeros(64, device="cuda")
        row[0] = -2.0 ** 19
        if cache == "e4m3":
            code, byte = ref.quantise(row[None])
            c.k[page, slot] = code.float().to(E4M3)
            c.ks[page, slot] = byte
        else:
            c.k[page, slot] = row.to(BF16)
    words = (max(T) + 31) // 32
    c.mask = torch.full((c.N, words), -1, dtype=torch.int32, device="cuda")
    without = c.mask.clone()
    for b, t in enumerate(T):
        rows = slice(int(c.first[b]), int(c.first[b + 1]))
        if t > 1 or c.L[b] > 0:
            without[rows, (t - 1) // 32] ^= torch.tensor(1 << (t - 1) % 32, dtype=torch.int64).int().item() \
                if (t - 1) % 32 < 31 else -2 ** 31
    out, lse = c.attend(scale=1.0, softcap=1e6)
    check_capped(c, out, lse, 1.0, 1e6, mask=without)


@pytest.mark.parametrize("T,L", [([1, 3, 2, 1], [200, 45, 1, 0]), ([30, 100, 40], [200, 1, 0])])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_attend_infinite_scores_meet_the_cap(tree, T, L, dtype, bad):
    """A score of either infinity is the cap or its negative, where nothing else is visible too."""
    c = Case(tree, 4, 2, 64, 20, dtype, "16", T, L, seed=233, mask="tree")
    def put(x):  # noqa: E306
        for b, n in enumerate(L):                  # the request's first key, and its last node
            for p in (0, n + T[b] - 1):
                c.k[c.pages[b, p // 20].long(), p % 20, :, 5] = x
    put(0.0)
    sums = ref.attend(c.q, c.k, c.v, None, None, c.pages, 20, c.length, c.first, c.mask, 0.2, 2.0)[3]
    put(bad)
    assert (c.q[:, :, 5] != 0).all()
    out, lse = c.attend(scale=0.2, softcap=2.0)
    check_capped(c, out, lse, 0.2, 2.0, sums=sums)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_smallest_scale_of_keys(tree, D):
    """Keys under scale byte 0, 2^-127, with queries that reach them."""
    c = Case(tree, 4, 2, D, 20, BF16, "e4m3", FEW, [200, 45, 0], seed=234)
    c.ks[c.ks != 255] = 0
    c.q = (c.q.float() * 2.0 ** 118).to(BF16)
    c.check(*c.attend(scale=0.25), scale=0.25)


# -------------------------------------------------- invisible rows of the draft --


@pytest.mark.parametrize("T,L", [([3, 2], [130, 20]), ([4, 3, 2], [3000, 0, 7]), ([1, 5], [500, 33]),
                                 ([9, 150], [130, 20]), ([40, 20], [5000, 250])])
@pytest.mark.parametrize("dtype,cache", [(BF16, "16"), (F16, "16"), (BF16, "e4m3"), (F16, "e4m3")])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attend_invisible_rows_hold_anything_in_both_kernels(tree, T, L, dtype, cache, bad, where):
    """What a node holds reaches the nodes that see it and no other: few rows and tiles, items in one
    piece and in parts, every type."""
    if cache == "e4m3" and not math.isnan(bad):
        pytest.skip("an e4m3 row that is not finite is NaN")
    c = Case(tree, 4, 2, 64, 20, dtype, cache, T, L, seed=235, mask=None)
    parent = torch.tensor([-1 if i == 0 else 0 for t in T for i in range(t)], dtype=torch.int32, device="cuda")
    c.mask = tree.ancestor_bits(parent, c.first)   # all nodes are children of node 0
    nodes = [(b, j) for b, t in enumerate(T) for j in {t - 1, t // 2} if j > 0]
    clean_out, clean_lse = c.attend()
    for b, j in nodes:
        p = L[b] + j
        page, slot = c.pages[b, p // 20].long(), p % 20
        if cache == "e4m3":
            getattr(c, where).view(torch.uint8)[page, slot] = 0x7f
            getattr(c, where + "s")[page, slot] = 255
        else:
            getattr(c, where)[page, slot, :, 3] = bad
    out, lse = c.attend()
    hit = torch.zeros(c.N, dtype=torch.bool, device="cuda")
    for b, j in nodes:
        hit[int(c.first[b]) + j] = True
    assert torch.equal(out[~hit], clean_out[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    if where == "v":
        assert torch.equal(lse[hit], clean_lse[hit])
        if cache == "e4m3":
            assert torch.isnan(out[hit]).all()
        else:
            got = out[hit][..., 3].float()
            assert torch.isnan(got).all() if math.isnan(bad) else (got == bad).all()
            other = [i for i in range(64) if i != 3]
            assert torch.equal(out[hit][..., other], clean_out[hit][..., other])
    elif math.isnan(bad):
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()


@pytest.mark.parametrize("T,L", [([3, 2], [130, 20]), ([4, 3, 2], [3000, 0, 7]), ([40, 20], [600, 250])])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("byte", [0, 60, 112, 135, 150])
def test_attend_scales_of_invisible_rows(tree, T, L, dtype, byte):
    """The scale that an invisible row of the draft has (finite in the rows' type) changes no bit."""
    if dtype == F16 and byte > 134:
        byte = 134
    c = Case(tree, 4, 2, 64, 20, dtype, "e4m3", T, L, seed=236, mask=None)
    parent = torch.tensor([-1 if i == 0 else 0 for t in T for i in range(t)], dtype=torch.int32, device="cuda")
    c.mask = tree.ancestor_bits(parent, c.first)
    clean_out, clean_lse = c.attend()
    hit = torch.zeros(c.N, dtype=torch.bool, device="cuda")
    for b, t in enumerate(T):
        p = L[b] + t - 1
        page, slot = c.pages[b, p // 20].long(), p % 20
        c.ks[page, slot] = byte
        c.vs[page, slot] = byte
        hit[int(c.first[b]) + t - 1] = True
    out, lse = c.attend()
    assert torch.equal(out[~hit], clean_out[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


# -------------------------------------------------------------- parts --


@pytest.mark.parametrize("T,cache", [(1, "16"), (4, "e4m3"), (20, "16"), (60, "16"), (40, "e4m3")])
def test_attend_one_item_over_all_workers(tree, T, cache):
    """One cached head and a long context: an item of as many parts as there are SMs."""
    c = Case(tree, 4, 1, 64, 16, BF16, cache, [T], [60000], seed=240)
    out, lse = c.attend()
    c.check(out, lse)
    for _ in range(5):
        o2, l2 = c.attend()
        assert torch.equal(out, o2) and torch.equal(lse, l2)


# ------------------------------------------------------------- arguments --


def test_attend_refuses_a_mask_without_words(tree):
    c = Case(tree, 4, 2, 64, 16, BF16, "16", [4], [40], seed=250)
    with pytest.raises((ValueError, tree.WalkError)):
        c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=c.mask[:, :0])
    assert c.tree.status() == 0


def test_attend_takes_a_mask_of_many_words(tree):
    """More words a row than nodes need, as many as 2^26."""
    for T in (1, 20):
        c = Case(tree, 4, 2, 64, 16, BF16, "16", [T], [40], seed=251)
        out, lse = c.attend()
        wide = torch.zeros(T, 1 << 26, dtype=torch.int32, device="cuda")
        wide[:, :1] = c.mask
        o2, l2 = c.tree.attend(c.q, c.cache, c.pages, c.length, c.first, mask=wide)
        assert c.tree.status() == 0
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        del wide


@pytest.mark.parametrize("T", [2, 40])
def test_attend_where_no_request_has_rows(tree, T):
    """All requests fail, or none has a row: nothing is written."""
    from serial_draft_head_gb300 import walk
    c = Case(tree, 4, 2, 64, 16, BF16, "16", [T, T], [40, 9], seed=252)
    for length, first, code in ((-1, c.first, walk.EPAGES), (3, torch.zeros_like(c.first), 0)):
        out = torch.full_like(c.q, 3.0)
        c.tree.attend(c.q, c.cache, c.pages, torch.full_like(c.length, length), first, mask=c.mask, out=out)
        assert c.tree.status() == code and (out == 3).all()


FIRSTS = [[0, 2 ** 31 - 1, 9, 15], [0, -1, 9, 15], [3, 1, 9, 15], [0, 12, 9, 15], [0, 4, 2, 15]]


@pytest.mark.parametrize("first", FIRSTS)
@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_a_bad_row_range_leaves_the_other_requests_alone(tree, first, cache):
    """Requests behind one whose rows are out of range are written, read and attended to."""
    from serial_draft_head_gb300 import walk
    T, L = [9, 9, 6], [40, 50, 60]
    c = Case(tree, 4, 2, 64, 16, BF16, cache, T, L, seed=253, garbage=None, mask=None)
    c.tree = tree.Tree(4, 2, 64, BF16, max_requests=3, max_nodes=16)
    N = 15
    f = torch.tensor(first, dtype=torch.int32, device="cuda")
    ok = [0 <= a <= b <= N for a, b in zip(first, first[1:])]
    assert not all(ok) and ok[2]
    new = torch.randn(N, 2, 64, generator=c.g, device="cuda").to(BF16)
    c.tree.write(c.cache, c.pages, c.length, f, new, new)
    assert c.tree.status() == walk.EPAGES
    code, byte = ref.quantise(new)
    want = (code * ref.scale_of(byte)[..., None]).to(BF16) if cache == "e4m3" else new
    alone = torch.tensor([0, first[3] - first[2]], dtype=torch.int32, device="cuda")
    rows = slice(first[2], first[3])
    got = c.tree.read(c.cache, c.pages[2:], c.length[2:], alone, first[3] - first[2])
    assert c.tree.status() == 0
    assert all(torch.equal(x, want[rows]) for x in got)
    back = tuple(torch.full((N, 2, 64), 5.0, dtype=BF16, device="cuda") for _ in range(2))
    c.tree.read(c.cache, c.pages, c.length, f, N, out=back)
    assert c.tree.status() == walk.EPAGES
    assert all(torch.equal(x[rows], want[rows]) for x in back)
    q = torch.randn(N, 4, 64, generator=c.g, device="cuda").to(BF16)
    out, _ = c.tree.attend(q, c.cache, c.pages, c.length, f)
    assert c.tree.status() == walk.EPAGES
    one, _ = c.tree.attend(q[rows], c.cache, c.pages[2:], c.length[2:], alone)
    assert c.tree.status() == 0
    if all(b <= first[2] for a, b, o in zip(first[:2], first[1:], ok) if o):
        # rows of one request only; the kernel's choice goes by all requests' rows: within roundings
        assert (out[rows].double() - one.double()).abs().max() < 2.0 ** -6


def test_cache_calls_report_bad_requests_without_rows(tree):
    """As attend does: a request that has no rows but numbers that do not fit."""
    from serial_draft_head_gb300 import walk
    c = Case(tree, 2, 2, 64, 16, BF16, "e4m3", [4, 0, 5], [40, 7, 50], seed=254, garbage=None, mask=None)
    new = torch.randn(9, 2, 64, generator=c.g, device="cuda").to(BF16)
    for length in (-1, 1 << 20):
        bad = c.length.clone()
        bad[1] = length
        c.tree.write(c.cache, c.pages, bad, c.first, new, new)
        assert c.tree.status() == walk.EPAGES
        k, v = c.tree.read(c.cache, c.pages, bad, c.first, 9)
        assert c.tree.status() == walk.EPAGES
        code, byte = ref.quantise(new)
        want = (code * ref.scale_of(byte)[..., None]).to(BF16)
        assert torch.equal(k, want) and torch.equal(v, want)
        q = torch.randn(9, 2, 64, generator=c.g, device="cuda").to(BF16)
        c.tree.attend(q, c.cache, c.pages, bad, c.first)
        assert c.tree.status() == walk.EPAGES


def test_keep_of_many_requests(tree):
    """More requests than a grid is wide in its second direction."""
    B, page, Hkv, D = 70001, 4, 1, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(255)
    t = tree.Tree(1, Hkv, D)
    k = torch.randn(B, page, Hkv, D, generator=g, device="cuda").to(BF16)
    v = torch.randn(B, page, Hkv, D, generator=g, device="cuda").to(BF16)
    want = [x.clone() for x in (k, v)]
    for x in want:
        x[:, 1] = x[:, 3]
    pages = torch.randperm(B, generator=g, device="cuda").int()[:, None].contiguous()
    start = torch.ones(B, dtype=torch.int32, device="cuda")
    path = torch.full((B, 1), 2, dtype=torch.int32, device="cuda")
    t.keep(tree.KVCache(k, v), pages, start, path, torch.ones_like(start))
    assert t.status() == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.parametrize("T,L", [([1], [600]), ([2, 3], [45, 0]), ([20], [600])])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attend_slots_past_the_end_change_no_bit(tree, T, L, dtype):
    """Codes and scales of a page's slots that a request has not reached."""
    c = Case(tree, 4, 2, 64, 64, dtype, "e4m3", T, L, seed=256, garbage=None)
    out, lse = c.attend()
    free = torch.ones(c.n_pages, 64, dtype=torch.bool, device="cuda")
    for b in range(c.B):
        at = torch.arange(L[b] + T[b], device="cuda")
        free[c.pages[b][at // 64].long(), at % 64] = False
    for code, byte in ((0, 0), (0x7f, 255), (0x55, 200), (0x7e, 254)):
        for x in (c.k, c.v):
            x.view(torch.uint8)[free] = code
        for x in (c.ks, c.vs):
            x[free] = byte
        o2, l2 = c.attend()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
