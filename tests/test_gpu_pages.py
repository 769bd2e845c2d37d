"""Page tables on the GPU against lists, and rounds of a serving loop with everything together."""
import random

import pytest
import torch

import e2m1_reference as e2m1
import tree_reference as ref
from test_gpu_rotate import formula, frequencies
from test_gpu_tree import BF16, F16, tree  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def Pages():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    from serial_draft_head_gb300 import Pages
    return Pages


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Lists:
    """The definition, request by request."""

    def __init__(self, n_pages, page, requests, max_pages):
        self.n_pages, self.page, self.R, self.P = n_pages, page, requests, max_pages
        self.table = [[-1] * max_pages for _ in range(requests)]
        self.held = [0] * requests
        self.free = list(range(n_pages))[::-1]         # the last is handed out first
        self.gone = []                                 # what stands behind the free ones

    def grow(self, length, count, N, depth=None):
        first, slot, position, bad = [0], [-1] * N, [-1] * N, False
        wanted, free_before = 0, len(self.free)
        for r in range(self.R):
            n, t = length[r], count[r]
            ok = n >= 0 and t >= 0 and n + t <= self.P * self.page
            t = max(t, 0)
            need = max(-(-(n + t) // self.page) - self.held[r], 0) if ok else 0
            wanted += need
            served = need == 0 or wanted <= free_before
            fits = first[r] + t <= N
            bad |= not (ok and served and fits)
            if ok and served:
                for _ in range(need):
                    self.table[r][self.held[r]] = self.free.pop()
                    self.held[r] += 1
            for i in range(min(t, max(N - first[r], 0))):
                at, m = n + i, first[r] + i
                if ok and fits:
                    position[m] = at if depth is None else n + depth[m] - 1
                    if served:
                        slot[m] = self.table[r][at // self.page] * self.page + at % self.page
            first.append(first[r] + t)
        return first, slot, position, bad

    def trim(self, length):
        bad, back = False, []
        for r in range(self.R):
            if not 0 <= length[r] <= self.P * self.page:
                bad = True
                continue
            keep = min(self.held[r], -(-length[r] // self.page))
            back += self.table[r][keep:self.held[r]]
            self.table[r][keep:] = [-1] * (self.P - keep)
            self.held[r] = keep
        self.free += back[::-1]
        return bad

    def check(self, pool):
        assert pool.table.tolist() == self.table and pool.held.tolist() == self.held
        n = pool.n_free.item()
        assert n == len(self.free) and pool.free[:n].tolist() == self.free


@pytest.mark.parametrize("requests,page,max_pages,seed", [(1, 1, 5, 0), (3, 16, 8, 1), (16, 24, 20, 2), (256, 7, 12, 3),
                                                          (257, 64, 3, 4), (1024, 16, 9, 5), (1000, 100, 4, 6)])
@pytest.mark.parametrize("scarce", [False, True])
def test_grow_and_trim_as_lists_say(Pages, requests, page, max_pages, seed, scarce):
    """Many rounds of random lengths and counts, with numbers that do not fit and pools that run out."""
    from serial_draft_head_gb300 import walk
    rng = random.Random(seed)
    n_pages = max(requests * max_pages // (3 if scarce else 1), 1)
    pool, lists = Pages(n_pages, page, requests, max_pages), Lists(n_pages, page, requests, max_pages)
    lists.check(pool)
    most = max_pages * page
    for step in range(8):
        length = [min(rng.randint(0, most), h * page) if rng.random() < 0.9 else rng.randint(0, most) for h in lists.held]
        count = [rng.choice((0, 1, rng.randint(0, most - n))) for n in length]
        if step % 3 == 2:                              # numbers that do not fit
            r = rng.randrange(requests)
            length[r] = rng.choice((-1, most + 1, 2 ** 31 - 1, length[r]))
            count[rng.randrange(requests)] = rng.choice((-3, 2 ** 31 - 1, most))
        total = sum(max(t, 0) for t in count if t < 2 ** 30)
        N = min(total + rng.choice((0, 5, -3)), 200000)
        N = max(N, 0)
        first, slot, position = pool.grow(ints(length), ints(count), N)
        w_first, w_slot, w_position, bad = lists.grow(length, count, N)
        assert first.tolist() == [min(x, 2 ** 31 - 1) for x in w_first]
        assert slot.tolist() == w_slot and position.tolist() == w_position
        assert pool.status() == (walk.EPAGES if bad else 0) and pool.status() == 0
        lists.check(pool)
        after = [rng.choice((0, n, n + max(t, 0), rng.randint(0, most))) if rng.random() < 0.95 else -1
                 for n, t in zip(length, count)]
        pool.trim(ints([min(x, 2 ** 31 - 1) for x in after]))
        assert pool.status() == (walk.EPAGES if lists.trim(after) else 0)
        lists.check(pool)


def test_grow_then_trim_changes_nothing(Pages):
    pool = Pages(50, 16, 4, 20)
    pool.grow(ints([0, 0, 0, 0]), ints([33, 1, 0, 100]), 134)
    before = [x.clone() for x in (pool.table, pool.held, pool.free, pool.n_free)]
    length = ints([33, 1, 0, 100])
    for _ in range(3):
        first, slot, position = pool.grow(length, ints([20, 15, 17, 8]), 64)
        assert (slot[:60] >= 0).all() and (slot[60:] == -1).all() and first[-1] == 60
        assert len(set(slot[:60].tolist())) == 60
        pool.trim(length)
        assert all(torch.equal(x, y) for x, y in zip(before, (pool.table, pool.held, pool.free, pool.n_free)))
    assert pool.status() == 0


@pytest.mark.parametrize("T,words", [([5, 1, 40, 0, 31], 2), ([256, 3], 8), ([7], 1)])
def test_positions_by_depth(Pages, tree, T, words):
    """With a mask a node's position is its depth, whatever its place among the rows; strided masks."""
    first = ints([sum(T[:b]) for b in range(len(T) + 1)])
    parent = [-1 if i == 0 else max(0, i - 1 - (i * 7 + t) % 5) for t in T for i in range(t)]
    mask = tree.ancestor_bits(ints(parent), first)
    depth = []
    for b, t in enumerate(T):
        d = []
        for i in range(t):
            p = parent[sum(T[:b]) + i]
            d.append(0 if p < 0 else d[p] + 1)
        depth += d
    wide = torch.full((len(mask), words + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :mask.shape[1]] = mask
    pool = Pages(200, 16, len(T), 40)
    length = [17 * b + 3 for b in range(len(T))]
    first2, slot, position = pool.grow(ints(length), ints(T), sum(T), mask=wide[:, :mask.shape[1]])
    assert torch.equal(first, first2) and pool.status() == 0
    assert position.tolist() == [length[b] + depth[sum(T[:b]) + i] for b, t in enumerate(T) for i in range(t)]
    at = [length[b] + i for b, t in enumerate(T) for i in range(t)]
    table, b = pool.table.tolist(), [b for b, t in enumerate(T) for _ in range(t)]
    assert slot.tolist() == [table[r][x // 16] * 16 + x % 16 for r, x in zip(b, at)]


def test_many_rows_repeat_and_graph(Pages):
    """Rows enough for all blocks; the same every time; replayed from a graph with other lengths; two pools
    on two streams at once."""
    rng = random.Random(9)
    R, page, P = 700, 16, 40
    pools = [Pages(R * P, page, R, P) for _ in range(2)]
    length, count = ints([rng.randint(0, 300) for _ in range(R)]), ints([rng.randint(0, 300) for _ in range(R)])
    N = int(count.sum())
    streams = [torch.cuda.Stream() for _ in pools]
    torch.cuda.synchronize()
    got = [p.grow(length, count, N, stream=s) for p, s in zip(pools, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert len(set(got[0][1].tolist())) == N and pools[0].status() == 0
    out = [torch.empty_like(x) for x in got[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pools[0].trim(length)
        pools[0].grow(length, count, N, out=out)
    for step in range(3):
        if step:
            length += 7
            pools[1].trim(length)
            got[1] = pools[1].grow(length, count, N)
        else:
            pools[1].trim(length)
            got[1] = pools[1].grow(length, count, N)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, got[1])), step
        for name in ("table", "held", "n_free"):
            assert torch.equal(getattr(pools[0], name), getattr(pools[1], name))
        n = pools[0].n_free.item()
        assert torch.equal(pools[0].free[:n], pools[1].free[:n])


def test_refusals(Pages):
    pool = Pages(8, 16, 3, 4)
    z = ints([0, 0, 0])
    for bad in (lambda: pool.grow(z.long(), z, 4), lambda: pool.grow(z[:2], z, 4), lambda: pool.grow(z, z.cpu(), 4),
                lambda: pool.grow(z, z, 4, mask=torch.zeros(3, 1, dtype=torch.int32, device="cuda")),
                lambda: pool.grow(z, z, 4, mask=torch.zeros(4, 0, dtype=torch.int32, device="cuda")),
                lambda: pool.grow(z, z, 4, mask=torch.zeros(4, 2, dtype=torch.int32, device="cuda")[:, ::2].T.contiguous()),
                lambda: pool.grow(z, z, 4, out=(z, z, z)), lambda: pool.trim(z.float())):
        with pytest.raises(ValueError):
            bad()
    first, slot, position = pool.grow(z, z, 0)
    assert first.tolist() == [0, 0, 0, 0] and len(slot) == len(position) == 0 and pool.status() == 0


@pytest.mark.parametrize("n", [-1, 9, 2 ** 31 - 1])
def test_a_wrong_count_of_free_pages_hands_none_out(Pages, n):
    """A count that the pool cannot have, and a table that holds what is no page: reported, nothing given."""
    from serial_draft_head_gb300 import walk
    pool = Pages(8, 16, 3, 4)
    before = [x.clone() for x in (pool.table, pool.held, pool.free)]
    pool.n_free.fill_(n)
    z, c = ints([0, 0, 0]), ints([20, 1, 0])
    first, slot, position = pool.grow(z, c, 21)
    assert pool.status() == walk.EPAGES
    assert first.tolist() == [0, 20, 21, 21] and (slot == -1).all() and position.tolist() == list(range(20)) + [0]
    pool.trim(z)
    assert all(torch.equal(x, y) for x, y in zip(before, (pool.table, pool.held, pool.free))) and pool.n_free.item() == n
    pool.status()
    pool.reset()
    pool.held.fill_(5)                                 # more than a request's row has
    first, slot, position = pool.grow(z, c, 21)
    assert pool.status() == walk.EPAGES and (slot == -1).all()
    pool.trim(z)
    assert pool.status() == walk.EPAGES and pool.n_free.item() == 8
    pool.reset()
    pool.held.fill_(1)                                 # held, but -1 in the table
    first, slot, position = pool.grow(z, c, 21)
    assert pool.status() == walk.EPAGES and (slot[:16] == -1).all() and (slot[16:20] >= 0).all()


def test_all_pages_there_can_be_at_once(Pages):
    """2^31 - 1 pages of one slot (8.6 GB of them free, 8.6 GB of table) go to one request and back."""
    n, some = 2 ** 31 - 1, 100000
    pool = Pages(n, 1, 1, n)
    first, slot, position = pool.grow(ints([0]), ints([n]), n)
    assert pool.status() == 0 and int(pool.held) == n and int(pool.n_free) == 0
    assert first.tolist() == [0, n]
    for at in (0, n // 2, n - some):
        want = torch.arange(at, at + some, dtype=torch.int32, device="cuda")
        assert torch.equal(slot[at:at + some], want)
        assert torch.equal(position[at:at + some], want)
        assert torch.equal(pool.table[0, at:at + some], want)
    del slot, position
    pool.free[:some] = -7                            # what comes back is written again
    pool.free[n - some:] = -7
    pool.trim(ints([0]))
    assert pool.status() == 0 and int(pool.held) == 0 and int(pool.n_free) == n
    for at in (0, n // 2, n - some):
        want = n - 1 - torch.arange(at, at + some, dtype=torch.int32, device="cuda")
        assert torch.equal(pool.free[at:at + some], want)
        assert bool((pool.table[0, at:at + some] == -1).all())
    for many in (-1, 2 ** 31):
        with pytest.raises(ValueError):
            pool.grow(ints([0]), ints([0]), many)


@pytest.mark.parametrize("held", ["e2m1", "e4m3", "16"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rounds_together(Pages, tree, held, dtype):
    """Prompts and then rounds of a serving loop: pages and slots for a round's rows, norms and rotation on
    the way into the cache, attention of trees over it, the accepted path kept, pages given back; the
    requests come and go.  Each round's attention is that of the cached values, and the cache holds what
    the requests' tokens are worth at their positions."""
    Hq, Hkv, D, page, R, P = 8, 2, 64, 16, 4, 20
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rng = random.Random(5)
    pool = Pages(40, page, R, P)
    cache = tree.KVCache.zeros(40, page, Hkv, D, {"e2m1": torch.uint8, "e4m3": torch.float8_e4m3fn, "16": dtype}[held])
    t = tree.Tree(Hq, Hkv, D, dtype, max_requests=R, max_nodes=70)
    freq = frequencies(D)
    norms = [0.5 + torch.rand(D, generator=g, device="cuda") for _ in range(2)]
    rotation = tree.Rotation(D, freq, *norms)
    length = [0] * R
    texts = [[] for _ in range(R)]                     # (k, v) rows of the requests' tokens, before rotation
    for step in range(6):
        T = [rng.randint(30, 70) if n == 0 else rng.randint(0, 20) for n in length]
        N = sum(T)
        first = ints([sum(T[:b]) for b in range(R + 1)])
        parent = [-1 if i == 0 else i - 1 if length[b] == 0 else max(0, i - rng.randint(1, 4)) for b, n in enumerate(T)
                  for i in range(n)]
        mask = tree.ancestor_bits(ints(parent), first)
        q, k, v = (torch.randn(N, h, D, generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
        at = ints(length)
        first2, slot, position = pool.grow(at, ints(T), N, mask=mask)
        q2 = t.place(cache, slot, q, k, v, position, rotation)
        out, lse = t.attend(q2, cache, pool.table, at, first2, mask=mask)
        assert torch.equal(first, first2) and t.status() == 0 and pool.status() == 0
        # attention is that of what the cache holds
        everything = ints(sum(([b] * (n + x) for b, (n, x) in enumerate(zip(length, T))), []))
        kk, vv = (torch.zeros(40, page, Hkv, D, dtype=torch.float64, device="cuda") for _ in range(2))
        f = ints([sum(length[:b]) + sum(T[:b]) for b in range(R + 1)])
        back = t.read(cache, pool.table, ints([0] * R), f, len(everything))
        for b in range(R):
            j = torch.arange(length[b] + T[b], device="cuda")
            where = pool.table[b][j // page].long(), j % page
            kk[where], vv[where] = (x[f[b]:f[b + 1]].double() for x in back)
        want, want_lse, weight, sums = ref.attend(q2, kk, vv, None, None, pool.table, page, at, first, mask, D ** -0.5, 0.0)
        tol, tol_lse = ref.bounds(want, weight, sums, D, dtype, 0.0)
        extra = 0 if held != "e2m1" else (max(T) + max(length)) * 2.0 ** -31 * vv.abs().max()
        assert ((out.double() - want).abs() <= tol + extra).all() and ((lse.double() - want_lse).abs() <= tol_lse).all()
        # the longest chain of each tree is kept, and all of a prompt
        path, count = torch.zeros(R, 70, dtype=torch.int32), []
        for b in range(R):
            chain, i = [], T[b] - 1
            while i >= 0:
                chain.append(i)
                i = parent[sum(T[:b]) + i]
            path[b, :len(chain)] = torch.tensor(chain[::-1], dtype=torch.int32)
            count.append(len(chain))
            rows = [sum(T[:b]) + i for i in chain[::-1]]
            texts[b] += [(k[i], v[i]) for i in rows]
        t.keep(cache, pool.table, at, path.cuda(), ints(count))
        length = [n + x for n, x in zip(length, count)]
        if step in (2, 4):                             # a request ends, its pages are free for the next
            length[step // 2], texts[step // 2] = 0, []
        pool.trim(ints(length))
        assert t.status() == 0 and pool.status() == 0
        assert pool.held.tolist() == [-(-n // page) for n in length]
        assert pool.n_free.item() == 40 - sum(pool.held.tolist())
        # the cache holds the tokens at their positions, in order
        f = ints([sum(length[:b]) for b in range(R + 1)])
        got_k, got_v = t.read(cache, pool.table, ints([0] * R), f, sum(length))
        raw_k, raw_v = (torch.stack([x[i] for text in texts for x in text]) for i in range(2))
        places = ints([i for n in length for i in range(n)])
        want_k, size = formula(raw_k, places, freq.cuda(), norms[1], 1e-6, False)
        half = torch.finfo(dtype).eps / 2
        off = (got_k.double() - want_k).abs() - (half * want_k.abs() + 2.0 ** -18 * size + 2.0 ** -24)
        if held == "16":
            assert torch.equal(got_v, raw_v) and (off <= 0).all()
        elif held == "e4m3":
            # half a step of the row's largest code, 448, is 16
            top = want_k.abs().amax(-1, keepdim=True)
            assert (off <= 2 * top * 16 / 448).all()
        else:
            # half a step at the block's largest code, 6, is 1; a scale is up to 9 / 8 of what it has to be
            top = want_k.unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
            assert (off <= top * 1.13 / 6 + 2.0 ** -17).all()
            value, byte = e2m1.quantise(raw_v)
            assert torch.equal(got_v.double(), value * e2m1.scale_of(byte).repeat_interleave(16, -1))


@pytest.mark.parametrize("cache,rotary", [("e2m1", False), ("e2m1", True), ("e4m3", True), ("16", True)])
def test_example_runs(tree, cache, rotary):
    """The example's loop over a 4-bit cache, and with pages from the pool and turned heads: it ends with the
    requests' rows in the cache, and with no more pages held than they need."""
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import draft_and_check as ex
    finally:
        sys.path.pop(0)
    target = ex.Target(vocab=2048)
    texts, cached, pages, length = ex.decode(target, [5, 9, 77], rounds=4, gamma=5, cache=cache, rotary=rotary)
    assert [len(t) - 1 for t in texts] == length.tolist()
    if rotary:
        assert (pages >= 0).sum(1).tolist() == [-(-n // 16) for n in length.tolist()]
    t = tree.Tree(8, 2, 64, max_requests=3)
    n = int(length.sum())
    first = torch.tensor([0] + length.cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    k, v = t.read(cached, pages, torch.zeros_like(length), first, n)
    assert t.status() == 0
    tokens = torch.tensor([x for text in texts for x in text[:-1]], device="cuda")
    if cache == "e2m1":
        value, byte = e2m1.quantise(target.v[tokens])
        assert torch.equal(v.double(), value * e2m1.scale_of(byte).repeat_interleave(16, -1))
    elif cache == "16":
        assert torch.equal(v, target.v[tokens])
    if not rotary:
        value, byte = e2m1.quantise(target.k[tokens])
        assert torch.equal(k.double(), value * e2m1.scale_of(byte).repeat_interleave(16, -1))
