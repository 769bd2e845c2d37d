"""Page tables at their edges: pools that run out and tables that hold what is no page."""
import pytest
import torch

from test_gpu_pages import Pages, ints  # noqa: F401

pytestmark = pytest.mark.gpu


def test_free_pages_go_out_in_the_order_of_the_requests(Pages):  # noqa: F811
    """No request overtakes one that the free pages do not serve; those that lack no page get their slots,
    and the pages that are left go to whoever is first the next time."""
    from serial_draft_head_gb300 import walk
    pool = Pages(8, 16, 5, 8)
    length, count = ints([0, 0, 0, 3, 0]), ints([20, 100, 1, 2, 1])
    pool.grow(ints([0, 0, 0, 3, 0]), ints([0, 0, 0, 0, 0]), 0)      # request 3 holds its page: 7 are left
    assert pool.held.tolist() == [0, 0, 0, 1, 0] and pool.status() == 0
    first, slot, position = pool.grow(length, count, 124)           # 2, 7, 1, 0 and 1 pages are lacking
    assert pool.status() == walk.EPAGES and pool.status() == 0
    assert first.tolist() == [0, 20, 120, 121, 123, 124]
    assert pool.held.tolist() == [2, 0, 0, 1, 0] and pool.n_free.item() == 5
    assert (slot[:20] >= 0).all() and (slot[20:121] == -1).all() and slot[121:].tolist() == [3, 4, -1]
    assert position.tolist() == list(range(20)) + list(range(100)) + [0, 3, 4, 0]
    first, slot, _ = pool.grow(length, ints([20, 0, 1, 2, 1]), 24)  # without the one in the way
    assert pool.status() == 0 and (slot >= 0).all() and pool.held.tolist() == [2, 0, 1, 1, 1]


def test_trim_gives_no_entry_back_that_is_no_page(Pages):  # noqa: F811
    """Entries past the pool and below it leave the table, are reported, and are never handed out."""
    from serial_draft_head_gb300 import walk
    pool = Pages(8, 16, 3, 4)
    z = ints([0, 0, 0])
    pool.grow(z, ints([48, 32, 0]), 80)                            # pages 0, 1, 2 and 3, 4
    pool.table[0, 1], pool.table[1, 1] = -1, 8
    pool.trim(z)
    assert pool.status() == walk.EPAGES and pool.status() == 0
    assert (pool.table == -1).all() and pool.held.tolist() == [0, 0, 0]
    assert pool.n_free.item() == 6 and pool.free[:6].tolist() == [7, 6, 5, 3, 2, 0]
    _, slot, _ = pool.grow(z, ints([64, 32, 0]), 96)
    assert pool.status() == 0 and (slot.view(6, 16)[:, 0] // 16).tolist() == [0, 2, 3, 5, 6, 7]


@pytest.mark.parametrize("requests,each,share", [(1024, 90, 0.01), (700, 3, 0.5), (5, 20000, 0.2), (3, 7, 1.0)])
def test_trim_of_many_entries_that_are_no_pages(Pages, requests, each, share):  # noqa: F811
    """Any share of them, in all blocks: the rest comes back in its order, in a replayed graph as well."""
    from serial_draft_head_gb300 import walk
    g = torch.Generator(device="cuda")
    g.manual_seed(requests)
    n = requests * each + 9
    pool = Pages(n, 1, requests, each)
    z = torch.zeros(requests, dtype=torch.int32, device="cuda")
    count = torch.randint(0, each + 1, (requests,), generator=g, device="cuda").int()
    pool.grow(z, count, 0)
    pool.status()                                                  # rows past none: not what is tested
    for _ in range(2):
        free = pool.free[:pool.n_free.item()].clone()
        held = pool.table >= 0
        bad = held & (torch.rand(requests, each, generator=g, device="cuda") < share)
        wrong = torch.where(torch.rand(requests, each, generator=g, device="cuda") < 0.5, -3, n)
        pool.table[bad] = wrong[bad].int()
        want = torch.cat([free, pool.table[held & ~bad].flip(0)])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pool.trim(z)
        graph.replay()
        assert pool.status() == (walk.EPAGES if bad.any() else 0)
        assert (pool.table == -1).all() and (pool.held == 0).all()
        assert pool.n_free.item() == len(want) and torch.equal(pool.free[:len(want)], want)
        graph.replay()                                             # nothing is held any more
        assert pool.status() == 0 and torch.equal(pool.free[:len(want)], want)
        count = torch.minimum(count, torch.full_like(count, len(want) // requests))
        pool.grow(z, count, 0)
        pool.status()


def test_trim_takes_pages_held_before_the_rows_came(Pages):  # noqa: F811
    """A request that held more than its length needs gives that back as well; the others end as they began."""
    pool = Pages(20, 16, 2, 10)
    pool.grow(ints([0, 0]), ints([100, 20]), 120)                  # 7 and 2 pages
    length = ints([40, 20])
    pool.grow(length, ints([5, 30]), 35)                           # none and 2 more
    assert pool.held.tolist() == [7, 4] and pool.n_free.item() == 9
    pool.trim(length)
    assert pool.held.tolist() == [3, 2] and pool.n_free.item() == 15 and pool.status() == 0
    assert pool.table[0].tolist() == [0, 1, 2] + [-1] * 7 and pool.table[1].tolist() == [7, 8] + [-1] * 8
    assert pool.free[:15].tolist() == list(range(19, 10, -1)) + [10, 9, 6, 5, 4, 3]
