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
