"""dfl2_cache_evict of sequences that are no longer than `keep`: nothing moves, and their pages are
looked at all the same."""
import numpy as np
import pytest

import draft_selection_gb300 as dfl2
from test_gpu_evict import Held
from test_gpu_tree_attn import _lib  # noqa: F401  (the fixture builds and loads the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [8, 64])
def test_short_sequences_that_lack_pages_are_not_served(page):
    """The first, a middle and the last page missing, one out of range; a page past the length
    may be missing, and a sequence of none needs none."""
    n = 5 * page - 3
    h = Held([n, n, n, n, n, n - 2 * page, 0, 3000], page, seed=page, extra=1)
    for b, entry, value in [(0, 0, -1), (1, 2, -1), (2, 4, -1), (3, 1, 1 << 20), (5, 4, -1)]:
        h.cache.table[b, entry] = value
        h.table[b, entry] = value
    h.check(5 * page, 1, 2, unserved=(0, 1, 2, 3))
    assert dfl2.dfl2_device_error() == 0


def test_short_sequences_may_share_pages():
    h = Held([60, 0, 100], 16, seed=2, spare=10)
    served = h.i32([0])
    dfl2.dfl2_cache_fork(h.cache, h.i32([0]), h.i32([1]), h.i32([60]), served)
    assert served.item() == 1
    h.lens[1] = 60
    h.table, h.refs = h.cache.table.cpu().numpy(), h.cache.refs.cpu().numpy()
    h.check(60, 4, 10)
    assert np.array_equal(h.cache.refs.cpu().numpy(), h.refs)


def test_a_long_row_of_pages():
    """More pages than a block has threads, one of the last missing."""
    h = Held([8 * 3000, 8 * 3000], 8, H=1, D=64, layers=1, seed=4)
    h.cache.table[1, 2998] = -1
    h.table[1, 2998] = -1
    h.check(8 * 3000, 1, 1, unserved=(1,))
