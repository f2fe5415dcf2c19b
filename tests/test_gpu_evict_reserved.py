"""dfl2_cache_evict with pages reserved past the length: they stay, and serve again later."""
import numpy as np
import pytest

import draft_selection_gb300 as dfl2
from test_gpu_evict import Held
from test_gpu_tree_attn import _lib  # noqa: F401  (the fixture builds and loads the library)

pytestmark = pytest.mark.gpu


def test_pages_past_the_length_stay():
    h = Held([150, 64], 16, seed=12, extra=4, spare=20)
    length, served = h.i32(h.lens), h.i32([0, 0])
    dfl2.dfl2_cache_reserve(h.cache, length, 40, served)  # positions .. 189 and .. 103
    assert served.tolist() == [1, 1]
    h.table, h.refs = h.cache.table.cpu().numpy(), h.cache.refs.cpu().numpy()
    assert (h.table[0, 10:12] >= 0).all() and (h.table[1, 4:7] >= 0).all()
    h.check(64, 3, 20)  # (its model gives back the pages of positions 64 .. 149 alone)
    assert (h.table[0, 4:10] == -1).all() and (h.table[0, 10:12] >= 0).all()
    held = h.table.copy()
    dfl2.dfl2_cache_reserve(h.cache, h.i32(h.lens), 128, served)  # positions 64 .. 191
    assert served.tolist() == [1, 1]
    table = h.cache.table.cpu().numpy()
    assert (table[:, :12] >= 0).all() and np.array_equal(table[held >= 0], held[held >= 0])
    dfl2.dfl2_cache_free(h.cache, h.i32([0, 1]))
    assert int(h.cache.refs.sum()) == 0 and dfl2.dfl2_device_error() == 0
