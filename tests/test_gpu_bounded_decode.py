"""The example that decodes sampled texts in a cache of bounded size."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import bounded_decode as ex  # noqa: E402

import draft_selection_gb300 as dfl2  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,keep,page", [(3, 64, 16), (1, 50, 8)])
def test_the_cache_stays_within_its_budget(batch, keep, page):
    from draft_selection_gb300 import build
    build.build()
    emitted, length, cache, gone = ex.decode(batch, 40, keep, page=page, recent=20, seed=batch)
    assert dfl2.dfl2_device_error() == 0
    total = [len(t) - 1 for t in emitted]
    lost = [sum(g[b] for g in gone) for b in range(batch)]
    assert [n + g for n, g in zip(length.tolist(), lost)] == total
    assert length.tolist() == [min(keep, n) for n in total] and max(lost) > 0
    assert all(0 <= x < 2048 for t in emitted for x in t)
    used = (cache.table >= 0).sum(1).tolist()
    assert used == [-(-n // page) for n in length.tolist()]
    dfl2.dfl2_cache_free(cache, torch.arange(batch, dtype=torch.int32, device="cuda"))
    assert int(cache.refs.sum()) == 0
