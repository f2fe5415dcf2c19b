"""The example that runs the serving operators together: trees drafted, verified over
the paged cache and accepted, turn after turn, on forks of one prompt."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import tree_decode as ex  # noqa: E402

import draft_selection_gb300 as dfl2  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,prompt,page", [(5, 45, 16), (1, 3, 8), (3, 64, 32)])
def test_the_text_is_the_targets_own(batch, prompt, page):
    from draft_selection_gb300 import build
    build.build()
    turns = 8
    target, emitted, kept, cache, length = ex.decode(batch, turns, prompt, page=page, seed=prompt)
    assert dfl2.dfl2_device_error() == 0
    total = [prompt - 1 + sum(k[b] for k in kept) for b in range(batch)]
    assert length.tolist() == total
    # the last token of each text has no row in the cache yet
    assert [len(t) for t in emitted] == [n + 1 for n in total]
    # some drafts are kept and some are not, or the turns prove nothing
    flat = [x for k in kept for x in k]
    assert max(flat) > 1 and min(flat) < 7
    # bf16 activations round to 2^-8; three layers and the head stay within 0.1 of the spread
    for text, gap, spread in ex.check(target, emitted):
        assert float(gap[prompt - 1:].max()) <= 0.1 * float(spread)
    # each sequence holds the pages of its length and no other
    used = (cache.table >= 0).sum(1).tolist()
    assert used == [-(-n // page) for n in total]
    refs = torch.zeros_like(cache.refs)
    held = cache.table[cache.table >= 0].long()
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    assert torch.equal(refs, cache.refs)
    dfl2.dfl2_cache_free(cache, torch.arange(batch, dtype=torch.int32, device="cuda"))
    assert int(cache.refs.sum()) == 0 and (cache.table == -1).all()
