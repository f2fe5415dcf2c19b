"""GPU tests of dfl2_tree_attn where a sequence's last tiles, its missing pages or its lengths
are out of the ordinary, against the 64-bit definition or a run on data without the oddity."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_gpu_tree_attn import Case, _lib  # noqa: F401  (the fixture builds and loads the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,G,D", [(17, 48, 64), (40, 71, 128), (150, 5, 64)])
def test_nan_in_nodes_of_two_last_tiles(T, G, D):
    """Two streams of rows, in the first one (G = 48, 71) a warp that has none, and nodes on
    both sides of a tile's end: NaN and Inf in the values of nodes of the first of the two tiles
    reach the nodes that see them only."""
    B = 100 if T == 40 else 400
    c = Case([48 + b % 10 for b in range(B)], T, 2 * G, 2, D, 16, seed=G)
    clean, clean_lse = c.run()
    table = c.cache.table.cpu()
    hit = [(b % 5) + 1 for b in range(B)]
    for b in range(B):
        pos = c.lens[b] + hit[b]
        assert pos < 64 < c.lens[b] + T
        c.cache.v[0, int(table[b, pos // 16]), :, pos % 16, b % 7::9] = (float("nan"),
                                                                         float("inf"))[b % 2]
    for _ in range(3):
        out, lse = c.run()
        assert torch.equal(lse, clean_lse)
        for b in range(B):
            blind = torch.from_numpy(np.nonzero(~c.seen[b][:, hit[b]])[0]).cuda()
            assert torch.equal(out[b, blind], clean[b, blind]), b
            sees = torch.from_numpy(np.nonzero(c.seen[b][:, hit[b]])[0]).cuda()
            assert not torch.isfinite(out[b, sees][..., b % 7::9]).any(), b
