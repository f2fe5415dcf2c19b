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


def slow_nodes():
    """NaN in the values of one node of 256 in every sequence, several heads to a CTA."""
    c = Case([100, 300, 37, 64] * 16, 256, 8, 8, 128, 16, seed=3, mask="chain")
    table = c.cache.table.cpu()
    for b, n in enumerate(c.lens):
        c.cache.v[0, int(table[b, (n + 5) // 16]), :, (n + 5) % 16] = float("nan")
    return c


def test_a_recorded_index_ends_no_wait():
    """An index out of range in the error word is an ordinary state: what is merely slow then
    still ends whole."""
    c = slow_nodes()
    want, want_lse = c.run()
    bad = torch.tensor([-1], dtype=torch.int32, device="cuda")
    dfl2.dfl2_cache_free(c.cache, bad)
    assert dfl2.dfl2_device_error(clear=False) == 5
    q, out, lse = c.q.cuda(), torch.zeros_like(want), torch.zeros_like(want_lse)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(*q.shape[:3], 8, 128, c.dtype))
    dfl2.dfl2_tree_attn(q, c.cache, 0, c.length, c.mask, out, ws, lse=lse)
    assert dfl2.dfl2_device_error() == 5
    assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(lse, want_lse)
    assert torch.isnan(out[:, 5:]).all() and torch.isfinite(out[:, :5]).all()


def test_nan_in_a_node_costs_no_more_than_its_nodes():
    """Looking for the values that are no numbers takes time by the nodes that are seen, not by
    nodes times channels: the limit is a tenth of what the latter took, 50 ms."""
    c = slow_nodes()
    q = c.q.cuda()
    out = torch.empty_like(q)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(*q.shape[:3], 8, 128, c.dtype))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        begin.record()
        dfl2.dfl2_tree_attn(q, c.cache, 0, c.length, c.mask, out, ws)
        end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) < 5.0
    assert dfl2.dfl2_device_error() == 0
