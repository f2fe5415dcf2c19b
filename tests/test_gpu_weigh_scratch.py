"""dfl2_cache_weigh without a workspace of the caller's: the call takes its own from torch."""
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_gpu_tree_attn import _lib  # noqa: F401  (the fixture builds and loads the library)
from test_gpu_weigh import Weighed

pytestmark = pytest.mark.gpu


def case():
    # (groups that several ranges share, so that the scratch is used)
    return Weighed([900, 40, 2100, 0, 517], 33, 8, 2, 128, 16, path=True, kept=[33, 2, 9, 0, 17], seed=3)


def weigh(c, w, q, lse, **kw):
    dfl2.dfl2_cache_weigh(q, lse, c.cache, c.layer, c.length, w, path=c.path, n_path=c.n_path,
                          first=True, rows=c.rows, scale=c.scale, **kw)


def test_the_same_bits():
    c = case()
    want = c.run(first=True)
    q, lse = c.q.cuda(), c.lse.cuda()
    for _ in range(3):
        torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda")  # what the allocator gives next
        w = c.weight.clone()
        weigh(c, w, q, lse)
        assert torch.equal(w, want)
    assert dfl2.dfl2_device_error() == 0


def test_streams():
    """Two streams at once, named and current, each call with scratch of its own."""
    c = case()
    want = c.run(first=True)
    q, lse = c.q.cuda(), c.lse.cuda()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [[c.weight.clone() for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        weigh(c, ws[0][i], q, lse, stream=streams[0])
        with torch.cuda.stream(streams[1]):
            weigh(c, ws[1][i], q, lse)
    torch.cuda.synchronize()
    assert all(torch.equal(w, want) for many in ws for w in many)


def test_captured():
    """Two graphs, replayed at once on two streams."""
    c = case()
    want = c.run(first=True)
    q, lse = c.q.cuda(), c.lse.cuda()
    ws, graphs = [c.weight.clone(), c.weight.clone()], []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            weigh(c, w, q, lse)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for w in ws:
            w.copy_(c.weight)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ws[0], want) and torch.equal(ws[1], want)
