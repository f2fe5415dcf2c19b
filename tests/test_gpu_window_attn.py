"""GPU tests of dfl2_window_attn against the 64-bit definition: windows and sinks that end
inside tiles and pages, trees longer than the window, rows that see nothing, and anything at
all in the positions that no node, or not every node, sees."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _tree_ref import attention, attention_bounds
from test_gpu_tree_attn import Case, _lib  # noqa: F401  (the fixture builds and loads the library)

pytestmark = pytest.mark.gpu


class Windowed(Case):
    def __init__(self, lens, T, Hq, Hkv, D, page, dtype=torch.bfloat16, sinks=4, window=64,
                 depth=True, mask="tree", **kw):
        super().__init__(lens, T, Hq, Hkv, D, page, dtype, mask=mask, **kw)
        self.sinks, self.window = sinks, window
        self.deep = [np.arange(T) if mask == "chain" else s.sum(1) - s.diagonal() for s in self.seen]
        self.depth = None
        if mask != "chain" or depth == "given":
            self.depth = torch.tensor(np.stack(self.deep), dtype=torch.int32, device="cuda")

    def sees(self, b):
        n, c = self.lens[b], self.counts[b]
        seen = np.ones((self.T, n + c), bool)
        seen[:, n:] = self.seen[b][:, :c]
        seen[c:] = False
        at = np.concatenate([np.arange(n), n + self.deep[b][:c]])
        return seen & ((at < self.sinks) | (at > (n + self.deep[b] - self.window)[:, None]))

    def run(self, q=None, out=None, ws=None):
        q = self.q.cuda() if q is None else q
        B, T, Hq, D = q.shape
        out = torch.full((B, T, Hq, D), float("nan"), dtype=self.dtype, device="cuda") if out is None else out
        lse = torch.full((B, T, Hq), float("nan"), device="cuda")
        if ws is None:
            nb = dfl2.dfl2_tree_attn_workspace_size(B, T, Hq, self.cache._s.kv_heads, D, self.dtype)
            ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
        dfl2.dfl2_window_attn(q, self.cache, self.layer, self.length, self.mask, self.depth,
                              self.sinks, self.window, out, ws, rows=self.rows, count=self.count,
                              lse=lse)
        torch.cuda.synchronize()
        assert dfl2.dfl2_device_error() == 0
        return out, lse

    def check(self, out, lse):
        o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            kv = self.kv[b].double().numpy()
            ref = attention(self.q[b].double().numpy(), kv[0], kv[1], self.sees(b), self.D ** -0.5)
            ob, lb = attention_bounds(ref, self.dtype, self.D, n + c)
            bad = ~(np.abs(o[b] - ref[0]) <= ob)
            assert not bad.any(), (b, n, np.abs(o[b] - ref[0]).max(), bad.mean())
            dead = ~np.isfinite(ref[1])
            assert np.array_equal(z[b][dead], ref[1][dead])
            far = ~(np.abs(z[b][~dead] - ref[1][~dead]) <= lb[~dead])
            assert not far.any(), (b, n, np.abs(z[b][~dead] - ref[1][~dead]).max())

    def put(self, b, pos, k=None, v=None):
        """Other keys or values at a position, in the cache only."""
        ps = self.cache.k.shape[3]
        page = int(self.cache.table[self.table_rows[b], pos // ps])
        if k is not None:
            self.cache.k[self.layer, page, :, pos % ps] = k
        if v is not None:
            self.cache.v[self.layer, page, :, pos % ps] = v


def go(*a, **k):
    c = Windowed(*a, **k)
    c.check(*c.run())
    return c


LENS = [0, 1, 63, 64, 65, 130, 517, 1000]


@pytest.mark.parametrize("sinks,window", [(0, 1), (0, 64), (4, 100), (64, 64), (65, 63), (130, 17),
                                          (0, 1 << 30), (1 << 30, 1), (1, 517)])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 2, 128), (33, 4, 1, 64), (40, 8, 1, 128)])
def test_windows(sinks, window, T, Hq, Hkv, D):
    go(LENS, T, Hq, Hkv, D, 16, sinks=sinks, window=window, seed=T + window % 97)
    go(LENS, T, Hq, Hkv, D, 64, torch.float16, sinks=sinks, window=window, mask="chain", seed=T)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 4), (5, 3), (64, 4), (256, 2), (3, 128)])
def test_shapes(T, G, D):
    go([300, 0, 77, 640], T, G, 1, D, 32, sinks=7, window=90, seed=T)
    go([300, 0, 77, 640], T, 2 * G, 2, D, 8, torch.float16, sinks=7, window=90, seed=G,
       counts=[T, max(0, T - 1), max(1, T // 3), 0])


@pytest.mark.parametrize("window", [1, 2, 7, 31, 64, 100])
def test_windows_shorter_than_the_tree(window):
    for mask, depth in (("tree", True), ("chain", True), ("chain", "given"), ("random", True)):
        go([200, 0, 5, 60], 100, 4, 2, 128, 16, sinks=3, window=window, mask=mask, depth=depth,
           seed=window)
    go([10, 40, 70], 70, 4, 2, 64, 16, sinks=60, window=window, seed=window)  # nodes among the sinks


def test_many_sequences_and_long_ones():
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 900, 75)]
    go(lens, 17, 8, 2, 128, 16, sinks=5, window=200, rows=True, seed=1,
       counts=[int(x) for x in rng.integers(0, 18, 75)])
    go([20011, 7], 17, 4, 1, 128, 64, sinks=100, window=5000, seed=2)
    go([20011], 1, 4, 2, 64, 16, sinks=4, window=300, seed=3)


@pytest.mark.parametrize("T", [1, 9, 40])
def test_a_window_past_everything_is_the_plain_attention(T):
    c = Windowed([1000, 3, 77, 0, 512], T, 8, 2, 128, 16, sinks=0, window=5000, seed=T)
    want = Case.run(c)
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [3, 50])
def test_rows_that_see_nothing(T):
    """No mask bit, no sinks, and a window that ends before the committed positions do."""
    c = Windowed([0, 200, 40], T, 4, 2, 128, 16, mask="none", sinks=0, window=2, seed=T)
    c.depth.fill_(T - 1)
    c.deep = [np.full(T, T - 1)] * 3
    out, lse = c.run()
    c.check(out, lse)
    assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("page", [8, 16, 64, 128])
@pytest.mark.parametrize("T,mask", [(1, "chain"), (12, "tree"), (40, "chain")])
def test_unseen_positions_hold_anything(T, mask, page):
    """NaN and Inf in every position that no node sees; pages that lie wholly among them gone,
    without a record of it."""
    c = Windowed([700, 350, 90], T, 8, 2, 128, page, sinks=20, window=130, mask=mask, seed=page)
    want = c.run()
    for b, n in enumerate(c.lens):
        dark = np.flatnonzero(~c.sees(b).any(0))
        for pos in dark:
            c.put(b, int(pos), float("nan"), float("nan") if pos % 2 else float("inf"))
        gone = [x for x in range(n // page) if set(range(x * page, x * page + page)) <= set(dark)]
        for x in gone:
            c.cache.table[b, x] = -1
        assert gone or n < 200 or page == 128
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,G,D", [(6, 1, 128), (33, 4, 64), (64, 4, 128), (20, 4, 256)])
def test_values_that_some_nodes_see(T, G, D):
    """NaN and Inf in the values of positions that leave the window within the block: they reach
    the nodes that see them only."""
    c = Windowed([300, 161, 64], T, 2 * G, 2, D, 16, sinks=5, window=100, mask="chain", seed=T)
    clean = c.run()
    hit = {}
    for b, n in enumerate(c.lens):
        hit[b] = [n - 100 + 2, n - 100 + T // 2, n + 1]
        hit[b] = [p for p in hit[b] if p >= 5]
        for p, x in zip(hit[b], (float("inf"), float("nan"), float("-inf"))):
            y = c.kv[b][1, p].clone()
            y[:, 3::7] = x
            c.put(b, p, v=y.cuda())
    out, lse = c.run()
    assert torch.equal(lse, clean[1])
    for b in hit:
        sees = c.sees(b)[:, hit[b]].any(1)
        assert sees.any()
        at = torch.from_numpy(np.flatnonzero(~sees)).cuda()
        assert torch.equal(out[b, at], clean[0][b, at]), b
        on = torch.from_numpy(np.flatnonzero(sees)).cuda()
        assert not torch.isfinite(out[b, on][..., 3::7]).any(), b
        assert torch.isfinite(out[b, on][..., 4::7]).all(), b


def test_values_in_the_sinks():
    """An Inf among the sinks of a tile that is half sinks is everybody's."""
    c = Windowed([400], 9, 4, 2, 64, 16, sinks=70, window=50, seed=1)
    y = c.kv[0][1, 66].clone()
    y[:, 11] = float("inf")
    c.put(0, 66, v=y.cuda())
    c.put(0, 71, float("nan"), float("nan"))
    out, _ = c.run()
    assert (out[..., 11] == float("inf")).all()
    assert torch.isfinite(out[..., :11]).all() and torch.isfinite(out[..., 12:]).all()


def test_missing_pages_that_are_seen_are_recorded_and_left_out():
    c = Windowed([300], 5, 4, 2, 128, 16, sinks=4, window=100, seed=1)
    q = c.q.cuda()
    out = torch.empty_like(q)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(1, 5, 4, 2, 128, c.dtype))
    c.cache.table[0, 290 // 16] = -1
    dfl2.dfl2_window_attn(q, c.cache, 0, c.length, c.mask, c.depth, 4, 100, out, ws)
    assert dfl2.dfl2_device_error() == 5
    sees = c.sees(0)
    sees[:, 288:304] = False
    kv = c.kv[0].double().numpy()
    ref = attention(c.q[0].double().numpy(), kv[0], kv[1], sees, 128 ** -0.5)
    ob, _ = attention_bounds(ref, c.dtype, 128, 305)
    assert (np.abs(out[0].double().cpu().numpy() - ref[0]) <= ob).all()


def test_depths_out_of_range_are_taken_to_the_nearer_end():
    c = Windowed([300], 6, 4, 2, 128, 16, sinks=4, window=40, mask="chain", depth="given", seed=1)
    c.depth[0, 0] = -1000
    c.depth[0, 5] = 1 << 30
    c.check(*c.run())


def test_lengths_out_of_range_are_recorded():
    c = Windowed([300, 20], 6, 4, 2, 128, 16, sinks=4, window=40, seed=1)
    want, _ = c.run()
    q = c.q.cuda()
    out = torch.empty_like(q)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(2, 6, 4, 2, 128, c.dtype))
    for bad in (-1, (1 << 30) + 1, -(1 << 31)):
        n = torch.tensor([bad, 20], dtype=torch.int32, device="cuda")
        dfl2.dfl2_window_attn(q, c.cache, 0, n, c.mask, c.depth, 4, 40, out, ws)
        assert dfl2.dfl2_device_error() == 5
        assert (out[0] == 0).all() and torch.equal(out[1], want[1])


@pytest.mark.parametrize("T", [1, 20, 64])
def test_same_bits_again_and_in_a_graph_on_another_stream(T):
    c = Windowed([1000, 3, 77, 0, 512], T, 8, 2, 128, 16, sinks=4, window=150, seed=T)
    a, al = c.run()
    q = c.q.cuda()
    out, lse = torch.empty_like(a), torch.empty_like(al)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(*q.shape[:3], 2, 128, c.dtype))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dfl2.dfl2_window_attn(q, c.cache, 0, c.length, c.mask, c.depth, 4, 150, out, ws, lse=lse)
    for n in ([1000, 3, 77, 0, 512], [990, 2, 70, 0, 500]):
        c.length.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, wl = c.run()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("T", [4, 40])
def test_layouts(T):
    """Pages as [page_size, kv_heads, head_dim], another layer, q and out parts of wider rows."""
    c = Windowed([100, 337], T, 8, 2, 128, 16, nhd=True, layers=3, layer=1, rows=True, sinks=5,
                 window=70, seed=5)
    wide = torch.randn(2, T, 12, 128, device="cuda").to(torch.bfloat16)
    wide[:, :, :8] = c.q.cuda()
    hold = torch.full((2, 8, T, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = c.run(q=wide[:, :, :8], out=hold.transpose(1, 2))
    c.check(out, lse)
    part = torch.full((2, T, 8, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    c.run(out=part[..., 8:])  # rows that begin on 16 bytes and not on 32
    assert torch.equal(part[..., 8:], out) and torch.isnan(part[..., :8]).all()
