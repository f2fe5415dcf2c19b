"""GPU tests of dfl2_cache_weigh against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_gpu_tree_attn import Case, _lib  # noqa: F401  (the fixture builds and loads the library)

pytestmark = pytest.mark.gpu


class Weighed(Case):
    """Case's sequences after a turn: lens committed positions, then the kept queries' own."""

    def __init__(self, lens, T, Hq, Hkv, D, page, dtype=torch.bfloat16, kept=None, path=False, seed=0,
                 scale=None, **kw):
        self.n = [T] * len(lens) if kept is None else list(kept)
        super().__init__(lens, T, Hq, Hkv, D, page, dtype, counts=self.n, mask="chain", seed=seed, **kw)
        rng = np.random.default_rng(seed + 1)
        B, i32 = len(lens), dict(dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5 if scale is None else scale
        self.nodes = [list(range(n)) for n in self.n]
        self.path = self.n_path = None
        if path:
            p = np.full((B, T), -1, np.int32)
            for b, n in enumerate(self.n):
                self.nodes[b] = [int(x) for x in rng.permutation(T)[:n]]
                p[b, :n] = self.nodes[b]
            self.path = torch.tensor(p, device="cuda")
        if path or kept is not None:
            self.n_path = torch.tensor(self.n, **i32)
        self.lse = torch.randn(B, T, Hq)
        for b, n in enumerate(lens):
            k = self.kv[b][0].double()
            for i, node in enumerate(self.nodes[b]):
                for h in range(Hq):
                    s = k[:n + i + 1, h * Hkv // Hq] @ self.q[b, node, h].double() * self.scale
                    self.lse[b, node, h] = torch.logsumexp(s, 0).float()
        self.weight = torch.rand(self.cache.table.shape[0], self.cache.table.shape[1] * page,
                                 device="cuda")
        self.ws = torch.full((dfl2.dfl2_cache_weigh_workspace_size(),), 0xFF, dtype=torch.uint8,
                             device="cuda")

    def run(self, first=False, q=None, error=0):
        w = self.weight.clone()
        dfl2.dfl2_cache_weigh(self.q.cuda() if q is None else q, self.lse.cuda(), self.cache, self.layer,
                              self.length, w, self.ws, path=self.path, n_path=self.n_path, first=first,
                              rows=self.rows, scale=self.scale)
        torch.cuda.synchronize()
        assert dfl2.dfl2_device_error() == error
        return w

    def want(self, first=False, left_out=()):
        """The weights and how far they may be off.  A term 2^(s - l) is off by its exponent's
        error, of the product's D sums and two roundings of s and of l each (2^-24 of their
        sizes), and by 2^x's two units; a position's N terms and its old weight are added in
        float32, each addition off by 2^-24 of the sum."""
        w, bound = self.weight.double().cpu().numpy(), None
        bound = np.zeros_like(w)
        for b, n in enumerate(self.lens):
            row, k = self.table_rows[b], self.kv[b][0].double().numpy()
            got, err, count = np.zeros(n + self.n[b]), np.zeros(n + self.n[b]), 0
            for i, node in enumerate(self.nodes[b]):
                for h in range(self.q.shape[2]):
                    l = float(self.lse[b, node, h])
                    if (b, i, h) in left_out or not np.isfinite(l):
                        continue
                    kk = k[:n + i + 1, h * k.shape[1] // self.q.shape[2]]
                    q = self.q[b, node, h].double().numpy()
                    s = kk @ q * self.scale
                    mag = np.abs(kk) @ np.abs(q) * abs(self.scale)
                    t = np.exp(s - l)
                    got[:n + i + 1] += t
                    e = 2.0**-24 * ((self.D + 8) * mag + 2 * np.abs(s) + 2 * abs(l)) + 2.0**-22
                    err[:n + i + 1] += t * e * 1.01
                    count += 1
            if first:
                w[row, n:n + self.n[b]] = 0
            w[row, :n + self.n[b]] += got
            bound[row, :n + self.n[b]] = err + (count + 4) * 2.0**-24 * got + \
                2.0**-23 * w[row, :n + self.n[b]]
        return w, bound

    def check(self, first=False, **kw):
        w, bound = self.want(first, **kw)
        got = self.run(first).double().cpu().numpy()
        bad = ~(np.abs(got - w) <= bound)
        assert not bad.any(), (np.abs(got - w).max(), bad.mean(), np.argwhere(bad)[:4])


LENS = [0, 1, 127, 128, 129, 517]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 4), (1, 8, 1), (3, 6, 2), (17, 8, 2), (33, 8, 1)])
def test_shapes(T, Hq, Hkv, D, dtype):
    Weighed(LENS, T, Hq, Hkv, D, 16, dtype, seed=T * D + Hq).check()
    Weighed(LENS, T, Hq, Hkv, D, 32, dtype, seed=T, path=True, rows=True,
            kept=[T, 0, 1, max(1, T // 2), T, T // 3]).check(first=True)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_page_sizes(page):
    for D in (64, 256):
        Weighed([0, page - 1, page, 3 * page + 5, 300], 5, 4, 2, D, page, seed=page).check(first=True)


@pytest.mark.parametrize("T,G", [(256, 1), (256, 3), (100, 5), (2, 128), (1, 127), (64, 8)])
def test_many_columns(T, G):
    """Columns in several chunks, which begin inside a token's heads."""
    Weighed([0, 150], T, G, 1, 64, 16, seed=T, kept=[T, T - 1]).check()
    Weighed([200], T, G, 1, 128, 32, seed=G, path=True).check(first=True)


def test_many_and_long_sequences():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 300, 70)]
    Weighed(lens, 3, 4, 2, 64, 16, seed=1, rows=True,
            kept=[int(x) for x in rng.integers(0, 4, 70)], path=True).check()
    Weighed([20011, 3], 2, 4, 2, 64, 64, seed=2).check()


@pytest.mark.parametrize("H,D,B", [(8, 64, 100), (8, 128, 170), (16, 256, 60), (4, 64, 90)])
def test_groups_of_tiles(H, D, B):
    """Enough work for groups of two and four tiles, the last of them with fewer, several heads
    and sequences to a range."""
    rng = np.random.default_rng(H + D)
    lens = [int(x) for x in rng.integers(100, 900, B)]
    Weighed(lens, 3, H, H, D, 32, seed=D, kept=[int(x) for x in rng.integers(1, 4, B)], path=True).check()


def test_layouts():
    """Another layer, pages as [page_size, kv_heads, head_dim], q a part of wider rows."""
    c = Weighed([100, 37], 4, 8, 2, 128, 16, nhd=True, layers=3, layer=1, rows=True, seed=5)
    c.check()
    wide = torch.randn(2, 4, 12, 128, device="cuda").to(torch.bfloat16)
    wide[:, :, :8] = c.q.cuda()
    assert torch.equal(c.run(q=wide[:, :, :8]), c.run())
    one = Weighed([100], 4, 8, 1, 64, 32, nhd=True, seed=6, spare=0)
    one.check()


def test_scales():
    Weighed([300, 5], 7, 4, 2, 128, 16, seed=9, scale=0.01).check()
    Weighed([300, 5], 7, 4, 2, 128, 16, seed=9, scale=-0.3).check()
    Weighed([300, 5], 7, 4, 2, 128, 16, seed=9, amp=5.0).check()


def test_rows_without_a_finite_sum():
    c = Weighed([200, 40], 6, 4, 2, 128, 16, seed=2)
    c.lse[0, 1, 2], c.lse[0, 3, 0], c.lse[1, 5, 3] = -np.inf, np.nan, np.inf
    c.q[0, 3, 0] = np.nan
    c.check()


def test_positions_that_no_query_sees():
    """NaN keys behind a query's own position do not reach it, and those past the kept queries
    nobody; keys of NaN where a query looks make its lse no number, so it adds nothing."""
    c = Weighed([70, 130], 5, 4, 2, 128, 16, seed=3, kept=[3, 2])
    clean = c.run()
    w0 = c.weight.clone()
    for b, n in enumerate(c.lens):
        c.cache.k[0, int(c.cache.table[b, (n + c.n[b] - 1) // 16]), :, (n + c.n[b] - 1) % 16] = float("nan")
        c.lse[b, c.n[b] - 1] = float("nan")
    got = c.run()
    for b, n in enumerate(c.lens):
        last = n + c.n[b] - 1
        assert torch.isfinite(got[b]).all() and got[b, last] == w0[b, last]
        assert (got[b, :last] <= clean[b, :last]).all() and (got[b, :last] > w0[b, :last]).any()


def test_counts_paths_and_pages_out_of_range():
    c = Weighed([100, 50, 60], 4, 4, 2, 128, 16, seed=4, path=True, kept=[4, 4, 2])
    c.n_path.copy_(torch.tensor([9, 4, -3], dtype=torch.int32))
    c.n[2], c.nodes[2] = 0, []
    c.check()
    c.path[0, 2] = 4
    w, bound = c.want(left_out=[(0, 2, h) for h in range(4)])
    got = c.run(error=5).double().cpu().numpy()
    assert (np.abs(got - w) <= bound).all()
    c.path[0, 2] = c.nodes[0][2]
    c.cache.table[1, 1] = -1
    w, bound = c.want()
    w[1, 16:32] = c.weight[1, 16:32].double().cpu().numpy()
    got = c.run(error=5).double().cpu().numpy()
    assert (np.abs(got - w) <= bound)[[0, 2]].all() and np.array_equal(got[1, 16:32], w[1, 16:32])
    assert (np.abs(got - w) <= bound)[1].all()
    for bad in (-1, (1 << 30) + 1, 16 * c.cache.table.shape[1] - 3):
        c.length[0] = bad
        got = c.run(error=5)
        assert torch.equal(got[0], c.weight[0])
    assert dfl2.dfl2_device_error() == 0


def test_same_bits_and_captured():
    c = Weighed([1000, 3, 77, 0, 512], 6, 8, 2, 128, 16, seed=8)
    a = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), a)
    q, lse, w = c.q.cuda(), c.lse.cuda(), c.weight.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dfl2.dfl2_cache_weigh(q, lse, c.cache, 0, c.length, w, c.ws)
    w.copy_(c.weight)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, a)


def test_offsets_past_32_bits():
    H, ps, D = 8, 64, 128
    pages = (1 << 31) // (H * ps * D) + 40
    k = torch.empty(1, pages, H, ps, D, dtype=torch.bfloat16, device="cuda")
    c = Weighed([150, 90], 5, 16, 8, 128, 64, seed=3, spare=0)
    want = c.run()
    n = c.cache.k.shape[1]
    k[:, pages - n:] = c.cache.k
    table = torch.where(c.cache.table >= 0, c.cache.table + (pages - n), c.cache.table)
    c.cache = dfl2.Cache(k, k, table, torch.zeros(pages, dtype=torch.int32, device="cuda"),
                         torch.zeros((pages + 31) // 32, dtype=torch.int32, device="cuda"))
    assert torch.equal(c.run(), want)
