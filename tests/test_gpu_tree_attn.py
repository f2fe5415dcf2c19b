"""GPU tests of dfl2_tree_attn against the 64-bit definition, through the C ABI:
types, head layouts, lengths from nothing to long, page sizes, strides, masks
that hide everything, and Inf/NaN where a node does not look."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _tree_ref import ancestors, attention, attention_bounds, pack_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from draft_selection_gb300 import build
    build.build()
    dfl2.load()


def random_parents(rng, T):
    return [-1] + [int(max(0, i - rng.geometric(0.5))) for i in range(1, T)]


class Case:
    """A cache with its sequences' pages in random order, NaN wherever no position
    of a sequence lies, and the same positions as plain arrays."""

    def __init__(self, lens, T, Hq, Hkv, D, page, dtype=torch.bfloat16, counts=None, mask="tree",
                 seed=0, layers=1, layer=0, nhd=False, rows=False, amp=1.0, spare=2, device="cuda"):
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.lens, self.T, self.dtype, self.D, self.layer = lens, T, dtype, D, layer
        self.counts = list(counts) if counts is not None else [T] * B
        used = [-(-(n + c) // page) for n, c in zip(lens, self.counts)]
        pages = max(1, sum(used)) + spare
        g = torch.Generator().manual_seed(seed)
        self.kv = [(amp * torch.randn(2, n + c, Hkv, D, generator=g)).to(dtype)
                   for n, c in zip(lens, self.counts)]
        shape = (layers, pages, page, Hkv, D) if nhd else (layers, pages, Hkv, page, D)
        kv = torch.full((2,) + shape, float("nan"), dtype=dtype)
        view = kv.transpose(3, 4) if nhd else kv  # [2, layers, pages, Hkv, page, D]
        order = rng.permutation(pages)
        self.table_rows = rng.permutation(B + 2)[:B].astype(np.int32) if rows else np.arange(B)
        table = np.full((B + 2 if rows else B, max(1, max(used)) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(used):
            table[self.table_rows[b], :n] = order[at:at + n]
            at += n
            for c in range(n):
                part = self.kv[b][:, c * page:(c + 1) * page]
                view[:, layer, int(table[self.table_rows[b], c]), :, :part.shape[1]] = \
                    part.transpose(1, 2)
        dev = kv.to(device)
        view = dev.transpose(3, 4) if nhd else dev
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=device)
        bits = pack_bits(np.isin(np.arange(pages), order[at:])[None])[0]
        self.refs = np.isin(np.arange(pages), order[:at]).astype(np.int32)
        self.cache = dfl2.Cache(view[0], view[1], i32(table), i32(self.refs), i32(bits))
        self.rows = i32(self.table_rows) if rows else None
        self.length = i32(lens)
        self.count = i32(self.counts) if counts is not None else None
        self.q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
        self.seen = []
        if mask == "chain":
            self.mask = None
            self.seen = [np.tril(np.ones((T, T), bool))] * B
        else:
            for _ in range(B):
                if mask == "tree":
                    self.seen.append(ancestors(random_parents(rng, T)))
                elif mask == "random":
                    self.seen.append(rng.random((T, T)) < 0.5)
                else:  # "none"
                    self.seen.append(np.zeros((T, T), bool))
            self.mask = i32(pack_bits(np.stack(self.seen)))

    def run(self, q=None, out=None, lse=True, scale=None, ws=None, stream=None):
        q = self.q.cuda() if q is None else q
        B, T, Hq, D = q.shape
        out = torch.full((B, T, Hq, D), float("nan"), dtype=self.dtype, device="cuda") if out is None else out
        lse = torch.full((B, T, Hq), float("nan"), device="cuda") if lse else None
        if ws is None:
            nb = dfl2.dfl2_tree_attn_workspace_size(B, T, Hq, self.cache._s.kv_heads, D, self.dtype)
            ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN: must not matter
        dfl2.dfl2_tree_attn(q, self.cache, self.layer, self.length, self.mask, out, ws,
                            rows=self.rows, count=self.count, lse=lse, scale=scale, stream=stream)
        torch.cuda.synchronize()
        assert dfl2.dfl2_device_error() == 0
        return out, lse

    def check(self, out, lse, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        o, z = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            seen = np.ones((self.T, n + c), bool)
            seen[:, n:] = self.seen[b][:, :c]
            seen[c:] = False
            kv = self.kv[b].double().numpy()
            ref = attention(self.q[b].double().numpy(), kv[0], kv[1], seen, scale)
            ob, lb = attention_bounds(ref, self.dtype, self.D, n + c)
            fin = np.isfinite(ref[0])
            assert np.array_equal(fin, np.isfinite(o[b])), f"sequence {b}: finite elsewhere"
            bad = np.abs(o[b] - ref[0])[fin] > ob[fin]
            assert not bad.any(), (b, np.abs(o[b] - ref[0])[fin].max(), bad.mean())
            if z is not None:
                dead = ~np.isfinite(ref[1])
                assert np.array_equal(z[b][dead], ref[1][dead], equal_nan=True)
                far = np.abs(z[b][~dead] - ref[1][~dead]) > lb[~dead]
                assert not far.any(), (b, np.abs(z[b][~dead] - ref[1][~dead]).max())


def go(*a, **k):
    c = Case(*a, **k)
    out, lse = c.run()
    c.check(out, lse)
    return c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 4), (1, 8, 1), (3, 6, 2), (17, 8, 2), (33, 4, 1),
                                      (40, 8, 1)])
def test_shapes(T, Hq, Hkv, D, dtype):
    go([0, 1, 63, 64, 65, 200, 517], T, Hq, Hkv, D, 16, dtype, seed=T * D + Hq)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_page_sizes(page):
    go([0, page - 1, page, page + 1, 3 * page - 5, 777], 9, 8, 2, 128, page, seed=page)
    go([5, 300], 70, 8, 2, 128, page, seed=page + 1, mask="random")


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 100, 255, 256])
def test_tree_sizes(T):
    go([0, 130], T, 2, 1, 64, 16, seed=T)
    go([77], T, 2, 2, 128, 32, seed=T, mask="chain")
    go([3, 129], T, 4, 2, 128, 16, seed=T, mask="random")


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16])
def test_group_sizes(G):
    go([50, 1000, 0], 13, 2 * G, 2, 128, 16, seed=G)
    go([50, 1000, 0], 13, G, 1, 64, 64, seed=G, dtype=torch.float16)


@pytest.mark.parametrize("T,G", [(1, 1), (16, 4), (33, 4), (64, 8)])
def test_ragged_batch(T, G):
    """Sequences of very different lengths, so that the ranges of work cut them anywhere."""
    rng = np.random.default_rng(T)
    lens = [int(x) for x in rng.integers(0, 700, 21)] + [2500, 0, 1]
    counts = [int(x) for x in rng.integers(0, T + 1, len(lens))]
    counts[3] = T
    go(lens, T, 2 * G, 2, 128, 16, counts=counts, seed=T, rows=True)


@pytest.mark.parametrize("T,G", [(100, 5), (61, 7), (256, 3), (3, 128), (2, 100), (129, 1), (9, 48)])
def test_row_tiles(T, G):
    """Rows in several tiles and streams, whole nodes in each; some of them past the count."""
    go([200, 0, 70], T, G, 1, 64, 16, counts=[T, T, max(1, T // 3)], seed=T)
    go([333], T, 2 * G, 2, 128, 32, seed=G, mask="random")


def test_many_sequences():
    """More sequences than a warp looks up at once, most of them without work."""
    lens = [0] * 40 + [5, 300, 64] + [0] * 30 + [17] + [0] * 26
    counts = [0] * 40 + [3, 2, 1] + [0] * 30 + [3] + [0] * 26
    go(lens, 3, 4, 2, 128, 16, counts=counts, rows=True)
    rng = np.random.default_rng(8)
    go([int(x) for x in rng.integers(0, 90, 133)], 2, 4, 2, 64, 8, seed=8)


def test_counts_past_their_ends():
    c = Case([40, 9], 4, 4, 2, 128, 16, counts=[4, 0], seed=2)
    want, wl = c.run()
    c.count.copy_(torch.tensor([9, -3], dtype=torch.int32))
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_one_long_sequence():
    go([20011], 17, 4, 1, 128, 16, seed=1)
    go([20011], 1, 4, 2, 64, 64, seed=2, dtype=torch.float16)
    go([9001], 64, 8, 2, 128, 64, seed=3)


@pytest.mark.parametrize("T", [4, 40])
def test_layouts(T):
    """Pages as [page_size, kv_heads, head_dim], another layer, q and out parts of wider rows."""
    c = Case([100, 37], T, 8, 2, 128, 16, nhd=True, layers=3, layer=1, rows=True, seed=5)
    wide = torch.randn(2, T, 12, 128, device="cuda").to(torch.bfloat16)
    wide[:, :, :8] = c.q.cuda()
    hold = torch.full((2, 8, T, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = c.run(q=wide[:, :, :8], out=hold.transpose(1, 2))
    c.check(out, lse)
    a, _ = c.run(lse=False)
    assert torch.equal(a, out)
    part = torch.full((2, T, 8, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    c.run(out=part[..., 8:])  # rows that begin on 16 bytes and not on 32
    assert torch.equal(part[..., 8:], out) and torch.isnan(part[..., :8]).all()
    b, _ = c.run(q=c.q.cuda().transpose(1, 2).contiguous().transpose(1, 2))  # heads outside nodes
    assert torch.equal(b, out)
    one = Case([100], T, 8, 1, 64, 32, nhd=True, seed=6, spare=0)  # dimensions of one entry
    out, lse = one.run()
    one.check(out, lse)


@pytest.mark.parametrize("T", [5, 48])
def test_rows_that_see_nothing(T):
    c = Case([0, 0, 40], T, 4, 2, 128, 16, mask="none", counts=[T, 0, T], seed=2)
    out, lse = c.run()
    c.check(out, lse)
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,G", [(6, 1), (24, 4), (64, 4)])
def test_unseen_nodes_hold_anything(T, G, dtype):
    """NaN and Inf in the keys and values of nodes: only the nodes that see them have them."""
    c = Case([90, 0, 31], T, 2 * G, 2, 128, 16, dtype, seed=T, mask="tree")
    clean, clean_lse = c.run()
    hit = [2, 5, T - 1]
    for b in range(3):
        n = c.lens[b]
        for j, x in zip(hit, (float("nan"), float("inf"), float("-inf"))):
            page = int(c.cache.table[b, (n + j) // 16])
            c.cache.v[0, page, :, (n + j) % 16, 3::5] = x
            if j == 2:
                c.cache.k[0, page, :, (n + j) % 16] = x
    out, lse = c.run()
    for b in range(3):
        sees = c.seen[b][:, hit]
        blind = ~sees.any(1)
        at = torch.from_numpy(np.nonzero(blind)[0]).cuda()
        assert torch.equal(out[b, at], clean[b, at]) and torch.equal(lse[b, at], clean_lse[b, at])
        only5 = sees[:, 1] & ~sees[:, 0] & ~sees[:, 2]
        for i in np.nonzero(only5)[0]:
            assert (out[b, i, :, 3::5] == float("inf")).all()
            assert torch.isfinite(out[b, i, :, 4::5]).all()
        for i in np.nonzero(sees[:, 0])[0]:
            assert torch.isnan(out[b, i]).all() and torch.isnan(lse[b, i]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_inf_in_many_short_sequences(D):
    """Every sequence is one tile with an Inf of its own: two streams of rows, one of which
    may be several sequences ahead of the other."""
    B, T = 3000, 20
    c = Case([b % 44 for b in range(B)], T, 8, 1, D, 64, seed=D)
    table = c.cache.table.cpu()
    for b in range(B):
        page = int(table[b, 0])
        c.cache.v[0, page, 0, c.lens[b] + b % T, b % D] = float("inf")
    out = c.run()[0].cpu()
    for b in range(B):
        want = torch.zeros(T, 8, D, dtype=torch.bool)
        want[torch.from_numpy(np.nonzero(c.seen[b][:, b % T])[0]), :, b % D] = True
        assert torch.equal(out[b] == float("inf"), want), b
        assert torch.isfinite(out[b][~want]).all(), b


def test_large_scores_and_scale():
    c = Case([300, 5], 7, 4, 2, 128, 16, amp=6.0, seed=9)
    out, lse = c.run()
    c.check(out, lse)
    out, lse = c.run(scale=0.01)
    c.check(out, lse, scale=0.01)
    out, lse = c.run(scale=-0.2)
    c.check(out, lse, scale=-0.2)


def test_sharp_rows_after_flat_ones():
    """The maximum far behind: what came before is scaled down to nothing."""
    c = Case([640, 64], 3, 2, 1, 128, 16, seed=4)
    for b, n in enumerate(c.lens):
        j = n - 2
        page = int(c.cache.table[b, j // 16])
        k = (c.q[b, 0, 0] * 30).to(torch.bfloat16)
        c.kv[b][0, j, 0] = k
        c.cache.k[0, page, 0, j % 16] = k.cuda()
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("T", [1, 20, 64])
def test_same_bits_again_and_in_a_graph_on_another_stream(T):
    c = Case([1000, 3, 77, 0, 512], T, 8, 2, 128, 16, seed=T)
    a, al = c.run()
    b, bl = c.run()
    assert torch.equal(a, b) and torch.equal(al, bl)
    q = c.q.cuda()
    out, lse = torch.empty_like(a), torch.empty_like(al)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(*q.shape[:3], 2, 128, c.dtype))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dfl2.dfl2_tree_attn(q, c.cache, 0, c.length, c.mask, out, ws, lse=lse)
    for n in ([1000, 3, 77, 0, 512], [990, 2, 70, 0, 500]):  # the lengths are read when it runs
        c.length.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, wl = c.run()
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_offsets_past_32_bits():
    """A cache whose last pages lie more than 2^32 bytes and 2^31 elements in."""
    H, ps, D = 8, 64, 128
    pages = (1 << 31) // (H * ps * D) + 40
    k = torch.empty(1, pages, H, ps, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = Case([150, 90], 5, 16, 8, 128, 64, seed=3, spare=0)
    n = small.cache.k.shape[1]
    k[:, pages - n:] = small.cache.k
    v[:, pages - n:] = small.cache.v
    table = torch.where(small.cache.table >= 0, small.cache.table + (pages - n), small.cache.table)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    bits = torch.zeros((pages + 31) // 32, dtype=torch.int32, device="cuda")
    small.cache = dfl2.Cache(k, v, table, refs, bits)
    out, lse = small.run()
    small.check(out, lse)


def test_page_numbers_out_of_range_are_recorded():
    c = Case([100], 3, 4, 2, 128, 16, seed=1)
    c.cache.table[0, 2] = 1 << 20
    q = c.q.cuda()
    out = torch.empty_like(q)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(1, 3, 4, 2, 128, c.dtype))
    dfl2.dfl2_tree_attn(q, c.cache, 0, c.length, c.mask, out, ws)
    assert dfl2.dfl2_device_error() == 5
    rows = torch.tensor([7], dtype=torch.int32, device="cuda")
    dfl2.dfl2_tree_attn(q, c.cache, 0, c.length, c.mask, out, ws, rows=rows)
    assert dfl2.dfl2_device_error() == 5
    assert (out == 0).all()
