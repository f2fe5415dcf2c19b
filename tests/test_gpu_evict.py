"""GPU tests of dfl2_cache_evict against its definition, position by position: everything it
moves is compared bit by bit, and everything else has to stay as it was."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _tree_ref import pack_bits
from test_gpu_tree_attn import _lib  # noqa: F401  (the fixture builds and loads the library)

pytestmark = pytest.mark.gpu


def stays(w, n, keep, sinks, recent):
    """The positions of a sequence of n that stay."""
    if n <= keep:
        return list(range(n))
    w = np.where(np.isnan(w), -np.inf, w)
    mid = sorted(range(sinks, n - recent), key=lambda j: (-w[j], j))[:keep - sinks - recent]
    return sorted([*range(sinks), *mid, *range(n - recent, n)])


class Held:
    """A cache of sequences in pages of random order, and what it should hold."""

    def __init__(self, lens, page, H=2, D=64, dtype=torch.bfloat16, layers=2, nhd=False, rows=False,
                 seed=0, extra=0, spare=3):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.lens = rng, page, list(lens)
        B = len(lens)
        used = [-(-n // page) for n in lens]
        pages = sum(used) + spare
        cols = max(1, max(used)) + extra
        order = rng.permutation(pages)
        self.rows = rng.permutation(B + 2)[:B] if rows else np.arange(B)
        self.table = np.full((B + 2 if rows else B, cols), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        at = 0
        for r, n in zip(self.rows, used):
            self.table[r, :n] = order[at:at + n]
            self.refs[order[at:at + n]] = 1
            at += n
        shape = (layers, pages, page, H, D) if nhd else (layers, pages, H, page, D)
        g = torch.Generator(device="cuda").manual_seed(seed)
        kv = torch.randn((2,) + shape, generator=g, device="cuda").to(dtype)
        view = kv.transpose(3, 4) if nhd else kv
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        self.cache = dfl2.Cache(view[0], view[1], i32(self.table), i32(self.refs),
                                i32(pack_bits((self.refs == 0)[None])[0]))
        self.weight = torch.rand(self.table.shape[0], cols * page, generator=g, device="cuda")
        self.i32 = i32

    def call(self, keep, sinks, recent, lens=None, alias=False, ws=None):
        B = len(self.lens)
        length = self.i32(self.lens if lens is None else lens)
        kept = torch.full((B, keep), -9, dtype=torch.int32, device="cuda")
        new = length if alias else torch.full((B,), -9, dtype=torch.int32, device="cuda")
        served = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        if ws is None:
            ws = torch.full((dfl2.dfl2_cache_evict_workspace_size(B, keep),), 0xFF, dtype=torch.uint8,
                            device="cuda")
        dfl2.dfl2_cache_evict(self.cache, length, keep, sinks, recent, self.weight, kept, new, served,
                              ws, rows=self.i32(self.rows))
        torch.cuda.synchronize()
        return kept.cpu().numpy(), new.cpu().numpy(), served.cpu().numpy()

    def check(self, keep, sinks, recent, unserved=(), **kw):
        k0, v0, w0 = self.cache.k.clone(), self.cache.v.clone(), self.weight.clone()
        wn = w0.cpu().numpy()
        kept, new, served = self.call(keep, sinks, recent, **kw)
        ps = self.page
        table, refs = self.table.copy(), self.refs.copy()
        for b, (r, n) in enumerate(zip(self.rows, self.lens)):
            assert served[b] == (b not in unserved), b
            if b in unserved:
                assert (kept[b] == -1).all() and new[b] == n
                continue
            want = stays(wn[r], n, keep, sinks, recent)
            assert kept[b].tolist() == want + [-1] * (keep - len(want)), b
            assert new[b] == min(n, keep)
            if n <= keep:
                continue
            a = np.array([(table[r, p // ps], p % ps) for p in want]).reshape(-1, 2)
            z = np.array([(table[r, i // ps], i % ps) for i in range(keep)]).reshape(-1, 2)
            moved = np.flatnonzero(np.array(want) != np.arange(keep))
            a, z = torch.from_numpy(a[moved]).cuda().long(), torch.from_numpy(z[moved]).cuda().long()
            for x in (k0, v0):
                y = x.permute(1, 3, 0, 2, 4)
                y[z[:, 0], z[:, 1]] = y[a[:, 0], a[:, 1]]
            w0[int(r), :keep] = w0[int(r), torch.tensor(want, device="cuda")]
            for x in range(-(-keep // ps), -(-n // ps)):
                refs[table[r, x]] -= 1
                table[r, x] = -1
        bits = lambda t: t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)  # noqa: E731
        assert torch.equal(bits(self.cache.k), bits(k0)) and torch.equal(bits(self.cache.v), bits(v0))
        assert torch.equal(bits(self.weight), bits(w0))
        assert np.array_equal(self.cache.table.cpu().numpy(), table)
        assert np.array_equal(self.cache.refs.cpu().numpy(), refs)
        assert np.array_equal(self.cache.free_bits.cpu().numpy(), pack_bits((refs == 0)[None])[0])
        self.table, self.refs, self.lens = table, refs, new.tolist()


LENS = [0, 1, 19, 20, 21, 64, 200, 333]


@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("keep,sinks,recent", [(20, 4, 6), (20, 0, 0), (20, 20, 0), (20, 0, 20),
                                               (1, 0, 0), (1, 1, 0), (199, 3, 100), (64, 0, 63)])
def test_sizes(keep, sinks, recent, page):
    h = Held(LENS, page, seed=keep + page, rows=True)
    h.check(keep, sinks, recent)
    assert dfl2.dfl2_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,D,layers", [(1, 8, 1), (3, 24, 2), (8, 128, 5), (1, 256, 1)])
def test_types_and_layouts(H, D, layers, dtype):
    for nhd in (False, True):
        Held(LENS, 16, H, D, dtype, layers, nhd=nhd, seed=D, extra=2).check(20, 4, 6)


@pytest.mark.parametrize("kind", ["few", "same", "odd"])
def test_equal_weights_and_no_numbers(kind):
    """Ties stay from the lowest position on; NaN counts as -inf; zeros of both signs are equal."""
    h = Held([300, 40, 61, 1000], 16, seed=3)
    if kind == "few":
        h.weight.mul_(4).floor_()
    elif kind == "same":
        h.weight.fill_(0.25)
    else:
        x = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, -3.0],
                         device="cuda")
        h.weight.copy_(x[torch.randint(0, 8, h.weight.shape, device="cuda")])
    h.check(33, 2, 9)


def test_long_sequences():
    """More positions than a block holds at once, ties across its chunks; few columns, so that
    many warps share the rows."""
    h = Held([20011, 8193, 8192 + 5, 40000], 64, H=1, D=64, layers=1, seed=5)
    h.weight.mul_(50).floor_()
    h.check(6000, 5, 500)
    h = Held([30000], 16, H=2, D=64, layers=1, seed=6)
    h.weight[:, :20000] = 2.0  # the first position that goes lies in the third chunk
    h.check(25000, 0, 10)


def test_again_and_again():
    """Positions come in behind those that stayed, and go again."""
    h = Held([150, 90, 30], 16, seed=7, extra=4, spare=40)
    for step in range(4):
        h.check(64, 3, 20)
        count = h.i32([40 + step, 17, 60])
        served = h.i32([0, 0, 0])
        length = h.i32(h.lens)
        dfl2.dfl2_cache_reserve(h.cache, length, count, served, rows=h.i32(h.rows))
        assert served.tolist() == [1, 1, 1]
        h.lens = (length + count).tolist()
        h.table, h.refs = h.cache.table.cpu().numpy(), h.cache.refs.cpu().numpy()
        h.weight.uniform_()


def test_shared_pages():
    """A sequence that would write pages it shares stays as it is; one that only gives shared
    pages back does not."""
    h = Held([100, 0, 100], 16, seed=8, spare=10)
    i = h.i32
    served = i([0])
    dfl2.dfl2_cache_fork(h.cache, i([0]), i([1]), i([100]), served)
    assert served.item() == 1
    h.lens[1] = 100
    h.table, h.refs = h.cache.table.cpu().numpy(), h.cache.refs.cpu().numpy()
    h.check(50, 4, 10, unserved=(0, 1))
    # what goes lies behind position 48, whose pages are shared but not written
    h.weight[:, :48] = 2.0
    h.lens[2] = 50
    h.check(48, 4, 0)
    assert h.refs.max() == 2 and dfl2.dfl2_device_error() == 0


def test_missing_pages_and_bad_rows():
    h = Held([100, 100, 100, 100], 16, seed=9, extra=1)
    h.cache.table[0, 3] = -1
    h.table[0, 3] = -1
    h.cache.table[1, 6] = 1 << 20
    h.table[1, 6] = 1 << 20
    h.check(40, 4, 10, unserved=(0, 1))
    assert dfl2.dfl2_device_error() == 0
    h = Held([100, 100, 100, 100], 16, seed=9, extra=1)
    h.rows[1] = 77
    h.lens = [-1, 100, (1 << 30) + 1, 7 * 16 + 1 + 16]  # too long for the row: unserved only
    kept, new, served = h.call(40, 4, 10)
    assert dfl2.dfl2_device_error() == 5
    assert served.tolist() == [0, 0, 0, 0] and new.tolist() == h.lens and (kept == -1).all()
    assert np.array_equal(h.cache.table.cpu().numpy(), h.table)


def test_new_length_may_be_length():
    h = Held([100, 30, 200], 16, seed=10)
    h.check(40, 4, 10, alias=True)


def test_captured():
    h = Held([100, 30, 200], 16, seed=11)
    length, kept = h.i32(h.lens), torch.zeros(3, 40, dtype=torch.int32, device="cuda")
    new, served = torch.zeros_like(length), torch.zeros_like(length)
    ws = dfl2.workspace(dfl2.dfl2_cache_evict_workspace_size(3, 40))
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        dfl2.dfl2_cache_evict(h.cache, length, 40, 4, 10, h.weight, kept, new, served, ws)
    twin = Held([100, 30, 200], 16, seed=11)
    want = twin.call(40, 4, 10)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[0]) and new.tolist() == want[1].tolist()
    assert torch.equal(h.cache.k, twin.cache.k) and torch.equal(h.cache.table, twin.cache.table)


def test_offsets_past_32_bits():
    """A cache whose pages lie more than 2^32 bytes and 2^31 elements apart."""
    H, ps, D = 8, 64, 128
    pages = (1 << 31) // (H * ps * D) + 40
    k = torch.zeros(1, pages, H, ps, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    use = [0, pages - 1, 1, pages - 2]
    table = torch.tensor([use], dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[use] = 1
    free = pack_bits((refs.cpu().numpy() == 0)[None])[0]
    cache = dfl2.Cache(k, v, table, refs, torch.tensor(free, device="cuda"))
    n, keep = 250, 100
    rows = torch.randn(n, 2, H, D, device="cuda").to(torch.bfloat16)
    zero, i32 = torch.zeros(1, dtype=torch.int32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    dfl2.dfl2_cache_write(cache, rows[None, :, 0], rows[None, :, 1], zero)
    weight = torch.rand(1, 256, device="cuda")
    want = stays(weight[0].cpu().numpy(), n, keep, 2, 30)
    kept, new, served = torch.zeros(1, keep, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    ws = dfl2.workspace(dfl2.dfl2_cache_evict_workspace_size(1, keep))
    dfl2.dfl2_cache_evict(cache, torch.full((1,), n, **i32), keep, 2, 30, weight, kept, new, served, ws)
    assert kept[0].tolist() == want
    for i, p in enumerate(want):
        assert torch.equal(k[0, use[i // ps], :, i % ps], rows[p, 0])
        assert torch.equal(v[0, use[i // ps], :, i % ps], rows[p, 1])
