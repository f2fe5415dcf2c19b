"""GPU tests of the cache's pages and of the trees' masks and acceptance, through
the C ABI: every table entry, count, bit and moved row equal to the one-at-a-time
model's."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _tree_ref import CacheModel, ancestors, pack_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from draft_selection_gb300 import build
    build.build()
    dfl2.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Pair:
    """A device cache and its model.  A position's row is filled with numbers that
    are exact in every type and different per layer, head and K/V; the model holds
    one number per position."""

    def __init__(self, rows, cols, pages, ps, layers=2, H=2, D=64, dtype=torch.bfloat16, nhd=False):
        self.m = CacheModel(rows, cols, pages, ps)
        self.layers, self.H, self.D, self.dtype = layers, H, D, dtype
        if nhd:
            c = dfl2.cache(layers, pages, ps, H, D, rows, cols, dtype)  # [.., ps, H, D]
            self.c = dfl2.Cache(c.k.transpose(2, 3), c.v.transpose(2, 3), c.table, c.refs,
                                c.free_bits)
        else:
            self.c = dfl2.cache(layers, pages, H, ps, D, rows, cols, dtype)
        self.next = 1

    def spread(self, vals):
        """Numbers [...] -> rows [layers, ..., 2, H, D]: a position's number in base 64,
        a digit per channel, and where the row is."""
        v = torch.as_tensor(vals, device="cuda")
        x = torch.zeros((self.layers,) + v.shape + (2, self.H, self.D), device="cuda")
        for d in range(4):
            x[..., d::8] = ((v >> (6 * d)) & 63).float()[None, ..., None, None, None]
        for n in range(self.layers):
            x[n, ..., 4::8] = n + 1
        x[..., 1, :, 5::8] = 1
        for h in range(self.H):
            x[..., h, 6::8] = h + 1
        x[..., 7::8] = torch.arange(self.D // 8, device="cuda", dtype=torch.float32)
        x = torch.where((v == 0)[None, ..., None, None, None], torch.zeros_like(x), x)
        return x.to(self.dtype)

    def fresh(self, *shape):
        n = int(np.prod(shape))
        out = np.arange(self.next, self.next + n).reshape(shape)
        self.next += n
        return out

    def same(self):
        torch.cuda.synchronize()
        assert dfl2.dfl2_device_error() == 0
        m, c = self.m, self.c
        assert np.array_equal(c.table.cpu().numpy(), m.table)
        assert np.array_equal(c.refs.cpu().numpy(), m.refs)
        assert np.array_equal(c.free_bits.cpu().numpy(), m.bits())
        want = self.spread(m.val).permute(0, 1, 3, 4, 2, 5)  # [layers, pages, 2, H, ps, D]
        assert torch.equal(c.k, want[:, :, 0]) and torch.equal(c.v, want[:, :, 1])

    def reserve(self, rows, length, count):
        served = i32([7] * len(rows))
        dfl2.dfl2_cache_reserve(self.c, i32(length), i32(count), served, rows=i32(rows))
        assert served.tolist() == self.m.reserve(rows, length, count)
        return served.tolist()

    def write(self, rows, length, count):
        T = max(max(count), 1)
        vals = self.fresh(len(rows), T)
        new = self.spread(vals)
        dfl2.dfl2_cache_write(self.c, new[:, :, :, 0], new[:, :, :, 1], i32(length),
                              count=i32(count), rows=i32(rows))
        self.m.write(rows, length, count, vals)

    def compact(self, rows, length, count, path, n_path):
        T = max(count)
        full = np.full((len(rows), T), -1)
        for b, p in enumerate(path):
            full[b, :len(p)] = p
        new = i32(length)
        dfl2.dfl2_cache_compact(self.c, new, i32(count), i32(full), i32(n_path), new, rows=i32(rows))
        want = self.m.compact(rows, length, count, path, n_path)
        assert new.tolist() == want
        return want

    def fork(self, src, dst, length):
        served = i32([7] * len(src))
        dfl2.dfl2_cache_fork(self.c, i32(src), i32(dst), i32(length), served)
        assert served.tolist() == self.m.fork(src, dst, length)
        return served.tolist()

    def free(self, rows):
        dfl2.dfl2_cache_free(self.c, i32(rows))
        self.m.free(rows)


@pytest.mark.parametrize("seed,ps,dtype,nhd", [(0, 8, torch.bfloat16, False),
                                               (1, 16, torch.float32, True),
                                               (2, 32, torch.float16, False),
                                               (3, 128, torch.bfloat16, True)])
def test_a_life_of_turns(seed, ps, dtype, nhd):
    """Random admissions, turns, forks and ends, the state compared after each; the
    pages run out at times."""
    rng = np.random.default_rng(seed)
    rows, cols, pages = 9, 14, 20
    p = Pair(rows, cols, pages, ps, dtype=dtype, nhd=nhd)
    length = {}
    short = 0
    for step in range(40):
        idle = [r for r in range(rows) if r not in length]
        kind = rng.integers(0, 10)
        if kind < 3 and idle:  # admit
            n = min(len(idle), int(rng.integers(1, 4)))
            who = [int(x) for x in rng.permutation(idle)[:n]]
            count = [int(x) for x in rng.integers(0, ps * 5, n)]
            got = p.reserve(who, [0] * n, count)
            if any(got):
                p.write([r for r, g in zip(who, got) if g], [0] * sum(got),
                        [c for c, g in zip(count, got) if g])
            for r, c, g in zip(who, count, got):
                short += not g
                if g:
                    length[r] = c
        elif kind < 7 and length:  # a turn
            who = [int(x) for x in rng.permutation(sorted(length))[:int(rng.integers(1, 6))]]
            T = int(rng.integers(1, 2 * ps + 2))
            count = [int(x) for x in rng.integers(0, T + 1, len(who))]
            got = p.reserve(who, [length[r] for r in who], count)
            short += sum(not g for g in got)
            who, count = [r for r, g in zip(who, got) if g], [c for c, g in zip(count, got) if g]
            if who and max(count):
                base = [length[r] for r in who]
                p.write(who, base, count)
                path = [sorted(int(x) for x in rng.permutation(c)[:rng.integers(0, c + 1)])
                        for c in count]
                new = p.compact(who, base, count, path, [len(x) for x in path])
                length.update(zip(who, new))
        elif kind < 9 and length and idle:  # fork
            n = min(len(idle), int(rng.integers(1, 4)))
            src = [int(rng.choice(sorted(length))) for _ in range(n)]
            dst = idle[:n]
            at = [int(rng.integers(0, length[r] + 1)) for r in src]
            got = p.fork(src, dst, at)
            for z, a, g in zip(dst, at, got):
                short += not g
                if g:
                    length[z] = a
        elif length:
            who = [int(x) for x in rng.permutation(sorted(length))[:int(rng.integers(1, 3))]]
            p.free(who)
            for r in who:
                del length[r]
        p.same()
    assert short, "the pages never ran out: the test lost its point"
    p.free(sorted(length) or [0])
    p.same()
    assert (p.m.refs == 0).all()


def test_a_long_prompt_takes_thousands_of_pages():
    """More pages than one round of the list holds, over several sequences."""
    p = Pair(5, 6000, 12345, 8, layers=1, H=1, D=64)
    p.reserve([3, 1, 4], [0, 0, 0], [8 * 4000 + 3, 8 * 5990, 8 * 1500])
    p.free([1])
    p.reserve([0, 1], [0, 0], [8 * 2000 - 7, 8 * 100])
    p.reserve([2, 0], [0, 0], [8 * 5999, 8 * 6000 + 1])  # too few pages; too few entries
    p.same()


def test_many_sequences():
    B = 4096
    p = Pair(B, 2, 5000, 8, layers=1, H=1, D=64)
    rng = np.random.default_rng(0)
    count = [int(x) for x in rng.integers(0, 17, B)]
    got = p.reserve(list(range(B)), [0] * B, count)
    assert 0 < sum(got) < B
    p.same()


def test_counts_as_a_number_and_no_rows():
    p = Pair(2, 8, 9, 16)
    served, length = i32([0, 0]), i32([0, 0])
    dfl2.dfl2_cache_reserve(p.c, length, 33, served)
    assert served.tolist() == p.m.reserve([0, 1], [0, 0], [33, 33]) == [1, 1]
    vals = p.fresh(2, 33)
    new = p.spread(vals)
    for layer in range(2):
        dfl2.dfl2_cache_write(p.c, new[layer, :, :, 0], new[layer, :, :, 1], length, layer=layer)
    p.m.write([0, 1], [0, 0], [33, 33], vals)
    p.same()
    # everything dropped again
    path, n = i32(np.full((2, 33), -1)), i32([0, 0])
    dfl2.dfl2_cache_compact(p.c, length, 33, path, n, length)
    p.m.compact([0, 1], [0, 0], [33, 33], [[], []], [0, 0])
    p.same()
    assert length.tolist() == [0, 0]


def test_counts_no_row_can_hold():
    p = Pair(3, 8, 40, 16)
    big = (1 << 31) - 1
    assert p.reserve([0, 1, 2], [5, 0, 100], [big, 1 << 30, 29]) == [0, 0, 0]
    p.same()
    assert p.reserve([0, 2], [0, 100], [128, 28]) == [1, 1]  # the last entries, to the brim
    p.same()
    served = i32([7])
    dfl2.dfl2_cache_reserve(p.c, i32([-3]), 4, served)
    assert served.tolist() == [0]
    p.same()


def test_no_rows():
    p = Pair(2, 4, 6, 8)
    none = torch.zeros(2, 2, 0, p.c.kv_heads, p.c.head_dim, dtype=p.c.dtype, device="cuda")
    length, served = i32([0, 0]), i32([7, 7])
    dfl2.dfl2_cache_reserve(p.c, length, 0, served)
    dfl2.dfl2_cache_write(p.c, none, none, length)
    p.same()
    assert served.tolist() == [1, 1]


@pytest.mark.parametrize("pages", [1, 31, 33, 40])
def test_map_bits_past_the_pages_are_no_pages(pages):
    c = dfl2.cache(1, pages, 1, 8, 64, 2, 64)
    c.free_bits.fill_(-1)
    served = i32([7, 7])
    dfl2.dfl2_cache_reserve(c, i32([0, 0]), i32([8 * pages - 8, 16]), served)
    assert served.tolist() == [1, 0]
    dfl2.dfl2_cache_reserve(c, i32([0, 0]), i32([8 * pages, 8]), served)
    assert served.tolist() == [1, 0]
    assert c.table[0, :pages].tolist() == list(range(pages)) and (c.table[1] == -1).all()
    assert (c.refs == 1).all()


def test_odd_rows():
    """Rows whose 16-byte pieces are no power of two, in a part of a wider tensor."""
    k = torch.zeros(2, 7, 3, 8, 96, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    c0 = dfl2.cache(2, 7, 3, 8, 96, 3, 4, torch.float16)
    c = dfl2.Cache(k[..., :40], v[..., :40], c0.table, c0.refs, c0.free_bits)
    served, length = i32([0, 0, 0]), i32([0, 0, 0])
    dfl2.dfl2_cache_reserve(c, length, 11, served)
    new = torch.randn(2, 3, 11, 2, 3, 40, device="cuda").half()
    dfl2.dfl2_cache_write(c, new[:, :, :, 0], new[:, :, :, 1], length)
    torch.cuda.synchronize()
    assert dfl2.dfl2_device_error() == 0
    for b in range(3):
        for t in range(11):
            page = int(c.table[b, t // 8])
            assert torch.equal(k[:, page, :, t % 8, :40], new[:, b, t, 0])
            assert torch.equal(v[:, page, :, t % 8, :40], new[:, b, t, 1])
    assert (k[..., 40:] == 0).all()


def test_what_is_out_of_range_is_recorded_and_left_out():
    p = Pair(3, 4, 6, 8)
    p.reserve([0], [0], [9])
    p.same()
    served = i32([7, 7])
    dfl2.dfl2_cache_reserve(p.c, i32([0, 0]), 3, served, rows=i32([3, -1]))
    assert dfl2.dfl2_device_error() == 5 and served.tolist() == [0, 0]
    new = p.spread(p.fresh(1, 3))
    dfl2.dfl2_cache_write(p.c, new[:, :, :, 0], new[:, :, :, 1], i32([30]))  # no page there
    assert dfl2.dfl2_device_error() == 5
    dfl2.dfl2_cache_free(p.c, i32([-5, 99]))
    assert dfl2.dfl2_device_error() == 5
    dfl2.dfl2_cache_compact(p.c, i32([0]), 3, i32([[1, 0, 2]]), i32([2]), i32([0]))
    assert dfl2.dfl2_device_error() == 5
    torch.cuda.synchronize()
    assert p.c.table[0].tolist() == [0, 1, -1, -1]  # page 1 lies behind the three nodes' range


def test_fork_leaves_a_used_row_alone():
    p = Pair(3, 4, 8, 8)
    p.reserve([0, 1], [0, 0], [20, 5])
    assert p.fork([0, 1, 1], [1, 2, 2], [20, 17, 5]) == [0, 0, 1]
    p.same()


def random_parents(rng, T, roots=1):
    return [-1] * min(T, roots) + [int(max(0, i - rng.geometric(0.4))) for i in range(roots, T)]


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 200, 256])
def test_tree_mask(T):
    rng = np.random.default_rng(T)
    B = 5
    par = np.array([random_parents(rng, T, 1 + b % 2) for b in range(B)])
    par[1] = np.arange(T) - 1  # a chain
    count = [T, T, int(rng.integers(0, T + 1)), 0, T]
    anc = np.stack([ancestors(list(x)) for x in par])
    for b, n in enumerate(count):
        anc[b, n:] = False
    mask, depth = i32(np.full((B, T, (T + 31) // 32), 9)), i32(np.full((B, T), 9))
    dfl2.dfl2_tree_mask(i32(par), mask, depth, count=i32(count))
    torch.cuda.synchronize()
    assert dfl2.dfl2_device_error() == 0
    assert np.array_equal(mask.cpu().numpy(), pack_bits(anc))
    assert np.array_equal(depth.cpu().numpy(), np.maximum(anc.sum(-1) - 1, 0))


def test_tree_mask_records_bad_parents():
    par = i32([[-1, 0, 2, 1, -7]])  # node 2 names itself, node 4 nothing that exists
    mask = i32(np.zeros((1, 5, 1)))
    dfl2.dfl2_tree_mask(par, mask)
    assert dfl2.dfl2_device_error() == 5
    assert mask[0, :, 0].tolist() == [1, 3, 4, 11, 16]


def accept(tokens, parents, target, n):
    path = []
    if n == 0:
        return path, -1
    path, cur = [0], 0
    while True:
        kids = [i for i in range(cur + 1, n) if parents[i] == cur and tokens[i] == target[cur]]
        if not kids:
            return path, target[cur]
        cur = kids[0]
        path.append(cur)


@pytest.mark.parametrize("T", [1, 2, 17, 32, 33, 100, 256])
@pytest.mark.parametrize("vocab", [2, 50])
def test_tree_accept(T, vocab):
    rng = np.random.default_rng(T + vocab)
    B = 23
    par = np.array([random_parents(rng, T) for _ in range(B)])
    par[4] = np.arange(T) - 1
    tok, tgt = rng.integers(0, vocab, (B, T)), rng.integers(0, vocab, (B, T))
    tgt[4, :-1] = tok[4, 1:]  # a chain accepted whole
    count = rng.integers(0, T + 1, B)
    count[:10] = T
    path, n, nxt = i32(np.full((B, T), 9)), i32([9] * B), i32([9] * B)
    dfl2.dfl2_tree_accept(i32(tok), i32(par), i32(tgt), path, n, nxt, count=i32(count))
    torch.cuda.synchronize()
    for b in range(B):
        want, last = accept(tok[b], par[b], tgt[b], count[b])
        assert n[b] == len(want) and nxt[b] == last
        assert path[b].tolist() == want + [-1] * (T - len(want))
