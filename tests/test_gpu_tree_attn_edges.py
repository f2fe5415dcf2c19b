"""GPU tests of dfl2_tree_attn where a sequence's last tiles, its missing pages or its lengths
are out of the ordinary, against the 64-bit definition or a run on data without the oddity."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _tree_ref import attention, attention_bounds
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
    nodes times channels: the limit is half of what the latter took, 50 ms."""
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
    assert begin.elapsed_time(end) < 25.0
    assert dfl2.dfl2_device_error() == 0


def check_without(c, out, lse, gone):
    """As Case.check, without the positions gone[b] of sequence b."""
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (n, cnt) in enumerate(zip(c.lens, c.counts)):
        seen = np.ones((c.T, n + cnt), bool)
        seen[:, n:] = c.seen[b][:, :cnt]
        seen[cnt:] = False
        seen[:, gone[b]] = False
        kv = c.kv[b].double().numpy()
        ref = attention(c.q[b].double().numpy(), kv[0], kv[1], seen, c.D ** -0.5)
        ob, lb = attention_bounds(ref, c.dtype, c.D, n + cnt)
        assert (np.abs(o[b] - ref[0]) <= ob).all(), (b, np.abs(o[b] - ref[0]).max())
        dead = np.isneginf(ref[1])
        assert np.array_equal(z[b][dead], ref[1][dead])
        assert (np.abs(z[b][~dead] - ref[1][~dead]) <= lb[~dead]).all(), b


@pytest.mark.parametrize("page", [8, 16, 32, 64, 256])
@pytest.mark.parametrize("T,Hq,Hkv,D,dtype", [(1, 4, 2, 128, torch.bfloat16),
                                              (20, 8, 1, 64, torch.float16),
                                              (70, 4, 1, 128, torch.bfloat16),
                                              (9, 8, 2, 256, torch.bfloat16)])
def test_positions_without_a_page_are_left_out(T, Hq, Hkv, D, dtype, page):
    """Entries that are -1 or name no page, among the committed positions, among the nodes and
    everywhere: those positions count for nothing, and the index is recorded."""
    lens = [700, 515, 300, 0, 1500, 64, 2000]
    c = Case(lens, T, Hq, Hkv, D, page, dtype, seed=page + T)
    rng = np.random.default_rng(page)
    table = c.cache.table.cpu().numpy()
    gone = []
    for b, n in enumerate(lens):
        used = -(-(n + T) // page)
        if b == 4:
            cols = np.arange(used)                    # a sequence that was given no pages
        elif b == 5:
            cols = np.arange(n // page, used)         # no pages for its nodes
        elif b == 6:
            cols = np.arange(max(1, used // 2))       # none for its first half
        else:
            cols = rng.permutation(used)[:1 + used // 7]
        table[b, cols] = rng.choice([-1, 1 << 20, -7, c.cache.k.shape[1]], len(cols))
        gone.append(np.concatenate([np.arange(x * page, min((x + 1) * page, n + T)) for x in cols]))
    c.cache.table.copy_(torch.from_numpy(table))
    q = c.q.cuda()
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(*q.shape[:3], Hkv, D, dtype))
    dfl2.dfl2_tree_attn(q, c.cache, 0, c.length, c.mask, out, ws, lse=lse)
    assert dfl2.dfl2_device_error() == 5
    check_without(c, out, lse, gone)


@pytest.mark.parametrize("T", [3, 50])
def test_nan_keys_of_committed_positions(T):
    """A number that is none is no missing page: every node of that key head has it."""
    c = Case([500, 300, 70], T, 8, 2, 128, 16, seed=T)
    want, want_lse = c.run()
    page = int(c.cache.table[1, 5])
    c.cache.k[0, page, 1, 3] = float("nan")
    out, lse = c.run()
    assert torch.isnan(out[1, :, 4:]).all() and torch.isnan(lse[1, :, 4:]).all()
    out[1, :, 4:], lse[1, :, 4:] = want[1, :, 4:], want_lse[1, :, 4:]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("T,D,dtype", [(2, 64, torch.bfloat16), (40, 128, torch.float16),
                                       (3, 256, torch.bfloat16)])
def test_rows_with_scores_of_minus_infinity_only(T, D, dtype):
    """Out is 0 and lse -inf whatever the values hold, in a sequence of one tile and in one that
    is cut into parts."""
    c = Case([20, 9000], T, 4, 2, D, 16, dtype, seed=D, mask="chain")
    table = c.cache.table.cpu()
    c.cache.k.fill_(float("-inf"))
    q = torch.rand(2, T, 4, D, device="cuda").to(dtype) + 1
    for b, n in enumerate(c.lens):
        for j, x in ((3, float("inf")), (n - 1, float("nan")), (n + T - 1, float("-inf"))):
            c.cache.v[0, int(table[b, j // 16]), :, j % 16, ::3] = x
    out, lse = c.run(q=q)
    assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("length", [-1, -(1 << 31), (1 << 30) + 1, (1 << 31) - 1])
def test_lengths_out_of_range_are_recorded(length):
    c = Case([100, 30, 50], 3, 4, 2, 128, 16, seed=1)
    want, want_lse = c.run()
    c.length[1] = length
    q, out, lse = c.q.cuda(), torch.empty_like(want), torch.empty_like(want_lse)
    ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(3, 3, 4, 2, 128, c.dtype))
    dfl2.dfl2_tree_attn(q, c.cache, 0, c.length, c.mask, out, ws, lse=lse)
    assert dfl2.dfl2_device_error() == 5
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
    assert torch.equal(out[::2], want[::2]) and torch.equal(lse[::2], want_lse[::2])


@pytest.mark.parametrize("at", [0, 30000])
def test_a_long_tail_of_small_weights(at):
    """float16: one position has nearly all the weight of each, the others, of 2^-19 each, a tenth
    of the weight together.  Sums as attention_bounds has them, and half a unit of each weight
    and of the result, which small weights have too.  So many sequences (of the same pages) that
    a block has most of one: a part of its own has a maximum of its own, and larger weights."""
    n, X, B = 60000, 13.25, 400
    c = Case([n], 1, 2, 1, 64, 64, torch.float16, seed=1)
    c.cache.k.zero_()
    c.cache.v.fill_(1.0)
    page = int(c.cache.table[0, at // 64])
    c.cache.k[0, page, 0, at % 64, 0] = X
    c.cache.v[0, page, 0, at % 64] = 0.0
    c.cache = dfl2.Cache(c.cache.k, c.cache.v, c.cache.table.repeat(B, 1), c.cache.refs,
                         c.cache.free_bits)
    c.length, c.mask = c.length.repeat(B), None
    q = torch.zeros(B, 1, 2, 64, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    out, lse = c.run(q=q, scale=1.0)
    tail = n * np.exp(-X)                     # n + 1 positions, one of them the large one
    want = tail / (1 + tail)
    far = (2 * 2.0**-11 + 2 * (n * 2.0**-24 + 8 * X * 2.0**-24)) * want
    assert (out.double() - want).abs().max() <= far
    assert (lse.double() - X - np.log1p(tail)).abs().max() <= n * 2.0**-24 + 2.0**-20
