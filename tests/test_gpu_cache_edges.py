"""GPU tests of the cache's calls on lengths, rows and sizes out of the ordinary."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_gpu_cache import Pair, _lib, i32  # noqa: F401  (the fixture builds and loads the library)

pytestmark = pytest.mark.gpu

BAD_LENGTHS = [(1 << 31) - 1, (1 << 31) - 20, (1 << 30) + 1, -1, -5, -(1 << 31)]


def recorded():
    torch.cuda.synchronize()
    return dfl2.dfl2_device_error()


def test_compaction_leaves_out_a_length_out_of_range():
    """Neither entries far from the table nor rows that a length below 0 reaches with its last
    nodes are touched; the other sequences are compacted, and the length stays."""
    p = Pair(7, 6, 40, 8)
    rows = list(range(7))
    p.reserve(rows, [0] * 7, [40] * 7)
    p.write(rows, [0] * 7, [40] * 7)
    p.same()
    path = np.tile([0, 2, 5, 6, 16, -1], (7, 1))
    path = np.concatenate([path, np.full((7, 11), -1)], 1)
    length = i32(BAD_LENGTHS + [20])
    dfl2.dfl2_cache_compact(p.c, length, 17, i32(path), i32([5] * 7), length)
    assert recorded() == 5
    want = p.m.compact([6], [20], [17], path[6:], [5])
    assert length.tolist() == BAD_LENGTHS + want
    p.same()


def test_compaction_of_a_row_out_of_range_keeps_the_length():
    p = Pair(2, 4, 9, 8)
    p.reserve([0, 1], [0, 0], [9, 30])
    length = i32([3, 20])
    dfl2.dfl2_cache_compact(p.c, length, 4, i32([[0, 1, 2, 3]] * 2), i32([4, 2]), length,
                            rows=i32([2, 1]))
    assert recorded() == 5
    p.m.compact([1], [20], [4], [[0, 1]], [2])
    assert length.tolist() == [3, 22]
    p.same()


def test_writes_leave_out_a_length_out_of_range():
    """The last tokens behind a length just below 0 would lie at positions 0, 1, .."""
    p = Pair(7, 6, 40, 8)
    rows = list(range(7))
    p.reserve(rows, [0] * 7, [40] * 7)
    p.write(rows, [0] * 7, [40] * 7)
    vals = p.fresh(7, 9)
    new = p.spread(vals)
    dfl2.dfl2_cache_write(p.c, new[:, :, :, 0], new[:, :, :, 1], i32(BAD_LENGTHS + [20]))
    assert recorded() == 5
    p.m.write([6], [20], [9], vals[6:])
    p.same()


def test_rows_with_room_past_the_longest_sequence():
    """Entries for more than 2^30 positions do not make a length above that one."""
    cols = (1 << 22) + 16
    c = dfl2.cache(1, 4, 1, 256, 64, 2, cols)
    served = i32([7, 7])
    dfl2.dfl2_cache_reserve(c, i32([(1 << 30) + 1, 1 << 30]), 3, served)
    assert recorded() == 0 and served.tolist() == [0, 1]
    assert c.table[1, 1 << 22] == 0 and (c.table[0] == -1).all() and int(c.refs.sum()) == 1


def test_fork_into_a_row_with_pages_is_refused_wherever_they_are():
    """Also where the fork itself needs fewer entries, or none."""
    p = Pair(6, 40, 60, 8)
    p.reserve([0, 1, 2], [0, 0, 200], [100, 5, 9])      # row 2: pages behind position 200 only
    before = p.c.table.clone()
    served = i32([7] * 4)
    dfl2.dfl2_cache_fork(p.c, i32([0, 0, 0, 0]), i32([1, 2, 3, 4]), i32([0, 20, 0, 20]), served)
    assert served.tolist() == [0, 0, 1, 1]
    assert torch.equal(p.c.table[:4], before[:4])
    assert p.m.fork([0, 0], [3, 4], [0, 20]) == [1, 1]
    p.same()


@pytest.mark.parametrize("src,dst", [(6, 3), (-1, 3), (1 << 30, 3), (0, 6), (0, -2)])
def test_forks_of_rows_out_of_range_are_recorded(src, dst):
    p = Pair(6, 4, 20, 8)
    p.reserve([0], [0], [20])
    served = i32([7, 7])
    dfl2.dfl2_cache_fork(p.c, i32([src, 0]), i32([dst, 2]), i32([20, 20]), served)
    assert recorded() == 5 and served.tolist() == [0, 1]
    p.m.fork([0], [2], [20])
    p.same()


def test_writes_compactions_and_ends_of_5000_sequences():
    B = 5000
    p = Pair(B, 2, 2 * B, 8, layers=1, H=1, D=64)
    for a in range(0, B, 4000):
        n = min(B - a, 4000)
        p.reserve(list(range(a, a + n)), [0] * n, [11] * n)
    rows = [int(x) for x in np.random.default_rng(0).permutation(B)]
    p.write(rows, [0] * B, [11] * B)
    path = [[0, 2, 5] if b % 3 else [0, 3, 4, 5, 6, 7, 8, 9, 10] for b in range(B)]
    p.compact(rows, [0] * B, [11] * B, path, [len(x) for x in path])
    p.same()
    p.free(rows[:4500])
    p.same()


@pytest.mark.parametrize("layers,H,D,ps,dtype,nhd", [
    (3, 8, 128, 16, torch.bfloat16, False),    # 768 columns of 16 bytes: two blocks a sequence
    (7, 8, 128, 16, torch.float16, True),      # 1792: four, some threads without a column
    (33, 5, 104, 8, torch.bfloat16, False),    # 4290: eight, some with two columns
    (20, 8, 128, 32, torch.float32, False),    # 10240: eight, two or three columns each
    (2, 33, 128, 8, torch.bfloat16, True)])    # more than 128 pieces of a row: 528
def test_wide_rows_and_many_layers(layers, H, D, ps, dtype, nhd):
    """Writes, compactions, forks and the pages that a compaction gives back, where a sequence's
    rows are the work of several blocks and a warp takes a row in several turns."""
    rng = np.random.default_rng(layers)
    n = 7
    p = Pair(2 * n, 14, 90, ps, layers=layers, H=H, D=D, dtype=dtype, nhd=nhd)
    rows = [int(x) for x in rng.permutation(2 * n)]
    rows, others = rows[:n], rows[n:]
    length = [int(x) for x in rng.integers(0, 4 * ps, n)]
    p.reserve(rows, [0] * n, length)
    p.write(rows, [0] * n, length)
    p.same()
    for _ in range(3):
        T = 3 * ps + 1
        count = [int(x) for x in rng.integers(1, T + 1, n)]
        count[0] = T
        assert all(p.reserve(rows, length, count))
        p.write(rows, length, count)
        path = [sorted(int(x) for x in rng.permutation(c)[:rng.integers(0, min(c, ps) + 1)])
                for c in count]
        path[1] = list(range(len(path[1])))     # nothing moves
        length = p.compact(rows, length, count, path, [len(x) for x in path])
        p.same()
        got = p.fork(rows, others, length)
        p.same()
        p.free([r for r, g in zip(others, got) if g])
        p.same()


@pytest.mark.parametrize("B", [33, 64, 127, 128, 129, 300])
def test_more_sequences_than_a_pass_of_the_bookkeeping(B):
    """More than 32 sequences share the block's warps: their tables' entries, several steps of
    lanes each, and forks, which run short of pages."""
    rng = np.random.default_rng(B)
    p = Pair(3 * B, 70, 25 * B, 8, layers=1, H=1, D=64)
    rows = [int(x) for x in rng.permutation(3 * B)]
    a, b, c = rows[:B], rows[B:2 * B], rows[2 * B:]
    length = [int(x) for x in rng.integers(0, 8 * 34, B)]
    p.reserve(a, [0] * B, length)
    p.same()
    count = [int(x) for x in rng.integers(0, 8 * 34, B)]
    got = p.reserve(a, length, count)           # on from pages that are there
    p.same()
    assert any(got)
    p.write(a, [0] * B, length)
    p.same()
    at = [int(rng.integers(0, n + 1)) for n in length]
    src = [int(x) for x in rng.integers(0, B, B)]
    p.fork([a[i] for i in src], b, [at[i] for i in src])
    p.same()
    left = len(p.m.free_pages())
    if left > B // 2:                            # all but a few pages away, then forks again
        p.reserve([c[0]], [0], [min(70, left - B // 3) * 8])
    big = p.fork([a[i] for i in src], c[1:] + [c[0]], [length[i] for i in src])
    p.same()
    assert any(big)
    p.free(a)
    p.same()
    p.free(b + c)
    p.same()
    assert (p.m.refs == 0).all()
