"""dfl2_tree_verify where what is left of the target's distribution is little or nothing, against
its definition in 64 bits: rows whose mass lies on the candidates alone, several of them in one
16-byte vector, draws at both ends of [0, 1)."""
import numpy as np
import pytest

import draft_selection_gb300 as dfl2
from test_gpu_tree_verify import call, check, make

pytestmark = pytest.mark.gpu
LAST = np.float32(1 - 2.0**-24)  # the largest float32 below 1


def roots(rng, B, T, V, mass, first=None, of=16):
    """Roots with T - 1 children; `mass` adjacent candidates have all of p, `of` of them all of
    q.  Both are spread over eight decades, as those of a filtered softmax."""
    first = rng.randint(0, V - 16, B) if first is None else np.asarray(first)
    cand = first[:, None] + np.argsort(rng.rand(B, 16), 1)
    e = np.where(cand - first[:, None] < mass, np.exp(rng.uniform(-18, 0, (B, 16))), 0)
    p = np.zeros((B, T, V), np.float32)
    q = np.exp(rng.uniform(-18, 0, (B, T, 16))).astype(np.float32)
    q[np.broadcast_to((cand - first[:, None] >= of)[:, None], q.shape)] = 0
    for i in range(T):
        np.put_along_axis(p[:, i], cand, (e / e.sum(1, keepdims=True)).astype(np.float32), 1)
    order = np.argsort(-(np.log(q[:, 0] + 1e-30) + rng.gumbel(size=(B, 16))), 1)
    tokens = np.zeros((B, T), np.int32)
    tokens[:, 1:] = np.take_along_axis(cand, order[:, :T - 1], 1)
    parents = np.zeros((B, T), np.int32)
    parents[:, 0] = -1
    return dict(p=p, tokens=tokens, parents=parents, q=q,
                cand=np.broadcast_to(cand[:, None], (B, T, 16)).astype(np.int32),
                u=rng.randint(0, 1 << 24, (B, T)).astype(np.float32) * np.float32(2.0**-24))


def test_a_row_that_lies_on_four_candidates():
    """A miss of the last child leaves nothing: the draw is from p itself."""
    V, T = 1024, 5
    x = make(1, T, V, False, seed=1)
    x["p"][:], x["q"][:] = 0, 0
    x["cand"][:] = [153, 170, 168, 169, *range(600, 612)]
    x["p"][:, :, [153, 170, 168, 169]] = [.395767868, .604232073, 4.66871475e-09, 2.26337651e-08]
    x["q"][:, :, :4] = [6.7732342e-10, 2.69362272e-06, .999927402, 6.99239754e-05]
    x["parents"][:] = [-1, 0, 0, 0, 0]
    x["tokens"][:] = [0, 168, 169, 170, 153]
    x["u"][:] = [.914233387, .5, .5, .9, LAST]
    got = call(x, False)
    check(x, False, got)
    assert got[2].tolist() == [170]


@pytest.mark.parametrize("replace", [False, True])
@pytest.mark.parametrize("mass", [2, 3, 4, 9, 16])
@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("u0", [0.0, LAST, None])
def test_rows_that_lie_on_adjacent_candidates(mass, narrow, u0, replace):
    """Every u at its largest value, so that nearly every child is passed by."""
    rng = np.random.RandomState(mass)
    x = roots(rng, 1500, 5, 101, mass, of=mass if narrow else 16)
    x["u"][:, 1:] = LAST
    if u0 is not None:
        x["u"][:, 0] = u0
    check(x, replace, call(x, replace))
    assert dfl2.dfl2_device_error(clear=True) == 0


@pytest.mark.parametrize("V", [17, 18, 19, 37, 4099])
def test_candidates_in_the_first_and_last_vectors(V):
    """Rows begin 0 to 3 elements past 16 bytes, and what is left lies at either end."""
    rng = np.random.RandomState(V)
    for end in (0, V - 16):
        x = roots(rng, 400, 4, V, 16, first=np.full(400, end))
        x["u"][:, 1:] = LAST
        for u0 in (0.0, 0.5, LAST):
            x["u"][:, 0] = u0
            check(x, False, call(x, False))


def test_what_is_left_lies_far_from_the_rejected():
    """Four candidates of one vector are rejected; r is 0 there and on the rest of the row's
    first blocks, and a draw of 0 takes the first element that has any."""
    V, B = 151936, 6
    x = make(B, 5, V, False, seed=4)
    rng = np.random.RandomState(5)
    x["p"][:], x["q"][:] = 0, 0
    x["cand"][:] = [8, 9, 10, 11, *range(120000, 120012)]
    x["p"][:, :, 8:12] = (rng.rand(B, 1, 4) * [0.2, 2e-9, 5e-8, 3e-8]).astype(np.float32)
    x["p"][:, :, 150000] = 1 - x["p"].sum(2)
    x["q"][:, :, :4] = 0.25
    x["parents"][:], x["tokens"][:] = [-1, 0, 0, 0, 0], [0, 8, 9, 10, 11]
    for u0 in (0.0, 0.3, LAST):
        x["u"][:] = LAST
        x["u"][:, 0] = u0
        got = call(x, False)
        check(x, False, got)
        assert (got[2] == 150000).all()


def test_a_row_of_very_different_sizes():
    """Candidates of 1e30 beside elements of 1e-17: what is left of these, as floats, is 0 element
    by element and not 0 in sums.  The first of them is drawn all the same."""
    x = make(1, 2, 8192, False, seed=6)
    x["p"][:], x["q"][:] = 0, 0
    x["cand"][:] = np.arange(8000, 8016)
    x["p"][:, :, 5:256] = 1e-17
    x["p"][:, :, 8000:8002] = [1e30, 1e29]
    x["q"][:, :, 0] = 1
    x["parents"][:], x["tokens"][:] = [-1, 0], [0, 8000]
    x["u"][:] = [0, LAST]
    got = call(x, False)
    check(x, False, got)
    assert got[2].tolist() == [5]
