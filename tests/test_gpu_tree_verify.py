"""dfl2_tree_verify against its definition in 64 bits, and against the target's distribution."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _sampled_ref import accept

pytestmark = pytest.mark.gpu


def trees(rng, B, T):
    p = np.full((B, T), -1, np.int32)
    for i in range(1, T):
        p[:, i] = np.maximum(0, i - rng.geometric(0.4, B))
    return p


def make(B, T, V, replace, seed, spread=3.0):
    """Rows of p, candidates among the likely tokens, siblings drawn from q."""
    rng = np.random.RandomState(seed)
    z = rng.randn(B, T, V) * spread
    p = np.exp(z - z.max(-1, keepdims=True))
    p = (p / p.sum(-1, keepdims=True)).astype(np.float32)
    cand = np.argsort(-z, -1)[:, :, :16].astype(np.int32)
    if cand.shape[2] < 16:
        cand = np.pad(cand, ((0, 0), (0, 0), (0, 16 - cand.shape[2])), constant_values=0)
    q = np.take_along_axis(p, cand.astype(np.int64), 2) ** rng.uniform(0.5, 1.5, (B, T, 1))
    q = (q * np.exp(0.5 * rng.randn(B, T, 16))).astype(np.float32)
    par = trees(rng, B, T)
    order = np.argsort(-(np.log(q + 1e-30) + rng.gumbel(size=q.shape)), -1)
    tokens = rng.randint(0, V, (B, T)).astype(np.int32)
    rank = np.zeros((B, T), np.int64)
    for i in range(1, T):
        for b in range(B):
            up = par[b, i]
            r = order[b, up, 0] if replace else order[b, up, min(rank[b, up], 15)]
            if replace:
                w = q[b, up].astype(np.float64)
                r = rng.choice(16, p=w / w.sum())
            tokens[b, i] = cand[b, up, r]
            rank[b, up] += 1
    u = rng.random_sample((B, T)).astype(np.float32)
    u[u >= 1.0] = 0.5
    return dict(p=p, tokens=tokens, parents=par, cand=cand, q=q, u=u)


def outputs(B, T):
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.full((B, T), -7, **i32), torch.full((B,), -7, **i32), torch.full((B,), -7, **i32)


def call(x, replace, count=None, out=None, **kw):
    t = {n: torch.from_numpy(np.ascontiguousarray(a)).cuda() for n, a in x.items()}
    out = out or outputs(*x["tokens"].shape)
    n = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
    dfl2.dfl2_tree_verify(t["p"], t["tokens"], t["parents"], t["cand"], t["q"], t["u"], *out,
                          count=n, replace=replace, **kw)
    return [o.cpu().numpy() for o in out]


def check(x, replace, got, count=None):
    path, n_path, nxt = got
    B, T = x["tokens"].shape
    for b in range(B):
        n = T if count is None else max(0, min(T, count[b]))
        if n == 0:
            assert n_path[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
            continue
        want, token = accept(lambda i: x["p"][b, i], x["tokens"][b, :n], x["parents"][b, :n],
                             x["cand"][b], x["q"][b], x["u"][b], replace)
        assert path[b].tolist() == want + [-1] * (T - len(want)), b
        assert n_path[b] == len(want) and nxt[b] == token, b


@pytest.mark.parametrize("replace", [False, True])
@pytest.mark.parametrize("B,T,V", [(1, 1, 16), (2, 1, 1003), (3, 2, 17), (9, 33, 129), (5, 61, 4099),
                                   (2, 256, 5001), (3, 17, 40962), (1, 9, 151936), (700, 3, 50)])
def test_paths_and_draws(B, T, V, replace):
    x = make(B, T, V, replace, seed=B + T + V)
    check(x, replace, call(x, replace))
    assert dfl2.dfl2_device_error(clear=True) == 0


@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 9])
def test_vocabularies_smaller_than_the_candidates(V):
    x = make(6, 5, V, False, seed=V)
    check(x, False, call(x, False))


def test_counts():
    x = make(8, 12, 300, False, seed=3)
    count = [0, 1, 2, 5, 12, 40, -3, 11]
    check(x, False, call(x, False, count), count)


def test_first_and_last_elements_of_rows():
    """All the mass on one token, wherever it lies: rows begin 0 to 3 elements past 16 bytes."""
    V = 1031
    at = [0, 1, 2, 3, 4, 127, 128, 511, 512, 1028, 1029, 1030]
    x = make(len(at), 3, V, False, seed=1)
    x["p"][:] = 0
    for b, i in enumerate(at):
        x["p"][b, :, i] = 1.0
    x["cand"][:] = np.arange(600, 616)
    for u0 in (0.0, 0.37, 1 - 2.0**-24):
        x["u"][:, 0] = u0
        got = call(x, False)
        check(x, False, got)
        assert got[2].tolist() == at


def test_equal_numbers_are_exact():
    """Powers of two, so that every product is exact: u d R = r D does not keep."""
    V = 64
    x = make(4, 3, V, False, seed=1)
    x["p"][:] = 0
    x["p"][:, :, :4] = [0.25, 0.25, 0.375, 0.125]
    x["cand"][:] = np.arange(16)
    x["q"][:] = 0
    x["q"][:, :, :4] = [0.5, 0.25, 0.125, 0.125]
    x["parents"][:] = [-1, 0, 0]
    x["tokens"][:] = [9, 0, 1]          # 0.25 / 0.5; then what is left: 0, 0, 0.25, 0
    x["u"][:, 0] = 0
    x["u"][:, 1] = [0.5, np.nextafter(np.float32(0.5), np.float32(0)), 0.0, 0.75]
    x["u"][:, 2] = 0
    got = call(x, False)
    check(x, False, got)
    assert got[1].tolist() == [1, 2, 2, 1] and got[2].tolist()[0] == 2


def test_what_is_left_may_be_nothing():
    """p equal to q on all its mass: a miss leaves nothing, and the draw is from p itself."""
    V = 40
    x = make(3, 4, V, True, seed=5)
    x["p"][:] = 0
    x["p"][:, :, 3], x["p"][:, :, 7] = 0.25, 0.75
    x["cand"][:] = np.arange(16)
    x["q"][:] = 0
    x["q"][:, :, 3], x["q"][:, :, 7] = 1, 3
    x["parents"][:] = [-1, 0, 0, 0]
    x["tokens"][:] = [0, 3, 7, 3]
    x["u"][:] = np.float32(1.0)         # past the range, so that equal probabilities miss
    x["u"][:, 0] = [0.0, 0.3, 0.99]
    for replace in (True, False):
        got = call(x, replace)
        check(x, replace, got)
        assert got[1].tolist() == [1, 1, 1] and got[2].tolist() == [3, 7, 7]


def test_rows_without_mass_and_odd_candidates():
    x = make(4, 5, 100, False, seed=9)
    x["p"][0] = 0                                    # nothing to draw
    x["cand"][1, :, 5] = x["cand"][1, :, 2]          # a candidate named twice
    x["q"][2, :, 3] = -1.0
    x["q"][2, :, 4] = np.nan
    x["parents"][3] = [-1, 1, 7, -5, 3]              # parents that are not below their node
    check(x, False, call(x, False))
    assert dfl2.dfl2_device_error(clear=True) == 0
    x["cand"][1, 0, 6] = 100                         # past the vocabulary: recorded, left out
    x["cand"][1, 0, 7] = -1
    check(x, False, call(x, False))
    assert dfl2.dfl2_device_error(clear=True) == 5


@pytest.mark.parametrize("replace", [False, True])
def test_the_first_token_follows_the_target(replace):
    """Three siblings at the root: the first emitted token's frequencies against p (chi
    squared of 23 degrees of freedom is above 75 with a probability below 1e-6)."""
    B, V = 40000, 24
    rng = np.random.RandomState(17)
    p = rng.dirichlet(np.full(V, 0.6)).astype(np.float32) + np.float32(2e-3)
    p /= p.sum()
    cand = rng.permutation(V)[:16].astype(np.int32)
    q = rng.dirichlet(np.full(16, 0.7)).astype(np.float32) + np.float32(1e-3)
    if replace:
        pick = rng.choice(16, (B, 3), p=q.astype(np.float64) / q.astype(np.float64).sum())
    else:
        pick = np.argsort(-(np.log(q) + rng.gumbel(size=(B, 16))), -1)[:, :3]
    tokens = np.zeros((B, 4), np.int32)
    tokens[:, 1:] = cand[pick]
    x = dict(p=np.broadcast_to(p, (B, 4, V)), tokens=tokens,
             parents=np.broadcast_to(np.array([-1, 0, 0, 0], np.int32), (B, 4)),
             cand=np.broadcast_to(cand, (B, 4, 16)), q=np.broadcast_to(q, (B, 4, 16)),
             u=(rng.randint(0, 1 << 24, (B, 4)) * 2.0**-24).astype(np.float32))
    path, n_path, nxt = call(x, replace)
    first = np.where(n_path > 1, tokens[np.arange(B), path[:, 1].clip(min=0)], nxt)
    seen = np.bincount(first, minlength=V)
    want = p.astype(np.float64) / p.astype(np.float64).sum() * B
    assert ((seen - want) ** 2 / want).sum() < 75
    assert 0.2 < (n_path > 1).mean() < 1


def test_captured_and_on_another_stream():
    x, y = make(3, 9, 500, False, seed=1), make(3, 9, 500, False, seed=2)
    t = {n: torch.from_numpy(a).cuda() for n, a in x.items()}
    out = outputs(3, 9)
    args = [t[n] for n in ("p", "tokens", "parents", "cand", "q", "u")]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dfl2.dfl2_tree_verify(*args, *out)
    s.synchronize()
    check(x, False, [o.cpu().numpy() for o in out])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfl2.dfl2_tree_verify(*args, *out)
    for n, a in y.items():
        t[n].copy_(torch.from_numpy(a))
    g.replay()
    torch.cuda.synchronize()
    check(y, False, [o.cpu().numpy() for o in out])
