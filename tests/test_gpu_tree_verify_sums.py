"""The running sums of dfl2_tree_verify's last draw over long rows."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_gpu_tree_verify import outputs

pytestmark = pytest.mark.gpu


def draw(p, u):
    """next_token of trees of one node each: p [B,1,V] on the GPU, u a number for each."""
    B = p.shape[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    out = outputs(B, 1)
    dfl2.dfl2_tree_verify(p, torch.zeros(B, 1, **i32), torch.full((B, 1), -1, **i32),
                          torch.arange(16, **i32).expand(B, 1, 16).contiguous(),
                          torch.zeros(B, 1, 16, device="cuda"),
                          torch.tensor(u, dtype=torch.float32, device="cuda").view(B, 1), *out)
    return out[2].tolist()


def test_a_flat_row_of_2_to_26_elements():
    """Two values, so that the exact sums are known: 2^-26 (1 + 0.9 2^-14) in the first half,
  XX
    fraction of 2^-6 of an element here; every draw below falls 2^-5 of one from the nearest
    border at least."""
    V = 1 << 26
    a = Fraction(float(np.float32(2.0**-26 * (1 + 0.9 * 2.0**-14))))
    b = Fraction(1, 1 << 26)
    total = (a + b) * (V // 2)
    p = torch.full((1, 1, V), float(b), device="cuda")
    p[:, :, :V // 2] = float(a)
    tried = 0
    for u in np.float32([0.0, 0.013, 0.1, 0.25, 0.3, 0.49, 0.5, 0.61, 0.75, 0.9, 1 - 2.0**-20]):
        t = Fraction(float(u)) * total
        half = a * (V // 2)
        at = t / a if t < half else V // 2 + (t - half) / b
        if u > 0 and min(at % 1, 1 - at % 1) < Fraction(1, 32):
            continue
        tried += 1
        assert draw(p, [u]) == [int(at)], u
    assert tried >= 8


@pytest.mark.parametrize("B,V", [(1, 262144), (30, 151937), (70, 40001), (140, 32003), (310, 131075)])
def test_draws_of_every_cluster_size(B, V):
    """One block a sequence where there are many, up to 16 where there are few; against sums in 64
    bits (a draw within 2^-36 of a border, of which there is about one in 2^36 / V draws, is left
    out)."""
    g = torch.Generator(device="cuda").manual_seed(V)
    p = torch.softmax(3 * torch.randn(B, 1, V, generator=g, device="cuda"), 2)
    u = torch.rand(B, generator=g, device="cuda")
    run = p[:, 0].double().cumsum(1)
    t = u.double() * run[:, -1]
    want = (run > t[:, None]).int().argmax(1)
    near = torch.minimum(run.gather(1, want[:, None])[:, 0] - t,
                         t - run.gather(1, (want - 1).clamp(min=0)[:, None])[:, 0])
    got = draw(p, u.tolist())
    sure = near > 2.0**-36
    assert sure.float().mean() > 0.99
    assert torch.equal(torch.tensor(got, device="cuda")[sure], want[sure])
