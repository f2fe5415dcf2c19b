"""dfl2_tree_verify without a GPU: what is refused, and with which status."""
import pytest
import torch

import draft_selection_gb300 as dfl2
from draft_selection_gb300 import build as dbuild

INVALID, UNSUPPORTED = 1, 2
A = 0x10000  # an aligned stand-in address: never dereferenced by these tests


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dfl2.load()


def verify(lib, p=A, B=2, T=4, V=100, tokens=A, parents=A, count=A, cand=A, q=A, u=A, path=A, n=A,
           nxt=A):
    return lib.dfl2_tree_verify(p, B, T, V, tokens, parents, count, cand, q, u, 0, path, n, nxt, None)


def test_refusals(lib):
    for kw, status in [
            (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(V=0), INVALID),
            (dict(B=65536), UNSUPPORTED), (dict(T=257), UNSUPPORTED),
            (dict(V=(1 << 30) + 1), UNSUPPORTED), (dict(p=A + 4), INVALID),
            (dict(cand=A + 8), INVALID), (dict(count=A + 2), INVALID), (dict(q=A + 1), INVALID),
            *((dict([(n, None)]), INVALID)
              for n in ("p", "tokens", "parents", "cand", "q", "u", "path", "n", "nxt"))]:
        assert verify(lib, **kw) == status, kw
        assert dfl2.dfl2_last_error()
    # (what is in range fails later, for want of a device or of its memory)
    assert verify(lib) not in (0, UNSUPPORTED)
    assert verify(lib, count=None) not in (0, UNSUPPORTED)


def test_binding_refuses():
    B, T, V = 2, 3, 50
    i = torch.zeros(B, dtype=torch.int32)
    ij = torch.zeros(B, T, dtype=torch.int32)
    x = dict(p=torch.zeros(B, T, V), tokens=ij, parents=ij, cand_idx=torch.zeros(B, T, 16).int(),
             q=torch.zeros(B, T, 16), u=torch.zeros(B, T), path=ij, n_path=i, next_token=i)
    for n, bad, why in [
            ("p", x["p"].half(), TypeError), ("p", x["p"][0], ValueError),
            ("p", torch.zeros(B, V, T).transpose(1, 2), ValueError), ("p", None, TypeError),
            ("tokens", ij.long(), TypeError), ("parents", ij[:, :2], ValueError),
            ("cand_idx", x["cand_idx"][:, :, :8], ValueError), ("q", x["q"].double(), TypeError),
            ("q", torch.zeros(B, T, 15), ValueError), ("u", torch.zeros(B), ValueError),
            ("path", i, ValueError), ("n_path", ij, ValueError), ("next_token", i.long(), TypeError)]:
        with pytest.raises(why):
            dfl2.dfl2_tree_verify(**{**x, n: bad}, stream=1)
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_verify(**x, count=ij, stream=1)
    with pytest.raises(dfl2.Dfl2Error):     # host memory
        dfl2.dfl2_tree_verify(**x, stream=1)
