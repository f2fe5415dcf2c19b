"""dfl2_cache_evict without a GPU: what is refused, and with which status."""
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_cache_abi import A, BAD_CACHES, INVALID, UNSUPPORTED, WORKSPACE, cache, lib  # noqa: F401


def evict(lib, c=None, B=2, rows=None, length=A, keep=40, sinks=4, recent=10, weight=A, kept=A, new=A,
          served=A, ws=A, n=1 << 40):
    return lib.dfl2_cache_evict(c or cache(), B, rows, length, keep, sinks, recent, weight, kept, new,
                                served, ws, n, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_the_cache_is_checked(lib, bad, status):
    assert evict(lib, cache(**bad)) == status


def test_refusals(lib):
    for kw, status in [
            (dict(B=0), INVALID), (dict(B=65536), UNSUPPORTED), (dict(keep=0), INVALID),
            (dict(keep=(1 << 30) + 1), UNSUPPORTED), (dict(sinks=-1), INVALID),
            (dict(recent=-1), INVALID), (dict(sinks=31), INVALID),
            (dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), INVALID), (dict(rows=A + 2), INVALID),
            *((dict([(n, None)]), INVALID) for n in ("length", "weight", "kept", "new", "served")),
            (dict(weight=A + 1), INVALID), (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE)]:
        assert evict(lib, **kw) == status, kw
        assert dfl2.dfl2_last_error()
    need = dfl2.dfl2_cache_evict_workspace_size(2, 40)
    assert evict(lib, n=need - 1) == WORKSPACE
    # (what is in range fails later, for want of a device or of its memory)
    assert evict(lib, n=need) not in (0, WORKSPACE, UNSUPPORTED)
    assert evict(lib, sinks=40, recent=0, n=need) not in (0, WORKSPACE, UNSUPPORTED)


def test_workspace_size_of_a_refused_shape_is_zero(lib):
    for bad in ((0, 4), (1, 0), (65536, 4), (1, -3)):
        assert dfl2.dfl2_cache_evict_workspace_size(*bad) == 0


def test_binding_refuses():
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    i, kept = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 5, dtype=torch.int32)
    w = torch.zeros(2, 48)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    ok = dict(cache=c, length=i, keep=5, sinks=1, recent=1, weight=w, kept=kept, new_length=i,
              served=i, ws=ws)
    for n, bad, why in [("weight", w.half(), TypeError), ("weight", w[:, :32], ValueError),
                        ("weight", w[:1], ValueError), ("weight", None, TypeError),
                        ("kept", kept[:, :4], ValueError), ("kept", kept.long(), TypeError),
                        ("length", i.long(), TypeError), ("served", kept, ValueError),
                        ("keep", 6, ValueError), ("keep", "5", TypeError), ("ws", None, TypeError)]:
        with pytest.raises(why):
            dfl2.dfl2_cache_evict(**{**ok, n: bad}, stream=1)
    with pytest.raises(dfl2.Dfl2Error):  # host memory
        dfl2.dfl2_cache_evict(**ok, stream=1)
