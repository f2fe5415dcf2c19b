"""dfl2_cache_weigh without a GPU: what is refused, and with which status."""
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_cache_abi import A, BAD_CACHES, INVALID, QS, S3, UNSUPPORTED, cache, lib  # noqa: F401


def weigh(lib, c=None, q=A, qs=QS, lse=A, layer=0, B=2, T=4, hq=8, rows=None, length=A, path=A,
          n_path=A, scale=0.1, first=0, weight=A, ws=A, n=1 << 40):
    return lib.dfl2_cache_weigh(q, qs, lse, c or cache(), layer, B, T, hq, rows, length, path, n_path,
                                scale, first, weight, ws, n, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_the_cache_is_checked(lib, bad, status):
    assert weigh(lib, cache(**bad)) == status


def test_refusals(lib):
    for kw, status in [
            (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(hq=0), INVALID), (dict(hq=6), INVALID),
            (dict(T=257), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(hq=129 * 4), UNSUPPORTED),
            (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(q=None), INVALID),
            (dict(q=A + 8), INVALID), (dict(lse=None), INVALID), (dict(lse=A + 2), INVALID),
            (dict(length=None), INVALID), (dict(weight=None), INVALID), (dict(weight=A + 1), INVALID),
            (dict(path=A + 2), INVALID), (dict(n_path=A + 1), INVALID), (dict(rows=A + 1), INVALID),
            (dict(qs=None), INVALID), (dict(qs=S3(4096, 1028, 128)), INVALID),
            (dict(qs=S3(4096, -1024, 128)), INVALID), (dict(scale=float("nan")), INVALID),
            (dict(c=cache(dtype=0)), UNSUPPORTED), (dict(c=cache(head_dim=96)), UNSUPPORTED),
            (dict(c=cache(slot_stride=0)), UNSUPPORTED)]:
        assert weigh(lib, **kw) == status, kw
        assert dfl2.dfl2_last_error()
    # (what is in range fails later, for want of a device or of its memory)
    for kw in (dict(), dict(path=None), dict(n_path=None), dict(path=None, n_path=None, first=1)):
        assert weigh(lib, **kw) not in (0, UNSUPPORTED)


def test_binding_refuses():
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    i, ij = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.float16)
    w, lse = torch.zeros(2, 48), torch.zeros(2, 3, 4)
    ok = dict(q=q, lse=lse, cache=c, layer=0, length=i, weight=w, ws=torch.zeros(4096).byte())
    for n, bad, why in [("q", q.float(), ValueError), ("q", q[0], ValueError),
                        ("q", q.transpose(2, 3), ValueError), ("lse", lse.half(), TypeError),
                        ("lse", lse[:, :2], ValueError), ("lse", None, TypeError),
                        ("weight", w[:, :40], ValueError), ("weight", w.double(), TypeError),
                        ("length", ij, ValueError), ("path", i, ValueError),
                        ("n_path", i.long(), TypeError), ("layer", "0", TypeError),
                        ("ws", None, TypeError), ("scale", "x", TypeError)]:
        with pytest.raises(why):
            dfl2.dfl2_cache_weigh(**{**ok, n: bad}, stream=1)
    with pytest.raises(dfl2.Dfl2Error):  # host memory
        dfl2.dfl2_cache_weigh(**ok, stream=1)
