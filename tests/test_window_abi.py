"""dfl2_window_attn without a GPU: what is refused, and with which status."""
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_cache_abi import A, INVALID, QS, S3, UNSUPPORTED, cache, lib  # noqa: F401


def attn(lib, c=None, q=A, qs=QS, layer=0, B=2, T=4, hq=8, length=A, mask=A, depth=A, sinks=4,
         window=100, scale=0.1, out=A, os_=QS, lse=A, ws=A, n=1 << 40):
    return lib.dfl2_window_attn(q, qs, c or cache(), layer, B, T, hq, None, length, None, mask, depth,
                                sinks, window, scale, out, os_, lse, ws, n, None)


def test_refusals(lib):
    for kw, status in [
            (dict(window=0), INVALID), (dict(window=-5), INVALID), (dict(sinks=-1), INVALID),
            (dict(window=(1 << 30) + 1), UNSUPPORTED), (dict(sinks=(1 << 30) + 1), UNSUPPORTED),
            (dict(depth=None), INVALID), (dict(depth=A + 2), INVALID),
            (dict(mask=None, depth=A + 1), INVALID), (dict(B=0), INVALID), (dict(T=257), UNSUPPORTED),
            (dict(layer=2), INVALID), (dict(q=None), INVALID), (dict(length=None), INVALID),
            (dict(out=A + 4), INVALID), (dict(qs=S3(4096, 1028, 128)), INVALID),
            (dict(scale=float("nan")), INVALID), (dict(c=cache(dtype=0)), UNSUPPORTED),
            (dict(c=cache(page_size=12)), UNSUPPORTED), (dict(c=cache(k=None)), INVALID)]:
        assert attn(lib, **kw) == status, kw
        assert dfl2.dfl2_last_error()
    # (what is in range fails later, for want of a device or of its memory)
    for kw in (dict(), dict(mask=None, depth=None), dict(mask=None), dict(window=1, sinks=0),
               dict(window=1 << 30, sinks=1 << 30)):
        assert attn(lib, **kw) not in (0, UNSUPPORTED), kw
        assert "window" not in dfl2.dfl2_last_error() and "depth" not in dfl2.dfl2_last_error()


def test_binding_refuses():
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    ij = torch.zeros(2, 3, dtype=torch.int32)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.float16)
    call = dfl2.dfl2_window_attn
    with pytest.raises(ValueError):
        call(q, c, 0, i, None, i, 4, 100, q, i, stream=1)          # depth [2]
    with pytest.raises(TypeError):
        call(q, c, 0, i, None, ij.long(), 4, 100, q, i, stream=1)
    with pytest.raises(TypeError):
        call(q, c, 0, i, None, ij, "4", 100, q, i, stream=1)
    with pytest.raises(OverflowError):
        call(q, c, 0, i, None, ij, 4, 1 << 40, q, i, stream=1)
    with pytest.raises(ValueError):
        call(q.float(), c, 0, i, None, ij, 4, 100, q.float(), i, stream=1)
    with pytest.raises(dfl2.Dfl2Error, match="depth"):
        call(q, c, 0, i, torch.zeros(2, 3, 1, dtype=torch.int32), None, 4, 100, q, i, stream=1)
    with pytest.raises(dfl2.Dfl2Error, match="window"):
        call(q, c, 0, i, None, None, 4, 0, q, i, stream=1)
