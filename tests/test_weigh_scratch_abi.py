"""dfl2_cache_weigh's workspace may be left out of a call, but not be None; without a GPU."""
import pytest
import torch

import draft_selection_gb300 as dfl2
from test_cache_abi import lib  # noqa: F401


def test_left_out(lib):
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    x = (torch.zeros(2, 3, 4, 64, dtype=torch.float16), torch.zeros(2, 3, 4), c, 0,
         torch.zeros(2, dtype=torch.int32), torch.zeros(2, 48))
    with pytest.raises(dfl2.Dfl2Error):  # host memory, as with a workspace
        dfl2.dfl2_cache_weigh(*x, stream=1)
    with pytest.raises(dfl2.Dfl2Error):
        dfl2.dfl2_cache_weigh(*x, first=True, path=torch.zeros(2, 3, dtype=torch.int32), stream=1)
    with pytest.raises(TypeError):
        dfl2.dfl2_cache_weigh(*x, None, stream=1)
    with pytest.raises(ValueError):  # what else is wrong is said first
        dfl2.dfl2_cache_weigh(*x[:5], torch.zeros(2, 40), stream=1)
