"""dfl2_tree_verify with drafting weights of any size."""
import numpy as np
import pytest

import draft_selection_gb300 as dfl2
from test_gpu_tree_verify import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-133, -126, -100, 100, 120, 123, 124])
@pytest.mark.parametrize("replace", [False, True])
def test_drafting_weights_of_any_size(power, replace):
    """q need not sum to 1: its sums here reach from below float32's smallest normal number, where
    weights have a few bits only, to 2^127 and more."""
    x = make(60, 21, 97, replace, seed=abs(power))
    q = x["q"].astype(np.float64)
    x["q"] = (q / q.sum(2, keepdims=True) * 15 * 2.0**power).astype(np.float32)
    assert np.isfinite(x["q"].astype(np.float64).sum(2)).all()
    check(x, replace, call(x, replace))
    assert dfl2.dfl2_device_error(clear=True) == 0
