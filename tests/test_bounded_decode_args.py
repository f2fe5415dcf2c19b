"""The example that decodes in a cache of bounded size takes no window past what eviction keeps."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import bounded_decode as ex  # noqa: E402


@pytest.mark.parametrize("window,recent", [(32, 24), (26, 24), (2, 0)])
def test_a_window_past_the_recent_positions_is_refused(window, recent):
    with pytest.raises(ValueError, match="window"):
        ex.decode(1, 1, window=window, recent=recent)
