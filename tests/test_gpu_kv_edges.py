"""GPU checks of the paged cache and its attention at the edges of their arguments, against the numpy oracle (oracle/kv.py).

The bounds are those of test_gpu_kv.py, whose cases these build on."""

import numpy as np
import pytest

from oracle import kv as okv
from test_gpu_kv import Case, _run_plan, _status, env  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1])
@pytest.mark.parametrize("reqs", [[(2, 6), (40, 3), (0, 4), (300, 1)], [(90, 131), (200, 1)]])
def test_attention_windows_wider_than_any_length(env, window, reqs):
    """Rows before the cache's first position among them, whose position minus the window does not fit 32 bits: as without a window."""
    c = Case(env, 128, 128, 32, 1, 8, "float16", reqs)
    want = c.run()
    c.check(*want)
    c.window = window
    out, lse = c.run()
    assert np.array_equal(out, want[0]) and np.array_equal(lse, want[1])
