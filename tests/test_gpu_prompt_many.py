"""GPU parity of prompt attention over more requests than the kernel has threads, of up to some hundred tokens each, some of them empty, against the numpy
oracle (bounds: test_gpu_prompt.py)."""

import numpy as np
import pytest

from test_gpu_prompt import _check, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _lengths(n_req, longest, seed):
    rng = np.random.default_rng(seed)
    lengths = np.exp(rng.uniform(0, np.log(longest + 1), n_req)).astype(int)
    lengths[rng.random(n_req) < 0.1] = 0
    lengths[:: n_req // 3] = longest
    return [int(x) for x in lengths]


@pytest.mark.parametrize("n_req,longest", [(384, 300), (385, 300), (500, 290), (1200, 140)])
@pytest.mark.parametrize("dim,dtype,heads,ratio", [(64, "float16", 1, 2), (128, "bfloat16", 2, 1)])
def test_causal(env, n_req, longest, dim, dtype, heads, ratio):  # noqa: F811
    _check(env, _lengths(n_req, longest, n_req), heads, ratio, dim, dtype)


@pytest.mark.parametrize("n_req", [384, 600])
@pytest.mark.parametrize("how", ["all to all", "window", "padded", "padded, all to all"])
def test_other_forms(env, n_req, how):  # noqa: F811
    rng = np.random.default_rng(n_req)
    pad = [int(x) for x in rng.integers(0, 20, n_req)] if "padded" in how else None
    _check(env, _lengths(n_req, 270, 5), 1, 3, 64, "float16", causal="all" not in how, window=50 if how == "window" else 0, pad=pad)
