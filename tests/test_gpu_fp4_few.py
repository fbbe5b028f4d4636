"""GPU parity of 4-bit products of few tiles whose columns many CTAs share, each with more stages than its ring has places, against binary64 (bounds:
test_gpu_fp4.py)."""

import pytest

from test_gpu_fp4 import _check_product, _x, env  # noqa: F401

pytestmark = pytest.mark.gpu

# (tokens, rows, k)
SPLIT = [(17, 4096, 16384), (20, 4096, 13000), (32, 5120, 11008), (30, 1000, 14000), (25, 300, 30000), (32, 7000, 16384)]
OTHER = [(1, 4096, 11008), (8, 300, 30000), (16, 4096, 11008), (20, 4096, 11008), (33, 4096, 11008), (64, 5120, 8192), (48, 300, 30000)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("tokens,n,k", SPLIT + OTHER)
def test_shared_columns(env, tokens, n, k, block):  # noqa: F811
    sg, torch = env
    _check_product(env, _x(torch, tokens, k, "bfloat16", tokens), _x(torch, n, k, "float16", n, 0.3), block, "bfloat16")
