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


# (tokens, rows, k) that 2 to 8 CTAs share, with what is sent in a place of its own and where the ring was
CLUSTERS = {2: [(1, 18000, 2048), (64, 18000, 2048)], 3: [(20, 12500, 6000), (128, 12500, 4000)], 4: [(8, 9500, 4096), (40, 9500, 4096)], 5: [(30, 7600, 8192), (33, 7600, 8192)],
            6: [(1, 6200, 8192), (64, 6200, 8192)], 7: [(17, 5400, 8192), (50, 5400, 8192)], 8: [(32, 300, 20000), (64, 300, 20000)]}


@pytest.mark.parametrize("split", CLUSTERS)
def test_clusters_of_every_size(env, split):  # noqa: F811
    """The same bits again and again, alone and beside another call of another size of cluster on a stream of its own, and what binary64 says."""
    sg, torch = env
    calls = []
    for tokens, n, k in CLUSTERS[split] + CLUSTERS[10 - split if split != 5 else 8]:
        x, w = _x(torch, tokens, k, "float16", tokens), _x(torch, n, k, "float16", n, 0.3)
        y = _check_product(env, x, w, 16, "float16")
        calls.append((sg.fp4_quantize(w), sg.fp4_quantize(x), y, torch.empty_like(y)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(30):
        for (w, x, _, out), s in zip(calls, streams):
            sg.sgemv_fp4_product(*w, *x, out, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(out, y) for _, _, y, out in calls)
