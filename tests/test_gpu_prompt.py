"""GPU parity of attention over packed prompts against the numpy oracle (oracle/prompt.py).

Bound per output: the weights of a row are rounded to the type of V before they meet it (half a step of sum p |v|, and 2^-14 for exp and the
sums), a score is a sum of dim products in 32 bits (2 dim 2^-24 of the sum of their magnitudes), and the output is rounded once."""

import numpy as np
import pytest

from oracle import prompt as op

pytestmark = pytest.mark.gpu

HALF_STEP = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


@pytest.fixture(scope="module")
def env():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return sg, torch


def _check(env, lengths, heads, ratio, dim, dtype, causal=True, window=0, scale=None, pad=None, seed=0, edit=None):
    sg, torch = env
    rng = np.random.default_rng(seed + sum(lengths) + heads)
    pad = pad or [0] * len(lengths)
    start = np.concatenate([[0], np.cumsum([a + b for a, b in zip(lengths, pad)])]).astype(np.int32)
    n, hq = int(start[-1]) + (3 if any(pad) else 0), heads * ratio
    t = torch.tensor(rng.standard_normal((n, hq + 2 * heads, dim)), dtype=getattr(torch, dtype), device="cuda")
    q, k, v = t[:, :hq], t[:, hq:hq + heads], t[:, hq + heads:]
    if edit is not None:
        edit(q, k, v)
    length = None if not any(pad) else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = torch.full((n, hq, dim), 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n, hq), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = dim ** -0.5 if scale is None else scale
    sg.sgemv_prompt_attention(q, k, v, torch.tensor(start, device="cuda"), out, scale, length, lse, causal, window, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    ref, rlse, weight, size = op.attention(f(q), f(k), f(v), start.tolist(), lengths if any(pad) else None, scale, causal, window)
    used = ~np.isnan(rlse)
    got, glse = f(out), f(lse)
    assert np.all(got[~used] == 9.0) and np.all(glse[~used] == 9.0)  # rows of no request are left as they were
    noise = 2.0 ** -14 + 2 * dim * 2.0 ** -24 * size[..., None]
    tol = HALF_STEP[dtype] * np.abs(ref) + weight * (HALF_STEP[dtype] + noise) + TINY[dtype]
    err = np.abs(got - ref)
    bad = used[..., None] & ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), float(np.nanmax(err / tol)))
    terr = np.abs(glse - rlse)
    assert np.all((terr <= 2.0 ** -18 + 2 * dim * 2.0 ** -24 * size + 2.0 ** -22 * np.abs(rlse))[used]), float(np.nanmax(terr))
    return out


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lengths,heads,ratio", [([1], 1, 1), ([7], 2, 4), ([128], 1, 1), ([129], 1, 2), ([300], 2, 1), ([64, 0, 1, 65, 31], 2, 4),
                                                 ([257, 140], 1, 5), ([700], 1, 3), ([33], 1, 128), ([2], 1, 200)])
def test_causal(env, lengths, heads, ratio, dim, dtype):
    _check(env, lengths, heads, ratio, dim, dtype)


@pytest.mark.parametrize("window", [1, 5, 100, 128, 129, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("ratio", [1, 4])
def test_window(env, window, ratio):
    _check(env, [600, 20, 333], 1, ratio, 64, "float16", window=window)


@pytest.mark.parametrize("dim", [64, 128])
def test_all_to_all(env, dim):
    _check(env, [300, 1, 129, 128, 0, 64], 2, 2, dim, "bfloat16", causal=False)


@pytest.mark.parametrize("causal", [True, False])
def test_padded(env, causal):
    _check(env, [100, 0, 129, 1], 2, 2, 64, "float16", causal=causal, pad=[28, 5, 127, 0])


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 30.0])
def test_scales(env, scale):
    _check(env, [200, 150], 1, 2, 64, "bfloat16", scale=scale)


def test_many_requests(env):
    rng = np.random.default_rng(5)
    _check(env, [int(x) for x in rng.integers(0, 4, 1000)], 1, 2, 64, "float16")
