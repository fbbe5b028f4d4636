"""GPU parity of prompt attention at the ends of its weights' range, against binary64: values near the end of bf16 under many tiles of keys, small ones,
and fp16 weights far below a row's largest.

Bound per output as in test_gpu_prompt.py: half a step of sum p |v| for the weights, 2^-14 for exp and the sums, 2 dim 2^-24 of a score's sum of
magnitudes, half a step for the output; in fp16 each key's weight is held to 2^-27 of the row's largest at best, which n keys make n 2^-27 max |v|."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF_STEP = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


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


def _check(env, q, k, v, dtype, scale, rows, causal=True, small=0.0):
    """One request; only some rows are compared. small: what the weights' lowest steps may add to an output."""
    sg, torch = env
    q, k, v = (t.to(getattr(torch, dtype)) for t in (q, k, v))
    n, heads_q, dim = q.shape
    ratio = heads_q // k.shape[1]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lse = torch.empty((n, heads_q), device="cuda")
    out = sg.prompt_attention(q, k, v, start, scale, lse=lse, causal=causal, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for i in rows:
        to = i + 1 if causal else n
        for a in range(heads_q):
            kk, vv = k[:to, a // ratio].double(), v[:to, a // ratio].double()
            s = kk @ q[i, a].double() * scale
            p = torch.softmax(s, 0)
            ref, weight = p @ vv, p @ vv.abs()
            size = float((kk.abs() @ q[i, a].double().abs()).max()) * abs(scale)
            noise = 2.0 ** -14 + 2 * dim * 2.0 ** -24 * size
            tol = HALF_STEP[dtype] * ref.abs() + weight * (HALF_STEP[dtype] + noise) + small
            err = (out[i, a].double() - ref).abs()
            assert (err <= tol).all(), (i, a, float((err / tol).max()), out[i, a, :4], ref[:4])
            total = float(torch.logsumexp(s, 0))
            assert abs(float(lse[i, a]) - total) <= 2.0 ** -18 + 2 * dim * 2.0 ** -24 * size + 2.0 ** -22 * abs(total), (i, a)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_values_near_the_end_of_bf16(env, dim, causal):
    """Later tiles have scores 8 powers of two above the first one's, none of which moves a reference by itself; v is up to 1.5 * 2^127."""
    sg, torch = env
    n, rng = 3000, np.random.default_rng(dim)
    q, k = torch.zeros((n, 2, dim), device="cuda"), torch.zeros((n, 1, dim), device="cuda")
    q[:, :, 0] = 1.0
    k[128:, 0, 0] = 8 * 0.6931
    v = torch.tensor(rng.choice([1.0, 1.25, 1.5], (n, 1, dim)), device="cuda").float() * 2.0 ** 127
    _check(env, q, k, v, "bfloat16", 1.0, (0, 127, 128, 500, 1400, 2999), causal)


@pytest.mark.parametrize("power", [-80, 100])
def test_values_of_any_size(env, power):
    """bf16 values far from 1: the errors are relative to them."""
    sg, torch = env
    t = torch.randn((700, 4, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    _check(env, t[:, :2], t[:, 2:3], t[:, 3:] * 2.0 ** power, "bfloat16", 0.3, (0, 1, 100, 128, 300, 699))


@pytest.mark.parametrize("bits", [15, 20, 24, 26])
def test_fp16_weights_far_below_the_largest(env, bits):
    """A first key that most of the weight goes to, and 30000 others around 2^-bits of it."""
    sg, torch = env
    n, dim, rng = 30000, 64, np.random.default_rng(bits)
    q, k = torch.zeros((n, 1, dim), device="cuda"), torch.zeros((n, 1, dim), device="cuda")
    q[:, 0, 0] = 1.0
    k[0, 0, 0] = bits * 0.6931
    k[1:, 0, 0] = torch.tensor(rng.uniform(-0.7, 0.7, n - 1), device="cuda").float()
    v = torch.tensor(rng.standard_normal((n, 1, dim)) + 1.0, device="cuda").float()
    _check(env, q, k, v, "float16", 1.0, (0, 127, 128, 1000, 29999), small=n * 2.0 ** -27 * float(v.abs().max()))
