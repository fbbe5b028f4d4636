"""GPU parity of prompt attention where scores are infinite or no numbers: infinity or NaN among those that a row sees makes its output and its
log-sum-exp NaN, minus infinity beside finite ones has weight 0, and a row that sees nothing else is NaN (no row is empty: each sees itself).

The reference is the softmax in binary64. Bound per output as in test_gpu_prompt.py: half a step for the weights, 2^-14 for exp and the sums, 2 dim
2^-24 of a score's sum of magnitudes, half a step for the output; log-sum-exp 2^-18 + 2 dim 2^-24 of the same + 2^-22 of itself."""

import numpy as np
import pytest

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


def _inputs(torch, n, heads_q, heads, dim, dtype, seed):
    rng = np.random.default_rng(seed)
    t = rng.standard_normal((n, heads_q + 2 * heads, dim))
    t = np.where(np.abs(t) < 0.01, 0.01, t)  # (0 times infinity is left to the queries' test)
    t = torch.tensor(t, dtype=getattr(torch, dtype), device="cuda")
    return t[:, :heads_q], t[:, heads_q:heads_q + heads], t[:, heads_q + heads:]


def _run(env, q, k, v, start, scale, **kw):
    sg, torch = env
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sgemv_prompt_attention(q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), out, scale, lse=lse, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse


def _check(torch, q, k, v, out, lse, dtype, scale, causal, window):
    """One request. Rows whose scores hold infinity or NaN, or no number above -infinity: NaN. The others: the softmax in binary64."""
    n, heads_q, dim = q.shape
    ratio = heads_q // k.shape[1]
    i = torch.arange(n, device="cuda")
    seen = torch.ones((n, n), dtype=torch.bool, device="cuda")
    if causal:
        seen = i[:, None] >= i[None]
    if window:
        seen = seen & (i[:, None] - i[None] < window)
    empty = 0
    for a in range(heads_q):
        qq, kk, vv = q[:, a].double(), k[:, a // ratio].double(), v[:, a // ratio].double()
        s = (qq @ kk.t() * scale).masked_fill(~seen, -float("inf"))
        nan = (s.isnan() | (s == float("inf"))).any(1) | (s == -float("inf")).all(1)
        empty += int(((s == -float("inf")).all(1)).sum())
        assert out[nan, a].isnan().all() and lse[nan, a].isnan().all(), (a, out[nan, a].isnan().all(1), lse[nan, a])
        p = torch.softmax(s[~nan], 1)
        total = torch.logsumexp(s[~nan], 1)
        ref, weight = p @ vv, p @ vv.abs()
        size = (qq.abs() @ kk.abs().nan_to_num(posinf=0.0).t()).max(1, keepdim=True).values[~nan] * abs(scale)
        noise = 2.0 ** -14 + 2 * dim * 2.0 ** -24 * size
        tol = HALF_STEP[dtype] * ref.abs() + weight * (HALF_STEP[dtype] + noise) + TINY[dtype]
        err = (out[~nan, a].double() - ref).abs()
        assert (err <= tol).all(), (a, float((err / tol).max()))
        terr = (lse[~nan, a].double() - total).abs()
        assert (terr <= 2.0 ** -18 + 2 * dim * 2.0 ** -24 * size[:, 0] + 2.0 ** -22 * total.abs()).all(), a
    return empty


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 50), (False, 0)])
@pytest.mark.parametrize("at", [0, 5, 130, 299])
@pytest.mark.parametrize("sign", [1, -1])
def test_an_infinite_key(env, dtype, dim, causal, window, at, sign):
    """One element of one key, of either sign: half of the rows that see it have a score of infinity, the others of minus infinity."""
    sg, torch = env
    q, k, v = _inputs(torch, 300, 4, 2, dim, dtype, at)
    k = k.clone()
    k[at, 1, 7] = sign * float("inf")
    empty = 0
    for scale in (dim ** -0.5, -0.2):
        out, lse = _run(env, q, k, v, [0, 300], scale, causal=causal, window=window)
        empty += _check(torch, q, k, v, out, lse, dtype, scale, causal, window)
    # the scales have different signs, so that of the two query heads of a row that sees that key alone each is empty once
    assert empty == (2 if window == 1 or (causal and at == 0) else 0)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("value", ["inf", "-inf", "nan"])
@pytest.mark.parametrize("causal", [True, False])
def test_a_query_without_numbers(env, dtype, value, causal):
    """Output and log-sum-exp of such a row are NaN, whatever signs its scores have; the others are what they are without it."""
    sg, torch = env
    q, k, v = _inputs(torch, 300, 4, 2, 64, dtype, 3)
    q, k = q.clone(), k.clone()
    k[:, 0, 9] = -k[:, 0, 9].abs()  # (with infinity, all of KV head 0's scores are minus infinity)
    rows = (0, 17, 198, 200, 299)
    for i in rows:
        q[i, i % 4, 9] = float(value)
    out, lse = _run(env, q, k, v, [0, 200, 300], 0.125, causal=causal)
    for i in rows:
        assert out[i, i % 4].isnan().all() and lse[i, i % 4].isnan(), i
    for at in (slice(0, 200), slice(200, 300)):
        _check(torch, q[at], k[at], v[at], out[at], lse[at], dtype, 0.125, causal, 0)
    assert int(lse.isnan().sum()) == len(rows)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_leave_binary32(env, dim, sign):
    """Finite bf16 numbers whose product does not fit 32 bits: a first token that has no other score, and rows that have."""
    sg, torch = env
    n = 140
    q, k, v = _inputs(torch, n, 1, 1, dim, "bfloat16", 1)
    q, k = q.clone(), k.clone()
    q[0, 0], k[0, 0] = 0.0, 0.0
    q[0, 0, 3], k[0, 0, 3] = 2.0 ** 100, sign * 2.0 ** 100
    q[1:, 0, 3] = q[1:, 0, 3].abs()
    q[139, 0, 3] = 2.0 ** 100
    out, lse = _run(env, q, k, v, [0, n], 1.0)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert torch.isfinite(out[1:139]).all() and torch.isfinite(lse[1:139]).all()
    if sign > 0:  # the first key takes all the weight, but of the last row, whose score with it leaves binary32
        assert torch.equal(out[1:139, 0], v[0, 0].expand(138, dim))
        assert out[139].isnan().all() and lse[139].isnan().all()
    else:
        at = slice(1, 139)
        _check(torch, q[at], k[at], v[at], out[at], lse[at], "bfloat16", 1.0, True, 0)
        assert torch.isfinite(out[139]).all() and torch.isfinite(lse[139])
