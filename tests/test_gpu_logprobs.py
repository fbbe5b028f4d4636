"""GPU parity of sgemv_logprobs against binary64 (oracle/kv.py).

Bounds: a log-probability is (x - m) - ln S; S is a sum in 32 bits (relative error below 2^-18 for any order of at
most 2^18 terms a lane and a tree above, exp within 2^-21), so ln S is off by at most 2^-17, and the two subtractions
round once each (2^-23 of |x - m|). The entropy adds sum p (x - m), off by 2^-17 of sum p |x - m|."""

import numpy as np
import pytest

from oracle import kv as okv

pytestmark = pytest.mark.gpu


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


def _run(env, x, tokens=None, top=0, full=True):
    sg, torch = env
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = None if tokens is None else torch.tensor(tokens, dtype=torch.int32, device="cuda")
    got = sg.logprobs(x, t, top, full, status=st)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in got.items()}, int(st.item())


def _check(got, x, tokens, top):
    x = x.double().cpu().numpy()
    tok, lse, ent, top_tok, top_lp, lp = okv.logprobs(x, tokens, top)
    m = x.max(1)
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -17 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lp), lp, 0))
        def same(a, b, t):
            fin = np.isfinite(b)
            assert np.array_equal(np.isneginf(a), np.isneginf(b)) and not np.isnan(a).any()
            assert np.all(np.abs(a[fin] - b[fin]) <= np.broadcast_to(t, b.shape)[fin])
        same(got["lse"], lse, 2.0 ** -17 + 2.0 ** -23 * np.abs(np.where(np.isfinite(m), m, 0)))
        p = np.exp(lp)
        spread = np.where(p > 0, p * np.abs(lp), 0).sum(1)
        same(got["entropy"], ent, 2.0 ** -16 * (1 + spread))
        if "logp" in got:
            same(got["logp"], lp, tol)
        if tokens is not None:
            same(got["tok_logp"], tok, 2.0 ** -17 + 2.0 ** -22 * np.abs(np.where(np.isfinite(tok), tok, 0)))
        if top:
            assert np.array_equal(got["top_tok"], top_tok)
            same(got["top_logp"], top_lp, 2.0 ** -17 + 2.0 ** -22 * np.abs(np.where(np.isfinite(top_lp), top_lp, 0)))


def _logits(env, rows, vocab, dtype, seed, banned=0.0, spread=2.5, pad=0):
    _, torch = env
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, vocab + pad)) * spread
    if banned:
        x[rng.random(x.shape) < banned] = -np.inf
    return torch.tensor(x, dtype=torch.float32).to(getattr(torch, dtype)).cuda()[:, :vocab]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("rows,vocab,n_tok,top", [(1, 1, 1, 1), (3, 7, 2, 10), (2, 33, 0, 64), (5, 1000, 1, 5), (20, 32000, 1, 20),
                                                  (1, 50257, 3, 64), (300, 517, 1, 3), (2, 131075, 1, 64), (1, 262144, 1, 0),
                                                  (400, 4099, 1, 17)])
def test_logprobs_match_oracle(env, dtype, rows, vocab, n_tok, top):
    rng = np.random.default_rng(vocab)
    tokens = rng.integers(0, vocab, (rows, n_tok)).astype(np.int32) if n_tok else None
    if n_tok:
        tokens[-1, 0] = -1
    for banned, pad in ((0.0, 0), (0.6, 3)):  # pad: rows that start at odd addresses
        x = _logits(env, rows, vocab, dtype, rows + vocab, banned, pad=pad)
        got, status = _run(env, x, tokens, top)
        assert status == 0
        _check(got, x, tokens, top)


@pytest.mark.parametrize("vocab", [40, 5000, 140000])
def test_logprobs_ties_take_the_lowest_token(env, vocab):
    _, torch = env
    rng = np.random.default_rng(3)
    x = torch.tensor(np.round(rng.standard_normal((4, vocab))), dtype=torch.float32).half().cuda()
    x[1] = 0                                # every token the same
    x[2, ::2], x[2, 1::2] = 0.0, -0.0       # the two zeros are equal
    x[3] = -65504.0                         # the type's lowest value everywhere
    got, status = _run(env, x, None, 64)
    assert status == 0
    _check(got, x, None, 64)
    assert got["top_tok"][1].tolist()[:40] == list(range(40))


def test_logprobs_sharp_and_flat(env):
    _, torch = env
    x = _logits(env, 3, 30000, "float32", 1)
    x[0, 777] = 200.0                        # all weight on one token
    x[1] = x[1] * 1e-4 + 1e4                 # flat, far from zero
    x[2] = -3e38
    x[2, 5] = 3e38                           # differences that overflow binary32
    got, status = _run(env, x, np.array([[777], [0], [5]], dtype=np.int32), 4)
    assert status == 0
    assert got["tok_logp"][0, 0] == 0 and got["entropy"][0] >= 0 and got["entropy"][0] < 1e-30
    _check({k: v[:2] for k, v in got.items()}, x[:2], np.array([[777], [0]], dtype=np.int32), 4)
    assert got["tok_logp"][2, 0] == 0 and got["top_tok"][2].tolist() == [5, 0, 1, 2] and got["entropy"][2] == 0


def test_logprobs_banned_rows(env):
    _, torch = env
    for vocab in (50, 3000, 200000):
        x = _logits(env, 3, vocab, "float16", 9)
        x[1] = -float("inf")
        x[2] = -float("inf")
        x[2, vocab - 3] = 1.5
        tokens = np.array([[1], [2], [vocab - 3]], dtype=np.int32)
        got, status = _run(env, x, tokens, 6)
        assert status == 0
        _check(got, x, tokens, 6)
        assert got["entropy"][1] == 0 and np.isneginf(got["lse"][1]) and got["top_tok"][1].tolist() == list(range(6))
        assert got["tok_logp"][2, 0] == 0 and got["entropy"][2] == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("vocab", [60, 9001, 150000])
def test_logprobs_nonfinite_rows(env, bad, vocab):
    sg, torch = env
    x = _logits(env, 3, vocab, "float32", 2)
    clean, _ = _run(env, x, None, 5)
    x[1, vocab // 2] = bad
    got, status = _run(env, x, np.array([[0], [0], [vocab]], dtype=np.int32), 5)
    assert status in (sg.SGEMV_ERR_NONFINITE, sg.SGEMV_ERR_ARG)
    for k in ("lse", "entropy", "logp", "top_logp"):
        assert np.isnan(got[k][1]).all() and np.array_equal(got[k][[0, 2]], clean[k][[0, 2]]), k
    assert np.all(got["top_tok"][1] == -1)
    assert np.isnan(got["tok_logp"][1, 0]) and np.isnan(got["tok_logp"][2, 0]) and np.isfinite(got["tok_logp"][0, 0])


def test_logprobs_feed_the_beam_step(env):
    """The full rows are what sgemv_beam_step reads, and parts of the outputs can be left out."""
    sg, torch = env
    x = _logits(env, 4, 5000, "float16", 4)
    logp = torch.empty(4, 5000, device="cuda")
    sg.sgemv_logprobs(x, (None, None, None, None, None, logp))
    assert torch.allclose(logp, torch.log_softmax(x.float(), -1), atol=2e-5)
    with pytest.raises(sg.SgemvError) as e:
        sg.sgemv_logprobs(x.double(), (None,) * 6)
    assert e.value.code == sg.SGEMV_ERR_ARG
    with pytest.raises(ValueError):
        sg.sgemv_logprobs(x.t(), (None,) * 6)
    with pytest.raises(ValueError):
        sg.sgemv_logprobs(x, (None, torch.empty(3, device="cuda"), None, None, None, None))
    sg.sgemv_logprobs(x[:0], (None, logp.new_empty(0), None, None, None, None))


def test_logprobs_write_nothing_outside(env):
    sg, torch = env
    for rows, vocab, dtype in ((3, 1001, "float16"), (2, 70001, "bfloat16"), (200, 333, "float32")):
        x = _logits(env, rows, vocab, dtype, 8, pad=1)
        buf = torch.full((rows * vocab + 64,), 5.0, device="cuda")
        sizes = {"lse": rows, "entropy": rows}
        bufs = {k: torch.full((n + 64,), 5.0, device="cuda") for k, n in sizes.items()}
        sg.sgemv_logprobs(x, (None, bufs["lse"][32:32 + rows], bufs["entropy"][32:32 + rows], None, None,
                              buf[32:32 + rows * vocab].view(rows, vocab)))
        torch.cuda.synchronize()
        for b in (buf, *bufs.values()):
            assert torch.all(b[:32] == 5) and torch.all(b[-32:] == 5)
