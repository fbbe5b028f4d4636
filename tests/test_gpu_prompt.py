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


@pytest.mark.parametrize("ratio,heads", [(131, 1), (129, 1), (7, 3), (64, 2), (96, 1)])
def test_odd_groups(env, ratio, heads):
    """Groups of query heads that no row tile divides by, and more of them than a row tile has rows."""
    _check(env, [3, 150], heads, ratio, 64, "float16")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale", [0.125, -0.125])
def test_rising_scores(env, dtype, scale):
    """Scores that grow along the keys by hundreds: every tile moves the reference, in some rows and not in others."""
    def edit(q, k, v):
        n = k.shape[0]
        import torch
        ramp = torch.arange(n, device="cuda", dtype=torch.float32).view(n, 1, 1) / n
        k.copy_((k.float() * 0.1 + 14 * ramp).to(k.dtype))
        q.copy_((q.float() * 0.1 + 14 * torch.sign(q.float().mean(-1, keepdim=True))).to(q.dtype))
    _check(env, [900, 130], 1, 4, 64, dtype, scale=scale, edit=edit)
    _check(env, [900, 130], 2, 2, 128, dtype, scale=scale, edit=edit, window=200)
    _check(env, [600], 1, 2, 64, dtype, scale=scale, edit=edit, causal=False)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_huge_scores(env, dtype):
    """Scores past 2^26, where binary32 is coarser than 1: the largest one takes all the weight. q and k are powers of two, so that scores are
    exact, and the best two of a row differ by 2^20 at least."""
    sg, torch = env
    n, dim = 300, 64
    rng = np.random.default_rng(3)
    level = torch.tensor(rng.permutation(n) + 1, dtype=torch.float32, device="cuda")
    q, k = torch.zeros((n, 1, dim), device="cuda"), torch.zeros((n, 1, dim), device="cuda")
    q[:, 0, 0] = 2.0 ** 14
    k[:, 0, 0] = (level // 16) * 2.0 ** 10   # (both of few bits)
    k[:, 0, 1] = (level % 16) * 2.0 ** 6
    q[:, 0, 1] = 2.0 ** 14
    v = torch.randn((n, 1, dim), device="cuda")
    t = getattr(torch, dtype)
    q, k, v = q.to(t), k.to(t), v.to(t)
    out = sg.prompt_attention(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), 4.0)
    score = q.double()[:, 0] @ k.double()[:, 0].t() * 4.0
    best = score.masked_fill(torch.ones((n, n), device="cuda").triu(1).bool(), -1).argmax(1)
    assert torch.equal(out[:, 0], v[best, 0])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_what_is_not_seen_is_not_used(env, dtype, causal, window, what):
    """NaN and infinities in keys and values of other requests, of padding, of later tokens and of tokens before the window."""
    sg, torch = env
    lengths, pad, heads, ratio, dim = [200, 90, 131], [20, 0, 5], 2, 3, 64
    start = np.concatenate([[0], np.cumsum([a + b for a, b in zip(lengths, pad)])]).astype(np.int32)
    n, rng = int(start[-1]), np.random.default_rng(7)
    t = torch.tensor(rng.standard_normal((n, heads * (ratio + 2), dim)), dtype=getattr(torch, dtype), device="cuda")
    q, k, v = t[:, :heads * ratio], t[:, heads * ratio:heads * (ratio + 1)], t[:, heads * (ratio + 1):]
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    scale = dim ** -0.5
    clean = sg.prompt_attention(q, k, v, dev(start), scale, dev(lengths), causal=causal, window=window)
    odd = float(what)
    bad_v, bad_k = int(start[0]) + 150, int(start[2]) + 100  # a value of the first request, a key of the third
    k, v = k.clone(), v.clone()
    v[bad_v, 0, 5] = odd
    v[bad_v, 1, 60] = -odd
    k[bad_k, 1, 3] = odd
    k[bad_k, 1, 4] = float("nan")
    for r in range(3):
        for x in (k, v):
            x[start[r] + lengths[r]:start[r + 1]] = odd
    got = sg.prompt_attention(q, k, v, dev(start), scale, dev(lengths), causal=causal, window=window)
    for r in range(3):
        for i in range(lengths[r]):
            row = int(start[r]) + i
            sees = lambda at: start[r] <= at < start[r] + lengths[r] and (not causal or at - start[r] <= i) and (not window or i - (at - start[r]) < window)  # noqa: E731
            for a in range(heads * ratio):
                h, same = a // ratio, torch.ones(dim, dtype=torch.bool, device="cuda")
                if h == 1 and sees(bad_k):
                    assert torch.isnan(got[row, a]).all(), (r, i, a)
                    continue
                if sees(bad_v):
                    d = 5 if h == 0 else 60
                    same[d] = False
                    assert not torch.isfinite(got[row, a, d]), (r, i, a)
                assert torch.equal(got[row, a][same], clean[row, a][same]), (r, i, a)


def test_a_query_without_numbers(env):
    sg, torch = env
    t = torch.randn((100, 6, 64), device="cuda").half()
    start = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    clean = sg.prompt_attention(t[:, :4], t[:, 4:5], t[:, 5:], start, 0.125)
    q = t[:, :4].clone()
    q[17, 2, 9] = float("nan")
    got = sg.prompt_attention(q, t[:, 4:5], t[:, 5:], start, 0.125)
    assert torch.isnan(got[17, 2]).all()
    got[17, 2] = clean[17, 2]
    assert torch.equal(got, clean)


def test_strides(env):
    """Heads before tokens, rows of wider tensors, one token or head cut out of odd rows."""
    sg, torch = env
    rng = np.random.default_rng(2)
    n, heads, ratio, dim = 150, 2, 2, 64
    dense = lambda h: torch.tensor(rng.standard_normal((n, h, dim)), device="cuda").half()  # noqa: E731
    q, k, v = dense(4), dense(2), dense(2)
    start = torch.tensor([0, 100, n], dtype=torch.int32, device="cuda")
    want = sg.prompt_attention(q, k, v, start, 0.125)

    def heads_first(x):
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    def wide(x):
        y = torch.full((n, x.shape[1] + 1, dim + 8), float("nan"), dtype=x.dtype, device="cuda")
        y[:, 1:, 8:] = x
        return y[:, 1:, 8:]

    for f in (heads_first, wide):
        out = f(torch.zeros_like(q))
        sg.sgemv_prompt_attention(f(q), f(k), f(v), start, out, 0.125)
        assert torch.equal(out, want), f
    # out over q
    o = wide(q)
    sg.sgemv_prompt_attention(o, k, v, start, o, 0.125)
    assert torch.equal(o, want)
    # axes of length 1
    one = torch.randn((1, 4, 64), device="cuda").half()
    odd = torch.zeros((1, 4, 64 + 8), device="cuda").half()[:, :, :64]
    odd.copy_(one)
    s1 = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    a = sg.prompt_attention(one[:, :2], one[:, 2:3], one[:, 3:], s1, 0.125)
    b = sg.prompt_attention(odd[:, :2], odd[:, 2:3].as_strided((1, 1, 64), (7, 3, 1), odd[:, 2:3].storage_offset()), odd[:, 3:], s1, 0.125)
    assert torch.equal(a, b)
    assert torch.equal(a[0, 0], one[0, 3]) and torch.equal(a[0, 1], one[0, 3])  # a single token sees itself


@pytest.mark.parametrize("start,length,bad", [([0, 50, 20, 100], None, [1]), ([0, 50, 49, 49], None, [1]), ([-1, 50, 100, 100], None, [0]), ([0, 50, 60, 101], None, [2]),
                                              ([0, 50, 60, 100], [51, 10, 40], [0]), ([0, 50, 60, 100], [50, -1, 40], [1])])
def test_requests_out_of_range_are_reported(env, start, length, bad):
    sg, torch = env
    t = torch.randn((100, 4, 64), device="cuda").half()
    out, status = torch.full((100, 2, 64), 9.0, device="cuda").half(), torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sg.sgemv_prompt_attention(t[:, :2], t[:, 2:3], t[:, 3:], dev(start), out, 0.125, None if length is None else dev(length), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == sg.SGEMV_ERR_ARG
    for r in range(3):
        if r in bad:
            continue
        n = start[r + 1] - start[r] if length is None else length[r]
        at = slice(start[r], start[r] + n)
        # (requests that remain may share rows, where one between them is out of order: whose outputs those are is open)
        if n and not any(start[x] < start[r] + n and start[x + 1] > start[r] for x in range(3) if x != r and x not in bad):
            want = sg.prompt_attention(t[at, :2].contiguous(), t[at, 2:3].contiguous(), t[at, 3:].contiguous(), dev([0, n]), 0.125)
            assert torch.equal(out[at], want), r


@pytest.mark.parametrize("n_req", [301, 1001])
def test_overlapping_requests_do_nothing(env, n_req):
    """Starts that go back and forth: every second request is out of order, and the others are the same rows again and again."""
    sg, torch = env
    t = torch.randn((600, 4, 64), device="cuda").half()
    out, status = torch.full((600, 2, 64), 9.0, device="cuda").half(), torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 600] * (n_req // 2 + 1), dtype=torch.int32, device="cuda")[:n_req + 1].contiguous()
    sg.sgemv_prompt_attention(t[:, :2], t[:, 2:3], t[:, 3:], start, out, 0.125, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == sg.SGEMV_ERR_ARG and torch.all(out == 9.0)


def test_no_requests_and_no_tokens(env):
    sg, torch = env
    t = torch.randn((10, 4, 64), device="cuda").half()
    out = torch.full((10, 2, 64), 9.0, device="cuda").half()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for start in ([0], [0, 0, 0], [10, 10], [3, 3, 3, 3]):
        sg.sgemv_prompt_attention(t[:, :2], t[:, 2:3], t[:, 3:], torch.tensor(start, dtype=torch.int32, device="cuda"), out, 0.125, status=status)
    e = t[:0]
    sg.sgemv_prompt_attention(e[:, :2], e[:, 2:3], e[:, 3:], torch.tensor([0, 0], dtype=torch.int32, device="cuda"), out[:0], 0.125, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.all(out == 9.0)


def test_same_bits_alone_and_together(env):
    """A request's outputs depend neither on the others of its call nor on the run."""
    sg, torch = env
    rng = np.random.default_rng(11)
    lengths = [int(x) for x in rng.integers(0, 700, 37)]
    start = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    t = torch.tensor(rng.standard_normal((int(start[-1]), 12, 128)), device="cuda").bfloat16()
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v = t[:, :8], t[:, 8:10], t[:, 10:]
    all_out = sg.prompt_attention(q, k, v, dev(start), 0.1)
    for _ in range(3):
        assert torch.equal(sg.prompt_attention(q, k, v, dev(start), 0.1), all_out)
    for r in range(0, 37, 5):
        at = slice(int(start[r]), int(start[r + 1]))
        if lengths[r]:
            assert torch.equal(sg.prompt_attention(q[at], k[at], v[at], dev([0, lengths[r]]), 0.1), all_out[at]), r


def test_long_prompt(env):
    """One prompt of 9000 tokens, its last and some other rows against binary64."""
    sg, torch = env
    n, dim = 9000, 128
    t = torch.randn((n, 5, dim), device="cuda").half()
    lse = torch.empty((n, 3), device="cuda")
    out = sg.prompt_attention(t[:, :3], t[:, 3:4], t[:, 4:], torch.tensor([0, n], dtype=torch.int32, device="cuda"), dim ** -0.5, lse=lse)
    for i in (0, 1, 127, 128, 4095, 8191, 8999):
        s = t[i, :3].double() @ t[:i + 1, 3].double().t() * dim ** -0.5
        p = torch.softmax(s, 1)
        ref, weight = p @ t[:i + 1, 4].double(), p @ t[:i + 1, 4].double().abs()
        size = (t[i, :3].double().abs() @ t[:i + 1, 3].double().abs().t()).max(1, keepdim=True).values * dim ** -0.5
        tol = 2.0 ** -11 * ref.abs() + weight * (2.0 ** -11 + 2.0 ** -14 + 2 * dim * 2.0 ** -24 * size) + 2.0 ** -25
        assert ((out[i].double() - ref).abs() <= tol).all(), i
        assert ((lse[i].double() - torch.logsumexp(s, 1)).abs() <= 2.0 ** -18 + 2 * dim * 2.0 ** -24 * size[:, 0]).all(), i


def test_streams_and_graphs(env):
    """Two calls at once on two streams; captured, replayed with other inputs in the same place."""
    sg, torch = env
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    a, b = (torch.randn((700, 6, 64), device="cuda").half() for _ in range(2))
    start = dev([0, 300, 700])
    call = lambda t, o: sg.sgemv_prompt_attention(t[:, :4], t[:, 4:5], t[:, 5:], start, o, 0.125)  # noqa: E731
    outs = [torch.empty((700, 4, 64), device="cuda").half() for _ in range(4)]
    call(a, outs[0])
    call(b, outs[1])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            call(a, outs[2])
        with torch.cuda.stream(s2):
            call(b, outs[3])
    torch.cuda.synchronize()
    assert torch.equal(outs[2], outs[0]) and torch.equal(outs[3], outs[1])
    g = torch.cuda.CUDAGraph()
    x = a.clone()
    with torch.cuda.graph(g):
        call(x, outs[2])
        call(x, outs[3])
    x.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[2], outs[1]) and torch.equal(outs[3], outs[1])
