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


FACTORS = [1e-30, 1e-6, 1e8, 1e30, 2.0 ** 117, 2.0 ** -117]


def _check_rows(c, out, lse):
    """Case.check, and where a row's largest score stands out by more than what a score may be off: that key's values alone."""
    c.check(out, lse)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    q, cache = c.q.double().cpu().numpy(), c.cache.cpu().numpy()
    page, ratio, sharp = c.L.page, c.q.shape[1] // c.L.heads, 0
    for r, (n, new) in enumerate(c.reqs):
        j = np.arange(n)
        k, v, kmag, vmag = okv.values(c.O, cache, c.table[r][j // page].astype(np.int64) * page + j % page, 0)
        for i in range(new):
            for a in range(ratio):
                tok, see = c.starts[r] + i, n - new + i + 1
                s = k[:see] @ q[tok, a] * c.scale
                off = 4 * c.L.dim * 2.0 ** -24 * (kmag[:see] @ np.abs(q[tok, a])).max() * c.scale
                best = int(s.argmax())
                if see > 1 and s[best] - np.partition(s, -2)[-2] <= off + 40:
                    continue
                sharp += 1
                assert np.all(np.abs(out[tok, a] - v[best]) <= 2.0 ** -8 * np.abs(v[best]) + 2.0 ** -10 * vmag[best])
    return sharp


@pytest.mark.parametrize("shape", [(64, 64, 32, 1, 8), (128, 64, 32, 1, 8), (128, 128, 16, 1, 8), (256, 64, 32, 1, 4), (256, 128, 16, 1, 4)])
@pytest.mark.parametrize("reqs", [[(260, 1), (40, 1)], [(90, 20), (140, 3)]])
def test_attention_rows_of_any_size(env, shape, reqs):
    """Finite bf16 queries of very different sizes in one tile: each row as if it were alone."""
    c = Case(env, *shape, "bfloat16", reqs)
    good = c.run()
    other = np.ones(good[1].shape, dtype=bool)
    for n, f in enumerate(FACTORS):
        at = n % len(c.q), n % c.q.shape[1]
        c.q[at] *= f
        other[at] = False
    out, lse = c.run()
    assert np.array_equal(out[other], good[0][other]) and np.array_equal(lse[other], good[1][other])
    assert _check_rows(c, out, lse) > 0


@pytest.mark.parametrize("shape", [(64, 64, 32, 1, 8), (128, 64, 32, 1, 8), (128, 128, 16, 1, 8)])
@pytest.mark.parametrize("sign", [1, -1])
def test_attention_large_chunk_rows_of_any_size(env, shape, sign):
    """The same in a prompt chunk of 1048 rows, with scales of either sign."""
    c = Case(env, *shape, "bfloat16", [(190, 131), (60, 1)])
    good = c.run()
    other = np.ones(good[1].shape, dtype=bool)
    for n in range(24):
        at = (7 * n) % 131, n % 8
        c.q[at] *= FACTORS[n % 6]
        other[at] = False
    plain = c.run()
    assert np.array_equal(plain[0][other], good[0][other]) and np.array_equal(plain[1][other], good[1][other])
    if sign < 0:  # the signs of scale and queries cancel
        c.q *= -1
        c.scale = -c.scale
        out, lse = c.run()
        assert np.array_equal(out, plain[0]) and np.array_equal(lse, plain[1])
        return
    assert _check_rows(c, *plain) > 0


@pytest.mark.parametrize("shape", [(64, 64, 32, 1, 4), (128, 64, 16, 1, 4), (128, 128, 64, 1, 4), (256, 64, 32, 1, 4), (256, 128, 16, 1, 4)])
@pytest.mark.parametrize("new", [1, 3])
def test_attention_keys_without_values(env, shape, new):
    """Keys that take nearly all the weight and whose V is zero (its groups have scale 1) beside small values: what is left of those
    is the output, as exact as ever."""
    sg, torch = env
    c = Case(env, *shape, "bfloat16", [(1000, new)], vscale=1e-3)
    dim, page = c.L.dim, c.L.page
    # a key so far along every query that its score is 17 above the others' usual ones
    k = torch.linalg.lstsq(c.q.float().reshape(-1, dim).cpu(), torch.full((4 * new, 1), 17 / c.scale)).solution
    j = np.arange(5, 1000 - new, 32)
    slots = torch.tensor(c.table[0][j // page].astype(np.int64) * page + j % page, device="cuda")
    k = k.view(1, 1, dim).bfloat16().cuda().expand(len(j), 1, dim)
    sg.sgemv_kv_append(c.L, c.cache, k, torch.zeros_like(k), slots)
    out, lse = c.run()
    c.check(out, lse)
    # and by the bound without its last term, which is larger than these outputs
    ref, _, weight, size = okv.attention(c.O, c.cache.cpu().numpy(), c.q.float().cpu().numpy(), c.starts, [1000], c.table, c.scale)
    score = 2 * dim * 2.0 ** -24 * size[..., None]
    assert np.all(np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + weight * (2.0 ** -11 + 2.0 ** -14 + score))


def test_attention_whole_cache_without_values(env):
    """V zero everywhere: zeros, and the softmax's sum as it should be."""
    sg, torch = env
    for shape in ((128, 128, 16, 1, 4), (256, 64, 16, 1, 4)):
        c = Case(env, *shape, "float16", [(200, 1), (70, 5)], vscale=0.0)
        out, lse = c.run()
        c.check(out, lse)
        assert not out.any()


@pytest.mark.parametrize("shape", [(64, 64, 16, 2, 4, "float16"), (128, 128, 16, 1, 8, "bfloat16"), (128, 64, 32, 1, 8, "float16"),
                                   (256, 128, 16, 1, 2, "float16"), (128, 128, 128, 1, 8, "float16")])
@pytest.mark.parametrize("window", [1, 20, 75])
@pytest.mark.parametrize("new", [1, 5, 140])
def test_attention_window_behind_freed_pages(env, shape, window, new):
    """Pages that lie before everything that a row sees are free (-1 in the table): they are not looked at, and nothing is reported."""
    c = Case(env, *shape, [(300 + a, new) for a in (0, 9, 17, 31)], window=window)
    want = c.run()
    c.check(*want)
    for r, (n, _) in enumerate(c.reqs):
        c.table[r, :max(0, n - new - window + 1) // c.L.page] = -1
    out, lse = c.run()  # (asserts that the status stays 0)
    assert np.array_equal(out, want[0]) and np.array_equal(lse, want[1])


def test_plan_reports_bad_ids_of_released_pages(env):
    """A page id outside the cache in a block that a request gives up is reported by the step that finds it."""
    sg, _ = env
    for bad in (-1, 4):
        table = np.array([[2, bad, 1], [3, -1, -1]], dtype=np.int32)
        got, status = _run_plan(env, [40, 3], [5, 3], [0, 1], table, [0, -9, -9, -9], 1, 16, 1)
        assert status == sg.SGEMV_ERR_ARG
        assert got[3].tolist() == [3 * 16 + 3] and got[1][0] == 3 and got[6][:3].tolist() == [0, bad, 1]
    got, status = _run_plan(env, [40, 3], [5, 3], [0, 1], np.array([[2, 0, 1], [3, -1, -1]], dtype=np.int32), [-9] * 4, 0, 16, 1)
    assert status == 0 and got[6][:2].tolist() == [0, 1]


def test_strides_of_single_tokens_and_heads_are_not_used(env):
    """An axis of length 1 may have any stride."""
    sg, torch = env
    L = sg.sgemv_kv_layout_query(1, 128, 128, 16, 4)
    st = _status(torch)
    base = torch.randn(4000, device="cuda").half()
    for shape, strides in (((1, 1, 128), (129, 131, 1)), ((5, 1, 128), (136, 3, 1))):
        n = shape[0]
        k, v = base.as_strided(shape, strides), base[1600:].as_strided(shape, strides)
        slots = torch.arange(n, device="cuda")
        got = []
        for a, b in ((k, v), (k.contiguous(), v.contiguous())):
            cache = torch.zeros(L.total_bytes, dtype=torch.uint8, device="cuda")
            sg.sgemv_kv_append(L, cache, a, b, slots, status=st)
            got.append(cache)
        assert torch.equal(*got)
        i32 = dict(dtype=torch.int32, device="cuda")
        outs = []
        for q in (k, k.contiguous()):
            out = torch.empty(n * 300, dtype=torch.float16, device="cuda").as_strided(shape, strides)
            sg.sgemv_kv_attention(L, cache, q, torch.tensor([0, n], **i32), torch.tensor([n], **i32), torch.zeros((1, 1), **i32), out, n, 0.1,
                                  sg.kv_workspace(), status=st)
            outs.append(out.contiguous())
        assert torch.equal(*outs) and int(st.item()) == 0


def test_attention_out_in_place_of_q(env):
    """out may be q itself: the same bits."""
    sg, torch = env
    for reqs in ([(700, 1), (90, 7), (40, 1)], [(300, 131), (50, 1)]):
        c = Case(env, 128, 64, 32, 1, 8, "float16", reqs)
        out, _ = c.run()
        starts, lens, table, _ = c.tensors()
        q = c.q.clone()
        sg.sgemv_kv_attention(c.L, c.cache, q, starts, lens, table, q, c.max_q, c.scale, sg.kv_workspace())
        assert np.array_equal(q.float().cpu().numpy(), out)


def test_logprobs_in_place(env):
    """Full rows may take the place of fp32 logits."""
    sg, torch = env
    for rows, vocab in ((3, 70001), (300, 517)):
        x = torch.randn(rows, vocab, device="cuda")
        want = sg.logprobs(x, top=5, full=True)
        top = torch.empty(rows, 5, dtype=torch.int32, device="cuda"), torch.empty(rows, 5, device="cuda")
        sg.sgemv_logprobs(x, (None, None, None, *top, x))
        assert torch.equal(x, want["logp"]) and torch.equal(top[0], want["top_tok"]) and torch.equal(top[1], want["top_logp"])


def test_plan_arrays_between_the_rows_of_a_table(env):
    """A table of some columns of wider rows: what lies between its rows may be another array."""
    sg, torch = env
    i32 = dict(dtype=torch.int32, device="cuda")
    wide = torch.full((2, 40), -1, **i32)
    table, start = wide[:, :4], wide[0, 20:23]
    length, add = torch.zeros(2, **i32), torch.tensor([20, 5], **i32)
    out = (torch.empty(2, **i32), torch.empty(1, **i32), start, torch.empty(25, dtype=torch.int64, device="cuda"), torch.empty(25, **i32))
    sg.sgemv_kv_plan(length, None, add, table, torch.arange(8, **i32), torch.tensor([8], **i32), 16, out)
    assert start.tolist() == [0, 20, 25] and table.tolist() == [[7, 6, -1, -1], [5, -1, -1, -1]]


def many_requests(n_req):
    """Mostly decodes and idle requests, and prompt chunks of 560 rows (8 query heads a KV head), three of them neighbours."""
    rng = np.random.default_rng(n_req + 2)
    reqs = []
    for r in range(n_req):
        old, n = int(rng.integers(0, 40)), int(rng.integers(0, 2))
        reqs.append((old + 70, 70) if r % 97 in (50, 51, 52) else (old + n, n))
    return reqs


@pytest.mark.parametrize("n_req", [300, 700, 1400])
def test_attention_many_requests_and_prompt_chunks(env, n_req):
    """More requests than the tensor-core form has threads (640), so that a thread looks after several, with prompt chunks among them."""
    c = Case(env, 64, 64, 16, 1, 8, "float16", many_requests(n_req))
    c.check(*c.run())


MANY_ROWS = [(300, 300), (371, 260), (64, 1)]  # (tokens, new ones): 2400 and 2080 rows a KV head, and a decode


@pytest.mark.parametrize("dim,group,heads,dtype", [(128, 128, 2, "float16"), (64, 64, 1, "bfloat16"), (128, 64, 1, "float16"),
                                                   (256, 128, 1, "float16"), (256, 64, 1, "bfloat16")])
def test_attention_prompts_of_many_rows(env, dim, group, heads, dtype):
    """More than 2000 rows a KV head: many row tiles a request, a whole prompt and one behind a context."""
    c = Case(env, dim, group, 64, heads, 8, dtype, MANY_ROWS)
    c.check(*c.run())


def test_attention_shared_pages(env):
    """Two requests whose tables list the same pages for a common prefix."""
    c = Case(env, 128, 128, 16, 2, 4, "float16", [(90, 2), (75, 1), (200, 140)])
    c.table[1, :3] = c.table[0, :3]
    c.table[2, :4] = c.table[0, :4]
    c.check(*c.run())


def test_plan_with_more_pages_than_there_are(env):
    """Lengths that cannot be: requests give up and need more pages than the cache has, though as many as they give up. Nothing moves."""
    sg, _ = env
    table = np.array([[1, 2, 3, 0, 1, 2], [3, -1, -1, -1, -1, -1]], dtype=np.int32)
    length, keep, add = [96, 16], [16, 16], [0, 80]
    got, status = _run_plan(env, length, keep, add, table, [-9] * 4, 0, 16, 80)
    assert status == sg.SGEMV_ERR_SHAPE
    assert got[0].tolist() == length and got[1][0] == 0 and not got[2].any() and np.all(got[3] == -1) and np.all(got[4] == -1)
    assert np.array_equal(got[5], table) and np.all(got[6] == -9)
