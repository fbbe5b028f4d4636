"""GPU parity of the paged 4-bit KV cache (plan, append, read, attention) against the numpy oracle (oracle/kv.py).

Bytes, tables and slots are exact. Attention's bound per output follows from its arithmetic: the weights of a row are
rounded to 11 bits before they meet V (2^-11 of sum p |v|, and 2^-14 for exp and the sums), a score is a sum of dim
products in 32 bits (2 dim 2^-24 of the sum of their magnitudes), and the output is rounded once."""

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


def _status(torch):
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ plan

def _plan_case(rng, n_req, page, most, add_most, pad):
    length = [int(x) for x in rng.integers(0, most + 1, n_req)]
    keep, add = [], []
    for n in length:
        kind = rng.integers(0, 5)
        keep.append(0 if kind == 0 else max(0, n - int(rng.integers(0, 40))) if kind == 1 else n)
        add.append(0 if rng.integers(0, 6) == 0 else int(rng.integers(0, add_most + 1)))
    held = [-(-n // page) for n in length]
    need = [-(-(k + a) // page) for k, a in zip(keep, add)]
    pages = sum(max(a, b) for a, b in zip(held, need)) + 3
    ids = rng.permutation(pages)
    cols = max(held + need + [1]) + 2
    table = np.full((n_req, cols), -7, dtype=np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = ids[at:at + h]
        at += h
    free = np.full(pages, -9, dtype=np.int32)
    free[:pages - at] = ids[at:]
    return length, keep, add, table, free, pages - at, sum(add) + pad


def _run_plan(env, length, keep, add, table, free, count, page, n_slots, use_keep=True):
    sg, torch = env
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    n = len(length)
    t_table, t_free = dev(table), dev(free)
    out = (dev([77] * n), dev([77]), dev([77] * (n + 1)), torch.full((n_slots,), 77, dtype=torch.int64, device="cuda"),
           dev([77] * n_slots))
    status = _status(torch)
    sg.sgemv_kv_plan(dev(length), dev(keep) if use_keep else None, dev(add), t_table, t_free, dev([count]), page, out,
                     status=status)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in out] + [t_table.cpu().numpy(), t_free.cpu().numpy()], int(status.item())


@pytest.mark.parametrize("n_req,page,most,add_most,pad", [(1, 16, 0, 1, 0), (1, 64, 300, 1, 5), (7, 16, 100, 40, 0),
                                                          (64, 64, 4096, 1, 0), (513, 32, 200, 9, 3),
                                                          (1025, 16, 60, 30, 100), (3000, 256, 900, 300, 0)])
def test_plan_matches_oracle(env, n_req, page, most, add_most, pad):
    rng = np.random.default_rng(n_req * 7 + page)
    for _ in range(3):
        c = _plan_case(rng, n_req, page, most, add_most, pad)
        got, status = _run_plan(env, *c[:6], page, c[6])
        ref = okv.plan(c[0], c[1], c[2], c[3], c[4], c[5], page, c[6])
        assert status == 0
        for i, (a, b) in enumerate(zip(got, (ref[0], [ref[1]], ref[2], ref[3], ref[4], ref[5], ref[6]))):
            assert np.array_equal(a, np.asarray(b).reshape(a.shape)), i


def test_plan_without_keep_and_without_requests(env):
    c = _plan_case(np.random.default_rng(5), 9, 16, 80, 20, 4)
    length = c[0]
    got, status = _run_plan(env, length, length, [1] * 9, c[3], c[4], c[5], 16, 12, use_keep=False)
    ref = okv.plan(length, length, [1] * 9, c[3], c[4], c[5], 16, 12)
    assert status == 0 and np.array_equal(got[3], ref[3]) and np.array_equal(got[5], ref[5])
    got, status = _run_plan(env, [], [], [], np.zeros((0, 4), np.int32), c[4], c[5], 16, 6)
    assert status == 0 and got[1][0] == c[5] and got[2].tolist() == [0] and np.all(got[3] == -1)


def test_plan_releases_feed_growth_in_the_same_step(env):
    # the stack is empty: request 1 grows into what request 0 gives up, lowest block first
    table = np.array([[5, 6, 7, 0], [1, -1, -1, -1]], dtype=np.int32)
    got, status = _run_plan(env, [64, 16], [10, 16], [0, 20], table, [-1] * 8, 0, 16, 20)
    assert status == 0
    assert got[5][1].tolist() == [1, 6, 7, -1] and got[1][0] == 1 and got[6][0] == 0
    assert got[3].tolist() == [6 * 16 + i for i in range(16)] + [7 * 16 + i for i in range(4)]


@pytest.mark.parametrize("what", ["pages", "cols", "slots", "keep", "negative", "stack"])
def test_plan_failure_changes_nothing(env, what):
    sg, _ = env
    length, keep, add, count, n_slots, cols = [20, 5], [20, 5], [100, 3], 7, 103, 12
    if what == "pages":
        count = 2
    if what == "cols":
        cols = 4
    if what == "slots":
        n_slots = 102
    if what == "keep":
        keep = [21, 5]
    if what == "negative":
        add = [100, -3]
    if what == "stack":
        count = 99
    table = np.full((2, cols), -1, dtype=np.int32)
    table[0, :2], table[1, 0] = [3, 4], 5
    free = np.arange(10, 20).astype(np.int32)
    got, status = _run_plan(env, length, keep, add, table, free, count, 16, n_slots)
    assert status == (sg.SGEMV_ERR_SHAPE if what in ("pages", "cols") else sg.SGEMV_ERR_ARG)
    assert got[0].tolist() == length and got[1][0] == count and not got[2].any()
    assert np.all(got[3] == -1) and np.all(got[4] == -1)
    assert np.array_equal(got[5], table) and np.array_equal(got[6], free)


def test_plan_reports_bad_page_ids(env):
    sg, _ = env
    got, status = _run_plan(env, [3, 3], [3, 3], [1, 1], np.array([[99], [1]], dtype=np.int32), [0, 1, 2], 0, 16, 2)
    assert status == sg.SGEMV_ERR_ARG and got[3].tolist() == [-1, 19]


# ------------------------------------------------------------------------------------------------ append, read

def _fresh(torch, L, fill=255):
    return torch.full((L.total_bytes,), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 64), (128, 128), (256, 64), (256, 128)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (5, 3, 32), (37, 2, 64)])
def test_append_bytes_and_read(env, dim, group, dtype, tokens, heads, page):
    sg, torch = env
    rng = np.random.default_rng(dim + group + tokens)
    pages = tokens // page + 3
    L = sg.sgemv_kv_layout_query(heads, dim, group, page, pages)
    O = okv.layout(heads, dim, group, page, pages)
    assert L.as_dict() == O
    dt = getattr(torch, dtype)
    fused = rng.standard_normal((tokens, 3 * heads, dim)) * rng.choice([1e-6, 0.02, 1, 40], (tokens, 3 * heads, 1))
    fused[0, heads] = 0                       # a group of zeros
    fused[-1, 2 * heads, :group] = 3.25       # a constant, positive group
    t = torch.tensor(fused, dtype=torch.float32).to(dt).cuda()
    k, v = t[:, heads:2 * heads], t[:, 2 * heads:]
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 2:
        slots[1] = -1
    cache, status = _fresh(torch, L), _status(torch)
    sg.sgemv_kv_append(L, cache, k, v, torch.tensor(slots, device="cuda"), status=status)
    ref = np.full(L.total_bytes, 255, dtype=np.uint8)
    okv.append(O, ref, k.float().cpu().numpy(), v.float().cpu().numpy(), slots)
    assert int(status.item()) == 0
    assert np.array_equal(cache.cpu().numpy(), ref)
    for out_dtype in (torch.float32, dt):
        ko, vo = (torch.full((tokens, heads, dim), 7, dtype=out_dtype, device="cuda") for _ in range(2))
        sg.sgemv_kv_read(L, cache, torch.tensor(slots, device="cuda"), ko, vo, status=status)
        live = slots >= 0
        for h in range(heads):
            rk, rv = okv.values(O, ref, np.maximum(slots, 0), h)[:2]
            for got, want in ((ko, rk), (vo, rv)):
                # the value has at most 15 bits: exact in fp32, one rounding otherwise
                want = torch.tensor(np.where(live[:, None], want, 0.0)).float().to(out_dtype)
                assert torch.equal(got[:, h].cpu(), want)
    assert int(status.item()) == 0


def test_append_reports_nonfinite_and_far_slots(env):
    sg, torch = env
    L = sg.sgemv_kv_layout_query(2, 128, 64, 16, 2)
    for bad in (float("inf"), float("nan"), -float("inf")):
        k = torch.randn(3, 2, 128, device="cuda").half()
        v = k.clone()
        k[1, 1, 70] = bad
        cache, status = _fresh(torch, L, 0), _status(torch)
        slots = torch.tensor([0, 1, 2], device="cuda")
        sg.sgemv_kv_append(L, cache, k, v, slots, status=status)
        assert int(status.item()) == sg.SGEMV_ERR_NONFINITE
        ko, vo = torch.empty(3, 2, 128, device="cuda"), torch.empty(3, 2, 128, device="cuda")
        sg.sgemv_kv_read(L, cache, slots, ko, vo)
        assert not ko[1, 1, 64:].any() and ko[1, 1, :64].any() and torch.isfinite(ko).all() and torch.isfinite(vo).all()
    wide = torch.full((1, 2, 128), 3e38, device="cuda").bfloat16()  # (mx - mn) / 15 passes fp16
    status = _status(torch)
    sg.sgemv_kv_append(L, _fresh(torch, L), wide, wide, torch.tensor([3], device="cuda"), status=status)
    assert int(status.item()) == sg.SGEMV_ERR_NONFINITE
    cache, status = _fresh(torch, L), _status(torch)
    far = torch.tensor([32, 5], device="cuda")
    k = torch.randn(2, 2, 128, device="cuda").half()
    sg.sgemv_kv_append(L, cache, k, k, far, status=status)
    assert int(status.item()) == sg.SGEMV_ERR_ARG
    status.zero_()
    ko, vo = torch.ones(2, 2, 128, device="cuda"), torch.ones(2, 2, 128, device="cuda")
    sg.sgemv_kv_read(L, cache, far, ko, vo, status=status)
    assert int(status.item()) == sg.SGEMV_ERR_ARG and not ko[0].any() and ko[1].any()


# ------------------------------------------------------------------------------------------------ attention

class Case:
    """Requests with random K and V in a cache whose unwritten bytes are all ones (scales that are not numbers)."""

    def __init__(self, env, dim, group, page, heads, ratio, dtype, reqs, window=0, tree=False, seed=0, vscale=1.0):
        sg, torch = env
        self.env = env
        rng = np.random.default_rng(seed + dim + page + heads)
        self.reqs, self.window = reqs, window
        lens = [r[0] for r in reqs]
        blocks = [-(-n // page) for n in lens]
        pages = sum(blocks) + 2
        self.L = sg.sgemv_kv_layout_query(heads, dim, group, page, pages)
        self.O = okv.layout(heads, dim, group, page, pages)
        ids = rng.permutation(pages)
        self.table = np.full((len(reqs), max(blocks + [1]) + 1), -1, dtype=np.int32)
        at, slots = 0, []
        for r, b in enumerate(blocks):
            self.table[r, :b] = ids[at:at + b]
            at += b
            j = np.arange(lens[r])
            slots.append(self.table[r][j // page].astype(np.int64) * page + j % page)
        slots = np.concatenate(slots + [np.zeros(0, np.int64)])
        dt = getattr(torch, dtype)
        kv = rng.standard_normal((2, len(slots), heads, dim)) + 0.5 * rng.standard_normal((2, 1, heads, dim))
        kv[1] *= vscale
        k, v = torch.tensor(kv, dtype=torch.float32).to(dt).cuda()
        self.cache = _fresh(torch, self.L)
        st = _status(torch)
        if len(slots):
            sg.sgemv_kv_append(self.L, self.cache, k, v, torch.tensor(slots, device="cuda"), status=st)
        assert int(st.item()) == 0
        self.starts = np.concatenate([[0], np.cumsum([r[1] for r in reqs])]).astype(np.int32)
        t = int(self.starts[-1])
        self.max_q = max(r[1] for r in reqs)
        # q is cut out of wider rows, out too: strides other than the contiguous ones
        self.q_all = torch.tensor(rng.standard_normal((max(t, 1), heads * ratio + 3, dim)), dtype=torch.float32).to(dt).cuda()
        self.q = self.q_all[:t, 1:heads * ratio + 1]
        self.tree = None
        if tree:
            m = []
            for n in (r[1] for r in reqs):
                row = []
                for i in range(n):
                    par = int(rng.integers(0, i)) if i else -1
                    row.append((row[par] if i else 0) | (1 << i))
                m += row
            self.tree = np.array(m, dtype=np.uint64).astype(np.int64)
        self.scale = 1.0 / np.sqrt(dim)

    def tensors(self):
        _, torch = self.env
        dev = lambda x, d: torch.tensor(np.asarray(x), dtype=d, device="cuda")  # noqa: E731
        return (dev(self.starts, torch.int32), dev([r[0] for r in self.reqs], torch.int32), dev(self.table, torch.int32),
                dev(self.tree, torch.int64) if self.tree is not None else None)

    def run(self, workspace=None, status=None, stream=None, max_q=None):
        sg, torch = self.env
        starts, lens, table, tree = self.tensors()
        t, hq, d = self.q.shape
        wide = torch.full((t, hq, d + 8), 99, dtype=self.q.dtype, device="cuda")
        lse = torch.full((t, hq), 99, dtype=torch.float32, device="cuda")
        ws = sg.kv_workspace() if workspace is None else workspace
        st = _status(torch) if status is None else status
        sg.sgemv_kv_attention(self.L, self.cache, self.q, starts, lens, table, wide[:, :, :d],
                              self.max_q if max_q is None else max_q, self.scale, ws, lse=lse, window=self.window, tree=tree,
                              status=st, stream=stream)
        torch.cuda.synchronize()
        assert torch.all(wide[:, :, d:] == 99), "written past a row"
        if status is None:
            assert int(st.item()) == 0
        return wide[:, :, :d].float().cpu().numpy(), lse.cpu().numpy()

    def check(self, out, lse):
        ref, rlse, weight, size = okv.attention(self.O, self.cache.cpu().numpy(), self.q.float().cpu().numpy(), self.starts,
                                                [r[0] for r in self.reqs], self.table, self.scale, self.window, self.tree)
        u = 2.0 ** -11 if str(self.q.dtype) == "torch.float16" else 2.0 ** -8
        score = 2 * self.L.dim * 2.0 ** -24 * size
        tol = u * np.abs(ref) + weight * (2.0 ** -11 + 2.0 ** -14 + score[..., None]) + 2.0 ** -24
        err = np.abs(out - ref)
        assert np.all(err <= tol), float((err / tol).max())
        empty = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(lse), empty) and not out[empty].any()
        err = np.abs(lse[~empty] - rlse[~empty])
        assert np.all(err <= score[~empty] + 2.0 ** -20 + 2.0 ** -22 * np.abs(rlse[~empty]))


SHAPES = [  # dim, group, page, heads, query heads a head, type
    (64, 64, 16, 2, 1, "float16"), (64, 64, 64, 1, 8, "bfloat16"), (128, 128, 32, 2, 4, "float16"),
    (128, 64, 16, 1, 5, "bfloat16"), (128, 128, 256, 3, 1, "bfloat16"), (256, 128, 64, 1, 2, "float16"),
    (256, 64, 16, 2, 3, "bfloat16"), (128, 64, 128, 1, 16, "float16")]


@pytest.mark.parametrize("shape", SHAPES)
def test_attention_single_tokens(env, shape):
    c = Case(env, *shape, [(1, 1), (15, 1), (16, 1), (17, 1), (0, 0), (64, 1), (65, 1), (300, 1), (7, 0), (131, 1)])
    c.check(*c.run())


@pytest.mark.parametrize("shape", SHAPES)
def test_attention_several_tokens(env, shape):
    """Drafts and prompt chunks of 1 to 70 tokens behind contexts of 0 to 250, the whole prompt among them."""
    c = Case(env, *shape, [(5, 5), (33, 33), (120, 7), (250, 12), (64, 1), (70, 70), (16, 16), (91, 2)])
    c.check(*c.run())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window", [1, 16, 100])
def test_attention_window(env, shape, window):
    c = Case(env, *shape, [(1, 1), (40, 40), (200, 3), (333, 1), (100, 1), (101, 2)], window=window)
    c.check(*c.run())


@pytest.mark.parametrize("shape", SHAPES)
def test_attention_tree(env, shape):
    c = Case(env, *shape, [(12, 12), (90, 7), (200, 1), (77, 64), (64, 30)], tree=True)
    c.tree[3] = 1 << 3  # sees itself alone among the drafts, and no context
    c.tree[5] = 0       # sees nothing at all
    c.tree[40] = -1     # sees every draft, later ones too
    c.check(*c.run())


def test_attention_rows_that_see_nothing(env):
    """A request with more new tokens than cached positions: the first ones see nothing."""
    c = Case(env, 128, 128, 16, 2, 2, "float16", [(3, 5), (0, 2), (20, 4)])
    out, lse = c.run()
    c.check(out, lse)
    assert np.isneginf(lse[:2]).all() and np.isneginf(lse[5:7]).all() and np.isfinite(lse[2:5]).all()


@pytest.mark.parametrize("vscale", [1e-6, 3000.0])
def test_attention_extreme_values(env, vscale):
    """V of a size whose scales are near the ends of fp16."""
    c = Case(env, 128, 128, 16, 1, 4, "bfloat16", [(200, 1), (50, 3)], vscale=vscale)
    c.check(*c.run())


def test_attention_sharp_scores(env):
    """Queries so large that one key takes nearly all the weight, and the maximum moves along the keys."""
    c = Case(env, 128, 128, 32, 2, 4, "float16", [(500, 2), (260, 1)])
    c.q *= 30
    c.check(*c.run())


@pytest.mark.parametrize("queries,ratio,dim,group", [(150, 4, 128, 128), (333, 2, 64, 64), (130, 1, 256, 64), (40, 8, 128, 64)])
@pytest.mark.parametrize("window", [0, 37])
def test_attention_prompt(env, queries, ratio, dim, group, window):
    c = Case(env, dim, group, 32, 1, ratio, "float16", [(queries + 61, queries), (queries, queries), (50, 1), (queries // 2 + 9, queries // 2)],
             window=window)
    c.check(*c.run())


def test_attention_long_context(env):
    """Work that is split over the keys: one request of 40000 tokens, against the oracle on its own bytes."""
    c = Case(env, 64, 64, 64, 1, 4, "float16", [(40000, 1), (9000, 3)])
    c.check(*c.run())


@pytest.mark.parametrize("reqs", [[(700, 1)] * 5, [(5000, 2), (3, 1)], [(300, 90), (400, 1)]])
def test_attention_same_bits_every_time(env, reqs):
    sg, torch = env
    c = Case(env, 128, 128, 16, 2, 4, "float16", reqs)
    ws = sg.kv_workspace()
    first = c.run(ws)
    for _ in range(3):
        again = c.run(ws)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_attention_on_another_stream(env):
    sg, torch = env
    c = Case(env, 128, 64, 16, 2, 4, "float16", [(600, 1), (90, 30)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run(stream=s)
    c.check(*got)


def test_attention_pages_beyond_32_bit_offsets(env):
    """The same pages at the far end of a cache of more than 2^32 bytes give the same bits."""
    sg, torch = env
    c = Case(env, 128, 128, 256, 8, 2, "float16", [(700, 1), (300, 5)])
    first = c.run()
    far = (5 << 30) // c.L.page_bytes
    big = sg.sgemv_kv_layout_query(8, 128, 128, 256, far + c.L.n_pages)
    cache = torch.empty(big.total_bytes, dtype=torch.uint8, device="cuda")
    cache[far * c.L.page_bytes:] = c.cache
    c.table = np.where(c.table >= 0, c.table + far, -1)
    c.cache, c.L = cache, big
    again = c.run()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
    # and the same tokens written there and read back
    slots = torch.arange(far * 256, far * 256 + 9, device="cuda")
    k = torch.randn(9, 8, 128, device="cuda").half()
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    small, near = c.cache[:big.page_bytes], sg.sgemv_kv_layout_query(8, 128, 128, 256, 1)
    sg.sgemv_kv_append(big, cache, k, -k, slots)
    sg.sgemv_kv_append(near, small, k, -k, slots - far * 256)
    sg.sgemv_kv_read(big, cache, slots, ko, vo)
    k2, v2 = torch.empty_like(k), torch.empty_like(k)
    sg.sgemv_kv_read(near, small, slots - far * 256, k2, v2)
    assert torch.equal(ko, k2) and torch.equal(vo, v2) and ko.any()


def test_attention_reports_bad_requests(env):
    sg, torch = env
    c = Case(env, 128, 128, 16, 2, 4, "float16", [(60, 2), (90, 1), (40, 1)])
    good = c.run()
    # a page id outside the cache: its keys are left out, the request's neighbours are untouched
    st = _status(torch)
    keep = c.table.copy()
    c.table[1, 1] = c.L.n_pages
    out, lse = c.run(status=st)
    assert int(st.item()) == sg.SGEMV_ERR_ARG
    assert np.array_equal(out[:2], good[0][:2]) and np.array_equal(out[3:], good[0][3:]) and np.isfinite(out).all()
    c.table = keep
    # more tokens than max_q: that request's rows are not written
    st = _status(torch)
    out, lse = c.run(status=st, max_q=1)
    assert int(st.item()) == sg.SGEMV_ERR_ARG
    assert np.all(out[:2] == 99) and np.array_equal(out[2:], good[0][2:])
    # longer than the table
    st = _status(torch)
    c.reqs = [(60, 2), (1000, 1), (40, 1)]
    out, lse = c.run(status=st)
    assert int(st.item()) == sg.SGEMV_ERR_SHAPE
    assert np.all(out[2] == 99) and np.array_equal(out[3:], good[0][3:])


def test_attention_refusals(env):
    sg, torch = env
    c = Case(env, 128, 128, 16, 2, 4, "float16", [(60, 2)])
    starts, lens, table, _ = c.tensors()
    ws, out = sg.kv_workspace(), torch.empty(c.q.shape, dtype=c.q.dtype, device="cuda")
    ok = dict(q=c.q, q_start=starts, length=lens, table=table, out=out, max_q=2, scale=0.1, workspace=ws)

    def code(**kw):
        with pytest.raises(sg.SgemvError) as e:
            sg.sgemv_kv_attention(c.L, c.cache, **{**ok, **kw})
        return e.value.code

    assert code(workspace=ws[:1024]) == sg.SGEMV_ERR_ARG
    assert code(window=-1) == sg.SGEMV_ERR_ARG
    assert code(window=4, tree=torch.zeros(2, dtype=torch.int64, device="cuda")) == sg.SGEMV_ERR_ARG
    assert code(max_q=65, tree=torch.zeros(2, dtype=torch.int64, device="cuda")) == sg.SGEMV_ERR_ARG
    assert code(q=c.q[:, :7], out=out[:, :7]) == sg.SGEMV_ERR_SHAPE
    assert code(q=c.q.float(), out=out.float()) == sg.SGEMV_ERR_ARG
    odd = torch.zeros(2 * 8 * 129 + 8, dtype=torch.float16, device="cuda")[1:].as_strided((2, 8, 128), (1032, 129, 1))
    assert code(q=odd) == sg.SGEMV_ERR_ALIGN
    with pytest.raises(ValueError):
        sg.sgemv_kv_attention(c.L, c.cache, **{**ok, "q": c.q.cpu()})
    with pytest.raises(ValueError):
        sg.sgemv_kv_attention(c.L, c.cache[:100], **ok)
    with pytest.raises(ValueError):
        sg.sgemv_kv_attention(c.L, c.cache, **{**ok, "lse": torch.zeros(3, device="cuda")})


@pytest.mark.parametrize("n_req", [300, 700])
def test_attention_many_requests(env, n_req):
    """More requests than either kernel keeps in shared memory; every hundredth is a prompt chunk, some are empty."""
    rng = np.random.default_rng(n_req)
    reqs = []
    for r in range(n_req):
        old, n = int(rng.integers(0, 60)), int(rng.integers(0, 3))
        reqs.append((old + 70, 70) if r % 100 == 50 else (old + n, n))
    c = Case(env, 64, 64, 16, 2, 1, "float16", reqs)
    c.check(*c.run())


@pytest.mark.parametrize("dim,group,dtype", [(64, 64, "float16"), (128, 64, "bfloat16"), (128, 128, "float16")])
def test_attention_prompt_without_some_pages(env, dim, group, dtype):
    """Page ids outside the cache in a prompt chunk: reported, their keys are left out, all else is as it was."""
    sg, torch = env
    c = Case(env, dim, group, 16, 1, 2, dtype, [(90, 60), (200, 75)])
    good = c.run()
    lost = [1, 7]
    keep = c.table.copy()
    c.table[1, lost] = [-5, c.L.n_pages]
    st = _status(torch)
    out, lse = c.run(status=st)
    assert int(st.item()) == sg.SGEMV_ERR_ARG
    assert np.array_equal(out[:60], good[0][:60]) and np.array_equal(lse[:60], good[1][:60])
    # the formula on the keys that are left
    j = np.arange(200)
    slots = keep[1][j // 16].astype(np.int64) * 16 + j % 16
    k, v, kmag, vmag = okv.values(c.O, c.cache.cpu().numpy(), slots, 0)
    q = c.q.double().cpu().numpy()
    u = 2.0 ** -11 if dtype == "float16" else 2.0 ** -8
    for i in range(75):
        see = (j <= 125 + i) & ~np.isin(j // 16, lost)
        for a in range(2):
            s = k[see] @ q[60 + i, a] * c.scale
            e = np.exp(s - s.max())
            score = 2 * dim * 2.0 ** -24 * (kmag[see] @ np.abs(q[60 + i, a])).max() * c.scale
            ref, weight = e @ v[see] / e.sum(), e @ vmag[see] / e.sum()
            tol = u * np.abs(ref) + weight * (2.0 ** -11 + 2.0 ** -14 + score) + 2.0 ** -24
            assert np.all(np.abs(out[60 + i, a] - ref) <= tol)
            want = s.max() + np.log(e.sum())
            assert abs(lse[60 + i, a] - want) <= score + 2.0 ** -20 + 2.0 ** -22 * abs(want)


@pytest.mark.parametrize("vscale", [1e-6, 1e-3, 7e4])
def test_attention_prompt_extreme_values(env, vscale):
    """V whose scales are at either end of fp16, and so large that the values themselves are far outside it."""
    c = Case(env, 128, 128, 16, 1, 4, "bfloat16", [(200, 1), (150, 70)], vscale=vscale)
    c.check(*c.run())


def test_attention_prompt_sharp_scores(env):
    """One key takes nearly all the weight, and the maximum moves along the keys of a prompt chunk."""
    c = Case(env, 128, 128, 32, 2, 4, "float16", [(500, 100), (260, 40)])
    c.q *= 30
    c.check(*c.run())


@pytest.mark.parametrize("scale", [0.0, -0.11])
def test_attention_scale_of_any_sign(env, scale):
    c = Case(env, 128, 64, 32, 2, 4, "float16", [(300, 90), (260, 1), (40, 3)])
    c.scale = scale
    c.check(*c.run())


def test_attention_rows_do_not_meet(env):
    """A query that is not a number makes its own row so, and no other."""
    c = Case(env, 128, 128, 32, 1, 4, "float16", [(300, 90), (260, 4)])
    good = c.run()
    c.q[17, 2, 5] = float("nan")
    c.q[91, 1, 70] = float("nan")
    out, lse = c.run()
    bad = np.zeros(lse.shape, dtype=bool)
    bad[17, 2] = bad[91, 1] = True
    assert np.isnan(out[bad]).all()
    assert np.array_equal(out[~bad], good[0][~bad]) and np.array_equal(lse[~bad], good[1][~bad])


def test_attention_infinite_queries_stay_alone(env):
    """Tiny queries beside an infinite one of the same tile keep their accuracy."""
    c = Case(env, 128, 128, 32, 1, 8, "bfloat16", [(260, 1), (90, 20)])
    c.q *= 1e-6
    good = c.run()
    c.check(*good)
    c.q[0, 3, 70] = c.q[9, 1, 2] = float("inf")
    out, lse = c.run()
    bad = np.zeros(lse.shape, dtype=bool)
    bad[0, 3] = bad[9, 1] = True
    assert np.isnan(out[bad]).all()
    assert np.array_equal(out[~bad], good[0][~bad]) and np.array_equal(lse[~bad], good[1][~bad])


def test_attention_prompt_beyond_32_bit_offsets(env):
    sg, torch = env
    c = Case(env, 64, 64, 64, 8, 2, "float16", [(300, 90)])
    first = c.run()
    far = (5 << 30) // c.L.page_bytes
    big = sg.sgemv_kv_layout_query(8, 64, 64, 64, far + c.L.n_pages)
    cache = torch.empty(big.total_bytes, dtype=torch.uint8, device="cuda")
    cache[far * c.L.page_bytes:] = c.cache
    c.table = np.where(c.table >= 0, c.table + far, -1)
    c.cache, c.L = cache, big
    again = c.run()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


# 131 tokens of 8 query heads a KV head are 1048 rows, 300 of 4 are 1200: with those the tensor-core form runs whatever the
# number of segments (fewer rows go to it only where there is a segment for every SM).

@pytest.mark.parametrize("dim,group,dtype", [(64, 64, "float16"), (128, 64, "bfloat16"), (128, 128, "float16"), (128, 128, "bfloat16")])
@pytest.mark.parametrize("window", [0, 1, 37])
def test_attention_large_chunks(env, dim, group, dtype, window):
    """A whole prompt, a chunk behind a context, one that sees nothing at first, and decodes beside them."""
    c = Case(env, dim, group, 32, 1, 8, dtype, [(131, 131), (400, 140), (100, 135), (50, 1), (0, 0), (333, 9)], window=window)
    c.check(*c.run())


def test_attention_many_short_chunks(env):
    """Segments for every SM, 127 rows on average: requests of more than 64 go to the tensor-core form, the others do not."""
    rng = np.random.default_rng(3)
    reqs = [(int(o) + n, n) for o, n in zip(rng.integers(0, 90, 26), [33, 32, 1, 40, 65, 0, 34] * 3 + [64, 33, 50, 32, 36])]
    c = Case(env, 128, 64, 16, 6, 4, "float16", reqs)
    c.check(*c.run())


@pytest.mark.parametrize("vscale", [1e-6, 1e-3, 7e4])
def test_attention_large_chunk_extreme_values(env, vscale):
    c = Case(env, 128, 128, 16, 1, 8, "bfloat16", [(200, 1), (190, 131)], vscale=vscale)
    c.check(*c.run())


@pytest.mark.parametrize("scale,factor", [(0.0, 1), (-0.11, 1), (0.09, 30)])
def test_attention_large_chunk_scales(env, scale, factor):
    c = Case(env, 128, 128, 32, 1, 8, "float16", [(330, 131), (260, 1)])
    c.scale = scale
    c.q *= factor
    c.check(*c.run())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_large_chunk_rows_do_not_meet(env, bad):
    c = Case(env, 128, 64, 32, 1, 8, "bfloat16", [(300, 131), (260, 4)])
    good = c.run()
    c.q[17, 2, 5] = bad
    c.q[133, 1, 70] = bad
    out, lse = c.run()
    poisoned = np.zeros(lse.shape, dtype=bool)
    poisoned[17, 2] = poisoned[133, 1] = True
    assert np.isnan(out[poisoned]).all()
    assert np.array_equal(out[~poisoned], good[0][~poisoned]) and np.array_equal(lse[~poisoned], good[1][~poisoned])


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 64), (128, 128)])
def test_attention_large_chunk_without_some_pages(env, dim, group):
    """The keys of pages outside the cache are left out: the same as a context in which they never were."""
    sg, torch = env
    c = Case(env, dim, group, 16, 1, 8, "float16", [(160, 131)])
    lost = 1  # positions 16 .. 31, seen by every query but the first ones
    keep = c.table.copy()
    c.table[0, lost] = c.L.n_pages
    st = _status(torch)
    out, lse = c.run(status=st)
    assert int(st.item()) == sg.SGEMV_ERR_ARG
    # the context without them: 144 positions, of which the queries from position 32 on see what they saw but the page
    c.table = np.delete(keep, lost, axis=1)
    c.reqs, c.starts = [(144, 128)], np.array([0, 128], np.int32)
    c.q = c.q[3:]
    c.check(out[3:], lse[3:])


def test_attention_large_chunk_same_bits_and_far_offsets(env):
    sg, torch = env
    c = Case(env, 64, 64, 64, 8, 4, "float16", [(900, 300), (310, 270)])
    ws = sg.kv_workspace()
    first = c.run(ws)
    for _ in range(3):
        again = c.run(ws)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
    far = (5 << 30) // c.L.page_bytes
    big = sg.sgemv_kv_layout_query(8, 64, 64, 64, far + c.L.n_pages)
    cache = torch.empty(big.total_bytes, dtype=torch.uint8, device="cuda")
    cache[far * c.L.page_bytes:] = c.cache
    c.table = np.where(c.table >= 0, c.table + far, -1)
    c.cache, c.L = cache, big
    again = c.run(ws)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("n_req", [300, 700])
def test_attention_many_requests_with_chunks(env, n_req):
    rng = np.random.default_rng(n_req + 1)
    reqs = []
    for r in range(n_req):
        old, n = int(rng.integers(0, 40)), int(rng.integers(0, 2))
        reqs.append((old + 27, 27) if r % 60 == 50 else (old + n, n))
    c = Case(env, 64, 64, 16, 1, 8, "float16", reqs)
    c.check(*c.run())


@pytest.mark.parametrize("reqs", [[(300, 131), (40, 1)], [(300, 4)]])
def test_attention_scores_past_24_bits(env, reqs):
    """Scores so large that neighbouring ones differ by more than 1 in binary32: finite, and a weighted mean of the cached values."""
    c = Case(env, 128, 128, 32, 1, 8, "float16", reqs)
    c.q *= 4000
    c.scale = 4000.0
    out, lse = c.run()
    v = okv.values(c.O, c.cache.cpu().numpy(), np.array([c.table[r][j // 32] * 32 + j % 32 for r, (n, _) in enumerate(reqs) for j in range(n)]), 0)[1]
    assert np.isfinite(out).all() and np.isfinite(lse).all() and lse.max() > 2.0 ** 24
    assert np.all(out <= v.max() * 1.001) and np.all(out >= v.min() * 1.001)
