"""The kernels that use tensor memory, one after another without a pause and several at a time on streams of their own: products of few and of many
tiles, prompt attention, and the decode path's attention of prompt chunks. Every result is that of the call alone."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def calls():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(0)
    half = lambda *s: torch.tensor(rng.standard_normal(s), device="cuda").half()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = []
    for tokens, n, k in ((1, 4096, 4096), (40, 700, 3000), (100, 200, 9000), (300, 1500, 700), (900, 3000, 512)):
        (xl, x), (wl, w) = sg.fp4_quantize(half(tokens, k)), sg.fp4_quantize(half(n, k))
        y = torch.empty((tokens, n), device="cuda").half()
        got.append((lambda s=None, wl=wl, w=w, xl=xl, x=x, y=y: sg.sgemv_fp4_product(wl, w, xl, x, y, stream=s), y))
    for dim, lengths in ((64, [900, 3, 200]), (128, [500, 700]), (64, [20] * 200)):
        start = i32(np.concatenate([[0], np.cumsum(lengths)]))
        t = half(sum(lengths), 6, dim)
        out = torch.empty((sum(lengths), 4, dim), device="cuda").half()
        got.append((lambda s=None, t=t, start=start, out=out: sg.sgemv_prompt_attention(t[:, :4], t[:, 4:5], t[:, 5:], start, out, 0.1, stream=s), out))
    heads, ratio, dim, page, new = 4, 8, 64, 16, [260, 200, 300]
    blocks = [-(-m // page) for m in new]
    L = sg.sgemv_kv_layout_query(heads, dim, 64, page, sum(blocks))
    cache, table = sg.kv_cache(L), i32(np.full((3, max(blocks)), -1))
    length, q_start = i32(new), i32(np.concatenate([[0], np.cumsum(new)]))
    at, slots = 0, []
    for r, m in enumerate(new):
        table[r, :blocks[r]] = torch.arange(at, at + blocks[r], device="cuda")
        slots += [(at + i // page) * page + i % page for i in range(m)]
        at += blocks[r]
    n = sum(new)
    sg.sgemv_kv_append(L, cache, half(n, heads, dim), half(n, heads, dim), torch.tensor(slots, device="cuda"))
    q, out = half(n, heads * ratio, dim), torch.empty((n, heads * ratio, dim), device="cuda").half()
    ws = sg.kv_workspace()
    got.append((lambda s=None: sg.sgemv_kv_attention(L, cache, q, q_start, length, table, out, max(new), 0.1, ws, stream=s), out))
    torch.cuda.synchronize()
    want = []
    for f, y in got:
        f()
        torch.cuda.synchronize()
        want.append(y.clone())
    return torch, got, want


def test_one_after_another(calls):
    torch, got, want = calls
    order = np.random.default_rng(1)
    for _ in range(20):
        for i in order.permutation(len(got)):
            got[i][0]()
    torch.cuda.synchronize()
    for (_, y), w in zip(got, want):
        assert torch.equal(y, w)


def test_at_the_same_time(calls):
    torch, got, want = calls
    streams = [torch.cuda.Stream() for _ in got]
    for _, y in got:
        y.fill_(0)
    torch.cuda.synchronize()
    for _ in range(20):
        for (f, _), s in zip(got, streams):
            f(s)
    torch.cuda.synchronize()
    for (_, y), w in zip(got, want):
        assert torch.equal(y, w)


def test_captured_together(calls):
    torch, got, want = calls
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            for f, _ in got:
                f()
    for _, y in got:
        y.fill_(0)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for (_, y), w in zip(got, want):
        assert torch.equal(y, w)
