"""The prompt path as a decoder layer runs it: 4-bit products into a fused projection, attention over the packed prompts, their keys and values into
the paged cache, 4-bit products back; then one more token through the decode path over that cache. Each step is held to binary64 on the inputs that
it got."""

import numpy as np
import pytest

from oracle import prompt as op

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [16, 32])
def test_a_layer(block):
    import torch
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hidden, heads, ratio, dim, page = 320, 2, 3, 64, 16
    hq, lengths = heads * ratio, [70, 1, 129]
    rng = np.random.default_rng(block)
    half = lambda *s: torch.tensor(rng.standard_normal(s), device="cuda").half()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n = sum(lengths)
    w_qkv, w_out = half((hq + 2 * heads) * dim, hidden) * hidden ** -0.5, half(hidden, hq * dim) * (hq * dim) ** -0.5
    qkv_l, qkv_w = sg.fp4_quantize(w_qkv, block)
    out_l, out_w = sg.fp4_quantize(w_out, block)
    status = i32([0])

    def check_product(wl, wd, xl, xd, y):
        x, w = torch.empty((xl.rows, xl.k), device="cuda"), torch.empty((wl.rows, wl.k), device="cuda")
        sg.sgemv_fp4_read(xl, xd, x)
        sg.sgemv_fp4_read(wl, wd, w)
        ref, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
        assert ((y.double() - ref).abs() <= 2.0 ** -11 * ref.abs() + (xl.kp / 64 + 8) * 2.0 ** -22 * size + 2.0 ** -25).all()

    def layer(x, start, fused, mixed, y, x_bytes, m_bytes):
        xl = sg.sgemv_fp4_layout_query(x.shape[0], hidden, block)
        ml = sg.sgemv_fp4_layout_query(x.shape[0], hq * dim, block)
        sg.sgemv_fp4_quantize(xl, x_bytes, x, status)
        sg.sgemv_fp4_product(qkv_l, qkv_w, xl, x_bytes, fused, status)
        t = fused.view(x.shape[0], hq + 2 * heads, dim)
        sg.sgemv_prompt_attention(t[:, :hq], t[:, hq:hq + heads], t[:, hq + heads:], start, mixed, dim ** -0.5, status=status)
        sg.sgemv_fp4_quantize(ml, m_bytes, mixed.view(x.shape[0], hq * dim), status)
        sg.sgemv_fp4_product(out_l, out_w, ml, m_bytes, y, status)
        return xl, ml

    x = half(n, hidden)
    starts = [0, 70, 71, 200]
    fused = torch.empty((n, (hq + 2 * heads) * dim), device="cuda").half()
    mixed, y = torch.empty((n, hq, dim), device="cuda").half(), torch.empty((n, hidden), device="cuda").half()
    x_bytes = torch.empty(sg.sgemv_fp4_layout_query(n, hidden, block).total_bytes, dtype=torch.uint8, device="cuda")
    m_bytes = torch.empty(sg.sgemv_fp4_layout_query(n, hq * dim, block).total_bytes, dtype=torch.uint8, device="cuda")
    xl, ml = layer(x, i32(starts), fused, mixed, y, x_bytes, m_bytes)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check_product(qkv_l, qkv_w, xl, x_bytes, fused)
    check_product(out_l, out_w, ml, m_bytes, y)
    t = fused.view(n, hq + 2 * heads, dim).double().cpu().numpy()
    ref, _, weight, size = op.attention(t[:, :hq], t[:, hq:hq + heads], t[:, hq + heads:], starts, None, dim ** -0.5)
    tol = 2.0 ** -11 * np.abs(ref) + weight * (2.0 ** -11 + 2.0 ** -14 + 2 * dim * 2.0 ** -24 * size[..., None]) + 2.0 ** -25
    assert np.all(np.abs(mixed.double().cpu().numpy() - ref) <= tol)

    # the same steps captured, with other inputs in the same place
    first = [z.clone() for z in (fused, mixed, y)]
    x2 = half(n, hidden)
    layer(x2, i32(starts), fused, mixed, y, x_bytes, m_bytes)
    want = [z.clone() for z in (fused, mixed, y)]
    place, start = x.clone(), i32(starts)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(place, start, fused, mixed, y, x_bytes, m_bytes)
    for source, expect in ((x2, want), (x, first)):
        place.copy_(source)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((fused, mixed, y), expect))

    # the prompts' keys and values into the cache, and the last token of each again by the decode path: near the prompt path's row, as far as 4 bits go
    blocks = [-(-m // page) for m in lengths]
    L = sg.sgemv_kv_layout_query(heads, dim, 64, page, sum(blocks))
    cache, table = sg.kv_cache(L), torch.full((3, max(blocks)), -1, dtype=torch.int32, device="cuda")
    out = (i32([0] * 3), i32([0]), i32([0] * 4), torch.empty(n, dtype=torch.int64, device="cuda"), i32([0] * n))
    sg.sgemv_kv_plan(i32([0] * 3), None, i32(lengths), table, i32(list(range(sum(blocks)))), i32([sum(blocks)]), page, out, status)
    rows = fused.view(n, hq + 2 * heads, dim)
    sg.sgemv_kv_append(L, cache, rows[:, hq:hq + heads], rows[:, hq + heads:], out[3], status)
    cached_k, cached_v = (torch.empty((n, heads, dim), device="cuda").half() for _ in range(2))
    sg.sgemv_kv_read(L, cache, out[3], cached_k, cached_v, status)
    last = torch.tensor([s - 1 for s in starts[1:]], device="cuda")
    q = rows[:, :hq][last].contiguous()
    got = sg.kv_attention(L, cache, q, i32([0, 1, 2, 3]), out[0], table, 1, dim ** -0.5, sg.kv_workspace(), status=status)
    again = sg.prompt_attention(rows[:, :hq], cached_k, cached_v, start, dim ** -0.5)[last]
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # (the cache's values read back are rounded to fp16 where they have more bits: half a step of a score's terms and of V's values)
    ck, cv = cached_k.double().cpu().numpy(), cached_v.double().cpu().numpy()
    _, _, weight, size = op.attention(t[:, :hq], ck, cv, starts, None, dim ** -0.5)
    bound = (weight * (4 * 2.0 ** -11 + 2.0 ** -11 * 4 * size[..., None]) + 2.0 ** -20)[last.cpu().numpy()]
    assert np.all(np.abs(got.double().cpu().numpy() - again.double().cpu().numpy()) <= bound)
