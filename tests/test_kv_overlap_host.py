"""What a decode-path call writes may overlap neither its inputs nor what else it writes. The addresses are made up: every call here is
refused on the host, before anything is launched."""

import ctypes

import pytest

A = 0x1000000


@pytest.fixture(scope="module")
def sg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    from int4_weight_only_sgemv_gb300 import kv  # noqa: F401  (declares the argument types)
    return sg


def test_plan(sg):
    n, cols, stride, pages, n_slots = 100, 3, 5, 64, 50
    size = dict(ln=4 * n, keep=4 * n, add=4 * n, table=4 * stride * n, free=4 * pages, count=4, lo=4 * n, co=4, start=4 * n + 4,
                slots=8 * n_slots, pos=4 * n_slots, status=4)
    at = {name: A + 4096 * i for i, name in enumerate(size)}

    def plan(**kw):
        p = {**at, **kw}
        return sg._lib.sgemv_kv_plan(n, 16, pages, p["ln"], p["keep"], p["add"], p["table"], cols, stride, p["free"], p["count"], p["lo"],
                                     p["co"], p["start"], p["slots"], p["pos"], n_slots, p["status"], None)

    inputs = ("ln", "keep", "add", "count")
    for a in size:
        if a in inputs:
            continue
        for b in size:
            if a == b:
                continue
            # the first, an inner and the last of b's bytes
            for to in (at[b], at[b] + (size[b] // 2 & ~7), at[b] + size[b] - (8 if b == "slots" or a == "slots" else 4)):
                if b == "table" and (to - at[b]) % (4 * stride) >= 4 * cols:
                    to -= 4 * (stride - cols)  # onto a column, from between two rows
                to &= ~7 if a == "slots" else ~3
                assert plan(**{a: to}) == sg.SGEMV_ERR_ARG, (a, b, to - at[b])


def test_cache(sg):
    L = sg.sgemv_kv_layout_query(2, 128, 128, 16, 4)
    ref, n, row = ctypes.byref(L), 5, 256
    end = L.total_bytes

    def append(cache=A, k=A + 0x100000, v=A + 0x200000, slots=A + 0x300000, st=A + 0x400000, stride=row):
        return sg._lib.sgemv_kv_append(ref, cache, 0, k, stride, 128, v, row, 128, slots, n, st, None)

    for kw in (dict(k=A), dict(v=A + end - 16), dict(k=A - 2 * n * row + 16), dict(slots=A + 64), dict(st=A + 4), dict(st=A + 0x300004),
               dict(k=A + end + 1024, stride=-row)):
        assert append(**kw) == sg.SGEMV_ERR_ARG, kw

    def read(k=A + 0x100000, v=A + 0x200000, slots=A + 0x300000, st=A + 0x400000, dtype=2):
        return sg._lib.sgemv_kv_read(ref, A, slots, n, dtype, k, v, st, None)

    for kw in (dict(k=A), dict(v=A + end - 16), dict(k=A - 4 * n * row + 16), dict(v=A + 0x100000 + 4 * n * row - 16), dict(slots=A + 0x100008),
               dict(st=A + 0x200004), dict(st=A + 0x300000)):
        assert read(**kw) == sg.SGEMV_ERR_ARG, kw


def test_attention(sg):
    L = sg.sgemv_kv_layout_query(2, 128, 128, 16, 4)
    n, heads = 6, 4
    dense = 2 * n * heads * 128
    ok = dict(dtype=0, heads_q=heads, n_req=2, n_tokens=n, max_q=3, window=0, table_cols=4, scale=0.1, table_stride=4,
              q_token_stride=heads * 128, q_head_stride=128, out_token_stride=heads * 128, out_head_stride=128, q_dev=A + 0x100000,
              q_start_dev=A + 0x200000, len_dev=A + 0x300000, table_dev=A + 0x400000, tree_dev=A + 0x500000, out_dev=A + 0x600000,
              lse_dev=A + 0x700000, workspace_dev=A + 0x1000000, workspace_bytes=sg.KV_WORKSPACE)

    def attn(st=A + 0x800000, **kw):
        q = sg.KvQuery(**{**ok, **kw})
        return sg._lib.sgemv_kv_attention(ctypes.byref(L), A, ctypes.byref(q), st, None)

    ws = ok["workspace_dev"]
    for kw in (dict(out_dev=A + L.total_bytes - 16), dict(out_dev=A - dense + 16), dict(out_dev=ws + sg.KV_WORKSPACE - 16), dict(q_dev=ws),
               dict(lse_dev=A), dict(lse_dev=ws), dict(lse_dev=ok["len_dev"]), dict(lse_dev=ok["q_start_dev"] + 8), dict(workspace_dev=A + 1024),
               dict(lse_dev=ok["tree_dev"] + 8 * n - 4), dict(st=ok["len_dev"]), dict(st=ok["lse_dev"] + 4),
               dict(out_dev=ok["q_dev"] + 16), dict(out_dev=ok["q_dev"] - dense + 16)):
        assert attn(**kw) == sg.SGEMV_ERR_ARG, kw
    assert attn(n_req=(1 << 30) + 1, out_dev=A) == sg.SGEMV_ERR_SHAPE  # (before the overlap is looked at)


def test_logprobs(sg):
    rows, vocab, n_tok, top = 3, 1000, 2, 4
    at = dict(x=A, tok=A + 0x100000, tl=A + 0x200000, lse=A + 0x300000, ent=A + 0x400000, tt=A + 0x500000, tv=A + 0x600000,
              full=A + 0x700000, st=A + 0x800000)

    def lp(dtype=2, stride=vocab, **kw):
        p = {**at, **kw}
        return sg._lib.sgemv_logprobs(p["x"], dtype, rows, vocab, stride, p["tok"], n_tok, top, p["tl"], p["lse"], p["ent"], p["tt"], p["tv"],
                                      p["full"], p["st"], None)

    for kw in (dict(lse=A + 400), dict(ent=A + 4 * rows * vocab - 4), dict(full=A + 4), dict(full=A, dtype=0), dict(full=A, stride=vocab + 1),
               dict(tl=at["tok"]), dict(tt=at["tv"] + 8), dict(st=at["lse"] + 8), dict(ent=at["lse"]), dict(full=at["tl"] - 8), dict(tv=A)):
        assert lp(**kw) == sg.SGEMV_ERR_ARG, kw


def test_plan_sizes_that_leave_32_bits(sg):
    """(the addresses are apart, and refused for the sizes)"""
    def plan(pages=9, n_slots=5):
        return sg._lib.sgemv_kv_plan(4, 16, pages, A, None, A + 64, 2 * A, 3, 3, 3 * A, A + 128, A + 192, A + 256, A + 320, 1 << 40, 1 << 41,
                                     n_slots, None, None)

    assert plan(pages=(1 << 30) + 1) == sg.SGEMV_ERR_SHAPE
    assert plan(n_slots=(1 << 30) + 1) == sg.SGEMV_ERR_SHAPE and plan(n_slots=(1 << 31) - 1) == sg.SGEMV_ERR_SHAPE
