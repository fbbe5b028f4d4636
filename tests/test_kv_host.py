"""Host-side checks of the decode-path operators' C ABI (no GPU needed): layouts, the oracle's byte places, and the
refusals that come before anything is launched."""

import ctypes
import os
import re

import numpy as np
import pytest

from oracle import kv as okv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    return sg


def test_exports_match_the_header(sg):
    text = open(os.path.join(ROOT, "include", "sgemv_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(sgemv_[a-z_]+)\s*\(", text))
    assert names == set(sg.EXPORTED_KV)
    lib = ctypes.CDLL(sg.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 64), (128, 128), (256, 64), (256, 128)])
def test_layout_and_places(sg, dim, group):
    for heads, page, pages in ((1, 16, 1), (8, 64, 1000), (32, 256, 7)):
        assert sg.sgemv_kv_layout_query(heads, dim, group, page, pages).as_dict() == okv.layout(heads, dim, group, page, pages)
    L = okv.layout(1, dim, group, 16, 1)
    kb, ks, vb, vs = okv.places(L)
    nibbles = set((2 * kb + (ks > 0)).ravel()) | set((2 * vb + (vs > 0)).ravel())
    assert nibbles == set(range(2 * 16 * dim))  # every nibble before the scales, once


def test_layout_refusals(sg):
    for args in ((0, 128, 128, 16, 1), (1025, 128, 128, 16, 1), (8, 96, 64, 16, 1), (8, 64, 128, 16, 1), (8, 128, 32, 16, 1),
                 (8, 128, 128, 48, 1), (8, 128, 128, 16, 0)):
        with pytest.raises(sg.SgemvError) as e:
            sg.sgemv_kv_layout_query(*args)
        assert e.value.code == sg.SGEMV_ERR_SHAPE


A = 0x100000  # fake addresses, never dereferenced on these paths


def test_cache_refusals(sg):
    lib, L = sg._lib, sg.sgemv_kv_layout_query(8, 128, 128, 64, 10)
    ref = ctypes.byref

    def app(layout=L, cache=A, dtype=0, k=A, kt=1024, kh=128, v=A, vt=1024, vh=128, slots=A, n=4, st=None):
        return lib.sgemv_kv_append(None if layout is None else ref(layout), cache, dtype, k, kt, kh, v, vt, vh, slots, n, st, None)

    broken = sg.KvLayout.from_buffer_copy(L)
    broken.page_bytes += 16
    assert app(layout=None) == sg.SGEMV_ERR_ARG
    assert app(layout=broken) == sg.SGEMV_ERR_FORMAT
    assert app(dtype=2) == sg.SGEMV_ERR_ARG and app(n=-1) == sg.SGEMV_ERR_ARG
    assert app(cache=None) == sg.SGEMV_ERR_ARG and app(slots=None) == sg.SGEMV_ERR_ARG
    for kw in (dict(cache=A + 8), dict(k=A + 2), dict(v=A + 8), dict(slots=A + 4), dict(kt=1025), dict(vh=4), dict(st=A + 2)):
        assert app(**kw) == sg.SGEMV_ERR_ALIGN, kw
    assert app(n=0) == sg.SGEMV_OK

    def read(dtype=0, slots=A, n=4, k=A, v=A):
        return lib.sgemv_kv_read(ref(L), A, slots, n, dtype, k, v, None, None)

    assert read(dtype=3) == sg.SGEMV_ERR_ARG and read(k=None) == sg.SGEMV_ERR_ARG
    assert read(v=A + 4) == sg.SGEMV_ERR_ALIGN and read(n=0) == sg.SGEMV_OK


def test_plan_refusals(sg):
    def plan(n=4, page=16, pages=9, ln=A, keep=None, add=A + 64, table=A, cols=3, stride=3, free=A, count=A, lo=A + 128,
             co=A + 256, start=A, slots=A, pos=A, n_slots=5):
        return sg._lib.sgemv_kv_plan(n, page, pages, ln, keep, add, table, cols, stride, free, count, lo, co, start, slots, pos,
                                     n_slots, None, None)

    for kw in (dict(n=-1), dict(pages=0), dict(cols=0), dict(stride=2), dict(ln=None), dict(add=None), dict(table=None),
               dict(free=None), dict(count=None), dict(start=None), dict(slots=None), dict(pos=None), dict(n_slots=-1),
               dict(co=A), dict(lo=A), dict(lo=A + 64)):
        assert plan(**kw) == sg.SGEMV_ERR_ARG, kw
    assert plan(page=24) == sg.SGEMV_ERR_SHAPE
    for kw in (dict(ln=A + 2), dict(slots=A + 4), dict(pos=A + 1)):
        assert plan(**kw) == sg.SGEMV_ERR_ALIGN, kw


def test_attention_refusals(sg):
    L = sg.sgemv_kv_layout_query(8, 128, 128, 64, 10)
    ok = dict(dtype=0, heads_q=32, n_req=2, n_tokens=2, max_q=1, window=0, table_cols=4, scale=0.1, table_stride=4,
              q_token_stride=4096, q_head_stride=128, out_token_stride=4096, out_head_stride=128, q_dev=A, q_start_dev=A,
              len_dev=A, table_dev=A, tree_dev=None, out_dev=A, lse_dev=A, workspace_dev=A, workspace_bytes=sg.KV_WORKSPACE)

    def attn(layout=L, cache=A, st=None, **kw):
        q = sg.KvQuery(**{**ok, **kw})
        return sg._lib.sgemv_kv_attention(ctypes.byref(layout), cache, ctypes.byref(q), st, None)

    for kw in (dict(dtype=2), dict(n_req=-1), dict(n_tokens=-1), dict(max_q=-1), dict(window=-1), dict(table_cols=0),
               dict(table_stride=3), dict(scale=float("nan")), dict(tree_dev=A, window=3), dict(tree_dev=A, max_q=65),
               dict(cache=None), dict(q_dev=None), dict(q_start_dev=None), dict(len_dev=None), dict(table_dev=None),
               dict(out_dev=None), dict(workspace_dev=None), dict(workspace_bytes=sg.KV_WORKSPACE - 1)):
        assert attn(**kw) == sg.SGEMV_ERR_ARG, kw
    for kw in (dict(heads_q=12), dict(heads_q=0), dict(heads_q=32768)):
        assert attn(**kw) == sg.SGEMV_ERR_SHAPE, kw
    for kw in (dict(cache=A + 8), dict(q_dev=A + 2), dict(out_dev=A + 8), dict(q_head_stride=4), dict(out_token_stride=9),
               dict(len_dev=A + 2), dict(tree_dev=A + 4), dict(st=A + 1), dict(workspace_dev=A + 8)):
        assert attn(**kw) == sg.SGEMV_ERR_ALIGN, kw
    broken = sg.KvLayout.from_buffer_copy(L)
    broken.sub_bytes = 0
    assert attn(layout=broken) == sg.SGEMV_ERR_FORMAT
    assert attn(n_tokens=0) == sg.SGEMV_OK and attn(n_req=0) == sg.SGEMV_OK and attn(max_q=0) == sg.SGEMV_OK


def test_logprobs_refusals(sg):
    def lp(x=A, dtype=0, rows=2, vocab=100, stride=100, tok=None, n_tok=0, top=0, tl=None, tt=None, tv=None, full=A, st=None):
        return sg._lib.sgemv_logprobs(x, dtype, rows, vocab, stride, tok, n_tok, top, tl, A, A, tt, tv, full, st, None)

    for kw in (dict(x=None), dict(dtype=3), dict(rows=-1), dict(stride=99), dict(n_tok=65, tok=A, tl=A), dict(n_tok=1, tl=A),
               dict(n_tok=1, tok=A), dict(top=65, tt=A, tv=A), dict(top=3, tt=A), dict(top=3, tv=A)):
        assert lp(**kw) == sg.SGEMV_ERR_ARG, kw
    for kw in (dict(vocab=0), dict(vocab=(1 << 24) + 1, stride=1 << 25)):
        assert lp(**kw) == sg.SGEMV_ERR_SHAPE, kw
    for kw in (dict(x=A + 1), dict(dtype=2, x=A + 2), dict(full=A + 2), dict(st=A + 2)):
        assert lp(**kw) == sg.SGEMV_ERR_ALIGN, kw
    assert lp(rows=0) == sg.SGEMV_OK


def test_plan_oracle_keeps_pages_distinct():
    """The oracle itself: after random steps no page is in two places, and none is lost."""
    rng = np.random.default_rng(1)
    page, pages, n = 16, 60, 5
    table, free, count, length = [[-1] * 20 for _ in range(n)], list(range(pages)), pages, [0] * n
    for _ in range(50):
        keep = [max(0, x - int(rng.integers(0, 30))) if rng.random() < 0.5 else x for x in length]
        add = [int(rng.integers(0, 40)) if k < 100 else 0 for k in keep]
        length, count, start, slots, pos, table, free = okv.plan(length, keep, add, table, free, count, page, sum(add))
        used = [table[r][b] for r in range(n) for b in range(-(-length[r] // page))]
        assert sorted(used + free[:count]) == list(range(pages))
        assert len(set(slots)) == len(slots)


def test_size_refusals(sg):
    """Sizes past what the kernels index."""
    plan = lambda n: sg._lib.sgemv_kv_plan(n, 16, 9, A, None, A + 64, A, 3, 3, A, A, A + 128, A + 256, A, A, A, 5, None, None)  # noqa: E731
    assert plan(16385) == sg.SGEMV_ERR_SHAPE
    L = sg.sgemv_kv_layout_query(1, 128, 128, 64, 10)
    q = sg.KvQuery(dtype=0, heads_q=64, n_req=2, n_tokens=1 << 25, max_q=1, window=0, table_cols=4, scale=0.1, table_stride=4,
                   q_token_stride=8192, q_head_stride=128, out_token_stride=8192, out_head_stride=128, q_dev=A, q_start_dev=A,
                   len_dev=A, table_dev=A, tree_dev=None, out_dev=A, lse_dev=A, workspace_dev=A, workspace_bytes=sg.KV_WORKSPACE)
    assert sg._lib.sgemv_kv_attention(ctypes.byref(L), A, ctypes.byref(q), None, None) == sg.SGEMV_ERR_SHAPE
