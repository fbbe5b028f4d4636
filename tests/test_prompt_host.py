"""Host-side checks of the prompt-path operators' C ABI (no GPU needed): exports, layouts, the oracle's own pins, and the refusals that come
before anything is launched. The addresses are made up: every call here is refused, or has nothing to do."""

import ctypes
import os
import re

import numpy as np
import pytest

from oracle import prompt as op

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x1000000


@pytest.fixture(scope="module")
def sg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    from int4_weight_only_sgemv_gb300 import prompt  # noqa: F401  (declares the argument types)
    return sg


def test_exports_match_the_header(sg):
    text = open(os.path.join(ROOT, "include", "sgemv_prompt.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(sgemv_[a-z0-9_]+)\s*\(", text))
    assert names == set(sg.EXPORTED_PROMPT)
    lib = ctypes.CDLL(sg.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("block", [16, 32])
def test_layouts(sg, block):
    for rows in (0, 1, 2, 8, 9, 16, 17, 33, 64, 65, 127, 128, 129, 1000, 1 << 24):
        for k in (1, 16, 63, 64, 65, 100, 128, 129, 4096, 11008, 1 << 20):
            assert sg.sgemv_fp4_layout_query(rows, k, block).as_dict() == op.layout(rows, k, block), (rows, k)
    for rows, k, b in ((-1, 64, 16), (1, 0, 16), ((1 << 24) + 1, 64, 16), (1, (1 << 20) + 1, 16), (1, 64, 8), (1, 64, 64)):
        with pytest.raises(sg.SgemvError):
            sg.sgemv_fp4_layout_query(rows, k, b)
    assert sg._lib.sgemv_fp4_layout_query(1, 64, 16, None) == sg.SGEMV_ERR_ARG


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("rows,k", [(1, 1), (5, 70), (64, 64), (65, 200), (300, 130)])
def test_every_byte_has_one_place(block, rows, k):
    L = op.layout(rows, k, block)
    code, scale, row = op.places(L)
    nibbles = (2 * code + np.arange(L["kp"]) % 2).ravel()
    assert np.unique(nibbles).size == nibbles.size and code.max() < L["scale_off"]
    assert np.unique(scale).size == scale.size and scale.min() >= L["scale_off"] and scale.max() < L["row_off"]
    assert row.min() >= L["row_off"] and row.max() + 4 <= L["total_bytes"]


def test_oracle_quantisation_pins():
    """Worked numbers of the definition."""
    x = np.zeros((4, 32))
    x[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]       # midpoints: to the even code
    x[1, :8] = [-0.26, 0.74, -1.26, 1.74, -2.51, 3.49, -5.01, 7.9]  # beside them; past 6
    x[2, 16:] = 2688.0
    x[3, 0] = 2689.0
    code, byte, row = op.quantise(x, 32)
    assert byte[0, 0] == 127 and code[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    assert byte[1, 0] == 127 and code[1, :8].tolist() == [9, 1, 11, 3, 13, 5, 15, 7]
    assert byte[2, 0] == 127 + 9 and code[2, 16] == 7  # 2688 / 2^9 = 5.25 -> 6
    code, byte, row = op.quantise(x, 16)
    assert row.tolist() == [2.0 ** -8, 2.0 ** -8, 1.0, 2.0]
    assert op.E4M3[byte[0, 0]] == 256.0 and code[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    assert byte[2].tolist() == [0, 126, 0, 0] and code[2, 16] == 7  # a block of zeros beside one at the end of e4m3
    # 2689 / 2 / 6 = 224.08 -> 224, and 2689 / 2 / 224 = 6.002 -> 6
    assert op.E4M3[byte[3, 0]] == 224.0 and code[3, 0] == 7
    # values that the format holds come back as they are
    rng = np.random.default_rng(0)
    v = op.E2M1[rng.integers(0, 8, (3, 64))] * rng.choice([-1, 1], (3, 64)) * np.repeat(2.0 ** rng.integers(-3, 4, (3, 4)), 16, axis=1)
    v[:, ::16] = 6.0 * np.abs(v[:, ::16] / np.where(v[:, ::16] == 0, 1, v[:, ::16])) * np.repeat(2.0 ** np.arange(-2, 2), 1)[None, :]
    L = op.layout(3, 64, 16)
    assert np.abs(op.values(L, op.pack(L, *op.quantise(v, 16))[0]) - v).max() <= np.abs(v).max() / 8
    # (a block's scale has 4 bits, a code at most 3, its step at most a third of the value; half a step each)
    z = op.values(L, op.pack(L, *op.quantise(np.zeros((3, 64)), 16))[0])
    assert np.all(z == 0)


def test_refusals_of_matrices(sg):
    lib, E = sg._lib, sg
    L, W = sg.sgemv_fp4_layout_query(5, 100, 16), sg.sgemv_fp4_layout_query(200, 100, 16)
    r, w = ctypes.byref(L), ctypes.byref(W)

    def quantize(layout=r, x=A, dtype=0, stride=100, packed=A + 0x100000, status=None):
        return lib.sgemv_fp4_quantize(layout, x, dtype, stride, packed, status, None)

    def read(layout=r, packed=A, out=A + 0x100000, dtype=2, stride=100):
        return lib.sgemv_fp4_read(layout, packed, out, dtype, stride, None)

    def product(wl=w, wd=A, xl=r, xd=A + 0x200000, y=A + 0x400000, dtype=0, stride=200, status=None):
        return lib.sgemv_fp4_product(wl, wd, xl, xd, y, dtype, stride, status, None)

    for kw in (dict(layout=None), dict(x=None), dict(packed=None), dict(dtype=2), dict(dtype=-1), dict(stride=99), dict(stride=-100),
               dict(x=A + 0x100000), dict(x=A + 0x100000 + L.total_bytes - 2), dict(status=A), dict(status=A + 0x100000), dict(stride=1 << 50)):
        assert quantize(**kw) == E.SGEMV_ERR_ARG, kw
    for kw in (dict(x=A + 1), dict(packed=A + 0x100008), dict(status=A + 0x900002)):
        assert quantize(**kw) == E.SGEMV_ERR_ALIGN, kw
    for kw in (dict(layout=None), dict(packed=None), dict(out=None), dict(dtype=3), dict(stride=99), dict(out=A + 64), dict(out=A - 4 * 400 - 4)):
        assert read(**kw) == E.SGEMV_ERR_ARG, kw
    for kw in (dict(packed=A + 8), dict(out=A + 0x100002)):
        assert read(**kw) == E.SGEMV_ERR_ALIGN, kw
    for kw in (dict(wl=None), dict(xl=None), dict(wd=None), dict(xd=None), dict(y=None), dict(dtype=2), dict(stride=199), dict(y=A), dict(y=A + 0x200000),
               dict(status=A + 0x400000), dict(status=A + 4), dict(y=A + 0x200000 - 2 * 200)):
        assert product(**kw) == E.SGEMV_ERR_ARG, kw
    for kw in (dict(wd=A + 8), dict(xd=A + 0x200004), dict(y=A + 0x400001), dict(status=A + 0x900001)):
        assert product(**kw) == E.SGEMV_ERR_ALIGN, kw
    other_k, other_block = sg.sgemv_fp4_layout_query(5, 101, 16), sg.sgemv_fp4_layout_query(5, 100, 32)
    assert product(xl=ctypes.byref(other_k)) == E.SGEMV_ERR_FORMAT and product(xl=ctypes.byref(other_block)) == E.SGEMV_ERR_FORMAT
    for field in ("rows", "k", "block", "tile", "kp", "scale_off", "row_off", "total_bytes"):
        bad = sg.sgemv_fp4_layout_query(5, 100, 16)
        setattr(bad, field, getattr(bad, field) + {"rows": 4, "k": 29}.get(field, 1))  # (6 rows of 101 would have the same bytes)
        assert quantize(layout=ctypes.byref(bad)) in (E.SGEMV_ERR_FORMAT, E.SGEMV_ERR_ARG), field
        assert read(layout=ctypes.byref(bad)) in (E.SGEMV_ERR_FORMAT, E.SGEMV_ERR_ARG), field
        assert product(xl=ctypes.byref(bad)) == E.SGEMV_ERR_FORMAT, field
    # nothing to do
    none = ctypes.byref(sg.sgemv_fp4_layout_query(0, 100, 16))
    assert quantize(layout=none, x=None, packed=None) == 0 and read(layout=none, packed=None, out=None) == 0
    assert product(xl=none, xd=None, y=None) == 0 and product(wl=none, wd=None, y=None) == 0


def _query(sg, **kw):
    q = sg.PromptQuery(0, 8, 2, 64, 3, 100, 1, 0, 0.125, 0, 512, 64, 128, 64, 128, 64, 512, 64, A, A + 0x100000, A + 0x200000, A + 0x300000, None,
                       A + 0x400000, A + 0x500000)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def test_refusals_of_attention(sg):
    call = lambda status=None, **kw: sg._lib.sgemv_prompt_attention(ctypes.byref(_query(sg, **kw)), status, None)  # noqa: E731
    assert sg._lib.sgemv_prompt_attention(None, None, None) == sg.SGEMV_ERR_ARG
    for kw in (dict(dtype=2), dict(dtype=-1), dict(n_req=-1), dict(n_tokens=-1), dict(window=-1), dict(causal=2), dict(causal=0, window=5),
               dict(scale=float("nan")), dict(q_dev=None), dict(k_dev=None), dict(v_dev=None), dict(start_dev=None), dict(out_dev=None),
               dict(out_dev=A, out_token_stride=1024), dict(out_dev=A + 16), dict(out_dev=A + 0x100000), dict(out_dev=A + 0x200000 + 2 * 128 * 100 - 16),
               dict(out_dev=A + 0x300000), dict(lse_dev=A), dict(lse_dev=A + 0x100000), dict(lse_dev=A + 0x300000), dict(lse_dev=A + 0x400000),
               dict(out_token_stride=504), dict(out_head_stride=56), dict(out_token_stride=64, out_head_stride=64),
               dict(out_token_stride=64, out_head_stride=6392), dict(status=A + 0x300000), dict(status=A + 0x400000)):
        assert call(**kw) == sg.SGEMV_ERR_ARG, kw
    for kw in (dict(dim=32), dict(dim=256), dict(dim=96), dict(heads=0), dict(heads=3), dict(heads_q=0), dict(heads_q=16386, heads=2), dict(heads=16),
               dict(q_token_stride=0), dict(k_token_stride=0), dict(v_head_stride=0), dict(k_head_stride=-64), dict(v_token_stride=1 << 39),
               dict(n_tokens=1 << 28), dict(n_req=(1 << 30) + 1)):
        assert call(**kw) == sg.SGEMV_ERR_SHAPE, kw
    for kw in (dict(q_dev=A + 8), dict(k_dev=A + 0x100002), dict(v_dev=A + 0x200008), dict(out_dev=A + 0x400004), dict(start_dev=A + 0x300002),
               dict(length_dev=A + 0x600001), dict(lse_dev=A + 0x500002), dict(q_token_stride=516), dict(k_head_stride=68), dict(out_head_stride=66),
               dict(status=A + 0x700001)):
        assert call(**kw) == sg.SGEMV_ERR_ALIGN, kw
    assert call(n_req=0) == 0 and call(n_tokens=0) == 0 and call(n_tokens=0, q_dev=None, k_dev=None) == 0
