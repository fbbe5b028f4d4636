"""Scales and numbers of requests that prompt attention refuses, without a GPU: what is no number, what leaves binary32 in base 2 (every score of 0 would
become NaN), and more requests than a bounded wait allows for. The addresses are made up: every call is refused, or has nothing to do."""

import ctypes

import pytest

A = 0x1000000
FLT_MAX = float.fromhex("0x1.fffffep127")


@pytest.fixture(scope="module")
def sg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    from int4_weight_only_sgemv_gb300 import prompt  # noqa: F401  (declares the argument types)
    return sg


def _call(sg, scale, n_req, n_tokens=100):
    q = sg.PromptQuery(0, 8, 2, 64, n_req, n_tokens, 1, 0, scale, 0, 512, 64, 128, 64, 128, 64, 512, 64, A, A + 0x100000, A + 0x200000, A + 0x300000, None,
                       A + 0x400000, A + 0x500000)
    return sg._lib.sgemv_prompt_attention(ctypes.byref(q), None, None)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), FLT_MAX, -FLT_MAX, 3e38])
def test_refused(sg, scale):
    assert _call(sg, scale, 3) == sg.SGEMV_ERR_ARG and _call(sg, scale, 0) == sg.SGEMV_ERR_ARG


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, 2.0 ** 127, -2.0 ** 127])
def test_taken(sg, scale):
    assert _call(sg, scale, 0) == 0


@pytest.mark.parametrize("scale", [1e39, -1e39, 10 ** 400])
def test_the_binding_refuses_what_binary32_does_not_hold(sg, scale, monkeypatch):
    import torch
    from int4_weight_only_sgemv_gb300 import kv

    class Cuda(torch.Tensor):
        def get_device(self):
            return 0

    monkeypatch.setattr(kv, "_current", lambda: 0)
    t = torch.zeros((4, 4, 64), dtype=torch.float16).as_subclass(Cuda)
    start = torch.zeros(2, dtype=torch.int32).as_subclass(Cuda)
    with pytest.raises(ValueError):
        sg.sgemv_prompt_attention(t[:, :2], t[:, 2:3], t[:, 3:], start, torch.zeros((4, 2, 64), dtype=torch.float16).as_subclass(Cuda), scale)


def test_more_requests_than_can_be_looked_through(sg):
    assert _call(sg, 0.125, (1 << 26) + 1) == _call(sg, 0.125, (1 << 26) + 1, 0) == sg.SGEMV_ERR_SHAPE
    assert _call(sg, 0.125, 1 << 26, 0) == 0
