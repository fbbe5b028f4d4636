"""The prompt-path binding's checks of its tensors, without a GPU: tensors that say they are on one stand in for CUDA tensors, and the C entry
points are replaced by recorders, so that nothing is ever launched."""

import pytest


@pytest.fixture
def env(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import int4_weight_only_sgemv_gb300 as sg
    from int4_weight_only_sgemv_gb300 import kv, prompt

    class Cuda(torch.Tensor):
        """A CPU tensor that passes for one of device 0, or of the device that it is given."""
        device_index = 0
        is_cuda = property(lambda self: True)

        def get_device(self):
            return self.device_index

    class Lib:
        sgemv_fp4_layout_query = prompt._lib.sgemv_fp4_layout_query  # (host only)

        def __init__(self):
            self.calls = []

        def __getattr__(self, name):
            return lambda *args: self.calls.append((name, args)) or 0

    lib = Lib()
    monkeypatch.setattr(prompt, "_lib", lib)
    monkeypatch.setattr(kv, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(kv, "_current", lambda: 0)
    return sg, torch, lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype).as_subclass(Cuda), lib.calls


def _calls(sg, torch, cuda):
    """A call of every operator, with its tensors by name."""
    f16, u8, i32 = torch.float16, torch.uint8, torch.int32
    L, W = sg.sgemv_fp4_layout_query(5, 100, 16), sg.sgemv_fp4_layout_query(200, 100, 16)
    quant = dict(packed=cuda(L.total_bytes, dtype=u8), x=cuda(5, 100, dtype=f16), status=cuda(1, dtype=i32))
    read = dict(packed=cuda(L.total_bytes, dtype=u8), out=cuda(5, 100))
    prod = dict(w=cuda(W.total_bytes, dtype=u8), x=cuda(L.total_bytes, dtype=u8), y=cuda(5, 200, dtype=f16), status=cuda(1, dtype=i32))
    attn = dict(q=cuda(9, 4, 64, dtype=f16), k=cuda(9, 2, 64, dtype=f16), v=cuda(9, 2, 64, dtype=f16), start=cuda(3, dtype=i32),
                out=cuda(9, 4, 64, dtype=f16), length=cuda(2, dtype=i32), lse=cuda(9, 4), status=cuda(1, dtype=i32))
    return [(lambda **t: sg.sgemv_fp4_quantize(L, t["packed"], t["x"], t["status"]), quant),
            (lambda **t: sg.sgemv_fp4_read(L, t["packed"], t["out"]), read),
            (lambda **t: sg.sgemv_fp4_product(W, t["w"], L, t["x"], t["y"], t["status"]), prod),
            (lambda **t: sg.sgemv_prompt_attention(t["q"], t["k"], t["v"], t["start"], t["out"], 0.125, t["length"], t["lse"], True, 0, t["status"]), attn)]


def test_calls_reach_the_library(env):
    sg, torch, cuda, calls = env
    for call, tensors in _calls(sg, torch, cuda):
        call(**tensors)
    assert [c[0] for c in calls] == ["sgemv_fp4_quantize", "sgemv_fp4_read", "sgemv_fp4_product", "sgemv_prompt_attention"]


def test_every_tensor_is_looked_at(env):
    """Of another device, of another type, too few elements, not contiguous, no tensor at all."""
    sg, torch, cuda, calls = env
    for call, tensors in _calls(sg, torch, cuda):
        for name, t in tensors.items():
            other = t.clone()
            other.device_index = 1
            host = torch.zeros(t.shape, dtype=t.dtype)
            bad = [other, host, t.flatten()[:-1] if name != "status" else cuda(1, dtype=torch.float32)]
            if name not in ("x", "out", "y") and name != "q":
                bad.append(t.to(torch.float64))
            if name in ("packed", "w"):
                bad.append(cuda(2 * t.numel(), dtype=t.dtype)[::2])
            for b in bad:
                with pytest.raises(ValueError):
                    call(**{**tensors, name: b})
            if name not in ("status", "length", "lse"):
                with pytest.raises(TypeError):
                    call(**{**tensors, name: None})
            if name not in ("x", "out", "y", "packed", "w"):
                with pytest.raises((TypeError, ValueError)):
                    call(**{**tensors, name: 3.0})
    assert not calls


def test_rows(env):
    """Row strides go through; rows that overlap or columns apart do not."""
    sg, torch, cuda, calls = env
    L = sg.sgemv_fp4_layout_query(5, 100, 16)
    packed = cuda(L.total_bytes, dtype=torch.uint8)
    sg.sgemv_fp4_quantize(L, packed, cuda(5, 130, dtype=torch.float16)[:, 7:107])
    sg.sgemv_fp4_read(L, packed, cuda(5, 120, dtype=torch.bfloat16)[:, :100])
    assert calls[0][1][3] == 130 and calls[1][1][4] == 120
    del calls[:]
    x = cuda(5, 200, dtype=torch.float16)
    for bad in (x[:, ::2], x[:1, :100].expand(5, 100), cuda(600, dtype=torch.float16).as_strided((5, 100), (99, 1)), cuda(100, 5, dtype=torch.float16).t(),
                cuda(5, 99, dtype=torch.float16), cuda(500, dtype=torch.float16)):
        with pytest.raises(ValueError):
            sg.sgemv_fp4_quantize(L, packed, bad)
    # one row's stride is never used
    one = sg.sgemv_fp4_layout_query(1, 100, 16)
    sg.sgemv_fp4_quantize(one, packed, cuda(300, dtype=torch.float16).as_strided((1, 100), (7, 1)))
    assert calls[-1][1][3] == 100
    t = cuda(9, 8, 64, dtype=torch.float16)
    q, k, v, out, start = t[:, :4], t[:, 4:6], t[:, 6:], cuda(9, 4, 64, dtype=torch.float16), cuda(2, dtype=torch.int32)
    sg.sgemv_prompt_attention(q, k, v, start, out, 0.125)
    a = sg.PromptQuery.from_buffer_copy(calls[-1][1][0])
    assert (a.q_token_stride, a.k_token_stride, a.v_head_stride, a.out_token_stride, a.n_req, a.n_tokens, a.heads, a.heads_q) == (512, 512, 64, 256, 1, 9, 2, 4)
    n = len(calls)
    for bad in (dict(k=cuda(9, 2, 32, dtype=torch.float16)), dict(v=cuda(8, 2, 64, dtype=torch.float16)), dict(v=cuda(9, 1, 64, dtype=torch.float16)),
                dict(k=cuda(9, 2, 64, dtype=torch.bfloat16)), dict(k=cuda(9, 2, 128, dtype=torch.float16)[:, :, ::2])):
        with pytest.raises(ValueError):
            sg.sgemv_prompt_attention(q, bad.get("k", k), bad.get("v", v), start, out, 0.125)
    assert len(calls) == n
