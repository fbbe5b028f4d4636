"""Where the helpers that allocate do so when they are given a stream, without a GPU: stand-ins for CUDA tensors and streams, and recorders for the C
entry points."""

import contextlib

import pytest


@pytest.fixture
def env(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import int4_weight_only_sgemv_gb300 as sg
    from int4_weight_only_sgemv_gb300 import kv, prompt

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    made, kept, at = [], [], [7]  # (stream that each tensor was made on; tensors kept for a stream; the current stream)

    class Cuda(torch.Tensor):
        is_cuda = property(lambda self: True)

        def get_device(self):
            return 0

        def record_stream(self, stream):
            kept.append((self.data_ptr(), stream.cuda_stream))

    @contextlib.contextmanager
    def on(stream):
        at.append(stream.cuda_stream)
        yield
        at.pop()

    empty = torch.empty

    def make(*args, **kw):
        t = empty(*args, **kw).as_subclass(Cuda)
        made.append((t.data_ptr(), at[-1]))
        return t

    class Lib:
        def __getattr__(self, name):
            return getattr(sg_lib, name) if name.endswith("layout_query") else lambda *args: 0

    sg_lib = prompt._lib
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(at[-1]))
    monkeypatch.setattr(torch, "empty", make)
    for m in (sg, kv, prompt):
        monkeypatch.setattr(m, "_lib", Lib())
    monkeypatch.setattr(sg, "_addr", lambda t: 0 if t is None else t.data_ptr())
    monkeypatch.setattr(sg, "_check_tensor", lambda *a: None)
    monkeypatch.setattr(sg, "_check_packed", lambda *a: None)
    monkeypatch.setattr(kv, "_raw_stream", lambda device: 7)
    monkeypatch.setattr(kv, "_current", lambda: 0)
    return sg, torch, lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype).as_subclass(Cuda), made, kept, Stream


def _helpers(sg, torch, cuda):
    f16, u8, i32 = torch.float16, torch.uint8, torch.int32
    L, W = sg.sgemv_fp4_layout_query(5, 128, 16), sg.sgemv_fp4_layout_query(200, 128, 16)
    K = sg.sgemv_kv_layout_query(2, 64, 64, 16, 3)
    D = sg.sgemv_layout_query(sg.SGEMV_FMT_DENSE, 64, 128, 128)
    yield lambda s: sg.fp4_quantize(cuda(5, 128, dtype=f16), 16, stream=s), 1
    yield lambda s: sg.fp4_product(W, cuda(W.total_bytes, dtype=u8), L, cuda(L.total_bytes, dtype=u8), f16, stream=s), 1
    yield lambda s: sg.prompt_attention(cuda(9, 4, 64, dtype=f16), cuda(9, 2, 64, dtype=f16), cuda(9, 2, 64, dtype=f16), cuda(3, dtype=i32), 0.1, stream=s), 1
    yield lambda s: sg.kv_attention(K, cuda(K.total_bytes, dtype=u8), cuda(2, 4, 64, dtype=f16), cuda(2, dtype=i32), cuda(1, dtype=i32), cuda(1, 2, dtype=i32), 2, 0.1,
                                    cuda(sg.KV_WORKSPACE, dtype=u8), stream=s), 1
    yield lambda s: sg.logprobs(cuda(2, 50), cuda(2, dtype=i32), 3, True, stream=s), 6
    yield lambda s: sg.pack(cuda(64, 128, dtype=f16), sg.SGEMV_FMT_DENSE, 128, stream=s), 1
    yield lambda s: sg.gemv(D, cuda(D.total_bytes, dtype=u8), cuda(1, 128, dtype=f16), stream=s), 1


def test_tensors_are_made_on_the_stream_of_the_call(env):
    """And kept for the current one. On the current one (7), by itself or given, nothing is special."""
    sg, torch, cuda, made, kept, Stream = env
    for call, n in _helpers(sg, torch, cuda):
        for s, at in ((None, 7), (Stream(7), 7), (7, 7), (Stream(9), 9), (9, 9)):
            del made[:], kept[:]
            call(s)
            assert [x for _, x in made] == [at] * n, (n, s)
            assert kept == ([] if at == 7 else [(p, 7) for p, _ in made]), (n, s)
