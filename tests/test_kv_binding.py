"""The decode-path binding's checks of its tensors, without a GPU: tensors that say they are on one stand in for CUDA tensors, and
the C entry points are replaced by recorders, so that nothing is ever launched."""

import pytest


@pytest.fixture
def env(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import int4_weight_only_sgemv_gb300 as sg
    from int4_weight_only_sgemv_gb300 import kv

    class Cuda(torch.Tensor):
        """A CPU tensor that passes for one of device 0, or of the device that it is given."""
        device_index = 0
        is_cuda = property(lambda self: True)

        def get_device(self):
            return self.device_index

    class Lib:
        calls = []
        sgemv_kv_layout_query = kv._lib.sgemv_kv_layout_query  # (host only)

        def __getattr__(self, name):
            return lambda *args: self.calls.append((name, args)) or 0

    lib = Lib()
    lib.calls = []
    monkeypatch.setattr(kv, "_lib", lib)
    monkeypatch.setattr(kv, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(kv, "_current", lambda: 0, raising=False)
    return sg, torch, lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype).as_subclass(Cuda), lib.calls


def test_logprobs_rows_that_overlap_are_refused(env):
    """A row stride below the vocabulary, as of one row expanded to many: the rows that the call would read are not those of the tensor."""
    sg, torch, cuda, calls = env
    row = cuda(1, 50)
    out = (None, cuda(4), None, None, None, None)
    for x in (row.expand(4, 50), cuda(200).as_strided((4, 50), (49, 1)), cuda(200).as_strided((4, 50), (0, 1))):
        with pytest.raises(ValueError):
            sg.sgemv_logprobs(x, out)
    assert not calls
    # one row's stride is never used, and wider rows are fine
    sg.sgemv_logprobs(cuda(200).as_strided((1, 50), (7, 1)), (None, cuda(1), None, None, None, None))
    sg.sgemv_logprobs(cuda(4, 60)[:, :50], out)
    assert [(name, args[4]) for name, args in calls] == [("sgemv_logprobs", 50), ("sgemv_logprobs", 60)]


def _calls(sg, torch, cuda):
    """A call of every operator, with its tensors by name."""
    i32, i64, u8, f16 = torch.int32, torch.int64, torch.uint8, torch.float16
    L = sg.sgemv_kv_layout_query(2, 128, 128, 16, 4)
    z = lambda *shape, d=i32: cuda(*shape, dtype=d)  # noqa: E731
    plan = dict(length=z(3), keep=z(3), add=z(3), table=z(3, 2), free=z(4), free_count=z(1), o0=z(3), o1=z(1), o2=z(4), o3=z(5, d=i64),
                o4=z(5), status=z(1))
    kv = dict(cache=z(L.total_bytes, d=u8), k=z(5, 2, 128, d=f16), v=z(5, 2, 128, d=f16), slots=z(5, d=i64), status=z(1))
    attn = dict(cache=kv["cache"], q=z(3, 4, 128, d=f16), q_start=z(4), length=z(3), table=z(3, 2), out=z(3, 4, 128, d=f16),
                workspace=z(64, d=u8), lse=cuda(3, 4), tree=z(3, d=i64), status=z(1))
    logp = dict(logits=cuda(2, 9), tokens=z(2, 1), o0=cuda(2, 1), o1=cuda(2), o2=cuda(2), o3=z(2, 3), o4=cuda(2, 3), o5=cuda(2, 9), status=z(1))
    outs = lambda t, n: tuple(t.pop(f"o{i}") for i in range(n))  # noqa: E731
    return [
        (plan, lambda t: sg.sgemv_kv_plan(page=16, out=outs(t, 5), **t)),
        (kv, lambda t: sg.sgemv_kv_append(L, **t)),
        (kv, lambda t: sg.sgemv_kv_read(L, **t)),
        (attn, lambda t: sg.sgemv_kv_attention(L, max_q=1, scale=0.1, **t)),
        (logp, lambda t: sg.sgemv_logprobs(out=outs(t, 6), **t)),
    ]


def test_tensors_of_another_device_are_refused(env):
    """The library launches on the current device: a call all of whose tensors are elsewhere, or one of them, is refused."""
    sg, torch, cuda, calls = env
    for tensors, call in _calls(sg, torch, cuda):
        call(dict(tensors))
        done = len(calls)
        for name in tensors:
            other = tensors[name].clone()
            other.device_index = 1
            with pytest.raises(ValueError):
                call({**tensors, name: other})
            with pytest.raises(ValueError):
                call({**tensors, name: torch.zeros(tensors[name].shape, dtype=tensors[name].dtype)})  # on the CPU
        moved = {name: t.clone() for name, t in tensors.items()}
        for t in moved.values():
            t.device_index = 1
        with pytest.raises(ValueError):
            call(moved)
        assert len(calls) == done


def test_attention_helper_passes_lse_on(env, monkeypatch):
    sg, torch, cuda, calls = env
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: cuda(*shape, dtype=dtype))
    tensors, _ = _calls(sg, torch, cuda)[3]
    t = {k: v for k, v in tensors.items() if k not in ("out", "lse")}
    layout = sg.sgemv_kv_layout_query(2, 128, 128, 16, 4)
    out = sg.kv_attention(layout, max_q=1, scale=0.1, lse=tensors["lse"], **t)
    query = calls[-1][1][2]._obj
    assert query.lse_dev == tensors["lse"].data_ptr() and query.out_dev == out.data_ptr() and query.tree_dev == t["tree"].data_ptr()
    sg.kv_attention(layout, max_q=1, scale=0.1, **t)
    assert calls[-1][1][2]._obj.lse_dev is None
