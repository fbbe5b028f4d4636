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
        """A CPU tensor that passes for one of device 0."""
        is_cuda = property(lambda self: True)

        def get_device(self):
            return 0

    class Lib:
        calls = []

        def __getattr__(self, name):
            return lambda *args: self.calls.append((name, args)) or 0

    lib = Lib()
    lib.calls = []
    monkeypatch.setattr(kv, "_lib", lib)
    monkeypatch.setattr(kv, "_raw_stream", lambda device: 0)
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
