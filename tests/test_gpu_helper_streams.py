"""The helpers that allocate, on another stream than the current one: what they return is written while work of the current stream still reads memory that
has just been given back, and given back while work of the current stream still reads it."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_sgemv_gb300 as sg
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return sg, torch


def _helpers(sg, torch):
    half = lambda *s: torch.randn(s, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).half()  # noqa: E731
    w, x, t = half(4096, 1024), half(1000, 1024), half(3000, 6, 64)
    (wl, wd), (xl, xd) = sg.fp4_quantize(w), sg.fp4_quantize(x)
    start = torch.tensor([0, 1000, 3000], dtype=torch.int32, device="cuda")
    D, packed = sg.pack(w, sg.SGEMV_FMT_DENSE, 128)
    logits = half(1000, 3000)
    return {"fp4_quantize": lambda s: sg.fp4_quantize(w, stream=s)[1], "fp4_product": lambda s: sg.fp4_product(wl, wd, xl, xd, torch.float16, stream=s),
            "prompt_attention": lambda s: sg.prompt_attention(t[:, :4], t[:, 4:5], t[:, 5:], start, 0.125, stream=s),
            "pack": lambda s: sg.pack(w, sg.SGEMV_FMT_DENSE, 128, stream=s)[1], "gemv": lambda s: sg.gemv(D, packed, x[:8], stream=s),
            "logprobs": lambda s: sg.logprobs(logits, full=True, stream=s)["logp"]}


@pytest.mark.parametrize("name", ["fp4_quantize", "fp4_product", "prompt_attention", "pack", "gemv", "logprobs"])
@pytest.mark.parametrize("by_handle", [False, True])
def test_on_another_stream(env, name, by_handle):
    sg, torch = env
    call = _helpers(sg, torch)[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if by_handle else side
    # memory that the current stream will still read when the call writes its own
    size = want.numel() * want.element_size()
    a, b = torch.full((size,), 77, dtype=torch.uint8, device="cuda"), torch.zeros(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    b.copy_(a)
    del a
    got = call(s)
    side.synchronize()
    torch.cuda.synchronize()
    assert (b == 77).all() and torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    # what the call returned, read by the current stream while the next call on the side writes
    torch.cuda._sleep(50_000_000)
    copy = got.clone()
    del got
    again = [call(s) for _ in range(2)]
    with torch.cuda.stream(side):
        for t in again:
            t.fill_(0)
    torch.cuda.synchronize()
    assert torch.equal(copy.view(torch.uint8), want.view(torch.uint8))
