"""The prompt path where offsets pass 32 bits (rows far apart, matrices of more than 2^32 bytes), and captured into a graph by the first call of a process.
Bounds: test_gpu_fp4.py and test_gpu_prompt.py."""

import os
import subprocess
import sys

import pytest

from test_gpu_fp4 import _check_product, _x, env  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _far(torch, rows, cols, stride, dtype):
    """[rows, cols] with rows `stride` elements apart, in memory that holds nothing else."""
    return torch.empty((rows - 1) * stride + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (stride, 1))


@pytest.mark.parametrize("tokens,stride", [(70, (1 << 26) + 8), (9, (1 << 29) + 1)])
def test_rows_far_apart(env, tokens, stride):  # noqa: F811
    """Quantised from, read into and multiplied into rows whose last element is past 2^32 of the first."""
    sg, torch = env
    x, w = _x(torch, tokens, 300, "float16", 1), _x(torch, 200, 300, "float16", 2, 0.3)
    far = _far(torch, tokens, 300, stride, torch.float16)
    assert (tokens - 1) * stride > 1 << 32
    far.copy_(x)
    (l1, a), (l2, b) = sg.fp4_quantize(x), sg.fp4_quantize(far)
    want = torch.empty((tokens, 300), device="cuda").half()
    sg.sgemv_fp4_read(l1, a, want)
    sg.sgemv_fp4_read(l2, b, far)
    assert torch.equal(far, want)
    wl, wd = sg.fp4_quantize(w)
    y = far[:, :200]
    sg.sgemv_fp4_product(wl, wd, l1, a, y)
    assert torch.equal(y, sg.fp4_product(wl, wd, l1, a, torch.float16)) and torch.equal(far[:, 200:], want[:, 200:])


def test_attention_over_rows_far_apart(env):  # noqa: F811
    sg, torch = env
    n, stride = 140, 1 << 25
    t = torch.randn((n, 6, 64), device="cuda").half()
    start = torch.tensor([0, 100, n], dtype=torch.int32, device="cuda")
    want = sg.prompt_attention(t[:, :4], t[:, 4:5], t[:, 5:], start, 0.125)
    far = torch.empty((n - 1) * stride + 10 * 64, dtype=torch.float16, device="cuda").as_strided((n, 10, 64), (stride, 64, 1))
    assert (n - 1) * stride > 1 << 32
    far[:, :6] = t
    sg.sgemv_prompt_attention(far[:, :4], far[:, 4:5], far[:, 5:6], start, far[:, 6:], 0.125)
    assert torch.equal(far[:, 6:], want) and torch.equal(far[:, :6], t)
    # NaN in V that rows see: taken from where it lies
    far[120, 5, 3] = float("nan")
    sg.sgemv_prompt_attention(far[:, :4], far[:, 4:5], far[:, 5:6], start, far[:, 6:], 0.125)
    got = far[:, 6:]
    assert got[120:, :, 3].isnan().all() and int(got.isnan().sum()) == 20 * 4


@pytest.mark.parametrize("block", [16, 32])
def test_a_matrix_past_32_bits(env, block):  # noqa: F811
    """More than 2^32 bytes of codes: its last rows, for one token, for 40 and for 100 (the two kernels of products)."""
    sg, torch = env
    n, k = 131200, 65600
    w = torch.empty((n, k), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    wl, wd = sg.fp4_quantize(w, block)
    assert wl.scale_off > 1 << 32
    tail = w[-200:].clone()
    del w
    tl, td = sg.fp4_quantize(tail, block)
    vals = torch.empty((200, k), device="cuda")
    sg.sgemv_fp4_read(tl, td, vals)
    for tokens in (1, 40, 100):
        x = _x(torch, tokens, k, "bfloat16", tokens)
        xl, xd = sg.fp4_quantize(x, block)
        xv = torch.empty((tokens, k), device="cuda")
        sg.sgemv_fp4_read(xl, xd, xv)
        y = sg.fp4_product(wl, wd, xl, xd)[:, -200:].double()
        ref, size = xv.double() @ vals.double().t(), xv.double().abs() @ vals.double().abs().t()
        tol = 2.0 ** -8 * ref.abs() + (xl.kp / 64 + 8) * 2.0 ** -22 * size + 2.0 ** -134
        assert ((y - ref).abs() <= tol).all(), tokens
    out = torch.empty((n, k), dtype=torch.bfloat16, device="cuda")
    sg.sgemv_fp4_read(wl, wd, out)
    assert torch.equal(out[-200:].float(), vals)


FIRST = """
import torch, int4_weight_only_sgemv_gb300 as sg
torch.manual_seed(0)
w, xs, t = torch.randn((400, 320), device="cuda").half(), [torch.randn((n, 320), device="cuda").half() for n in (3, 100)], torch.randn((150, 6, 64), device="cuda").half()
start = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
def calls():
    for x in xs:
        for block in (16, 32):
            yield sg.fp4_product(*sg.fp4_quantize(w, block), *sg.fp4_quantize(x, block))
    yield sg.prompt_attention(t[:, :4], t[:, 4:5], t[:, 5:], start, 0.125)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = list(calls())
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls(), strict=True))
print("same")
"""


def test_first_calls_are_captured(env):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
