"""Bytes of 4-bit matrices whose rows hold infinities or NaN, against the numpy oracle: such a row has row scale NaN, codes and scales 0, whichever
kernel quantises it and wherever its elements lie; the other rows' bytes are what they are without it."""

import numpy as np
import pytest

from oracle import prompt as op

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


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("rows,k,offset,stride", [
    (1, 64, 0, 64), (3, 1, 0, 1), (9, 1000, 0, 1000), (64, 128, 0, 128), (8, 4096, 0, 4096),  # rows of one CTA or of one warp
    (70, 16, 1, 17), (100, 60, 0, 60), (129, 64, 8, 72), (300, 130, 0, 130), (66, 256, 3, 259),  # short rows, several a warp
    (130, 320, 0, 320), (131, 1025, 1, 1030), (129, 4104, 0, 4104),                            # tiles of 128 rows
    (2, 40000, 0, 40000), (2, 20001, 3, 20005),                                                # rows that registers do not hold
])
def test_bytes_of_rows_without_numbers(env, rows, k, offset, stride, dtype, block):
    sg, torch = env
    rng = np.random.default_rng(rows + k)
    x = torch.tensor(rng.standard_normal((rows, k)) * np.exp(rng.standard_normal((rows, 1))), dtype=getattr(torch, dtype), device="cuda")
    odd = [float("inf"), float("-inf"), float("nan")]
    bad = sorted(int(r) for r in set(rng.integers(0, rows, min(rows, 12))) | {rows - 1})
    for n, r in enumerate(bad):
        x[r, (0, k - 1, int(rng.integers(0, k)))[n % 3]] = odd[n // 3 % 3]
        if n % 4 == 3:
            x[r] = odd[n % 3]
    wide = torch.full((rows * stride + offset + 8,), float("nan"), dtype=x.dtype, device="cuda")
    y = wide.as_strided((rows, k), (stride, 1), offset)
    y.copy_(x)
    L = sg.sgemv_fp4_layout_query(rows, k, block)
    data = torch.full((L.total_bytes,), 255, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sgemv_fp4_quantize(L, data, y, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == sg.SGEMV_ERR_NONFINITE
    shape = op.layout(rows, k, block)
    ref, used = op.pack(shape, *op.quantise(x.double().cpu().numpy(), block))
    got, (codes, scales, row) = data.cpu().numpy(), op.places(shape)
    mask = np.full_like(got, 255)
    zero = np.zeros_like(got)
    for shift in (0, 4):  # (a code of magnitude 0 may have either sign)
        zero |= np.where((got >> shift) & 7, 0, 8 << shift).astype(np.uint8)
    mask[codes] &= ~zero[codes]
    wrong = np.nonzero(((got ^ ref) & mask) * used)[0]
    assert wrong.size == 0, (wrong[:8], got[wrong[:8]], ref[wrong[:8]])
    assert not got[codes[bad]].any() and not got[scales[bad]].any()
    assert np.all(np.ascontiguousarray(got[row[bad][:, None] + np.arange(4)]).view(np.uint32) == 0x7FC00000)
