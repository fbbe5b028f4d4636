"""GPU parity of 4-bit matrices (quantise, read, product) against the numpy oracle (oracle/prompt.py).

Bytes are exact, values read in fp32 and bf16 too. A product is a sum of exact products in 32 bits: kp / 64 steps of the tensor cores, each
off by no more than 2^-22 of the sum of magnitudes, and as much for a join of up to 8 parts; then y is rounded once."""

import numpy as np
import pytest

from oracle import prompt as op

pytestmark = pytest.mark.gpu

HALF_STEP = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


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


def _status(torch):
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _x(torch, rows, k, dtype, seed, spread=1.0):
    """Rows of different sizes, some columns much larger than the rest, some blocks of zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * np.exp(spread * rng.standard_normal((rows, 1)))
    x *= np.where(rng.random((1, k)) < 0.02, 30.0, 1.0)
    x *= np.repeat(rng.random((rows, (k + 15) // 16)) > 0.05, 16, axis=1)[:, :k]
    return torch.tensor(x, dtype=getattr(torch, dtype), device="cuda")


def _quantise(env, x, block, fill=255):
    sg, torch = env
    L = sg.sgemv_fp4_layout_query(x.shape[0], x.shape[1], block)
    data = torch.full((L.total_bytes,), fill, dtype=torch.uint8, device="cuda")
    status = _status(torch)
    sg.sgemv_fp4_quantize(L, data, x, status=status)
    torch.cuda.synchronize()
    return L, data, int(status.item())


def _check_bytes(env, x, block):
    L, data, status = _quantise(env, x, block)
    assert status == 0
    O = op.layout(x.shape[0], x.shape[1], block)
    ref, used = op.pack(O, *op.quantise(x.double().cpu().numpy(), block))
    got = data.cpu().numpy()
    # (a code of magnitude 0 may have either sign)
    pc = op.places(O)[0]
    zero = np.zeros_like(got)
    for shift in (0, 4):
        zero |= np.where((got >> shift) & 7, 0, 8 << shift).astype(np.uint8)
    mask = np.full_like(got, 255)
    mask[pc] &= ~zero[pc]
    bad = np.nonzero(((got ^ ref) & mask) * used)[0]
    assert bad.size == 0, (bad[:8], got[bad[:8]], ref[bad[:8]])
    return L, data, O


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 64), (1, 4096), (2, 33), (8, 200), (9, 1000), (64, 128), (65, 2056), (128, 96), (129, 1025),
                                    (300, 4104), (1, 40000), (513, 64)])
def test_quantise_matches_oracle(env, rows, k, dtype, block):
    sg, torch = env
    x = _x(torch, rows, k, dtype, rows * 7 + k)
    L, data, O = _check_bytes(env, x, block)
    want = torch.tensor(op.values(O, data.cpu().numpy()), device="cuda")
    for out in (torch.float32, torch.bfloat16, torch.float16):
        y = torch.full((rows, k), 7.0, dtype=out, device="cuda")
        sg.sgemv_fp4_read(L, data, y)
        assert torch.equal(y, want.to(out)), out


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("rows,k,offset,stride", [(65, 1, 0, 1), (70, 16, 1, 17), (100, 60, 0, 60), (129, 64, 8, 72), (200, 65, 3, 70), (300, 122, 0, 130), (66, 128, 1, 129),
                                                  (131, 129, 0, 129), (500, 250, 7, 251), (65, 256, 0, 256), (1000, 200, 0, 200)])
def test_short_rows(env, rows, k, offset, stride, dtype, block):
    """Several rows a warp, wherever they start; a row without numbers beside others."""
    sg, torch = env
    x = _x(torch, rows, k, dtype, rows + k)
    wide = torch.full((rows * stride + offset + 8,), float("nan"), dtype=x.dtype, device="cuda")
    y = wide.as_strided((rows, k), (stride, 1), offset)
    y.copy_(x)
    _check_bytes(env, y, block)
    clean = _quantise(env, y, block)[1]
    y[7, k - 1] = float("inf")
    L, data, status = _quantise(env, y, block)
    assert status == sg.SGEMV_ERR_NONFINITE
    a, b = (torch.empty((rows, k), device="cuda") for _ in range(2))
    sg.sgemv_fp4_read(L, clean, a)
    sg.sgemv_fp4_read(L, data, b)
    assert torch.isnan(b[7]).all()
    b[7] = a[7]
    assert torch.equal(a, b)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("rows,k,offset,stride", [(65, 1, 0, 1), (70, 16, 1, 17), (100, 60, 0, 60), (129, 64, 8, 72), (200, 65, 3, 70), (300, 122, 0, 130), (66, 128, 1, 129),
                                                  (131, 129, 0, 129), (500, 250, 7, 251), (65, 256, 0, 256), (1000, 200, 0, 200)])
def test_reading_short_rows(env, rows, k, offset, stride, block):
    """Each type is the fp32 form, rounded once; what lies between the rows stays."""
    sg, torch = env
    x = _x(torch, rows, k, "bfloat16", rows + 2 * k)
    x[5] = float("nan")
    L, data, status = _quantise(env, x, block)
    assert status == sg.SGEMV_ERR_NONFINITE
    want = torch.tensor(op.values(op.layout(rows, k, block), data.cpu().numpy()), device="cuda").float()
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        wide = torch.full((rows * stride + offset + 8,), 77.0, dtype=dtype, device="cuda")
        out = wide.as_strided((rows, k), (stride, 1), offset)
        sg.sgemv_fp4_read(L, data, out)
        assert torch.equal(out.nan_to_num(nan=-1e4), want.to(dtype).nan_to_num(nan=-1e4))
        out.fill_(77.0)
        assert (wide == 77.0).all()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantise_edges(env, block, dtype):
    """Ties between codes and between scales, signed zeros, rows of zeros, the smallest and the largest numbers of the type."""
    sg, torch = env
    info = torch.finfo(getattr(torch, dtype))
    rows = [np.zeros(96), np.full(96, -0.0), np.full(96, info.max), np.full(96, info.tiny), np.full(96, info.smallest_normal * 2.0 ** -5)]
    for s in (1.0, 1.125, 1.875, 3.0, 2.0 ** -9, 448.0):  # multiples of scales: codes and midpoints
        rows.append(np.concatenate([np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]) * s] * 6))
    for m in range(64):  # largest magnitudes of 6 times a midpoint between two e4m3 numbers, and beside it
        mid = (1 + (2 * (m % 8) + 1) / 16) * 2.0 ** (m // 8 - 4)
        row = np.zeros(96)
        row[::16] = 6 * mid * np.array([1, 1 + 2.0 ** -7, 1 - 2.0 ** -7, 448 / 6, 1, 1])
        row[3::16] = row[::16] / 3
        rows.append(row)
    rows.append(np.concatenate([[2688.0], np.zeros(95)]))
    rows.append(np.concatenate([[2704.0], np.full(95, 0.01)]))
    _check_bytes(env, torch.tensor(np.array(rows), dtype=getattr(torch, dtype), device="cuda"), block)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantise_every_number(env, block, dtype):
    """Every finite number of the type, beside a few scales' worth of neighbours."""
    sg, torch = env
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(getattr(torch, dtype))
    x = x[torch.isfinite(x)]
    x = x[torch.randperm(x.numel(), generator=torch.Generator().manual_seed(1))]
    _check_bytes(env, x.view(-1, 256).cuda(), block)
    x = x.sort().values  # neighbours in size share blocks
    _check_bytes(env, x.view(-1, 64).cuda(), block)


@pytest.mark.parametrize("block", [16, 32])
def test_rows_without_numbers(env, block):
    sg, torch = env
    x = _x(torch, 150, 300, "float16", 3)
    x[7, 3], x[20, 299], x[149, 0] = float("inf"), float("nan"), float("-inf")
    bad = [7, 20, 149]
    L, data, status = _quantise(env, x, block)
    assert status == sg.SGEMV_ERR_NONFINITE
    y = torch.empty((150, 300), dtype=torch.float32, device="cuda")
    sg.sgemv_fp4_read(L, data, y)
    ok = [r for r in range(150) if r not in bad]
    clean = x.clone()
    clean[bad] = 0
    L2, data2, _ = _quantise(env, clean, block)
    y2 = torch.empty_like(y)
    sg.sgemv_fp4_read(L2, data2, y2)
    assert torch.equal(y[ok], y2[ok]) and torch.isnan(y[bad]).all()
    # and in a product: those rows' outputs, on either side, and no others
    w = _x(torch, 140, 300, "float16", 4)
    wl, wd, _ = _quantise(env, w, block)
    a, b = sg.fp4_product(wl, wd, L, data), sg.fp4_product(wl, wd, L2, data2)
    assert torch.equal(a[ok], b[ok]) and torch.isnan(a[bad]).all()
    a, b = sg.fp4_product(L, data, wl, wd), sg.fp4_product(L2, data2, wl, wd)
    assert torch.equal(a[:, ok], b[:, ok]) and torch.isnan(a[:, bad]).all()


def _check_product(env, x, w, block, dtype, y=None):
    sg, torch = env
    xl, xd, _ = _quantise(env, x, block)
    wl, wd, _ = _quantise(env, w, block)
    status = _status(torch)
    if y is None:
        y = torch.full((x.shape[0], w.shape[0]), 5.0, dtype=getattr(torch, dtype), device="cuda")
    sg.sgemv_fp4_product(wl, wd, xl, xd, y, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # binary64 on the device: the values by the library's own reading, which the tests above hold to the oracle
    xv, wv = torch.empty(x.shape, device="cuda"), torch.empty(w.shape, device="cuda")
    sg.sgemv_fp4_read(xl, xd, xv)
    sg.sgemv_fp4_read(wl, wd, wv)
    ref, size = xv.double() @ wv.double().t(), xv.double().abs() @ wv.double().abs().t()
    tol = HALF_STEP[dtype] * ref.abs() + (xl.kp / 64 + 8) * 2.0 ** -22 * size + TINY[dtype]
    err = (y.double() - ref).abs()
    past = y.isinf() & (y == ref.to(y.dtype))  # (a sum past the type's end, rounded to infinity)
    bad = ~((err <= tol) | past)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), float((err / tol).max()))
    return y


@pytest.mark.parametrize("block,dtype", [(16, "float16"), (32, "bfloat16"), (16, "bfloat16"), (32, "float16")])
@pytest.mark.parametrize("tokens,n,k", [(1, 128, 64), (1, 1, 1), (1, 4096, 4096), (3, 100, 130), (8, 256, 256), (9, 129, 512), (20, 4096, 4096),
                                        (33, 1000, 320), (64, 11008, 704), (65, 300, 2050), (127, 64, 1000), (128, 40, 96), (129, 131, 5000),
                                        (333, 1024, 11008), (1000, 5003, 2050), (640, 7, 999), (1024, 1024, 8192)])
def test_product(env, tokens, n, k, block, dtype):
    sg, torch = env
    _check_product(env, _x(torch, tokens, k, dtype, tokens + k), _x(torch, n, k, "float16", n + k, 0.3), block, dtype)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("rows,k,offset,stride", [(3, 64, 8, 80), (3, 64, 1, 65), (5, 513, 3, 517), (70, 1030, 7, 1040), (2, 4099, 1, 5001), (9, 17, 0, 17),
                                                  (4, 16, 2, 31), (1, 20000, 1, 20001), (3, 2, 1, 3), (2, 511, 5, 512)])
def test_rows_that_start_anywhere(env, rows, k, offset, stride, dtype, block):
    """The same bytes whatever the rows' alignment; what lies around them is not read into them (it holds NaN) and not written."""
    sg, torch = env
    x = _x(torch, rows, k, dtype, rows + k)
    wide = torch.full((rows * stride + offset + 8,), float("nan"), dtype=x.dtype, device="cuda")
    y = wide.as_strided((rows, k), (stride, 1), offset)
    y.copy_(x)
    L, a, s1 = _quantise(env, x, block)
    _, b, s2 = _quantise(env, y, block)
    assert s1 == 0 and s2 == 0 and torch.equal(a, b)
    for out in (torch.float16, torch.bfloat16, torch.float32):
        want = torch.empty((rows, k), dtype=out, device="cuda")
        sg.sgemv_fp4_read(L, a, want)
        base = torch.full((rows * stride + offset + 8,), 77.0, dtype=out, device="cuda")
        got = base.as_strided((rows, k), (stride, 1), offset)
        sg.sgemv_fp4_read(L, a, got)
        assert torch.equal(got, want)
        got.fill_(77.0)
        assert torch.all(base == 77.0)


@pytest.mark.parametrize("tokens,n,stride,offset", [(3, 130, 133, 1), (20, 131, 131, 0), (70, 300, 301, 3), (300, 257, 1000, 5), (300, 264, 272, 8), (200, 5, 9, 1),
                                                    (64, 200, 204, 4)])
def test_product_into_rows_of_a_wider_tensor(env, tokens, n, stride, offset):
    sg, torch = env
    base = torch.full((tokens * stride + offset + 8,), 77.0, device="cuda").half()
    y = base.as_strided((tokens, n), (stride, 1), offset)
    _check_product(env, _x(torch, tokens, 200, "float16", 1), _x(torch, n, 200, "float16", 2, 0.3), 16, "float16", y)
    y.fill_(77.0)
    assert torch.all(base == 77.0)


@pytest.mark.parametrize("tokens,n,k", [(1, 256, 16384), (5, 100, 30000), (40, 128, 16384), (100, 200, 16384), (256, 300, 16384), (130, 130, 16384)])
@pytest.mark.parametrize("block", [16, 32])
def test_long_sums(env, tokens, n, k, block):
    """Few tiles and a long k: clusters of up to 8 CTAs share a tile."""
    sg, torch = env
    _check_product(env, _x(torch, tokens, k, "bfloat16", 5), _x(torch, n, k, "float16", 6, 0.3), block, "bfloat16")


@pytest.mark.parametrize("tokens,n", [(7, 300), (50, 300), (150, 200), (700, 4000)])
@pytest.mark.parametrize("block", [16, 32])
def test_exact_products(env, tokens, n, block):
    """Values that the format holds, whole numbers whose sums binary32 and the output hold exactly: the product is exact."""
    sg, torch = env
    k, rng = 128, np.random.default_rng(tokens)
    grid = np.array([0, 1, 2, 3, 4, 6]) * 1.0
    x, w = (rng.choice(grid, (m, k)) * rng.choice([-1, 1], (m, k)) * (rng.random((m, k)) < 0.2) for m in (tokens, n))
    x[:, ::16], w[:, ::16] = 6, 6  # every block's scale is then 1
    if block == 16:
        x[:, 0], w[:, 0] = 6, 6
    tx, tw = (torch.tensor(t, device="cuda").half() for t in (x, w))
    xl, xd = sg.fp4_quantize(tx, block)
    wl, wd = sg.fp4_quantize(tw, block)
    got = sg.fp4_product(wl, wd, xl, xd, torch.float16)
    want = x @ w.T
    assert np.abs(want).max() <= 2048
    assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("tokens,n", [(3, 140), (100, 140), (300, 200)])
def test_row_scales_of_any_size(env, tokens, n):
    """Row scales whose product leaves binary32's normal range, where the result does not, and where it does."""
    sg, torch = env
    k, rng = 64, np.random.default_rng(1)
    x, w = rng.standard_normal((tokens, k)), rng.standard_normal((n, k))
    ex, ew = rng.integers(-100, 100, tokens), rng.integers(-100, 100, n)
    tx = torch.tensor(x * 2.0 ** ex[:, None], device="cuda").bfloat16()
    tw = torch.tensor(w * 2.0 ** ew[:, None], device="cuda").bfloat16()
    xl, xd = sg.fp4_quantize(tx, 16)
    wl, wd = sg.fp4_quantize(tw, 16)
    got = sg.fp4_product(wl, wd, xl, xd, torch.bfloat16).double()
    xv, wv = torch.empty((tokens, k), device="cuda"), torch.empty((n, k), device="cuda")
    sg.sgemv_fp4_read(xl, xd, xv)
    sg.sgemv_fp4_read(wl, wd, wv)
    ref, size = xv.double() @ wv.double().t(), xv.double().abs() @ wv.double().abs().t()
    past = ref.to(torch.bfloat16).double()
    err = (got - ref).abs()
    ok = (err <= 2.0 ** -8 * ref.abs() + 16 * 2.0 ** -22 * size + 2.0 ** -134) | (got.isinf() & (got == past)) | (ref.abs() < 2.0 ** -126) & (got.abs() < 2.0 ** -125)
    assert ok.all(), ((~ok).nonzero()[:5].tolist(), got[~ok][:5], ref[~ok][:5])


def test_no_rows(env):
    sg, torch = env
    x = torch.randn((3, 64), device="cuda").half()
    xl, xd = sg.fp4_quantize(x)
    nl, nd = sg.fp4_quantize(x[:0])
    assert nd.numel() == 0 and sg.fp4_product(xl, xd, nl, nd).shape == (0, 3) and sg.fp4_product(nl, nd, xl, xd).shape == (3, 0)
    sg.sgemv_fp4_read(nl, nd, torch.empty((0, 64), device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens,n,k", [(1, 4096, 2048), (30, 1000, 5000), (100, 300, 8192), (400, 1500, 1000)])
def test_product_same_bits_streams_and_graphs(env, tokens, n, k):
    sg, torch = env
    w = _x(torch, n, k, "float16", 1, 0.3)
    xs = [_x(torch, tokens, k, "float16", s) for s in (2, 3)]
    wl, wd = sg.fp4_quantize(w)
    xq = [sg.fp4_quantize(x) for x in xs]
    want = [sg.fp4_product(wl, wd, *q) for q in xq]
    for _ in range(3):
        for q, y in zip(xq, want):
            assert torch.equal(sg.fp4_product(wl, wd, *q), y)
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, q, o in zip(streams, xq, outs):
            with torch.cuda.stream(s):
                sg.sgemv_fp4_product(wl, wd, *q, o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    x, (xl, xd), y = xs[0].clone(), xq[0], torch.empty_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sg.sgemv_fp4_quantize(xl, xd, x)
        sg.sgemv_fp4_product(wl, wd, xl, xd, y)
    for i in (1, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
