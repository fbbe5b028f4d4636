"""Cases of the prompt path: rows and weights in block-scaled 4-bit floating point (quantisation, reading back, the product of two such
matrices) and causal attention over packed prompts.

`run` computes them in their plain form (elementary torch operations in 32 bits) where `own` is false, and through the library's entry
points where it is true. `prepare` builds the inputs, the packed weights included, from the seed alone.

A 4-bit matrix of `rows` rows of `k` values holds, for every value, a code of one sign, two exponent and one mantissa bits (0, 0.5, 1, 1.5,
2, 3, 4, 6), a scale for every `block` of a row, and a scale for every row:
  block 32  scale 2^(floor(log2 max|x|) - 2) of the block, as the byte of its exponent plus 127; the row's scale is 1
  block 16  the row's scale is 2^e, the least with max|x| of the row <= 2688 * 2^e; a block's is max|x| / 2^e / 6, rounded to e4m3
A code is x / scale, rounded to the nearest (ties to the even code) and at most 6; the value it stands for is code * scale * row's scale.
Bytes, with k up to a multiple of 64 and T = 128 rows a tile (of up to 64 rows: the next power of two, 8 at least):
  codes   [rows / T][k / 32][T][16]: byte j of a row's 32 values holds values 2j (low nibble) and 2j + 1
  scales  [rows / 128][groups of 4 scales][32][4][4]: row 32 j + i of 128 at [i][j]
  rows    fp32 [rows up to a multiple of 128]
"""

import math

import torch

own = False

INF = float("inf")
FP = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    attn = dict(op="attention", dtype="fp16", dim=128, window=0)
    return [
        # one token's activations of a 7B-class decoder on their way into a product
        dict(name="quantize token", op="quantize", rows=1, k=4096, block=16, dtype="fp16"),
        # a long ragged prompt's activations, as wide as the feed-forward layer, cut from rows of two such projections
        dict(name="quantize prompt 4001", op="quantize", rows=4001, k=11008, block=32, dtype="bf16"),
        # a layer's weights, once, when a model is loaded
        dict(name="quantize weight", op="quantize", rows=11008, k=4096, block=16, dtype="fp16"),
        # one new token through the widest projection of a 7B-class decoder
        dict(name="linear token", op="linear", tokens=1, n=11008, k=4096, block=16, dtype="fp16"),
        # 20 beams through a square projection
        dict(name="linear beam 20", op="linear", tokens=20, n=4096, k=4096, block=32, dtype="bf16"),
        # a short prompt through the projection back from the feed-forward layer
        dict(name="linear prompt 333", op="linear", tokens=333, n=4096, k=11008, block=16, dtype="bf16"),
        # sizes that no tile divides: an odd vocabulary slice behind an odd hidden size
        dict(name="linear odd", op="linear", tokens=1000, n=5003, k=2050, block=16, dtype="fp16"),
        # a serving step's prompts through a wide feed-forward layer
        dict(name="linear prompts 8192", op="linear", tokens=8192, n=28672, k=8192, block=16, dtype="bf16"),
        # the smallest call: one short prompt
        dict(attn, name="attention short", requests=1, longest=7, heads=32, heads_q=32),
        # a serving step: 16 prompts of up to 2048 tokens, four query heads a KV head, cut from a fused projection
        dict(attn, name="attention packed", requests=16, longest=2048, heads=8, heads_q=32, dtype="bf16"),
        # one long document
        dict(attn, name="attention long", requests=1, longest=16384, heads=8, heads_q=32),
        # prompts of a small model with heads of 64 and a sliding window, five query heads a KV head
        dict(attn, name="attention window", requests=5, longest=4096, heads=4, heads_q=20, dim=64, window=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "attention", "attention"))
    block, dtype = rng.choice((16, 32)), rng.choice(("fp16", "bf16"))
    if op == "quantize":
        k = _log(rng, 40, 16384)
        return dict(op=op, rows=_log(rng, 1, max(1, 4001 * 11008 // k)), k=k, block=block, dtype=dtype)
    if op == "linear":
        tokens, n = _log(rng, 1, 8192), _log(rng, 100, 32768)
        k = _log(rng, 64, min(16384, 8192 * 28672 * 8192 // (tokens * n)))
        if rng.random() < 0.5:  # most layers are multiples of 64
            n, k = -(-n // 64) * 64, max(64, k // 64 * 64)
        return dict(op=op, tokens=tokens, n=n, k=k, block=block, dtype=dtype)
    heads = rng.choice((1, 2, 4, 8, 32))
    ratio = rng.choice((1, 2, 4, 5, 8)) if heads < 32 else 1
    dim = rng.choice((64, 128, 128))
    requests = _log(rng, 1, 64)
    # no more products than the long document
    most = int(math.sqrt(16384 * 16384 * 32 * 128 / (requests * heads * ratio * dim)))
    return dict(op=op, requests=requests, longest=_log(rng, 1, min(16384, most)), heads=heads, heads_q=heads * ratio, dim=dim,
                window=rng.choice((0, 0, 0, _log(rng, 8, 4096))), dtype=dtype)


def _lengths(case):
    """Tokens of every request: the longest first, the others spread evenly below it."""
    n = case["requests"]
    return [case["longest"] if i == 0 else int(case["longest"] * ((0.5 + i * 0.6180339887) % 1.0)) for i in range(n)]


def _held(rows, k, block):
    """Bytes of a 4-bit matrix, without what pads it."""
    return rows * k // 2 + rows * -(-k // block) + (4 * rows if block == 16 else 0)


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["k"]
        return {"bytes": 2 * n + 2 * _held(case["rows"], case["k"], case["block"]) + 2 * n, "flops": 0}
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": 2 * t * k + _held(n, k, case["block"]) + 2 * t * n, "flops": 2 * t * n * k}
    pairs = tokens = 0
    for length in _lengths(case):
        w = min(case["window"] or length, length)
        tokens += length
        pairs += w * (w + 1) // 2 + (length - w) * w
    return {"bytes": tokens * (case["heads_q"] * (4 * case["dim"] + 4) + case["heads"] * 4 * case["dim"]),
            "flops": 4 * case["dim"] * case["heads_q"] * pairs}


# ------------------------------------------------------------------------------------------------ 4-bit matrices, plain

LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _pow2(e):
    """2^e as fp32, e int32 in -126..127."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x, block):
    """x [rows, k] -> (codes uint8 [rows, k up], scales uint8 [rows, k up / block], row scales fp32 [rows]); k up to a multiple of block."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % block))
    g = x.unflatten(1, (-1, block))
    most = g.abs().amax(2)
    if block == 32:
        row = torch.ones_like(most[:, 0])
        byte = (torch.frexp(most).exponent - 1 - 2 + 127).clamp(0, 254)
        byte = torch.where(most == 0, torch.zeros_like(byte), byte)
        t = g * _pow2((127 - byte)).unsqueeze(2)
        scale = byte.to(torch.uint8)
    else:
        mantissa, exponent = torch.frexp(most.amax(1))  # 2688 = 0.65625 * 2^12
        e = torch.where(mantissa <= 0.65625, exponent - 12, exponent - 11).clamp(min=-100)
        e = torch.where(mantissa == 0, torch.zeros_like(e), e)
        row = _pow2(e)
        down = _pow2(-e)
        s8 = (most * down.unsqueeze(1) / torch.full_like(most, 6.0)).to(torch.float8_e4m3fn)
        s = s8.float()
        t = g * down.view(-1, 1, 1) / torch.where(s == 0, torch.full_like(s, INF), s).unsqueeze(2)
        scale = s8.view(torch.uint8)
    a = t.abs()
    code = (a > 0.25).to(torch.uint8)
    for limit, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= limit) if even else (a > limit)
    code += (t < 0).to(torch.uint8) * 8
    return code.flatten(1), scale, row


def _scale_values(byte, block):
    if block == 32:
        return torch.where(byte == 0, torch.full_like(byte, 2.0 ** -127, dtype=torch.float32), _pow2(byte.to(torch.int32).clamp(min=1) - 127))
    return byte.view(torch.float8_e4m3fn).float()


def _values(code, scale, row, block):
    """The values of codes, fp32 [rows, k up]."""
    lut = torch.tensor(LUT, device=code.device)
    v = lut[code.to(torch.int32)].unflatten(1, (-1, block))
    return (v * _scale_values(scale, block).unsqueeze(2) * row.view(-1, 1, 1)).flatten(1)


def _tile(rows):
    t = 8
    while t < rows and t < 128:
        t *= 2
    return t


def _pack(code, scale, row, k, block):
    """The bytes of a 4-bit matrix."""
    rows = row.numel()
    pad = torch.nn.functional.pad
    tile, kp, rp = _tile(rows), -(-k // 64) * 64, -(-rows // 128) * 128
    code = pad(code, (0, max(0, kp - code.shape[1])))[:, :kp]
    code = pad(code, (0, 0, 0, -rows % tile))
    b = code[:, 0::2] | (code[:, 1::2] << 4)
    data = b.view(-1, tile, kp // 32, 16).transpose(1, 2).reshape(-1)
    groups = -(-kp // (4 * block))
    scale = pad(scale, (0, max(0, 4 * groups - scale.shape[1])))[:, :4 * groups]
    scale = pad(scale, (0, 0, 0, rp - rows))
    sc = scale.view(rp // 128, 4, 32, groups, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return torch.cat((data, sc, pad(row, (0, rp - rows)).view(torch.uint8)))


def _unpack(packed, rows, k, block):
    """_quantise's three from the bytes."""
    tile, kp, rp = _tile(rows), -(-k // 64) * 64, -(-rows // 128) * 128
    rt, groups = -(-rows // tile) * tile, -(-kp // (4 * block))
    data, sc, row = packed.split((rt * kp // 2, rp * groups * 4, rp * 4))
    b = data.view(-1, kp // 32, tile, 16).transpose(1, 2).reshape(rt, kp // 2)[:rows]
    code = torch.stack((b & 15, b >> 4), 2).flatten(1)
    scale = sc.view(-1, groups, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, 4 * groups)[:rows, :kp // block]
    return code, scale, row.view(torch.float32)[:rows]


# ------------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _activations(gen, rows, k, dtype):
    """Rows of different sizes, some channels much larger than the rest, as activations are."""
    x = torch.randn((rows, k), generator=gen, device="cuda")
    channel = torch.rand((1, k), generator=gen, device="cuda")
    size = torch.exp(torch.randn((rows, 1), generator=gen, device="cuda") * 0.5)
    return (x * torch.where(channel < 0.01, 12.0, 1.0) * size).to(FP[dtype])


def _weights(gen, n, k):
    w = torch.randn((n, k), generator=gen, device="cuda")
    return w.mul_(0.02).half()


def _quantize_inputs(case, seed):
    gen = _generator(seed)
    x = _activations(gen, case["rows"], case["k"] + 8, case["dtype"])[:, :case["k"]]  # rows of a wider matrix
    if case["rows"] > 4:
        x[3] = 0  # a padded row
    return x


def _linear_inputs(case, seed):
    gen = _generator(seed)
    return _activations(gen, case["tokens"], case["k"], case["dtype"]), _weights(gen, case["n"], case["k"])


def _attention_inputs(case, seed):
    gen = _generator(seed)
    lengths = _lengths(case)
    h, hq, d = case["heads"], case["heads_q"], case["dim"]
    rows = torch.randn((sum(lengths), hq + 2 * h, d), generator=gen, device="cuda")
    rows += torch.randn((1, hq + 2 * h, d), generator=gen, device="cuda") * 0.5
    rows = rows.to(FP[case["dtype"]])
    return rows[:, :hq], rows[:, hq:hq + h], rows[:, hq + h:], lengths  # cut from a fused projection


def prepare(case, seed):
    s = {"case": case}
    if own:
        import int4_weight_only_sgemv_gb300 as sg
        s["sg"] = sg
    dev = torch.device("cuda")
    if case["op"] == "quantize":
        s["x"] = x = _quantize_inputs(case, seed)
        s["out"] = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
        if own:
            s["layout"] = sg.sgemv_fp4_layout_query(case["rows"], case["k"], case["block"])
            s["packed"] = torch.empty(s["layout"].total_bytes, dtype=torch.uint8, device=dev)
    elif case["op"] == "linear":
        s["x"], w = _linear_inputs(case, seed)
        s["w"] = torch.cat([_pack(*_quantise(w, case["block"]), case["k"], case["block"])])
        s["y"] = torch.empty((case["tokens"], case["n"]), dtype=FP[case["dtype"]], device=dev)
        if own:
            s["w_layout"] = sg.sgemv_fp4_layout_query(case["n"], case["k"], case["block"])
            s["layout"] = sg.sgemv_fp4_layout_query(case["tokens"], case["k"], case["block"])
            s["packed"] = torch.empty(s["layout"].total_bytes, dtype=torch.uint8, device=dev)
    else:
        s["q"], s["k"], s["v"], s["lengths"] = _attention_inputs(case, seed)
        start = [0]
        for n in s["lengths"]:
            start.append(start[-1] + n)
        s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
        s["out"] = torch.empty((start[-1], case["heads_q"], case["dim"]), dtype=FP[case["dtype"]], device=dev)
        s["lse"] = torch.empty((start[-1], case["heads_q"]), dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------------------------------------ the operators

def run(s):
    case = s["case"]
    if own:
        sg = s["sg"]
        if case["op"] == "quantize":
            sg.sgemv_fp4_quantize(s["layout"], s["packed"], s["x"])
            sg.sgemv_fp4_read(s["layout"], s["packed"], s["out"])
            return s["out"]
        if case["op"] == "linear":
            sg.sgemv_fp4_quantize(s["layout"], s["packed"], s["x"])
            sg.sgemv_fp4_product(s["w_layout"], s["w"], s["layout"], s["packed"], s["y"])
            return s["y"]
        sg.sgemv_prompt_attention(s["q"], s["k"], s["v"], s["start"], s["out"], case["dim"] ** -0.5, lse=s["lse"],
                                  window=case["window"])
        return s["out"], s["lse"]
    block = case.get("block")
    if case["op"] == "quantize":
        x = s["x"]
        s["out"].copy_(_values(*_quantise(x, block), block)[:, :x.shape[1]])
        return s["out"]
    if case["op"] == "linear":
        k = case["k"]
        x = _values(*_quantise(s["x"], block), block)[:, :k]
        w = _values(*_unpack(s["w"], case["n"], k, block), block)[:, :k]
        s["y"].copy_(x @ w.t())
        return s["y"]
    ratio, scale, window = case["heads_q"] // case["heads"], case["dim"] ** -0.5, case["window"]
    first = 0
    for n in s["lengths"]:
        for h in range(case["heads"]):
            at = slice(first, first + n)
            k, v = s["k"][at, h].float(), s["v"][at, h].float()
            j = torch.arange(n, device=k.device)
            for a in range(h * ratio, (h + 1) * ratio):
                t = (s["q"][at, a].float() @ k.t()) * scale
                hide = j.unsqueeze(0) > j.unsqueeze(1)
                if window:
                    hide |= j.unsqueeze(0) <= j.unsqueeze(1) - window
                t = t.masked_fill_(hide, -INF)
                if n == 0:
                    continue
                top = t.amax(1, keepdim=True)
                p = t.sub_(top).exp_()
                total = p.sum(1, keepdim=True)
                s["out"][at, a] = ((p @ v) / total).to(s["out"].dtype)
                s["lse"][at, a] = (top + total.log()).squeeze(1)
        first += n
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------------------------ from the definitions, in 64 bits

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest(x, grid):
    """Every x >= 0 as the nearest number of an ascending grid, ties to the one of even place, the last for anything past it."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(g, x).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = x - g[lo], g[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, g[hi], g[lo])


def _exact_values(x, block):
    """The values that the quantised rows stand for, in 64 bits."""
    rows, k = x.shape
    e4m3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]
    out = torch.empty((rows, k), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 25) // k)
    for a in range(0, rows, step):
        v = x[a:a + step].double()
        full = torch.zeros((v.shape[0], -(-k // block) * block), dtype=torch.float64, device=x.device)
        full[:, :k] = v
        full = full.view(v.shape[0], -1, block)
        big = full.abs().max(2).values
        if block == 32:
            safe = torch.where(big > 0, big, torch.ones_like(big))
            scale = torch.exp2(torch.floor(torch.log2(safe)) - 2)
            scale = torch.where(safe / scale >= 8, scale * 2, torch.where(safe / scale < 4, scale / 2, scale))
        else:
            top = big.max(1).values
            e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 2688.0)) / 2688))
            e = torch.where(top > 2688 * torch.exp2(e), e + 1, torch.where(2 * top <= 2688 * torch.exp2(e), e - 1, e))
            e = torch.where(top > 0, e, torch.zeros_like(e))
            unit = torch.exp2(e).unsqueeze(1)
            scale = _nearest(big / unit / 6, e4m3) * unit
        scale = scale.unsqueeze(2)
        ratio = torch.where(scale > 0, full.abs() / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(full))
        got = torch.copysign(_nearest(ratio, _E2M1) * scale, full)
        out[a:a + step] = got.flatten(1)[:, :k]
    return out


def exact(case, seed):
    if case["op"] == "quantize":
        return _exact_values(_quantize_inputs(case, seed), case["block"])
    if case["op"] == "linear":
        x, w = _linear_inputs(case, seed)
        return _exact_values(x, case["block"]) @ _exact_values(w, case["block"]).t()
    q, k, v, lengths = _attention_inputs(case, seed)
    ratio = case["heads_q"] // case["heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -INF, dtype=torch.float64, device=q.device)
    begin = 0
    for n in lengths:
        for i0 in range(0, n, 2048):
            i1 = min(n, i0 + 2048)
            j0 = max(0, i0 - case["window"] + 1) if case["window"] else 0
            i = torch.arange(i0, i1, device=q.device).view(-1, 1)
            j = torch.arange(j0, i1, device=q.device).view(1, -1)
            seen = j <= i
            if case["window"]:
                seen &= i - j < case["window"]
            for a in range(case["heads_q"]):
                kk, vv = (t[begin + j0:begin + i1, a // ratio].double() for t in (k, v))
                score = q[begin + i0:begin + i1, a].double() @ kk.t() / math.sqrt(case["dim"])
                score = torch.where(seen, score, torch.full_like(score, -INF))
                total = torch.logsumexp(score, 1)
                lse[begin + i0:begin + i1, a] = total
                out[begin + i0:begin + i1, a] = torch.exp(score - total.unsqueeze(1)) @ vv
        begin += n
    return out, lse
