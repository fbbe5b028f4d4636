"""Oracle of the prompt-path operators (numpy, binary64): 4-bit matrices and attention over packed prompts. Test infrastructure only; it
shares no code with the library.

Quantisation follows the definition number by number: every quotient is formed in binary64, where quotients of the few bits that the
operands have are decided as the exact ones are, and rounded by looking for the nearest member of the grid."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])


def layout(rows, k, block):
    """What sgemv_fp4_layout_query says."""
    tile = next(t for t in (8, 16, 32, 64, 128) if t >= rows or t == 128)
    kp = (k + 63) // 64 * 64
    big = (rows + 127) // 128
    scale_off = (rows + tile - 1) // tile * tile * kp // 2
    row_off = scale_off + big * 512 * ((kp + 4 * block - 1) // (4 * block))
    return {"rows": rows, "k": k, "block": block, "tile": tile, "kp": kp, "scale_off": scale_off, "row_off": row_off,
            "total_bytes": row_off + 512 * big}


def nearest(x, grid):
    """Places in an ascending grid of the members nearest to x >= 0; ties go to the even place, what is past the grid to its last."""
    hi = np.minimum(np.searchsorted(grid, x), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    below, above = x - grid[lo], grid[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def quantise(x, block):
    """x float64 [rows, k] -> codes [rows, kp], scale bytes [rows, groups * 4], row scales [rows] (NaN for a row with no number in it,
    whose other bytes are then 0 here)."""
    rows, k = x.shape
    kp = (k + 63) // 64 * 64
    width = (kp + 4 * block - 1) // (4 * block) * 4 * block
    bad = ~np.isfinite(x).all(axis=1)
    full = np.zeros((rows, width))
    full[:, :k] = np.where(bad[:, None], 0.0, x)
    b = full.reshape(rows, -1, block)
    m = np.abs(b).max(axis=2)
    if block == 32:
        with np.errstate(divide="ignore"):
            byte = np.where(m > 0, np.frexp(m)[1] - 1 - 2 + 127, 0)
        byte = np.clip(byte, 0, 254)
        scale, row = 2.0 ** (byte - 127.0), np.ones(rows)
    else:
        row = np.ones(rows)
        for r in range(rows):
            top = m[r].max()
            if top > 0:
                e = int(np.floor(np.log2(top / 2688))) - 2
                while top > 2688 * 2.0 ** e:
                    e += 1
                row[r] = 2.0 ** max(e, -100)
        byte = nearest(m / row[:, None] / 6, E4M3)
        scale = E4M3[byte] * row[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(scale[..., None] > 0, np.abs(b) / scale[..., None], 0.0)
    codes = nearest(t, E2M1) + 8 * (b < 0)
    return codes.reshape(rows, width)[:, :kp], byte, np.where(bad, np.nan, row)


def places(L):
    """Byte of every code [rows, kp] (values 2j in the low nibble), of every scale [rows, groups * 4] and of every row's scale [rows]."""
    r = np.arange(L["rows"])[:, None]
    c = np.arange(L["kp"])[None, :]
    t = L["tile"]
    code = ((r // t * (L["kp"] // 32) + c // 32) * t + r % t) * 16 + c % 32 // 2
    groups = (L["kp"] + 4 * L["block"] - 1) // (4 * L["block"])
    s = np.arange(4 * groups)[None, :]
    scale = L["scale_off"] + (r // 128 * groups + s // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + s % 4
    return code, scale, L["row_off"] + 4 * np.arange(L["rows"])


def pack(L, codes, scales, row):
    """(bytes, which of them mean something)."""
    out, used = np.zeros(L["total_bytes"], dtype=np.uint8), np.zeros(L["total_bytes"], dtype=bool)
    pc, ps, pr = places(L)
    np.add.at(out, pc, (codes << (4 * (np.arange(L["kp"]) % 2))).astype(np.uint8))
    out[ps] = scales
    words = row.astype(np.float32).view(np.uint8).reshape(-1, 4)
    out[pr[:, None] + np.arange(4)] = words
    used[pc], used[ps], used[pr[:, None] + np.arange(4)] = True, True, True
    return out, used


def values(L, data):
    """The values that the bytes stand for, float64 [rows, k]."""
    pc, ps, pr = places(L)
    code = (data[pc] >> (4 * (np.arange(L["kp"]) % 2)).astype(np.uint8)) & 15
    mag = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = 2.0 ** (data[ps] - 127.0) if L["block"] == 32 else E4M3[np.minimum(data[ps], 126)]
    row = np.ascontiguousarray(data[pr[:, None] + np.arange(4)]).view(np.float32)[:, 0].astype(np.float64)
    return (mag * np.repeat(scale, L["block"], axis=1)[:, :L["kp"]] * row[:, None])[:, :L["k"]]


def attention(q, k, v, start, length, scale, causal=True, window=0):
    """q [tokens, heads_q, dim], k, v [tokens, heads, dim], float64 -> out, lse, the weighted sums of |v|, and of every row the largest sum
    of score magnitudes; rows of no request are NaN."""
    ratio = q.shape[1] // k.shape[1]
    out, weight = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, size = np.full(q.shape[:2], np.nan), np.full(q.shape[:2], np.nan)
    for r in range(len(start) - 1):
        n = start[r + 1] - start[r] if length is None else length[r]
        for i in range(n):
            a = max(0, i - window + 1) if window else 0
            b = i + 1 if causal else n
            at = slice(start[r] + a, start[r] + b)
            row = start[r] + i
            kk, vv = k[at].repeat(ratio, axis=1), v[at].repeat(ratio, axis=1)
            t = np.einsum("hd,jhd->hj", q[row], kk) * scale
            top = t.max(axis=1, keepdims=True)
            p = np.exp(t - top)
            total = p.sum(axis=1, keepdims=True)
            p /= total
            out[row], weight[row] = np.einsum("hj,jhd->hd", p, vv), np.einsum("hj,jhd->hd", p, np.abs(vv))
            lse[row] = (top + np.log(total))[:, 0]
            size[row] = (np.einsum("hd,jhd->hj", np.abs(q[row]), np.abs(kk)) * abs(scale)).max(axis=1)
    return out, lse, weight, size
