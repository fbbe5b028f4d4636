"""Oracle of the decode-path operators (plain numpy): the paged 4-bit cache's bytes, block tables, attention and
log-probabilities. Bytes and tables are exact; attention and log-probabilities are in binary64."""

import numpy as np

SUB = 16


def layout(heads, dim, group, page, n_pages):
    sub = SUB * dim + 128 * (dim // group)
    head = sub * (page // SUB)
    return {"heads": heads, "dim": dim, "group": group, "page": page, "n_pages": n_pages, "sub_bytes": sub,
            "head_bytes": head, "page_bytes": head * heads, "total_bytes": head * heads * n_pages}


def quantise(v):
    """One group of binary32 values: (q, scale fp16, zero point)."""
    v = np.asarray(v, dtype=np.float32)
    mn, mx = min(np.float32(0), v.min()), max(np.float32(0), v.max())
    s16 = np.float16(np.float32(np.float32(mx - mn) / np.float32(15)))
    if s16 == 0:
        s16 = np.float16(1)
    s = np.float32(s16)
    z = min(max(np.rint(np.float32(-mn / s)), 0), 15)
    q = np.clip(np.rint((v / s).astype(np.float32)) + z, 0, 15)
    return q.astype(np.uint8), s16, np.float16(z + 0.0)  # a zero point of 0 is +0


def k_place(L, tau, d):
    """(byte in the subtile, nibble) of dim d of token tau of K."""
    p = min(L["dim"], 128)
    return d // p * 8 * p + tau * (p // 2) + d % p // 2, d % 2


def v_place(L, tau, d):
    dim = L["dim"]
    c, n, i = d % 8, d // 8 % 4, d // 32
    w = tau // 2 % 2 * (dim // 32) + i
    return 8 * dim + w // 4 * 512 + (4 * c + tau // 4) * 16 + w % 4 * 4 + tau % 2 * 2 + n // 2, n % 2


def places(L):
    """Index arrays of a subtile: K byte and shift [16, D], V byte and shift [16, D]."""
    out = []
    for f in (k_place, v_place):
        b = np.zeros((SUB, L["dim"]), dtype=np.int64)
        s = np.zeros((SUB, L["dim"]), dtype=np.uint8)
        for tau in range(SUB):
            for d in range(L["dim"]):
                at, nib = f(L, tau, d)
                b[tau, d], s[tau, d] = at, 4 * nib
        out += [b, s]
    return out


def append(L, cache, k, v, slots):
    """Writes k, v [T, heads, D] (any float type) into cache (uint8, modified) at slots."""
    pl = places(L)
    d, g = L["dim"], L["group"]
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        at, tau = slot % L["page"] // SUB, slot % SUB
        for h in range(L["heads"]):
            base = slot // L["page"] * L["page_bytes"] + h * L["head_bytes"] + at * L["sub_bytes"]
            for which, x in enumerate((k, v)):
                b, s = pl[2 * which][tau], pl[2 * which + 1][tau]
                for j in range(d // g):
                    q, s16, z = quantise(x[t, h, j * g:(j + 1) * g])
                    for i in range(g):
                        dim = j * g + i
                        o = base + b[dim]
                        cache[o] = (cache[o] & (0xF0 if s[dim] == 0 else 0x0F)) | (q[i] << s[dim])
                    o = base + 16 * d + which * 64 * (d // g) + 64 * j + 4 * tau
                    cache[o:o + 4] = np.array([s16, z], dtype=np.float16).view(np.uint8)


def values(L, cache, slots, head):
    """(K, V, zero-extended magnitudes s (q + z) of both) in binary64 of one head's tokens at slots: [T, D] each."""
    pl = places(L)
    d, g = L["dim"], L["group"]
    slots = np.asarray(slots, dtype=np.int64)
    tau = slots % SUB
    base = slots // L["page"] * L["page_bytes"] + head * L["head_bytes"] + slots % L["page"] // SUB * L["sub_bytes"]
    got, mags = [], []
    for which in (0, 1):
        q = (cache[base[:, None] + pl[2 * which][tau]] >> pl[2 * which + 1][tau]) & 15
        o = base[:, None] + 16 * d + which * 64 * (d // g) + 64 * (np.arange(d) // g) + 4 * tau[:, None]
        sz = np.stack([cache[o + i] for i in range(4)], -1).view(np.float16).astype(np.float64)
        got.append((q - sz[..., 1]) * sz[..., 0])
        mags.append((q + sz[..., 1]) * sz[..., 0])
    return got + mags


def plan(length, keep, add, table, free, count, page, n_slots):
    """List form of the step: returns (length, count, q_start, slots, pos, table, free), copies."""
    table, free = [list(r) for r in table], list(free)
    stack = free[:count]
    held = [-(-n // page) for n in length]
    need = [-(-(k + a) // page) for k, a in zip(keep, add)]
    given = [table[r][b] for r in range(len(length)) for b in range(need[r], held[r])]
    came = 0
    for r in range(len(length)):
        for b in range(held[r], need[r]):
            table[r][b] = given[came] if came < len(given) else stack.pop()
            came += 1
    stack += given[came:]
    free[:len(stack)] = stack
    start, slots, pos = [0], [], []
    for r in range(len(length)):
        start.append(start[-1] + add[r])
        for i in range(add[r]):
            p = keep[r] + i
            pos.append(p)
            slots.append(table[r][p // page] * page + p % page)
    pad = n_slots - len(slots)
    return ([k + a for k, a in zip(keep, add)], len(stack), start, slots + [-1] * pad, pos + [-1] * pad, table, free)


def attention(L, cache, q, q_start, length, table, scale, window=0, tree=None):
    """(out [T, Hq, D], lse [T, Hq], weight [T, Hq, D] = sum p |v|, size [T, Hq] = the largest sum of magnitudes that
    makes up one score), all binary64; NaN rows where no request has the token."""
    t, hq, d = q.shape
    ratio = hq // L["heads"]
    out, lse = np.full((t, hq, d), np.nan), np.full((t, hq), np.nan)
    weight, size = np.zeros((t, hq, d)), np.zeros((t, hq))
    q = q.astype(np.float64)
    for r in range(len(length)):
        n, ln = q_start[r + 1] - q_start[r], int(length[r])
        j = np.arange(ln)
        slots = np.asarray(table[r])[j // L["page"]].astype(np.int64) * L["page"] + j % L["page"]
        for h in range(L["heads"]):
            k, v, kmag, vmag = values(L, cache, slots, h)
            for i in range(n):
                tok, p = q_start[r] + i, ln - n + i
                if tree is not None:
                    see = np.array([x < ln - n or (int(tree[tok]) >> (x - (ln - n))) & 1 == 1 for x in j], dtype=bool)
                else:
                    see = (j <= p) & ((j > p - window) if window else True)
                for a in range(h * ratio, (h + 1) * ratio):
                    if not see.any():
                        out[tok, a], lse[tok, a] = 0, -np.inf
                        continue
                    s = k[see] @ q[tok, a] * scale
                    m = s.max()
                    e = np.exp(s - m)
                    out[tok, a], lse[tok, a] = e @ v[see] / e.sum(), m + np.log(e.sum())
                    weight[tok, a] = e @ vmag[see] / e.sum()
                    size[tok, a] = (kmag[see] @ np.abs(q[tok, a]) * abs(scale)).max()
    return out, lse, weight, size


def logprobs(x, tokens, top):
    """(tok_logp, lse, entropy, top_tok, top_logp, logp) of finite or -inf logits x [rows, vocab] in binary64."""
    x = np.asarray(x, dtype=np.float64)
    rows, vocab = x.shape
    m = x.max(1, keepdims=True)
    none = np.isneginf(m[:, 0])
    t = x - np.where(np.isneginf(m), 0, m)
    e = np.exp(t)
    s = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = m + np.log(s)
        lp = np.where(none[:, None], -np.inf, x - lse)
        entropy = np.where(none, 0, -np.where(e > 0, e / s * lp, 0).sum(1))
    order = np.argsort(-x, axis=1, kind="stable")[:, :top]
    top_tok = np.full((rows, top), -1, dtype=np.int32)
    top_lp = np.full((rows, top), -np.inf)
    top_tok[:, :order.shape[1]] = order
    top_lp[:, :order.shape[1]] = np.take_along_axis(lp, order, 1)
    tok_lp = None
    if tokens is not None:
        tok_lp = np.where(tokens == -1, 0.0, np.take_along_axis(lp, np.clip(tokens, 0, vocab - 1), 1))
    return tok_lp, lse[:, 0], entropy, top_tok, top_lp, lp
