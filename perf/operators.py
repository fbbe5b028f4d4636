"""Cases of the decode-path operators: the paged 4-bit KV cache (plan, append, read, attention) and the
log-probabilities that feed the beam step.

`run` computes them in their plain form (elementary torch operations in 32 bits) where `own` is false, and through the
library's entry points where it is true. `prepare` builds the inputs, packed cache included, from the seed alone.

The cache is a byte buffer of pages; a page holds, for each KV head, page/16 subtiles of 16 tokens:
  K nibbles  8*D bytes  [D/128 panels (one of D < 128)][16 tokens][panel/2 bytes], even dim in the low nibble
  V nibbles  8*D bytes  u16 [D/64][g = 8][t = 4][4][half = 2], 4 nibbles each: with w = 4 * first + fourth index,
             pair = w / (D/32), i = w % (D/32), the nibbles n = 0..3 are dims g + 8n + 32i of token 4t + 2 pair + half
  K scales   [D/group][16 tokens] {fp16 scale, fp16 zero point}, then V scales, the same
The value of a nibble q is (q - zero) * scale.
"""

import math

import torch

own = False

INF = float("inf")
FP = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    attn = dict(op="attention", window=0, tree=False, dtype="fp16", group=128)
    return [
        # block tables of one decode step: 64 running requests, one new token each, some finished
        dict(name="plan decode 64", op="plan", requests=64, page=64, most=4096, add=1, pad=0),
        # a large serving step: prompts of up to 512 tokens beside decodes, roll-backs and releases
        dict(name="plan mixed 4096", op="plan", requests=4096, page=16, most=1500, add=512, pad=1000),
        # one decode step of 8 beams of a 7B-class decoder (32 heads of 128), k and v cut from one fused projection
        dict(name="append decode 8", op="append", tokens=8, heads=32, dim=128, group=128, page=64, dtype="fp16"),
        # a long ragged prompt batch written at once, finer groups, small pages
        dict(name="append prompt 20011", op="append", tokens=20011, heads=8, dim=128, group=64, page=16, dtype="bf16"),
        # the smallest call: one request, one token, a short context of a 7B-class decoder
        dict(attn, name="attention single", requests=1, queries=1, most=333, heads=32, heads_q=32, dim=128, page=16),
        # a serving batch: 64 requests of 1 to 16384 tokens, four query heads a KV head
        dict(attn, name="attention batch 64", requests=64, queries=1, most=16384, heads=8, heads_q=32, dim=128, page=64),
        # one very long context, bf16, eight query heads a KV head
        dict(attn, name="attention long", requests=1, queries=1, most=262144, heads=8, heads_q=64, dim=128, page=128,
             dtype="bf16"),
        # tree verification: up to 12 draft tokens of a token tree a request, heads of 64
        dict(attn, name="attention tree", requests=24, queries=12, most=5000, heads=4, heads_q=16, dim=64, group=64,
             page=32, tree=True),
        # prompt chunks of up to 2048 tokens behind cached contexts
        dict(attn, name="attention chunk", requests=3, queries=2048, most=8192, heads=8, heads_q=32, dim=128, page=64),
        # the beam search's step: 20 beams, 32000 tokens, full rows for the beam step
        dict(name="logprobs beam 20", op="logprobs", rows=20, vocab=32000, dtype="fp16", given=1, top=20, full=True,
             banned=0.0),
        # one row of a large constrained vocabulary (most tokens banned), many alternatives
        dict(name="logprobs row 262144", op="logprobs", rows=1, vocab=262144, dtype="fp32", given=4, top=64, full=False,
             banned=0.9),
        # scoring a prompt: every position's given token, odd vocabulary
        dict(name="logprobs prompt 4096", op="logprobs", rows=4096, vocab=50001, dtype="bf16", given=1, top=5, full=False,
             banned=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "append", "attention", "attention", "attention", "logprobs"))
    if op == "plan":
        return dict(op=op, requests=_log(rng, 1, 4096), page=rng.choice((16, 32, 64, 128, 256)), most=_log(rng, 64, 8192),
                    add=_log(rng, 1, 512), pad=rng.randrange(0, 1000))
    dim = rng.choice((64, 128, 128, 256))
    group = rng.choice((64, 128)) if dim > 64 else 64
    page = rng.choice((16, 32, 64, 128, 256))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "append":
        heads = rng.choice((1, 2, 4, 8, 32))
        return dict(op=op, tokens=_log(rng, 1, 20011 * 8 * 128 // (max(heads, 8) * max(dim, 128))), heads=heads, dim=dim,
                    group=group, page=page, dtype=dtype)
    if op == "attention":
        heads = rng.choice((1, 2, 4, 8, 32))
        ratio = rng.choice((1, 2, 4, 5, 8)) if heads < 32 else 1
        requests = _log(rng, 1, 64)
        kind = rng.choice(("step", "step", "tree", "chunk"))
        queries = 1 if kind == "step" else (rng.randrange(2, 17) if kind == "tree" else _log(rng, 17, 2048))
        # no more cache than the large batch, no more products than the prompt chunks
        cap = min(262144, 64 * 16384 * 8 * 128 // (2 * requests * heads * dim),
                  3 * 2048 * 8192 * 32 * 128 // (2 * requests * queries * heads * ratio * dim))
        most = max(queries, 16, _log(rng, 16, max(17, cap)))
        window = rng.choice((0, 0, 0, _log(rng, 8, 4096))) if kind != "tree" else 0
        return dict(op=op, requests=requests, queries=queries, most=most, heads=heads, heads_q=heads * ratio, dim=dim,
                    group=group, page=page, dtype=dtype, window=window, tree=kind == "tree")
    vocab = _log(rng, 100, 262144)
    rows = _log(rng, 1, max(1, min(4096, 4096 * 50001 // (2 * vocab))))
    return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(("fp16", "bf16", "fp32")), given=rng.choice((0, 1, 3)),
                top=rng.choice((0, 1, 5, 20, 64)), full=rng.random() < 0.4, banned=rng.choice((0.0, 0.0, 0.5)))


def _spread(i, step):
    """The i-th of numbers spread evenly over [0, 1)."""
    return (0.5 + i * step) % 1.0


def _lengths(case):
    """(length, new tokens) of every request; the lengths hold the new tokens."""
    n, got = case["requests"], []
    for i in range(n):
        new = 1 if case["queries"] == 1 else max(1, int(case["queries"] * (1 - 0.8 * _spread(i, 0.7548776662)) + 0.5))
        most = case["most"] if n == 1 else int(case["most"] * _spread(i, 0.6180339887))
        if n > 3 and i == 2 and case["queries"] > 1:
            new = 0  # a request without queries in this step
        got.append((max(new, 1, most), new))
    return got


def _plan_counts(case):
    """(length, kept, added) of every request."""
    got = []
    for i in range(case["requests"]):
        length = int(case["most"] * _spread(i, 0.6180339887))
        added = 1 if case["add"] == 1 else (1 if i % 4 else 1 + int(case["add"] * _spread(i, 0.7548776662)))
        kept = length
        if i % 16 == 5:  # finished
            kept, added = 0, 0
        elif i % 16 == 9:  # the last draft tokens are taken back
            kept = max(0, length - 7)
        got.append((length, kept, added))
    return got


def work(case):
    op = case["op"]
    if op == "plan":
        c = _plan_counts(case)
        t, p = sum(x[2] for x in c), case["page"]
        moved = sum(abs(-(-(k + a) // p) + (-n // p)) for n, k, a in c)
        return {"bytes": 12 * len(c) + 8 * len(c) + 4 * len(c) + 12 * (t + case["pad"]) + 8 * moved, "flops": 0}
    if op == "append":
        n = case["tokens"] * case["heads"]
        held = n * (case["dim"] + 8 * case["dim"] // case["group"])
        return {"bytes": 2 * (2 * 2 * n * case["dim"] + held) + 16 * case["tokens"], "flops": 0}
    if op == "attention":
        d, w = case["dim"], case["window"]
        seen = pairs = tokens = 0
        for length, new in _lengths(case):
            tokens += new
            first = length - new
            seen += 0 if new == 0 else (length if w == 0 else min(length, w + new - 1))
            for i in range(new):
                pairs += min(first + i + 1, w) if w else first + i + 1
        return {"bytes": seen * case["heads"] * (d + 8 * d // case["group"]) + tokens * case["heads_q"] * (4 * d + 4),
                "flops": 4 * d * case["heads_q"] * pairs}
    size = 4 if case["dtype"] == "fp32" else 2
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (size + (4 if case["full"] else 0)) + case["rows"] * (8 * case["given"] + 8 * case["top"] + 8),
            "flops": 4 * n}


# ------------------------------------------------------------------------------------------------ inputs

def _quantise(x, group):
    """x fp32 [..., D] -> (q int32 [..., D], scale fp16 [..., D/group], zero fp32 [..., D/group])."""
    g = x.unflatten(-1, (-1, group))
    lo, hi = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    s16 = ((hi - lo) / torch.full_like(hi, 15.0)).half()
    s16 = torch.where(s16 == 0, torch.ones_like(s16), s16)
    s = s16.float()
    z = torch.round(-lo / s).clamp(0, 15)
    q = (torch.round(g / s.unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 15)
    return q.flatten(-2).to(torch.int32), s16, z


def _pack_k(q):
    """q int32 [..., 16, D] -> uint8 [..., 8 * D]."""
    d = q.shape[-1]
    b = (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8)  # [..., 16, D / 2]
    half = min(d, 128) // 2
    return b.unflatten(-1, (-1, half)).transpose(-3, -2).flatten(-3)


def _pack_v(q):
    """q int32 [..., 16, D] -> uint8 [..., 8 * D]."""
    d = q.shape[-1]
    x = q.unflatten(-2, (4, 2, 2)).unflatten(-1, (d // 32, 4, 8))  # ... t pair half i n g
    n = x.dim() - 6
    x = x.permute(*range(n), n + 1, n + 3, n + 5, n + 0, n + 2, n + 4)  # ... pair i g t half n
    x = x.flatten(n, n + 1).unflatten(n, (d // 64, 4))  # ... first fourth g t half n
    x = x.permute(*range(n), n + 0, n + 2, n + 3, n + 1, n + 4, n + 5)  # ... first g t fourth half n
    lo = (x[..., 0] | (x[..., 1] << 4)).to(torch.uint8)
    hi = (x[..., 2] | (x[..., 3] << 4)).to(torch.uint8)
    return torch.stack((lo, hi), -1).flatten(n)


def _pack_scales(s16, z):
    """[..., 16, groups] each -> uint8 [..., groups * 64]."""
    w = torch.stack((s16, z.half()), -1).transpose(-3, -2).contiguous()  # ... group token 2
    return w.flatten(-3).view(torch.uint8)


def _pack(k, v, group):
    """k, v fp32 [..., 16, D] -> the bytes of the subtiles, uint8 [..., 16 D + 128 D / group]."""
    kq, ks, kz = _quantise(k, group)
    vq, vs, vz = _quantise(v, group)
    return torch.cat((_pack_k(kq), _pack_v(vq), _pack_scales(ks, kz), _pack_scales(vs, vz)), -1)


def _sub(case):
    return 16 * case["dim"] + 128 * (case["dim"] // case["group"])


def _prepare_attention(case, gen, dev):
    h, d, page, nr = case["heads"], case["dim"], case["page"], case["requests"]
    pairs = _lengths(case)
    blocks = [-(-length // page) for length, _ in pairs]
    used, cap = sum(blocks), max(blocks)
    pages = used + 7
    order = torch.randperm(pages, generator=gen, device=dev)[:used]
    table = torch.full((nr, cap), -1, dtype=torch.int32, device=dev)
    at = torch.tensor([r * cap + b for r in range(nr) for b in range(blocks[r])], device=dev)
    table.view(-1)[at] = order.to(torch.int32)
    # what no token was written to holds bytes whose scales are not numbers
    cache = torch.full((pages, h, page // 16, _sub(case)), 255, dtype=torch.uint8, device=dev)
    bias = torch.randn((2, h, 1, 1, d), generator=gen, device=dev) * 0.5
    fill = torch.tensor([min(page, pairs[r][0] - b * page) for r in range(nr) for b in range(blocks[r])], device=dev)
    step = max(1, (1 << 27) // (h * page * d))
    for a in range(0, used, step):
        n = min(step, used - a)
        k = torch.randn((n, h, page // 16, 16, d), generator=gen, device=dev) + bias[0]
        v = torch.randn((n, h, page // 16, 16, d), generator=gen, device=dev) + bias[1]
        packed = _pack(k, v, case["group"])
        live = torch.arange(page, device=dev).view(1, page // 16, 16) < fill[a:a + n].view(n, 1, 1)
        ng = d // case["group"]
        scales = packed[..., 16 * d:].unflatten(-1, (2 * ng, 16, 4))
        scales.masked_fill_(~live.view(n, 1, page // 16, 1, 16, 1), 255)
        cache[order[a:a + n]] = packed
    tokens = sum(new for _, new in pairs)
    dtype = FP[case["dtype"]]
    starts = [0]
    for _, new in pairs:
        starts.append(starts[-1] + new)
    s = {"cache": cache.view(-1), "table": table, "pages": pages}
    # the queries are a slice of a fused projection's rows
    rows = torch.randn((tokens, case["heads_q"] + 2 * h, d), generator=gen, device=dev).to(dtype)
    s["q"] = rows[:, :case["heads_q"]]
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["length"] = torch.tensor([length for length, _ in pairs], dtype=torch.int32, device=dev)
    s["tree"] = None
    if case["tree"]:
        picks = torch.rand(tokens, generator=gen, device=dev).tolist()
        masks = []
        for r in range(nr):
            mine = []
            for i in range(pairs[r][1]):
                parent = int(picks[starts[r] + i] * i) if i else -1
                mine.append((mine[parent] if i else 0) | (1 << i))
            masks += mine
        s["tree"] = torch.tensor(masks, dtype=torch.int64, device=dev)
    s["out"] = torch.empty((tokens, case["heads_q"], d), dtype=dtype, device=dev)
    s["lse"] = torch.empty((tokens, case["heads_q"]), dtype=torch.float32, device=dev)
    s["workspace"] = torch.zeros(32 << 20, dtype=torch.uint8, device=dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if op == "attention":
        s.update(_prepare_attention(case, gen, dev))
    elif op == "plan":
        counts = _plan_counts(case)
        page, nr = case["page"], case["requests"]
        held = [-(-length // page) for length, _, _ in counts]
        cap = max(max(h, -(-(k + a) // page)) for h, (_, k, a) in zip(held, counts)) + 1
        pages = sum(max(h, -(-(k + a) // page)) for h, (_, k, a) in zip(held, counts)) + 16
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.full((nr, cap), -1, dtype=torch.int32, device=dev)
        at = torch.tensor([r * cap + b for r in range(nr) for b in range(held[r])], dtype=torch.int64, device=dev)
        table.view(-1)[at] = order[:sum(held)]
        free = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        free[:pages - sum(held)] = order[sum(held):]
        most = sum(a for _, _, a in counts) + case["pad"]
        s.update(table=table, free=free, most=most, count=torch.tensor([pages - sum(held)], dtype=torch.int32, device=dev))
        s["length"], s["keep"], s["add"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in zip(*counts))
        s["out"] = (torch.empty(nr, dtype=torch.int32, device=dev), torch.empty(1, dtype=torch.int32, device=dev),
                    torch.empty(nr + 1, dtype=torch.int32, device=dev), torch.empty(most, dtype=torch.int64, device=dev),
                    torch.empty(most, dtype=torch.int32, device=dev))
    elif op == "append":
        t, h, d, page = case["tokens"], case["heads"], case["dim"], case["page"]
        dtype = FP[case["dtype"]]
        # requests of up to 600 tokens, each in pages of its own in random order, the last token of each padded out
        pages = t // page + t // 600 + 2
        order = torch.randperm(pages, generator=gen, device=dev)
        i = torch.arange(t, device=dev)
        per = (600 // page) * page if page <= 600 else page
        at = i // per * (-(-per // page)) + (i % per) // page
        at = at.clamp(max=pages - 1)
        s["slots"] = order[at] * page + (i % per) % page
        if t > 2:
            s["slots"][t // 2] = -1  # a padded place of a step of fixed shape
        rows = torch.randn((t, 3 * h, d), generator=gen, device=dev)
        rows += torch.randn((1, 3 * h, d), generator=gen, device=dev) * 0.5
        rows = rows.to(dtype)
        s.update(k=rows[:, h:2 * h], v=rows[:, 2 * h:], pages=pages)
        s["cache"] = torch.full((pages * h * (page // 16) * _sub(case),), 255, dtype=torch.uint8, device=dev)
        s["out"] = (torch.empty((t, h, d), dtype=dtype, device=dev), torch.empty((t, h, d), dtype=dtype, device=dev))
    else:
        n, vocab = case["rows"], case["vocab"]
        x = torch.randn((n, vocab), generator=gen, device=dev) * 2.5
        if case["banned"]:
            x.masked_fill_(torch.rand((n, vocab), generator=gen, device=dev) < case["banned"], -INF)
        s["logits"] = x.to(FP[case["dtype"]])
        top = case["top"]
        s["tokens"] = None
        if case["given"]:
            s["tokens"] = torch.randint(0, vocab, (n, case["given"]), generator=gen, device=dev, dtype=torch.int32)
            if n > 2:
                s["tokens"][1, 0] = -1  # no token asked for here
        f = dict(dtype=torch.float32, device=dev)
        s["out"] = (torch.empty((n, case["given"]), **f) if case["given"] else None, torch.empty(n, **f), torch.empty(n, **f),
                    torch.empty((n, top), dtype=torch.int32, device=dev) if top else None,
                    torch.empty((n, top), **f) if top else None, torch.empty((n, vocab), **f) if case["full"] else None)
    return s


# ------------------------------------------------------------------------------------------------ the operators

def run(s):
    op = s["case"]["op"]
    if op == "plan":
        return _run_plan(s)
    if op == "append":
        return _run_append(s)
    if op == "attention":
        return _run_attention(s)
    return _run_logprobs(s)


def _layout(s):
    """The cache's layout, a plain struct that a program asks for once and keeps beside the cache."""
    if "layout" not in s:
        import int4_weight_only_sgemv_gb300 as sg
        c = s["case"]
        s["layout"] = sg.sgemv_kv_layout_query(c["heads"], c["dim"], c["group"], c["page"], s["pages"])
    return s["layout"]


def _run_plan(s):
    c = s["case"]
    if own:
        import int4_weight_only_sgemv_gb300 as sg
        sg.sgemv_kv_plan(s["length"], s["keep"], s["add"], s["table"], s["free"], s["count"], c["page"], s["out"],
                         status=s["status"])
        return list(s["out"]) + [s["table"], s["free"]]
    page, most = c["page"], s["most"]
    length, keep, add = s["length"].long(), s["keep"].long(), s["add"].long()
    table, free, dev = s["table"].clone(), s["free"].clone(), length.device
    nr, cap = table.shape
    held, new = (length + page - 1) // page, (keep + add + page - 1) // page
    start = torch.zeros(nr + 1, dtype=torch.int64, device=dev)
    start[1:] = torch.cumsum(add, 0)
    b = torch.arange(cap, device=dev)
    gone = (b >= new[:, None]) & (b < held[:, None])
    come = (b >= held[:, None]) & (b < new[:, None])
    released, rank = table[gone].long(), torch.cumsum(come.view(-1).long(), 0).view(nr, cap) - 1
    nrel, ntake = gone.sum(), come.sum()
    count = s["count"].long()[0]
    pool = torch.cat((released, free.long()))  # index i < nrel: released; then the stack from its top
    want = rank[come]
    take = torch.where(want < nrel, want, released.shape[0] + count - 1 - (want - nrel))
    table[come] = pool[take].to(torch.int32)
    i = torch.arange(released.shape[0], device=dev)
    left = i >= ntake
    free[(count + i - ntake)[left]] = released[left].to(torch.int32)
    t = torch.arange(most, device=dev)
    r = (torch.searchsorted(start, t, right=True) - 1).clamp(max=nr - 1)
    pos = keep[r] + t - start[r]
    live = t < start[-1]
    pos = torch.where(live, pos, 0)
    slots = table[r, pos // page].long() * page + pos % page
    return [(keep + add).to(torch.int32), (count + nrel - ntake).to(torch.int32).view(1), start.to(torch.int32),
            torch.where(live, slots, -1), torch.where(live, pos, -1).to(torch.int32), table, free]


def _place(case, slots):
    """Byte offset of the subtile and place in it of every (slot, head): [T, H], [T, 1]."""
    page, h = case["page"], case["heads"]
    head = torch.arange(h, device=slots.device)
    sub = slots[:, None] // page * (h * (page // 16)) + head * (page // 16) + slots[:, None] % page // 16
    return sub * _sub(case), slots[:, None] % 16


def _where(case, base, tok):
    """16-bit places in the cache of one token's values: K [T, H, D / 4], V [T, H, D / 4], scales [T, H, 2, groups, 2]."""
    d, dev = case["dim"], base.device
    ng, panel = d // case["group"], min(d, 128)
    x = torch.arange(d // 4, device=dev)  # four dims at a time: 4x .. 4x + 3
    k = base[..., None] + (4 * x // panel) * (8 * panel) + tok[..., None] * (panel // 2) + (4 * x % panel) // 2
    g, i = x % 8, x // 8  # dims g, g + 8, g + 16, g + 24 of block i
    w = (tok[..., None] // 2 % 2) * (d // 32) + i
    v = base[..., None] + 8 * d + w // 4 * 512 + (g * 4 + tok[..., None] // 4) * 16 + w % 4 * 4 + tok[..., None] % 2 * 2
    which, group, part = (torch.arange(n, device=dev) for n in (2, ng, 2))
    sz = base[..., None, None, None] + 16 * d + which[:, None, None] * 64 * ng + group[:, None] * 64 + part * 2
    return k // 2, v // 2, (sz + tok[..., None, None, None] * 4) // 2


def _four(q):
    """[..., n, 4] -> the 16-bit words that hold four nibbles each."""
    return q[..., 0] | (q[..., 1] << 4) | (q[..., 2] << 8) | (q[..., 3] << 12)


def _run_append(s):
    c = s["case"]
    if own:
        import int4_weight_only_sgemv_gb300 as sg
        layout = _layout(s)
        sg.sgemv_kv_append(layout, s["cache"], s["k"], s["v"], s["slots"], status=s["status"])
        sg.sgemv_kv_read(layout, s["cache"], s["slots"], *s["out"], status=s["status"])
        return s["out"]
    d, group = c["dim"], c["group"]
    live = s["slots"] >= 0
    base, tok = _place(c, s["slots"].clamp(min=0))
    at_k, at_v, at_s = _where(c, base, tok)
    words = s["cache"].view(torch.int16)
    kq, ks, kz = _quantise(s["k"].float(), group)
    vq, vs, vz = _quantise(s["v"].float(), group)
    words[at_k[live]] = _four(kq.unflatten(-1, (-1, 4)))[live].to(torch.int16)
    words[at_v[live]] = _four(vq.unflatten(-1, (-1, 4, 8)).transpose(-1, -2).flatten(-3, -2))[live].to(torch.int16)
    sz = torch.stack((torch.stack((ks, kz.half()), -1), torch.stack((vs, vz.half()), -1)), 2)
    words[at_s[live]] = sz.view(torch.int16)[live]
    # back out of the cache
    shift = torch.tensor([0, 4, 8, 12], device=words.device)
    k = (words[at_k].int()[..., None] >> shift & 15).flatten(-2).float()
    v = (words[at_v].int()[..., None] >> shift & 15).unflatten(-2, (-1, 8)).transpose(-1, -2).flatten(-3).float()
    sz = words[at_s].view(torch.float16).float()
    got = []
    for which, x in ((0, k), (1, v)):
        x = (x.unflatten(-1, (-1, group)) - sz[:, :, which, :, 1:]) * sz[:, :, which, :, :1]
        got.append(torch.where(live[:, None, None], x.flatten(-2), 0.0).to(s["out"][0].dtype))
    return tuple(got)


def _unpack(case, b):
    """uint8 [R, blocks, H, page / 16, sub] -> K, V fp32 [R, H, L, D]."""
    d, group = case["dim"], case["group"]
    ng, n = d // group, b.dim() - 1
    both = []
    kb = b[..., :8 * d].unflatten(-1, (-1, 16, min(d, 128) // 2)).transpose(-3, -2).flatten(-2)
    k = torch.stack((kb & 15, kb >> 4), -1).flatten(-2)  # ... 16 D
    vb = b[..., 8 * d:16 * d].unflatten(-1, (d // 64, 8, 4, 4, 2, 2))  # first g t fourth half byte
    v = torch.stack((vb & 15, vb >> 4), -1).flatten(-2)  # ... n
    v = v.permute(*range(n), n + 0, n + 3, n + 1, n + 2, n + 4, n + 5).flatten(n, n + 1).unflatten(n, (2, d // 32))
    # pair i g t half n -> t pair half i n g
    v = v.permute(*range(n), n + 3, n + 0, n + 4, n + 1, n + 5, n + 2).flatten(n, n + 2).flatten(n + 1)
    sz = b[..., 16 * d:].contiguous().view(torch.float16).unflatten(-1, (2, ng, 16, 2)).float()
    for which, x in ((0, k), (1, v)):
        s, z = (sz[..., which, :, :, j].transpose(-1, -2).unsqueeze(-1) for j in (0, 1))  # ... 16 groups 1
        x = ((x.float().unflatten(-1, (ng, group)) - z) * s).flatten(-2)  # R blocks H page/16 16 D
        both.append(x.transpose(1, 2).flatten(2, 4))
    return both


def _run_attention(s):
    c = s["case"]
    scale = 1.0 / math.sqrt(c["dim"])
    if own:
        import int4_weight_only_sgemv_gb300 as sg
        sg.sgemv_kv_attention(_layout(s), s["cache"], s["q"], s["starts"], s["length"], s["table"], s["out"],
                              c["queries"], scale, s["workspace"], lse=s["lse"], window=c["window"], tree=s["tree"],
                              status=s["status"])
        return s["out"], s["lse"]
    h, hq, d, page = c["heads"], c["heads_q"], c["dim"], c["page"]
    nr, nq = c["requests"], c["queries"]
    cache = s["cache"].view(-1, h, page // 16, _sub(c))
    k, v = _unpack(c, cache[s["table"].long().clamp(min=0)])
    size, dev = k.shape[2], k.device
    start, length = s["starts"].long(), s["length"].long()
    new = start[1:] - start[:-1]
    i, j = torch.arange(nq, device=dev), torch.arange(size, device=dev)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # [R, nq]
    q = s["q"].float()[row].unflatten(2, (h, hq // h)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # R H G*nq D
    first = (length - new)[:, None, None]
    place = first + i[:, None]
    if c["tree"]:
        bits = s["tree"][row][:, :, None]
        see = (j < first) | (((bits >> (j - first).clamp(0, 63)) & 1).bool() & (j < length[:, None, None]))
    else:
        see = j <= place
        if c["window"]:
            see = see & (j > place - c["window"])
    see = see[:, None, None]  # R 1 1 nq L
    v = torch.where((j < length[:, None])[:, None, :, None], v, 0.0)
    score = (torch.matmul(q, k.transpose(-1, -2)) * scale).unflatten(2, (hq // h, nq))
    score = torch.where(see, score, -INF)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -INF, 0.0, top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(2, 3), v).unflatten(2, (hq // h, nq)) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    live = i < new[:, None]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live]
    return o.to(s["out"].dtype), lse.permute(0, 3, 1, 2).flatten(2)[live]


def _run_logprobs(s):
    c = s["case"]
    if own:
        import int4_weight_only_sgemv_gb300 as sg
        sg.sgemv_logprobs(s["logits"], s["out"], tokens=s["tokens"], status=s["status"])
        return s["out"]
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    lp = x - lse
    p = e / total
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    given = top_tok = top_lp = None
    if c["given"]:
        given = torch.where(s["tokens"] < 0, 0.0, lp.gather(1, s["tokens"].long().clamp(min=0)))
    if c["top"]:
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        top_tok, top_lp = order.to(torch.int32), lp.gather(1, order)
        miss = c["top"] - order.shape[1]
        if miss > 0:
            top_tok = torch.nn.functional.pad(top_tok, (0, miss), value=-1)
            top_lp = torch.nn.functional.pad(top_lp, (0, miss), value=-INF)
    return given, lse.squeeze(-1), entropy, top_tok, top_lp, lp if c["full"] else None


# ------------------------------------------------------------------------------------------------ in 64 bits

def _fetch(case, cache, pages, places):
    """K and V in 64 bits of the tokens at (page, place in page): [T, H, D] each, byte by byte from the layout."""
    h, d, page, group = case["heads"], case["dim"], case["page"], case["group"]
    sub, dev = _sub(case), cache.device
    dims, head = torch.arange(d, device=dev), torch.arange(h, device=dev)
    start = ((pages[:, None] * h + head) * (page // 16) + (places // 16)[:, None]) * sub  # [T, H]
    tau = (places % 16)[:, None, None]
    width = min(d, 128)
    kat = start[..., None] + dims // width * (16 * width // 2) + tau * (width // 2) + dims % width // 2
    kq = (cache[kat] >> (4 * (dims % 2)).to(torch.uint8)) & 15
    block, n, g = dims // 32, dims // 8 % 4, dims % 8
    word = tau // 2 % 2 * (d // 32) + block
    vat = start[..., None] + 8 * d + word // 4 * 512 + g * 64 + tau // 4 * 16 + word % 4 * 4 + tau % 2 * 2 + n // 2
    vq = (cache[vat] >> (4 * (n % 2)).to(torch.uint8)) & 15
    half = cache.view(torch.float16)
    got = []
    for which, q in enumerate((kq, vq)):
        at = (start[..., None] + 16 * d + which * 64 * (d // group) + dims // group * 64 + tau * 4) // 2
        got.append((q.double() - half[at + 1].double()) * half[at].double())
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "append":
        live = s["slots"] >= 0
        got = []
        for x in (s["k"], s["v"]):
            g = x.double().reshape(x.shape[0], x.shape[1], -1, case["group"])
            lo, hi = g.min(-1, keepdim=True).values.clamp(max=0), g.max(-1, keepdim=True).values.clamp(min=0)
            scale = ((hi - lo) / 15).half().double()
            scale[scale == 0] = 1
            zero = (-lo / scale).round().clamp(0, 15)
            val = (((g / scale).round() + zero).clamp(0, 15) - zero) * scale
            got.append(val.reshape(x.shape) * live[:, None, None])
        return tuple(got)
    if op == "attention":
        h, hq, d, page, w = case["heads"], case["heads_q"], case["dim"], case["page"], case["window"]
        out, lse, at = [], [], 0
        for r, (length, new) in enumerate(_lengths(case)):
            if new == 0:
                continue
            q = s["q"][at:at + new].double().view(new, h, hq // h, d)
            first = length - new
            rows = torch.arange(new, device=q.device)
            low = torch.full((new, h, hq // h), -INF, dtype=torch.float64, device=q.device)
            total = torch.zeros_like(low)
            acc = torch.zeros((new, h, hq // h, d), dtype=torch.float64, device=q.device)
            step = max(16, min(16384, (1 << 27) // (new * hq)))
            begin = max(0, first - w + 1) if w else 0
            for a in range(begin, length, step):
                j = torch.arange(a, min(length, a + step), device=q.device)
                k, v = _fetch(case, s["cache"], s["table"][r, j // page].long(), j % page)
                sc = torch.einsum("nhgd,lhd->nhgl", q, k) / math.sqrt(d)
                if case["tree"]:
                    mine = s["tree"][at:at + new]
                    ok = torch.stack([(j < first) | ((mine[i] >> (j - first).clamp(min=0)) & 1 == 1) for i in range(new)])
                else:
                    ok = j[None] <= (first + rows)[:, None]
                    if w:
                        ok &= j[None] > (first + rows)[:, None] - w
                sc.masked_fill_(~ok[:, None, None], -INF)
                top = torch.maximum(low, sc.amax(-1))
                ref = torch.where(top == -INF, 0.0, top)
                p = torch.exp(sc - ref[..., None])
                fade = torch.exp(low - ref)
                total = total * fade + p.sum(-1)
                acc = acc * fade[..., None] + torch.einsum("nhgl,lhd->nhgd", p, v)
                low = top
            out.append((acc / total.clamp(min=1e-300)[..., None]).view(new, hq, d))
            lse.append((low + torch.log(total)).view(new, hq))
            at += new
        return torch.cat(out), torch.cat(lse)
    given, lse, entropy, tops, full = [], [], [], [], []
    n, top = case["rows"], min(case["top"], case["vocab"])
    step = max(1, (1 << 26) // case["vocab"])
    for a in range(0, n, step):
        x = s["logits"][a:a + step].double()
        z = torch.logsumexp(x, -1, keepdim=True)
        lp = x - z
        lse.append(z[:, 0])
        entropy.append(-torch.special.xlogy(torch.exp(lp), torch.exp(lp)).sum(-1))
        if case["given"]:
            t = s["tokens"][a:a + step].long()
            given.append(torch.where(t >= 0, torch.take_along_dim(lp, t.clamp(min=0), 1), torch.zeros_like(t).double()))
        if top:
            best = torch.topk(lp, top, -1).values
            tops.append(torch.cat((best, best.new_full((best.shape[0], case["top"] - top), -INF)), 1))
        if case["full"]:
            full.append(lp)
    join = lambda x: torch.cat(x) if x else None  # noqa: E731
    return join(given), join(lse), join(entropy), None, join(tops), join(full)
