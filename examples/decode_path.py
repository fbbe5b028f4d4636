"""One decode path with every operator: tree-based parallel verification on a small decoder.

A decoder with INT4 layers (2:4 sparse and dense, as the layer table says) writes its keys and values into a paged 4-bit
cache, attends over it, and its head's logits become the log-probabilities that the trie-constrained beam search reads:

  sgemv_kv_plan       pages and slots of the step's tokens (and of draft tokens taken back)
  sgemv_run_stack     q, k and v of a layer in one launch; o; gate and up; down
  sgemv_kv_append     k and v into the cache          sgemv_kv_attention  of the step's tokens over it
  sgemv_run_dense     the head                        sgemv_logprobs      entropy, alternatives, full rows
  sgemv_beam_decode   all positions' beam-score steps over the trie, and the traceback

The method is the one of "Efficient LLM-based Advertising via Model Compression and Parallel Verification" (§3.4): the draft
tokens of one pass are scored together, the trie filters them, and the pages of draft tokens that the best sequence does
not keep go back to the pool. Weights are random: the example shows the calls, not a language.

Run: python examples/decode_path.py
"""

from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import int4_weight_only_sgemv_gb300 as sg  # noqa: E402
import synth  # noqa: E402

MAX_ROWS = 8  # rows of a GEMV


class Decoder:
    """A pre-norm decoder with grouped query heads. Its seven linears a block and its head are packed INT4."""

    def __init__(self, vocab=4096, hidden=1024, heads_q=8, heads=2, ffn=2816, blocks=2, page=16, pages=64, requests=1, seed=0):
        self.vocab, self.hidden, self.heads_q, self.heads, self.blocks = vocab, hidden, heads_q, heads, blocks
        self.dim, self.page = hidden // heads_q, page
        dev = torch.device("cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.embed = torch.from_numpy(synth.activations(vocab, hidden, "example", "embed", seed)).to(dev)
        shapes = {"q": (heads_q * self.dim, hidden), "k": (heads * self.dim, hidden), "v": (heads * self.dim, hidden),
                  "o": (hidden, heads_q * self.dim), "gate": (ffn, hidden), "up": (ffn, hidden), "down": (hidden, ffn)}
        self.layers = []
        for b in range(blocks):
            layer = {}
            for name, (n, k) in shapes.items():
                w = torch.from_numpy(synth.weights(n, k, "example", b, name, seed, std=k ** -0.5)).to(dev)
                fmt = sg.SGEMV_FMT_SPARSE24 if name in ("gate", "up") else sg.SGEMV_FMT_DENSE
                layer[name] = sg.pack(w, fmt, 128, status=self.status)
            self.layers.append(layer)
        w = torch.from_numpy(synth.weights(vocab, hidden, "example", "head", seed, std=4 * hidden ** -0.5)).to(dev)
        self.head = sg.pack(w, sg.SGEMV_FMT_DENSE, 128, status=self.status)
        # a cache a block, all with the same block table; the pool of free pages
        self.kv = sg.sgemv_kv_layout_query(heads, self.dim, min(128, self.dim), page, pages)
        self.caches = [sg.kv_cache(self.kv) for _ in range(blocks)]
        self.workspace = sg.kv_workspace()
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((requests, pages), -1, **i32)
        self.free = torch.arange(pages, **i32)
        self.free_count = torch.tensor([pages], **i32)
        self.length = torch.zeros(requests, **i32)

    def plan(self, keep, add, n_slots):
        """Tokens kept and added a request; returns (q_start, slots). The lengths and the pool move on."""
        i32 = dict(dtype=torch.int32, device=self.table.device)
        keep = self.length if keep is None else torch.tensor(keep, **i32)
        out = (torch.empty_like(self.length), torch.empty_like(self.free_count), torch.empty(self.length.numel() + 1, **i32),
               torch.empty(n_slots, dtype=torch.int64, device=self.table.device), torch.empty(n_slots, **i32))
        sg.sgemv_kv_plan(self.length, keep, torch.tensor(add, **i32), self.table, self.free, self.free_count, self.page, out,
                         status=self.status)
        self.length, self.free_count = out[0], out[1]
        return out[2], out[3]

    def _linears(self, layer, names, x):
        """The named linears of x [rows, in], each a part of one tensor [rows, sum of outputs]; one launch of independent layers."""
        out = [torch.empty((x.shape[0], layer[n][0].n), dtype=torch.float16, device=x.device) for n in names]
        sg.sgemv_run_stack([(*layer[n], x, y) for n, y in zip(names, out)], x.shape[0], status=self.status)
        return out

    def attend(self, block, q, q_start):
        rows = q.shape[0]
        return sg.kv_attention(self.kv, self.caches[block], q, q_start, self.length, self.table, rows, 1 / math.sqrt(self.dim),
                               self.workspace, status=self.status)

    def step(self, tokens, keep=None, attend=None):
        """Runs tokens (ids, up to 8, of the one request) behind the cache; returns the logits [rows, vocab], fp16."""
        rows = len(tokens)
        assert rows <= MAX_ROWS
        q_start, slots = self.plan(keep, [rows], rows)
        x = self.embed[torch.tensor(tokens, device=self.embed.device)].float()
        norm = lambda t: (t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)).half()  # noqa: E731
        for b, layer in enumerate(self.layers):
            h = norm(x)
            q, k, v = self._linears(layer, ("q", "k", "v"), h)
            sg.sgemv_kv_append(self.kv, self.caches[b], k.view(rows, self.heads, self.dim), v.view(rows, self.heads, self.dim), slots,
                               status=self.status)
            o = (attend or self.attend)(b, q.view(rows, self.heads_q, self.dim), q_start)
            x = x + self._linears(layer, ("o",), o.reshape(rows, -1))[0].float()
            gate, up = self._linears(layer, ("gate", "up"), norm(x))
            x = x + self._linears(layer, ("down",), torch.nn.functional.silu(gate.float()).mul(up.float()).half())[0].float()
        return sg.gemv(*self.head, norm(x), status=self.status)


def verify(model, trie, logp, k):
    """Beam search over the trie with one row of log-probabilities a position: (sequences [k, steps], scores of the last step)."""
    steps = logp.shape[0]
    i32 = dict(dtype=torch.int32, device=logp.device)
    out = (torch.empty((steps, k), **i32), torch.empty((steps, k), dtype=torch.float32, device=logp.device), torch.empty((steps, k), **i32),
           torch.empty((steps, k), **i32), torch.empty(steps, **i32))
    seq = torch.empty((k, steps), **i32)
    sg.sgemv_beam_decode(trie, torch.zeros(1, **i32), torch.zeros(1, device=logp.device), [logp[t:t + 1] for t in range(steps)], k, out,
                         seq, shared_row=True, status=model.status)
    return seq, out[1][-1]


def run(prompt=40, drafts=4, beams=6, attend=None, seed=0):
    """A prompt into the cache, one verification pass of `drafts` positions, the best sequence kept. Returns what was found."""
    model = Decoder(seed=seed)
    attend = None if attend is None else attend(model)
    ids = [(7 * i + 3) % model.vocab for i in range(prompt)]
    for a in range(0, prompt, MAX_ROWS):
        logits = model.step(ids[a:a + MAX_ROWS], attend=attend)
    # the drafts: the most likely next token, then placeholders whose positions are scored in the same pass
    first = sg.logprobs(logits[-1:], top=1, status=model.status)["top_tok"]
    draft = [int(first[0, 0])] + [(11 * i + 5) % model.vocab for i in range(drafts - 1)]
    logits = model.step(draft, attend=attend)
    scored = sg.logprobs(logits, torch.tensor([[t] for t in draft], dtype=torch.int32, device="cuda"), top=5, full=True,
                         status=model.status)
    trie_arrays = synth.trie([16, 8, 4, 3][:drafts], model.vocab, "example", seed)
    trie, held = sg.make_trie(*trie_arrays)
    seq, score = verify(model, trie, scored["logp"], beams)
    # the draft tokens go back, the best sequence's tokens take their place
    best = [t for t in seq[0].tolist() if t >= 0]
    final = model.step(best, keep=[prompt], attend=attend)
    torch.cuda.synchronize()
    assert int(model.status.item()) == 0, sg.sgemv_status_str(int(model.status.item()))
    return {"model": model, "logits": logits, "scored": scored, "seq": seq, "score": score, "trie": trie_arrays, "best": best,
            "final": final, "held": held}


if __name__ == "__main__":
    got = run()
    model = got["model"]
    print("entropy of the positions:", [round(x, 3) for x in got["scored"]["entropy"].tolist()])
    print("best sequence:", got["best"], "score", round(float(got["score"][0]), 3))
    print("tokens in the cache:", model.length.tolist(), "free pages:", model.free_count.tolist())
