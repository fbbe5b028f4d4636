"""The example examples/decode_path.py on the GPU: every operator in one path, against the same path with attention, log-probabilities
and beam search from the oracles.

Logits of the two paths differ by attention's rounding alone (2^-11 of outputs of size 1, through two blocks of
norm-preserving fp16 linears whose own rounding is as large): 2^-6 of the logits' size bounds it with room."""

import os
import sys

import numpy as np
import pytest

from oracle import beam as obeam
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_path
    return decode_path, torch


def test_decode_path(example):
    path, torch = example

    def oracle_attend(model):
        def attend(block, q, q_start):
            L = okv.layout(model.kv.heads, model.kv.dim, model.kv.group, model.kv.page, model.kv.n_pages)
            out = okv.attention(L, model.caches[block].cpu().numpy(), q.float().cpu().numpy(), q_start.tolist(), model.length.tolist(),
                                model.table.tolist(), 1 / np.sqrt(model.dim))[0]
            return torch.tensor(out).half().cuda()
        return attend

    got, ref = path.run(), path.run(attend=oracle_attend)
    for name in ("logits", "final"):
        a, b = got[name].double().cpu().numpy(), ref[name].double().cpu().numpy()
        if got["best"] == ref["best"] or name == "logits":
            assert np.abs(a - b).max() <= 2.0 ** -6 * np.abs(b).max()
    # log-probabilities of the path's own logits, and the beam search over them
    logits = got["logits"].double().cpu().numpy()
    lse, ent, tops, top_lp, lp = okv.logprobs(logits, None, 5)[1:]
    s = {k: v.cpu().numpy() for k, v in got["scored"].items()}
    assert np.abs(s["logp"] - lp).max() < 2e-5 and np.abs(s["lse"] - lse).max() < 2e-5 and np.abs(s["entropy"] - ent).max() < 5e-5
    assert np.array_equal(s["top_tok"], tops)
    ptr, tok, nod = got["trie"]
    nodes, scores = np.array([0], dtype=np.int32), np.array([0.0], dtype=np.float32)
    for t in range(s["logp"].shape[0]):
        o = obeam.beam_step(ptr, tok, nod, nodes, scores, np.repeat(s["logp"][t:t + 1], len(nodes), 0), got["seq"].shape[0])
        nodes, scores = o["node"], o["score"]
    assert np.array_equal(got["score"].cpu().numpy()[:len(scores)], scores)
    # the rejected drafts' pages are back, and none is held twice
    model = got["model"]
    length, free = int(model.length[0]), int(model.free_count[0])
    used = model.table[0, :-(-length // model.page)].tolist()
    assert length == 40 + len(got["best"])
    assert sorted(used + model.free[:free].tolist()) == list(range(model.kv.n_pages))
