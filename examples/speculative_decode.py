"""Speculative decoding with trees of drafted tokens over the paged 8-bit cache: the
layer of decoder_layer.py between an embedding and a head, and as drafter the head
on the embedding alone.  One step, for every sequence at once:

    drafted: the tree's tokens, level by level, drawn by the drafter    sample_tokens
    bits, positions of the nodes                                         tree_plan
    the layer on all nodes; each sees its ancestors   kv_append, chain_attn(tree=...)
    targets: at each node a token drawn from the model's logits          sample_tokens
    the path whose drafts are the targets, and one token more            tree_accept
    its keys and values move to the front of the tree's slots            kv_keep

Every step adds 1 to DEPTH + 1 tokens to a sequence, drawn as the model alone would
draw them, up to roundings (a rejected draft may have raised the scale of a page, by
which small codes of other tokens on it were rounded once more).  Two sequences continue each prompt: the second shares its pages, but for
the last, partly filled one, which is copied (KvPages, kv_copy).  The step is captured
in a HIP graph and replayed; the host reads the tokens behind it.

    python examples/speculative_decode.py [--steps 32] [--temperature 0.3]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import decoder_layer as dl  # noqa: E402
from decoder_layer import fc  # noqa: E402

VOCAB = 512
# the tree's shape: every node's parent; node 0 is the token that the last step decided
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 4]
LEVELS = [[1, 2, 3], [4, 5, 6], [7]]
NODES, DEPTH = len(PARENTS), len(LEVELS)


def make_model(seed=0, device="cuda"):
    p = dl.make_weights(seed, device)
    g = torch.Generator()
    g.manual_seed(seed + 1)
    p["emb"] = torch.randn((VOCAB, dl.HIDDEN), generator=g).half().to(device)
    p["head"] = (4 * torch.randn((dl.HIDDEN, VOCAB), generator=g) / math.sqrt(dl.HIDDEN)).half().to(device)
    return p


class Batch:
    """What a step reads and writes, so that it can be captured: each sequence's length
    without the tree (``held``), its undecided token (``last``), the random numbers."""

    def __init__(self, cache, table, lens, last):
        dev = table.device
        B = len(lens)
        self.cache, self.table = cache, table
        self.held = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.last = last.clone()
        self.levels = [(torch.tensor(nodes, device=dev), torch.tensor([PARENTS[i] for i in nodes], device=dev))
                       for nodes in LEVELS]
        self.parents = torch.tensor(PARENTS * B, dtype=torch.int32, device=dev)
        self.cu = torch.arange(0, NODES * B + 1, NODES, dtype=torch.int32, device=dev)
        self.drafted = torch.zeros((B, NODES), dtype=torch.int32, device=dev)
        self.u = torch.zeros(2, B * NODES, dtype=torch.float32, device=dev)
        self.kept = torch.zeros(B, dtype=torch.int32, device=dev)
        self.path = torch.zeros((B, NODES), dtype=torch.int32, device=dev)   # the tokens decided, 0 behind them


def draft(p, b, temperature):
    """Fills b.drafted: children are drawn by the head on their parent's embedding."""
    B = b.drafted.shape[0]
    b.drafted[:, 0] = b.last
    u = b.u[0].view(B, NODES)
    for nodes, above in b.levels:
        x = p["emb"][b.drafted.index_select(1, above).view(-1).long()]
        logits = fc.gemm_bias_act(x, p["head"], None)
        drawn = fc.sample_tokens(logits, u.index_select(1, nodes).view(-1), temperature)
        b.drafted.index_copy_(1, nodes, drawn.view(B, -1))


def step(p, b, temperature, max_kv):
    """One step of all sequences; returns what was computed on the way."""
    draft(p, b, temperature)
    tokens = b.drafted.view(-1)
    kv = b.held + NODES
    tree = fc.tree_plan(b.parents, b.cu, kv, max_q=NODES)
    x = p["emb"][tokens.long()]
    y, mid = dl.layer(x, p, b.cache, b.table, b.cu, kv, NODES, max_kv, tree=tree)
    logits = fc.gemm_bias_act(y, p["head"], None)
    targets = fc.sample_tokens(logits, b.u[1], temperature)
    keep, kept, last, after = fc.tree_accept(b.parents, tokens, targets, b.cu, kv, max_q=NODES)
    fc.kv_keep(*b.cache, b.table, b.cu, kv, keep, kept)
    passed = torch.gather(b.drafted, 1, keep.clamp_min(0).long())
    b.path.copy_(torch.where(keep >= 0, passed, 0))
    b.kept.copy_(kept)
    b.last.copy_(last)
    b.held.copy_(after)
    return dict(mid, x=x, y=y, kv=kv, tree=tree, logits=logits, targets=targets, keep=keep)


def prompts(p, cache, pages, texts, temperature, u):
    """The whole prompts in one ragged call; returns the first token drawn after each."""
    lens = [len(t) for t in texts]
    for i, n in enumerate(lens):
        pages.add(i)
        pages.grow(i, n)
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    kv = torch.tensor(lens, dtype=torch.int32)
    table = pages.table(range(len(lens)))
    fc.kv_check(table, cu, kv, pages=cache[0].shape[0], page=dl.PAGE, writes=True)
    x = p["emb"][torch.cat(texts).cuda()]
    y, _ = dl.layer(x, p, cache, table.cuda(), cu.cuda(), kv.cuda(), max(lens), max(lens))
    return fc.sample_tokens(fc.gemm_bias_act(y[cu[1:].long() - 1], p["head"], None), u, temperature)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--temperature", type=float, default=0.3)
    a = ap.parse_args()
    g = torch.Generator()
    g.manual_seed(2)
    lens = [700, 33, 1500, 1, 256, 90]
    n, most = len(lens), max(lens) + NODES * (a.steps + 1)
    p = make_model()
    room = sum(-(-(l + NODES * (a.steps + 1)) // dl.PAGE) for l in lens)
    cache = fc.kv_cache(2 * room, dl.HKV, dl.PAGE, dl.D)
    pages = fc.KvPages(2 * room, dl.PAGE)
    texts = [torch.randint(0, VOCAB, (l,), generator=g) for l in lens]
    first = prompts(p, cache, pages, texts, a.temperature, torch.rand(n, generator=g).cuda())
    for i in range(n):
        pages.fork(i, n + i)
    # all the pages that the steps may need, beforehand: the captured step changes nothing but lengths
    for i in range(2 * n):
        fc.kv_copy(*cache, pages.grow(i, pages.length(i) + NODES * (a.steps + 1)))
    b = Batch(cache, pages.table(range(2 * n)).cuda(), lens + lens, first.repeat(2))

    def one():
        return step(p, b, a.temperature, most)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.u.copy_(torch.rand(b.u.shape, generator=g))
        one()                       # the first call of each kernel
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    before = b.held.tolist()
    text = [[] for _ in before]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        b.u.copy_(torch.rand(b.u.shape, generator=g))
        graph.replay()
        for s, row, m in zip(text, b.path.tolist(), b.kept.tolist()):
            s += row[:m]
    t = time.perf_counter() - t
    decided = sum(map(len, text))
    assert b.held.tolist() == [m + len(s) for m, s in zip(before, text)]
    print("%d sequences, %d steps: %.2f tokens a sequence and step, %.1f us a step" % (
        2 * n, a.steps, decided / (2 * n * a.steps), t / a.steps * 1e6))


if __name__ == "__main__":
    main()
