"""One decoder layer served from a paged 8-bit cache, out of the library's chains:

    qkv   = x Wqkv + b                         gemm_bias_act
    q, k  turned by their positions; k, v -> cache  kv_append (one launch)
    attn  = softmax(q K^T) V over the cache    chain_attn
    x     = x + attn Wo                        gemm_bias_act
    x     = x + act(x W0 + b0) W1 + b1         chain_gemm2

run over a ragged batch: prompts of several lengths first, then steps of one token
a sequence, captured in a HIP graph and replayed.  Synthetic weights, no norms.

    python examples/decoder_layer.py [--steps 64]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_conv_chain_amd as fc  # noqa: E402

HIDDEN, HQ, HKV, D, FFN = 256, 8, 2, 64, 256
PAGE = 32


def make_weights(seed=0, device="cuda"):
    g = torch.Generator()
    g.manual_seed(seed)

    def w(k, n):
        return (torch.randn((k, n), generator=g) / math.sqrt(k)).half().to(device)

    def b(n):
        return (torch.randn((n,), generator=g) / 16).half().to(device)
    turns, mscale = fc.rope_turns(D, device=device)
    return dict(wqkv=w(HIDDEN, (HQ + 2 * HKV) * D), bqkv=b((HQ + 2 * HKV) * D), wo=w(HQ * D, HIDDEN),
                w0=w(HIDDEN, FFN), b0=b(FFN), w1=w(FFN, HIDDEN), b1=b(HIDDEN), turns=turns, mscale=mscale)


def layer(x, p, cache, table, cu_q, kv_lens, max_q, max_kv):
    """x [tokens, HIDDEN] -> the same, its keys and values appended to the cache;
    returns (result, what was computed on the way)."""
    qkv = fc.gemm_bias_act(x, p["wqkv"], p["bqkv"])
    rows = qkv.view(-1, HQ + 2 * HKV, D)
    q = fc.kv_append(rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:], *cache, table, cu_q, kv_lens, turns=p["turns"],
                     mscale=p["mscale"], q=rows[:, :HQ], max_q=max_q)
    attn = fc.chain_attn(q, *cache, table, cu_q, kv_lens, max_q=max_q, max_kv=max_kv)
    h = x + fc.gemm_bias_act(attn.view(-1, HQ * D), p["wo"], None)
    mlp = fc.chain_gemm2(h, p["w0"], p["b0"], p["w1"], p["b1"], act="gelu_tanh")
    return h + mlp, dict(qkv=qkv, q=q, attn=attn, h=h, mlp=mlp)


class Pages:
    """Hands out the pool's pages and keeps the batch's table on the host."""

    def __init__(self, pages, batch, most):
        self.free = list(range(pages))
        self.table = torch.zeros((batch, most), dtype=torch.int32)
        self.held = [0] * batch

    def grow(self, lens):
        for b, n in enumerate(lens):
            while self.held[b] * PAGE < n:
                self.table[b, self.held[b]] = self.free.pop()
                self.held[b] += 1
        return self.table


def prompts(p, cache, pages, lens, seed=1):
    """The whole prompts in one ragged call; returns the last token's rows."""
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn((sum(lens), HIDDEN), generator=g).half().cuda()
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    kv = torch.tensor(lens, dtype=torch.int32)
    table = pages.grow(lens)
    fc.kv_check(table, cu, kv, pages=cache[0].shape[0], page=PAGE, writes=True)
    out, _ = layer(x, p, cache, table.cuda(), cu.cuda(), kv.cuda(), max(lens), max(lens))
    return out[cu[1:].long() - 1]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=64)
    steps = ap.parse_args().steps
    lens = [700, 33, 1500, 1, 256, 90, 1024, 411]
    B, most = len(lens), (max(lens) + steps) // PAGE + 1
    p = make_weights()
    cache = fc.kv_cache(sum(n // PAGE + 1 for n in lens) + B * (steps // PAGE + 2), HKV, PAGE, D)
    pages = Pages(cache[0].shape[0], B, most)
    x = prompts(p, cache, pages, lens).contiguous()

    # every page that the steps will need is handed out beforehand, so that the
    # captured step changes nothing but the lengths
    table = pages.grow([n + steps + 1 for n in lens]).cuda()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    one = torch.ones_like(kv)

    def step():
        kv.add_(one)
        y, _ = layer(x, p, cache, table, cu, kv, 1, max(lens) + steps)
        x.copy_(y / y.float().pow(2).mean(-1, keepdim=True).sqrt().half())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                      # the first call of each kernel
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps - 1):
        graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    assert torch.isfinite(x.float()).all()
    print("%d prompts (%d tokens), then %d steps of %d sequences: %.1f us a step" % (
        B, sum(lens), steps, B, t / max(steps - 1, 1) * 1e6))


if __name__ == "__main__":
    main()
