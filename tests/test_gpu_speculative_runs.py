"""Whole speculative runs against runs of single tokens: the example's greedy steps with
drafted trees give the tokens that the model gives one by one."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_attn import fc  # noqa: E402,F401
from test_gpu_speculative import ex, start  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# How far a logit of the two runs may differ.  They share weights, tokens and positions, but not the order
# of sums: a tree's path lies in other slots than consecutive tokens.  With y of about 1.2 (an embedding
# of 1, the layer's parts under 0.7) and a head of gain 4 the logits are under 32 (6 of their deviations), rounded
# to fp16 by 2^-7 at most in either run: 2^-6.  Six roundings before that (q, attention's result, its
# product, h, the hidden layer, y), each of 2^-11 / sqrt(3) of 1.2 rms, go through matrices of gain one and
# then the head: 4 * sqrt(6) * 3.4e-4 = 3.3e-3 rms, times sqrt(2) for two runs, times 6 deviations: 0.028.
# Scales that rejected drafts raised move codes by 2^-9 of a page's scale, 2^-16 of its largest value: nothing
# beside these.  A greedy choice compares two logits, each off by 0.016 + 0.028.
NEAR = 0.1


@pytest.mark.parametrize("lens,seed", [([70, 1, 33], 3), ([257], 11), ([15, 16, 17, 31], 12)])
def test_greedy_runs_agree(ex, monkeypatch, lens, seed):
    print("case greedy runs", lens, seed, flush=True)
    steps = 16
    p, b, pages, g = start(ex, lens, seed, steps)
    n = 2 * len(lens)
    drafted = ex.draft
    monkeypatch.setattr(ex, "draft", lambda p, b, t: drafted(p, b, 0.5))    # siblings differ
    texts = [[] for _ in range(n)]
    most = max(lens) + ex.NODES * (steps + 1)
    for _ in range(steps):
        b.u.copy_(torch.rand(b.u.shape, generator=g))
        ex.step(p, b, 0.0, most)
        for s, row, m in zip(texts, b.path.tolist(), b.kept.tolist()):
            s += row[:m]
    for s, t in zip(texts, b.last.tolist()):
        s.append(t)
    assert b.held.tolist() == [l + len(t) - 1 for l, t in zip(lens + lens, texts)]
    assert sum(map(len, texts)) > 1.2 * n * steps           # drafts were taken

    # the same prompts again, then a token at a time: after each the next has to be the model's choice
    q, c, _, _ = start(ex, lens, seed, steps)
    assert c.last.tolist() == [t[0] for t in texts]
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    clear = total = 0
    for i in range(max(map(len, texts)) - 1):
        token = torch.tensor([t[min(i, len(t) - 1)] for t in texts], device="cuda")
        y, _ = ex.dl.layer(q["emb"][token], q, c.cache, c.table, cu, c.held + (i + 1), 1, most)
        x = ex.fc.gemm_bias_act(y, q["head"], None).float().cpu()
        top = x.topk(2).values
        assert x.abs().max() < 32
        for s, t in enumerate(texts):
            if i + 1 >= len(t):
                continue
            assert x[s, t[i + 1]] >= top[s, 0] - NEAR, (s, i)
            total += 1
            clear += bool(top[s, 0] - top[s, 1] > NEAR)
    assert clear > total / 2
