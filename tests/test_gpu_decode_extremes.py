"""The operators around a decoding step at the ends of their ranges: more rows and sequences
than a grid has blocks, the largest vocabulary, the longest trees."""
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import decode_ref as D  # noqa: E402
from test_gpu_attn import BF16, F16, batch, fc, i32, on_gpu  # noqa: E402,F401
from test_gpu_sample import TYPES, expect, inside  # noqa: E402

pytestmark = pytest.mark.gpu
MANY = 2 ** 20 + 77


@pytest.mark.parametrize("vocab,settings", [(5, (1.0, 0, 0.9, 0.0)), (9, (1.0, 0, 1.0, 0.0)), (700, (1.0, 30, 0.9, 0.0)),
                                            (700, (1.0, 0, 1.0, 0.2)), (40000, (1.0, 0, 1.0, 0.0)), (40000, (0.5, 20, 1.0, 0.0))])
def test_more_rows_than_blocks(fc, vocab, settings):
    """One row of logits for all: each row's token by its own random number."""
    print("case rows", vocab, settings, flush=True)
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.standard_normal((1, vocab)) * 0.5).half()
    few = torch.cat([inside(x, rng, *settings) for _ in range(11)])
    want = torch.tensor(expect(x.expand(11, -1), few, *settings), dtype=torch.int32)
    at = torch.from_numpy(rng.integers(0, 11, MANY))
    got = fc.sample_tokens(x.cuda().expand(MANY, -1), few[at].cuda(), *settings)
    assert torch.equal(got.cpu(), want[at])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("settings", [(1.0, 0, 1.0, 0.0), (1.0, 0, 0.75, 0.0), (1.0, 300000, 1.0, 0.0), (1.0, 300001, 0.5, 0.0),
                                      (1.0, 0, 1.0, 0.9), (0.0, 0, 1.0, 0.0)], ids=str)
def test_the_largest_vocabulary(fc, dtype, settings):
    """2^20 logits, all equal (a mass of 2^62 units) and of a few levels."""
    print("case vocabulary", dtype, settings, flush=True)
    rng = np.random.default_rng(20)
    v = 2 ** 20
    x = torch.from_numpy(np.stack([np.full(v, 3.0), rng.integers(0, 3, v) * 0.25])).to(dtype)
    # (shares of 1e-6 are too narrow for middles(): eighths of the row, off the borders)
    for j in (0, 3, 7):
        u = torch.full((2,), (j + 0.37) / 8, dtype=torch.float32)
        want, near = [], []
        for r in range(2):
            w = D.weights_that_stay(x[r].double().numpy(), *[float(np.float32(s)) for s in settings])
            token, clear = D.draw(w, float(u[r]))
            want.append(token)
            near.append(clear)
        if not settings[0] > 0 or min(near) > 1e-10:
            assert fc.sample_tokens(x.cuda(), u.cuda(), *settings).tolist() == want, (j, settings)


@pytest.mark.parametrize("variant", ["rows", "tile"])
@pytest.mark.parametrize("d", [64, 128])
def test_the_longest_tree(fc, variant, d):
    """A chain of 4096 nodes gives what the causal call gives, bit for bit."""
    print("case longest", variant, d, flush=True)
    lens, new = [4200, 70, 4096], [4096, 3, 2000]
    b = batch(7, F16, lens, new, 2, 1, d, 64)
    g = on_gpu(b)
    par = i32([i - 1 for n in new for i in range(n)]).cuda()
    tree = fc.tree_plan(par, g["cu_q"], g["kv_lens"], max_q=4096)
    a = fc.chain_attn(**g, max_q=4096, variant=variant, splits=1)
    t = fc.chain_attn(**g, max_q=4096, variant=variant, splits=1, tree=tree)
    assert torch.equal(a, t)


def test_many_sequences(fc):
    """More sequences than blocks take at a time: trees of one and two nodes."""
    print("case sequences", flush=True)
    B = 300007
    rng = np.random.default_rng(3)
    new = rng.integers(0, 3, B)
    cu = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    first = np.zeros(cu[-1], dtype=bool)
    first[cu[:-1][new > 0]] = True
    par = np.where(first, -1, 0).astype(np.int32)
    lens = (new + rng.integers(0, 100, B)).astype(np.int32)
    tok, tgt = (rng.integers(0, 2, len(par)).astype(np.int32) for _ in range(2))
    p, k, g, c, n = (torch.from_numpy(v).cuda() for v in (par, tok, tgt, cu, lens))
    bits, pos = fc.tree_plan(p, c, n, max_q=2)
    start = np.repeat(lens - new, new)
    assert np.array_equal(bits[:, 0].cpu().numpy(), np.where(first, 1, 3)) and np.array_equal(pos.cpu().numpy(), start + ~first)
    keep, kept, nxt, after = (t.cpu().numpy() for t in fc.tree_accept(p, k, g, c, n, max_q=2))
    a = np.minimum(cu[:-1], len(par) - 1)
    z = np.minimum(a + 1, len(par) - 1)
    two = (new == 2) & (tok[z] == tgt[a])
    assert np.array_equal(kept, np.minimum(new, 1) + two) and np.array_equal(after, lens - new + kept)
    assert np.array_equal(nxt, np.where(new == 0, -1, np.where(two, tgt[z], tgt[a])))
    assert np.array_equal(keep, np.stack([np.where(new > 0, 0, -1), np.where(two, 1, -1)], 1))


@pytest.mark.parametrize("page", [16, 256])
def test_thousands_of_kept_tokens(fc, page):
    print("case keep many", page, flush=True)
    rng = random.Random(page)
    lens, new = [5000, 4096], [4096, 4096]
    b = batch(9, BF16, lens, new, 2, 1, 64, page)
    b["scales"] *= torch.tensor([2.0 ** rng.randint(-2, 2) for _ in range(b["scales"].numel())]).view(b["scales"].shape)
    keep, kept = torch.full((2, 4096), -1, dtype=torch.int32), i32([3000, 4095])
    keep[0, :3000] = i32(sorted(rng.sample(range(4096), 3000)))
    keep[1, :4095] = torch.arange(1, 4096)
    want = D.keep_tokens(b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], keep, kept)
    g = on_gpu(b)
    fc.kv_keep(g["codes"], g["scales"], g["table"], g["cu_q"], g["kv_lens"], keep.cuda(), kept.cuda())
    assert D.same_codes(g["codes"], want[0]) and torch.equal(g["scales"].cpu(), want[1])
