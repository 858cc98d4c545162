"""The LDS-poison build (see test_gpu_poison) of the operators around a decoding step: what
they leave is the product build's, bit for bit."""
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from test_gpu_attn import BF16, F16, fc, i32, on_gpu  # noqa: E402,F401
from test_gpu_sample import SETTINGS, TYPES, rows_of  # noqa: E402
from test_gpu_tree import cumulative, grow, tree_batch  # noqa: E402

pytestmark = pytest.mark.gpu


def both(fc, run):
    a = run()
    with fc.poison_build():
        p = run()
    torch.cuda.synchronize()
    assert len(a) == len(p)
    for x, y in zip(a, p):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [8, 512, 2048, 9000, 32000, 70001])
@pytest.mark.parametrize("kind", ["peaked", "levels", "masked", "flat"])
def test_sampling(fc, dtype, vocab, kind):
    """Lists that fit and that overflow, ties, whole rows by histograms; a row a block and, of 300, settings of each."""
    print("case poison sample", dtype, vocab, kind, flush=True)
    rng = np.random.default_rng(vocab)
    x = (rows_of(rng, 12, vocab, dtype, kind) if kind != "flat"
         else torch.from_numpy(rng.standard_normal((12, vocab)) * 0.05).to(dtype)).cuda()
    u = torch.from_numpy(rng.random(12)).float().cuda()
    for s in SETTINGS + [(1.0, 300, 1.0, 0.0), (1.0, 512, 0.9, 0.0)]:
        both(fc, lambda: [fc.sample_tokens(x, u, *s)])
    if vocab > 40000:
        return
    n = 300
    t, p, m = (torch.from_numpy(rng.choice(v, n)).float().cuda() for v in ([0.0, 0.7, 1.5], [0.3, 0.9, 1.0], [0.0, 0.0, 0.1]))
    k = torch.from_numpy(rng.choice([0, 5, 300, 2000], n)).int().cuda()
    both(fc, lambda: [fc.sample_tokens(x.repeat(25, 1), u.repeat(25), t, k, p, m)])


@pytest.mark.parametrize("new", [[5, 64, 1], [65, 0, 130], [1500, 64, 700]])
def test_bookkeeping(fc, new):
    print("case poison trees", new, flush=True)
    rng = random.Random(sum(new))
    n = sum(new)
    par = i32(sum((grow(rng, k, 70) for k in new), [])).cuda()
    tok, tgt = (i32([rng.randint(0, 1) for _ in range(n)]).cuda() for _ in range(2))
    cu, lens = cumulative(new).cuda(), i32([k + 9 for k in new]).cuda()
    both(fc, lambda: fc.tree_plan(par, cu, lens, max_q=max(new)))
    both(fc, lambda: fc.tree_accept(par, tok, tgt, cu, lens, max_q=max(new)))


@pytest.mark.parametrize("dtype,d,page", [(F16, 64, 16), (BF16, 128, 32), (BF16, 256, 256), (F16, 192, 128)])
def test_moves(fc, dtype, d, page):
    print("case poison keep", dtype, d, page, flush=True)
    rng = random.Random(d)
    new, lens = [60, 7, 130], [200, 7, 400]
    b, _, _ = tree_batch(d, dtype, lens, new, 4, 2, d, page)
    g = on_gpu(b)
    g["scales"] = g["scales"] * torch.tensor([2.0 ** rng.randint(-3, 3) for _ in range(g["scales"].numel())]).view(g["scales"].shape).cuda()
    keep = torch.full((3, 100), -1, dtype=torch.int32)
    kept = i32([40, 3, 100])
    for s in range(3):
        keep[s, :kept[s]] = i32(sorted(rng.sample(range(new[s]), int(kept[s]))))

    def run():
        codes, scales = g["codes"].clone(), g["scales"].clone()
        fc.kv_keep(codes, scales, g["table"], g["cu_q"], g["kv_lens"], keep.cuda(), kept.cuda())
        fc.kv_copy(codes, scales, [(0, codes.shape[0] - 1)])
        return codes, scales
    both(fc, run)
