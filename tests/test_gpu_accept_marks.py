"""tree_accept with targets that are no tokens: -1 from a row that sample_tokens cannot draw
from is not taken for a drafted -1, the drafter's own mark."""
import math

import pytest

torch = pytest.importorskip("torch")
from test_gpu_attn import fc, i32  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mark", [-1, -2, -2 ** 31])
@pytest.mark.parametrize("n", [1, 3, 64, 65, 200])
def test_a_path_ends_at_a_target_that_is_no_token(fc, mark, n):
    print("case accept marks", mark, n, flush=True)
    par = i32([-1] + list(range(n - 1))).cuda()
    for at in sorted({0, n // 2, n - 1, 63 if n > 63 else 0}):
        tok = torch.arange(n, dtype=torch.int32)
        tgt = tok + 1
        tgt[at] = mark
        tok[at + 1:at + 2] = mark                      # the draft behind it is marked too
        for most in (n, max(1, n // 3)):
            keep, kept, nxt, after = fc.tree_accept(par, tok.cuda(), tgt.cuda(), i32([0, n]).cuda(), i32([n + 7]).cuda(), max_q=most)
            m = min(at + 1, most)
            assert keep[0].tolist() == list(range(m)) + [-1] * (most - m)
            assert (kept.item(), nxt.item(), after.item()) == (m, int(tgt[m - 1]), 7 + m)


def test_bad_rows_of_drafter_and_model(fc):
    """Both draw from logits with a NaN: node 0 alone is kept, and the next token is marked."""
    print("case accept bad rows", flush=True)
    x = torch.randn((4, 1000), generator=torch.Generator().manual_seed(1))
    x[:2, 5] = math.nan
    u = torch.full((4,), 0.5).cuda()
    drawn = fc.sample_tokens(x.cuda(), u)
    assert drawn[:2].tolist() == [-1, -1] and drawn[2:].ge(0).all()
    par = i32([-1, 0, 1, 2]).cuda()
    tok = torch.cat((i32([9]).cuda(), drawn[:3]))      # the drafter's draws, one node on
    keep, kept, nxt, after = fc.tree_accept(par, tok, drawn, i32([0, 4]).cuda(), i32([50]).cuda())
    assert keep[0].tolist() == [0, -1, -1, -1] and kept.item() == 1 and nxt.item() == -1 and after.item() == 47
