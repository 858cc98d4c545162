"""top_p counts a row's whole mass, its far tail too, and alike in every launch: rows whose
cut falls between the mass with and without what lies under a unit of the largest weight."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from test_gpu_attn import fc  # noqa: E402,F401
from test_gpu_sample import TYPES, expect  # noqa: E402

pytestmark = pytest.mark.gpu
FAR = -30.5        # a weight of 2^-44: under half a unit of 2^-42, and exact in every type


def row(vocab, many, every):
    """`many` weights of 1, one in each `every` logits, in a tail of weights of 2^-44."""
    x = np.full(vocab, FAR)
    x[np.arange(many) * every] = 0.0
    return x


def how_many_stay(x, many):
    """Of the weights of 1, with top_p 0.5.  The weights before the (many / 2 + 1)-th are half of
    `many`: under half the mass, so that it stays, as soon as the tail adds anything.  It does where
    2048 adjacent logits have no weight of 1, as sums are in units of 2^-42 of their own largest: 2048
    of 2^-44 are 512 units of the row's.  Beside a weight of 1 each of them is a quarter of a unit,
    which counts as 0; then exactly half stays."""
    tail = any((x[i:i + 2048] < 0).all() for i in range(0, len(x), 2048))
    return many // 2 + tail


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,many,every", [
    (5000, 600, 1),       # at once whatever the rows, from all of the row
    (5000, 400, 8),       # at once, from the row's largest
    (16000, 400, 8),      # at once for up to two rows a CU, else apart
    (16000, 700, 2),
    (32000, 400, 8),      # apart, at once, apart: from all of it, its largest, all of it
    (32000, 400, 32),
    (32000, 1000, 32),
    (32768, 600, 3),
    (100003, 400, 8),     # always apart
    (100003, 2000, 50),
])
def test_a_share_of_the_whole_mass_in_any_company(fc, dtype, vocab, many, every):
    print("case shares", dtype, vocab, many, every, flush=True)
    half = many // 2
    x = torch.from_numpy(row(vocab, many, every)[None]).to(dtype)
    # the last of half + 1 tokens, or of half: u in the middle of the former's share and inside the latter's
    u = torch.tensor([(half + 0.5) / (half + 1)], dtype=torch.float32)
    want = expect(x, u, 1.0, 0, 0.5, 0.0)
    if how_many_stay(x[0], many) == half:      # (half of the weights, where 64 bits see the tail)
        assert want == [half * every]
        want = [(half - 1) * every]
    assert want == [(how_many_stay(x[0], many) - 1) * every]
    g, v = x.cuda(), u.cuda()
    for rows in (1, 2, 150) + ((600,) if vocab < 40000 else ()):
        assert fc.sample_tokens(g.repeat(rows, 1), v.repeat(rows), 1.0, 0, 0.5).tolist() == want * rows, rows
    # an array of settings, which reaches the same kernels with other rows beside
    p = torch.tensor([0.5, 1.0, 0.5], device="cuda")
    got = fc.sample_tokens(g.repeat(3, 1), v.repeat(3), 1.0, 0, p).tolist()
    assert got[0] == got[2] == want[0]
