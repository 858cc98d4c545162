"""sample_tokens where a row's list of elements in question (512 at most, of 512 groups at
most) is just full and where it overflows: the draw is decode_ref's in 64 bits either way,
in both launches (vocabularies to 8192 go at once, a few long rows by a pass apart)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from test_gpu_attn import fc  # noqa: E402,F401
from test_gpu_sample import TYPES, expect, inside  # noqa: E402

pytestmark = pytest.mark.gpu


def same(fc, x, rng, *settings, rows=None):
    """Every row's token, alone and beside many copies of the rows."""
    u = inside(x, rng, *settings)
    want = expect(x, u, *settings)
    assert fc.sample_tokens(x.cuda(), u.cuda(), *settings).tolist() == want, settings
    n = rows or 40
    got = fc.sample_tokens(x.cuda().repeat(n, 1), u.cuda().repeat(n), *settings)
    assert got.tolist() == want * n, settings


def spread(rng, vocab, many, every):
    """One row: `many` logits near 0, one in each of the first groups of `every`, the rest far below."""
    x = np.full(vocab, -30.0)
    at = np.arange(many) * every + (rng.integers(0, every, many) if every > 1 else 0)
    x[at] = -0.25 * rng.integers(0, 4, many)
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [8192, 32000])
@pytest.mark.parametrize("many", [511, 512, 513, 600])
def test_min_p_alone_with_a_full_list(fc, dtype, vocab, many):
    """min_p says nothing of how many stay, so that a second look at the groups would find the same."""
    print("case lists elements", dtype, vocab, many, flush=True)
    rng = np.random.default_rng(many)
    x = torch.from_numpy(np.stack([spread(rng, vocab, many, 1), spread(rng, vocab, many, 8)])).to(dtype)
    for m in (0.1, 0.4, 0.7):
        same(fc, x, rng, 1.0, 0, 1.0, m)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("many", [512, 513, 1000])
def test_min_p_alone_with_a_full_set_of_groups(fc, dtype, many):
    """The pass apart has groups of 32: one element in each of many of them."""
    print("case lists groups", dtype, many, flush=True)
    rng = np.random.default_rng(many)
    x = torch.from_numpy(spread(rng, 40000, many, 32)[None]).to(dtype)
    for m in (0.1, 0.7):
        same(fc, x, rng, 1.0, 0, 1.0, m, rows=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [8, 512, 513, 5000, 20000, 100003])
def test_min_p_alone_on_flat_rows(fc, dtype, vocab):
    print("case lists flat", dtype, vocab, flush=True)
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(np.stack([np.zeros(vocab), rng.integers(-1, 1, vocab) * 0.5])).to(dtype)
    for m in (0.05, 0.9, 1.0):
        same(fc, x, rng, 1.0, 0, 1.0, m, rows=4 if vocab > 50000 else 40)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [513, 600, 1024, 2047, 2048])
def test_more_wanted_than_there_are_groups(fc, dtype, vocab):
    """One batch has 256 groups of 8: they set no floor for a top_k past that, and more than 512 finite
    logits overflow the list."""
    print("case lists top_k", dtype, vocab, flush=True)
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.standard_normal((2, vocab)) * 2).to(dtype)
    for k in (256, 257, 300, 511, 512):
        same(fc, x, rng, 1.0, k, 1.0, 0.0)
    same(fc, x, rng, 0.8, 400, 0.9, 0.0)
    same(fc, x, rng, 1.2, 300, 1.0, 0.05)


@pytest.mark.parametrize("dtype", TYPES)
def test_the_second_look(fc, dtype):
    """Where the groups do set a floor and the first one, a bin's, lets too many in."""
    print("case lists second", dtype, flush=True)
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.integers(0, 100, (2, 30000)) / 128.0).to(dtype)   # all within a few bins
    for s in ((1.0, 40, 1.0, 0.0), (1.0, 300, 1.0, 0.0), (0.02, 0, 0.9, 0.0), (0.01, 200, 0.8, 0.01)):
        same(fc, x, rng, *s)
