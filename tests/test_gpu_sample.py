"""sample_tokens on the GPU: the very tokens that decode_ref draws in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import decode_ref as D  # noqa: E402
from test_gpu_attn import fc  # noqa: E402,F401

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16, torch.float32]
INF = math.inf


def rows_of(rng, rows, vocab, dtype, kind):
    x = rng.standard_normal((rows, vocab)) * 2
    if kind == "peaked":
        x[np.arange(rows), rng.integers(0, vocab, rows)] += 12
    elif kind == "levels":                # few values: ties everywhere
        x = np.floor(x)
    elif kind == "masked":
        x[rng.random((rows, vocab)) < 0.6] = -INF
        x[:, vocab // 2] = 0.5
    elif kind == "wide":
        x *= 30
    return torch.from_numpy(x).to(dtype)


def expect(x, u, temperature, top_k, top_p, min_p):
    """Tokens by decode_ref; every u has to be clear of the borders."""
    want = []
    for r in range(x.shape[0]):
        pick = [float(np.float32(v[r] if np.ndim(v) else v)) for v in (temperature, top_k, top_p, min_p)]
        w = D.weights_that_stay(x[r].double().numpy(), *pick)
        token, clear = D.draw(w, float(u[r]))
        assert clear > 1e-10 or not pick[0] > 0
        want.append(token)
    return want


def inside(x, rng, *settings):
    """A u for each row, in the middle of some token's share."""
    us = []
    for r in range(x.shape[0]):
        w = D.weights_that_stay(x[r].double().numpy(), *[float(np.float32(v)) for v in settings])
        us.append(D.middles(w, 4, rng)[1][r % 4])
    return torch.tensor(us, dtype=torch.float32)


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 0, 1.0, 0.0), (1.0, 1, 1.0, 0.0), (1.0, 7, 1.0, 0.0), (1.3, 300, 1.0, 0.0),
            (1.0, 0, 0.9, 0.0), (0.5, 0, 0.3, 0.0), (1.5, 0, 0.999, 0.0), (1.0, 0, 1.0, 0.05), (1.0, 0, 1.0, 1.0),
            (0.8, 50, 0.9, 0.02), (1.0, 1000, 0.5, 0.1), (0.0, 5, 0.5, 0.1), (1.0, 0, 0.0, 0.0), (3.0, 0, 0.97, 0.001)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 511, 512, 513, 8191, 32000, 100003])
@pytest.mark.parametrize("kind", ["peaked", "levels", "masked"])
def test_vocabularies(fc, dtype, vocab, kind):
    print("case sample", dtype, vocab, kind, flush=True)
    rng = np.random.default_rng(vocab)
    rows = 4
    x = rows_of(rng, rows, vocab, dtype, kind)
    g = x.cuda()
    for s in SETTINGS:
        u = inside(x, rng, *s)
        got = fc.sample_tokens(g, u.cuda(), *s)
        assert got.tolist() == expect(x, u, *s), s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["peaked", "levels", "masked", "wide"])
def test_settings_of_each_row(fc, dtype, kind):
    print("case sample mixed", dtype, kind, flush=True)
    rng = np.random.default_rng(5)
    rows, vocab = 60, 2500
    x = rows_of(rng, rows, vocab, dtype, kind)
    t = torch.tensor(rng.choice([0.0, -1.0, 0.3, 1.0, 2.0], rows), dtype=torch.float32)
    k = torch.tensor(rng.choice([0, -5, 1, 3, 100, 2499, 2500, 10 ** 9], rows), dtype=torch.int32)
    p = torch.tensor(rng.choice([0.0, 0.2, 0.9, 0.99, 1.0, 7.0], rows), dtype=torch.float32)
    m = torch.tensor(rng.choice([0.0, -1.0, 0.01, 0.3, 1.0], rows), dtype=torch.float32)
    u = torch.tensor(rng.random(rows), dtype=torch.float32)
    got = fc.sample_tokens(x.cuda(), u.cuda(), t.cuda(), k.cuda(), p.cuda(), m.cuda())
    want = expect(x, u, t.numpy(), k.numpy(), p.clamp(0, 1).numpy(), m.clamp(0, 1).numpy())
    assert got.tolist() == want


@pytest.mark.parametrize("vocab", [8, 1000, 4097])
def test_borders_of_equal_shares(fc, vocab):
    """Equal logits: u at j / 8 begins token j V / 8's share, exactly."""
    print("case sample borders", vocab, flush=True)
    x = torch.full((8, vocab), -3.0, dtype=torch.bfloat16).cuda()
    u = torch.arange(8, dtype=torch.float32).cuda() / 8
    want = [j * vocab // 8 for j in range(8)]      # the first i with i + 1 > j V / 8
    assert fc.sample_tokens(x, u).tolist() == want
    assert fc.sample_tokens(x, u, temperature=1e-30).tolist() == want
    inf = torch.full((8,), INF).cuda()
    assert fc.sample_tokens(x, u, temperature=inf).tolist() == want
    # half of the mass, and the first half by count: of equal ones the lowest
    half = -(-vocab // 2)
    want = [j * half // 8 for j in range(8)]
    assert fc.sample_tokens(x, u, top_p=0.5).tolist() == want
    assert fc.sample_tokens(x, u, top_k=half).tolist() == want
    assert fc.sample_tokens(x, u, top_k=half, top_p=1.0, min_p=1.0).tolist() == want


def test_numbers_at_the_ends(fc):
    print("case sample ends", flush=True)
    x = torch.tensor([[-INF, 1.0, 2.0, 0.0, -INF]] * 8)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 5.0, -3.0, INF, -INF, math.nan])
    for dtype in TYPES:
        assert fc.sample_tokens(x.to(dtype).cuda(), u.cuda()).tolist() == [1, 3, 3, 3, 1, 3, 1, -1]


def test_rows_that_are_no_distribution(fc):
    print("case sample bad rows", flush=True)
    for dtype in TYPES:
        x = torch.zeros((6, 3000), dtype=dtype)
        x[0, 2999] = math.nan
        x[1, 17] = INF
        x[2] = -INF
        x[3, 1:] = -INF
        x[4, :2999] = -INF
        for s in ((1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.7, 40, 0.9, 0.1)):
            got = fc.sample_tokens(x.cuda(), torch.full((6,), 0.4).cuda(), *s).tolist()
            assert got[:5] == [-1, -1, -1, 0, 2999] and got[5] >= 0, (dtype, s)


def test_zeros_of_both_signs_are_equal(fc):
    print("case sample zeros", flush=True)
    x = torch.full((1, 600), -5.0)
    x[0, 100:300:2], x[0, 101:300:2] = -0.0, 0.0
    for dtype in TYPES:
        g = x.to(dtype).cuda()
        u = torch.tensor([0.999]).cuda()
        assert fc.sample_tokens(g, u, temperature=0.0).tolist() == [100]
        assert fc.sample_tokens(g, u, top_k=3).tolist() == [102]
        assert fc.sample_tokens(g, u, top_k=50, top_p=0.5).tolist() == [124]


def test_many_ties_beyond_the_list(fc):
    """More equal logits at the border than are looked at one by one, in a row of 300000."""
    print("case sample ties", flush=True)
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.integers(-3, 3, (3, 300000)).astype(np.float32))
    for s in ((1.0, 100000, 1.0, 0.0), (1.0, 0, 0.8, 0.0), (1.0, 120000, 0.9, 0.05)):
        u = inside(x, rng, *s)
        assert fc.sample_tokens(x.cuda(), u.cuda(), *s).tolist() == expect(x, u, *s), s


def test_close_values_beyond_the_list(fc):
    """Thousands of different 32-bit logits inside one bin of the histogram."""
    print("case sample close", flush=True)
    rng = np.random.default_rng(9)
    x = torch.from_numpy((1.0 + 1e-3 * rng.random((4, 50000))).astype(np.float32))
    x[0] *= -1
    x[2:] *= 1e-30
    for s in ((1.0, 20000, 1.0, 0.0), (1.0, 0, 0.7, 0.0), (1.0, 30001, 0.33, 0.0)):
        u = inside(x, rng, *s)
        assert fc.sample_tokens(x.cuda(), u.cuda(), *s).tolist() == expect(x, u, *s), s


def test_strides_offsets_and_types_at_odd_places(fc):
    print("case sample strides", flush=True)
    rng = np.random.default_rng(10)
    for dtype in TYPES:
        wide = rows_of(rng, 6, 1111, dtype, "peaked")
        for a, z in ((1, 1000), (3, 1111), (8, 9)):
            x = wide[::2, a:z]
            u = inside(x, rng, 1.0, 20, 0.9, 0.0)
            assert fc.sample_tokens(wide.cuda()[::2, a:z], u.cuda(), 1.0, 20, 0.9).tolist() == expect(x, u, 1.0, 20, 0.9, 0.0)
        one = wide[:1].expand(5, -1)
        u = torch.tensor([0.1, 0.3, 0.5, 0.7, 0.9])
        assert fc.sample_tokens(wide.cuda()[:1].expand(5, -1), u.cuda()).tolist() == expect(one, u, 1.0, 0, 1.0, 0.0)


def test_offsets_past_32_bits(fc):
    print("case sample far", flush=True)
    rows, vocab = 2100, 2 ** 20
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    x[-1] = -20
    x[-1, 777777], x[-1, 1048575] = 5.0, 5.0
    u = torch.full((rows,), 0.5, device="cuda")
    u[-1] = 0.25
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 40, 0.9, 0.0)):
        got = fc.sample_tokens(x, u, *s)
        assert got[-1].item() == 777777
    assert fc.sample_tokens(x, u)[:-1].eq(vocab // 2).all()


def test_out_streams_and_repeats(fc):
    print("case sample streams", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((300, 9000), generator=g, device="cuda") * 3
    u = torch.rand(300, generator=g, device="cuda")
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 30, 0.95, 0.0), (1.2, 0, 0.9, 0.01)):
        a = fc.sample_tokens(x, u, *s)
        out = torch.full((302,), -9, dtype=torch.int32, device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            r = fc.sample_tokens(x, u, *s, out=out[1:301])
        st.synchronize()
        assert r.data_ptr() == out[1:301].data_ptr() and torch.equal(r, a) and out[0] == -9 and out[301] == -9
        for rows in (1, 2, 40, 299):            # a row's token does not depend on the rows beside it
            assert torch.equal(fc.sample_tokens(x[:rows], u[:rows], *s), a[:rows])
        for _ in range(3):
            assert torch.equal(fc.sample_tokens(x, u, *s), a)
    assert fc.sample_tokens(x[:0], u[:0]).shape == (0,)


def test_shares_come_out_as_drawn(fc):
    """Evenly spread numbers draw each token as often as its share says."""
    print("case sample shares", flush=True)
    n = 4000
    x = torch.tensor([0.0, 1.0, 2.0, -1.0, 0.5])
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    got = fc.sample_tokens(x.expand(n, -1).contiguous().cuda(), u.float().cuda(), temperature=0.9)
    share = torch.softmax(x.double() / 0.9, 0)
    many = torch.bincount(got.cpu().long(), minlength=5)
    assert (many - share * n).abs().max() <= 1          # a border falls inside one step of 1 / n


@pytest.mark.parametrize("vocab", [6000, 12000, 20000, 32768])
def test_a_row_is_drawn_alike_in_any_company(fc, vocab):
    """However many rows there are, and so whichever kernels take them."""
    print("case company", vocab, flush=True)
    g = torch.Generator()
    g.manual_seed(vocab)
    x = (3 * torch.randn((4, vocab), generator=g)).half().cuda()
    u = torch.rand(4, generator=g).cuda()
    for st in ((1.0, 0, 1.0, 0.0), (0.9, 40, 0.95, 0.0), (1.2, 0, 0.9, 0.0), (0.0, 0, 1.0, 0.0)):
        want = fc.sample_tokens(x, u, *st)
        assert want.ge(0).all()
        for n in (50, 150):
            assert torch.equal(fc.sample_tokens(x.repeat(n, 1), u.repeat(n), *st), want.repeat(n)), (st, n)
