"""chain_attn where its arithmetic is stretched, on the GPU against 64 bits: caps
far above the scores, long flat tails under a dominant key, scores near the end of
32-bit resolution, windows at the end of the 32-bit integers."""
import math

import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402
from test_gpu_attn import BF16, DTYPES, F16, FORMS, batch, fc, gen, i32, on_gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# How a capped score may be off.  Caps to 128 take the closed form cap (1 - 2 / (1 +
# e^2t)), t = score / cap, whose error is absolute: E = e^2t is off by 2^-23 (the
# exponential) and its argument's rounding, 1 / (1 + E) by 2^-23 + 2^-24, times 2 cap
# at most 1.25 cap / (1 + E) where the score is small: under cap 2^-21.  Larger ones
# take an odd series where |t| < 1/4 (cut off under 2^-26, six roundings of 2^-24 and
# 2^-23 for the argument) and the closed form elsewhere: 3e-7 cap of a result of at
# least 0.245 cap, under 2^-19 of it.
NEAR_CAP = 128.0


def cap_error(x, cap):
    if cap <= NEAR_CAP:
        return torch.full_like(x, cap * 2.0 ** -21)
    return cap * torch.tanh(x.abs() / cap) * 2.0 ** -19


def attention(b, scale=None, causal=True, softcap=0.0, window=0, slopes=None):
    """(out, tolerance before the output's rounding, lse, lse tolerance), for
    sequences of at least one key.  Weights are rounded to the type relative to
    their size, except that fp16's below 2^-14 lose a fixed 2^-25: the largest
    weight of a row is 2^7 or more, so that is 2^-32 of it for each key."""
    q, codes, scales, table, cu_q, kv_lens = (b[k] for k in ("q", "codes", "scales", "table", "cu_q", "kv_lens"))
    T, hq, d = q.shape
    G = hq // codes.shape[1]
    u = R.half_step(q.dtype)
    lost = 2.0 ** -32 if q.dtype == F16 else 0.0
    scale = d ** -0.5 if scale is None else scale
    out, tol = torch.zeros((2, T, hq, d), dtype=torch.float64)
    lse, ltol = torch.full((T, hq), -math.inf, dtype=torch.float64), torch.zeros((T, hq), dtype=torch.float64)
    for s in range(table.shape[0]):
        a, z, L = int(cu_q[s]), int(cu_q[s + 1]), int(kv_lens[s])
        K, V = R.gather(codes, scales, table[s], L, d)
        gap = torch.arange(L - (z - a), L)[:, None] - torch.arange(L)
        seen = gap >= 0 if causal else torch.ones_like(gap, dtype=torch.bool)
        if window:
            seen = seen & (gap < window)
        some = seen.any(-1)
        for h in range(hq):
            qq = q[a:z, h].double()
            x = qq @ K[h // G].T * scale
            # fp32 accumulation of d exact products, and the scale's own roundings
            dx = (d + 4) * 2.0 ** -24 * scale * (qq.abs() @ K[h // G].abs().T)
            if softcap:
                dx = dx + cap_error(x, softcap)
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                bias = float(slopes[h]) * gap.abs()
                x = x - bias
                dx = dx + bias.abs() * 2.0 ** -22
            dx = dx + x.abs() * 2.0 ** -22
            x = x.masked_fill(~seen, -math.inf)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
            l = p.sum(-1, keepdim=True)
            w = p / torch.where(l == 0, 1.0, l)
            err = torch.where(seen, dx, 0.0).amax(-1, keepdim=True) + 2.0 ** -20
            out[a:z, h] = w @ V[h // G]
            A = w @ V[h // G].abs()
            tol[a:z, h] = A * (u + 2 * err) + lost * (seen.double() @ V[h // G].abs())
            lse[a:z, h] = torch.where(some, (m + torch.log(l))[:, 0], -math.inf)
            ltol[a:z, h] = err[:, 0] + 2.0 ** -22 * lse[a:z, h].abs().nan_to_num(0, 0, 0)
    return out, tol, lse, ltol


def attend(fc, b, what, variant, splits, **kw):  # noqa: F811
    print("case scores", variant, splits, what, flush=True)
    ref, tol, lse, ltol = attention(b, **kw)
    dkw = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    out, le = fc.chain_attn(**on_gpu(b), lse=True, variant=variant, splits=splits, **dkw)
    R.assert_within(out, ref, R.rounded_tol(ref, tol, b["q"].dtype), what)
    R.assert_within(le, lse, ltol, what + " lse")
    # (the calls that ask for no lse are other code in the tile form)
    assert torch.equal(fc.chain_attn(**on_gpu(b), variant=variant, splits=splits, **dkw), out)


# ------------------------------------------------------------------------- caps
@pytest.mark.parametrize("variant,splits", FORMS)
@pytest.mark.parametrize("cap", [1e-18, 0.5, 30.0, 128.0, 129.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e18])
@pytest.mark.parametrize("slopes", [False, True])
def test_caps(fc, variant, splits, cap, slopes):  # noqa: F811
    """Scores of deviation 3 under any cap: one far above them is none."""
    b = batch(61, F16, [333, 20, 190], [3, 20, 1], 4, 2, 64, 16)
    kw = dict(scale=0.375, softcap=cap)
    if slopes:
        kw["slopes"] = torch.tensor([0.5, 0.0, 0.03, -0.02])
    attend(fc, b, "cap %g slopes %d" % (cap, slopes), variant, splits, **kw)


@pytest.mark.parametrize("variant,splits", FORMS)
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_caps_of_every_head_size(fc, variant, splits, d):  # noqa: F811
    b = batch(67, BF16, [150, 300], [40, 2], 4, 2, d, 32)
    for kw in (dict(softcap=2e5), dict(softcap=2e5, causal=False, slopes=torch.tensor([0.1, 0.0, 0.02, 0.3]))):
        attend(fc, b, "d %d %s" % (d, sorted(kw)), variant, splits, **kw)


@pytest.mark.parametrize("variant,splits", FORMS)
def test_caps_near_the_scores(fc, variant, splits):  # noqa: F811
    """Scores on both sides of a large cap."""
    b = batch(71, F16, [333, 90], [3, 40], 4, 2, 64, 16)
    attend(fc, b, "scores of the cap's size", variant, splits, scale=100.0, softcap=1000.0)


@pytest.mark.parametrize("variant,splits", FORMS)
def test_caps_with_most_keys_far_below(fc, variant, splits):  # noqa: F811
    """Three keys of four are at minus the cap, the others' scores are small:
    the latter alone decide, and carry the small scores' accuracy."""
    b = batch(73, F16, [400, 70], [2, 40], 4, 2, 64, 16)
    b["q"][:, :, 0] = 64.0
    K = R.unpack_k(b["codes"][:, :, 0], 64).clone()
    nan = K == 0x7f
    K[..., 0] = torch.where(torch.arange(K.shape[2]) % 4 == 0, 0x00, 0xfe)      # 0 and -448
    K[nan] = 0x7f
    b["codes"][:, :, 0] = R.pack_k(K.reshape(K.shape[0], 2, 1, 16, 64))
    b["scales"][:, :, 0] = 2.0 ** -4
    attend(fc, b, "most keys far below", variant, splits, scale=0.5, softcap=300.0)


# ------------------------------------------------------------------- flat tails
def tail_batch(dtype, n, d=64, page=128):
    """One sequence whose first key is 16, 17, 17.4 and 18 above the others for the
    four heads, with values near 1 behind the others and 0 behind it."""
    g = gen(79)
    pages = -(-n // page)
    K = torch.randn((pages, 1, page, d), generator=g) * 0.375
    V = 1.0 + torch.randn((pages, 1, page, d), generator=g) / 4
    K[:, :, :, 0] = 0.0
    K[0, 0, 0] = 0.0
    K[0, 0, 0, 0] = 16.0
    V[0, 0, 0] = 0.0
    codes = torch.empty((pages, 1, 2, page // 16, 16 * d), dtype=torch.uint8)
    codes[:, :, 0] = R.pack_k(R.encode(K).reshape(pages, 1, page // 16, 16, d))
    codes[:, :, 1] = R.pack_v(R.encode(V).reshape(pages, 1, page // 16, 16, d))
    q = torch.randn((1, 4, d), generator=g) / 4
    q[0, :, 0] = torch.tensor([8.0, 8.5, 8.7, 9.0])
    return dict(q=q.to(dtype), codes=codes, scales=torch.ones((pages, 1, 2)),
                table=torch.arange(pages, dtype=torch.int32)[None], cu_q=i32([0, 1]), kv_lens=i32([n]))


@pytest.mark.parametrize("variant,splits", FORMS + [("rows", 40), ("tile", 40)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [40000, 131071])
def test_flat_tail_under_a_dominant_key(fc, variant, splits, dtype, n):  # noqa: F811
    """The tail's small weights, of which there are many, are not lost."""
    attend(fc, tail_batch(dtype, n), "tail of %d %s" % (n, dtype), variant, splits)


@pytest.mark.parametrize("variant,splits", FORMS)
@pytest.mark.parametrize("every", [8, 64])
def test_scores_whose_steps_are_coarse(fc, variant, splits, every):  # noqa: F811
    """Scores of 2^27 and more, where neighbours in 32 bits are 16 apart (in units
    of log 2): weights stay inside fp16's range, results among the values."""
    n, d, page = 200, 64, 16
    pages = 13
    K, V = torch.zeros((pages, 1, page, d)), torch.randn((pages, 1, page, d), generator=gen(83))
    K[:, :, :, 0] = 128.0
    for p in range(pages):
        for t in range(page):
            K[p, 0, t, 1] = (p * page + t) // every          # a step of 16 above the keys before
    codes = torch.empty((pages, 1, 2, 1, 16 * d), dtype=torch.uint8)
    codes[:, :, 0] = R.pack_k(R.encode(K).reshape(pages, 1, 1, 16, d))
    codes[:, :, 1] = R.pack_v(R.encode(V).reshape(pages, 1, 1, 16, d))
    scales = torch.ones((pages, 1, 2))
    scales[:, :, 0] = 2.0 ** 7
    q = torch.zeros((1, 2, d))
    q[:, :, 0] = 2.0 ** 13
    q[:, :, 1] = 2.0 ** -3
    b = dict(q=q.half(), codes=codes, scales=scales, table=torch.arange(pages, dtype=torch.int32)[None],
             cu_q=i32([0, 1]), kv_lens=i32([n]))
    vals = R.values(R.encode(V)).abs().max()
    for scale in (0.69314, math.log(2.0), 0.6932, 4.0 * math.log(2.0)):
        print("case coarse", variant, splits, scale, flush=True)
        out = fc.chain_attn(**on_gpu(b), scale=scale, variant=variant, splits=splits).cpu().double()
        assert torch.isfinite(out).all(), scale
        assert out.abs().max() <= vals * (1 + 2.0 ** -10), scale


# ---------------------------------------------------------------------- windows
@pytest.mark.parametrize("variant,splits", FORMS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 31, 2 ** 32 + 3, 2 ** 63 - 1])
def test_windows_of_any_size(fc, variant, splits, window):  # noqa: F811
    """A window that no sequence fills is none, for queries before slot 0 too."""
    b = batch(89, BF16, [40, 300], [64, 3], 4, 2, 128, 16)
    want = fc.chain_attn(**on_gpu(b), variant=variant, splits=splits)
    print("case window", variant, splits, window, flush=True)
    assert torch.equal(fc.chain_attn(**on_gpu(b), variant=variant, splits=splits, window=window), want)
    ref, tol, _, _ = R.attention(**b)
    R.assert_within(want, ref, R.rounded_tol(ref, tol, BF16), "window %d" % window)
