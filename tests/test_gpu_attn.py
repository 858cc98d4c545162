"""rope, kv_append and chain_attn on the GPU against plain implementations in 64
bits (attn_ref), at the sizes, masks and layouts where they can go wrong."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
DTYPES = [F16, BF16]


@pytest.fixture(scope="module")
def fc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gemm_conv_chain_amd as m
    m.lib()
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


# ------------------------------------------------------------------------- rope
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot,inverse,mscale", [
    (1, 1, 64, 64, False, 1.0),
    (7, 3, 128, 128, True, 1.0),
    (33, 5, 192, 48, False, 1.25),
    (5, 2, 256, 16, True, 1.0),
    (19, 9, 80, 80, False, 1.0),
    (700, 40, 128, 128, False, 1.0),      # many blocks
    (900, 35, 128, 96, True, 0.5),        # and an odd number of heads
])
def test_rope(fc, dtype, interleaved, T, H, D, rot, inverse, mscale):
    print("case rope", dtype, interleaved, T, H, D, rot, inverse, flush=True)
    g = gen(T * 7 + D)
    x = torch.randn((T, H, D), generator=g).to(dtype)
    pos = torch.randint(-5000, 2 ** 20, (T,), generator=g, dtype=torch.int32)
    turns, _ = fc.rope_turns(rot)
    y = fc.rope(x.cuda(), pos.cuda(), turns.cuda(), interleaved=interleaved, mscale=mscale, inverse=inverse)
    ref, inner = R.rope(x, pos.tolist(), turns, interleaved, mscale, inverse)
    R.assert_within(y, ref, R.rounded_tol(ref, inner, dtype), "rope")
    assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


def test_rope_far_positions_strides_in_place(fc):
    # the ends of the 32-bit positions; rows inside wider rows; y = x
    print("case rope far", flush=True)
    g = gen(5)
    pos = i32([2 ** 31 - 1, -2 ** 31, 0, 2 ** 30 + 1, -1, 123456789])
    rows = torch.randn((6, 8, 128), generator=g).to(BF16)
    turns, mscale = fc.rope_turns(128, scaling="ramp", factor=8.0, original=4096, high=32.0, low=1.0)
    ref, inner = R.rope(rows[:, 2:7], pos.tolist(), turns, mscale=mscale)
    d = rows.cuda()
    y = fc.rope(d[:, 2:7], pos.cuda(), turns.cuda(), mscale=mscale)
    R.assert_within(y, ref, R.rounded_tol(ref, inner, BF16), "rope far")
    z = fc.rope(d[:, 2:7], pos.cuda(), turns.cuda(), mscale=mscale, out=d[:, 2:7])
    assert torch.equal(z, y)
    assert torch.equal(d.cpu()[:, :2], rows[:, :2]) and torch.equal(d.cpu()[:, 7:], rows[:, 7:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(fc, interleaved):
    """The inverse is the gradient: <rope(x), w> = <x, inverse(w)>, and the loss
    <rope(x), w> changes along a direction by its product with inverse(w)."""
    print("case rope gradient", flush=True)
    g = gen(9)
    T, H, D = 11, 3, 128
    x, w, dx = (torch.randn((T, H, D), generator=g).to(F16) for _ in range(3))
    pos = torch.randint(0, 9000, (T,), generator=g, dtype=torch.int32).cuda()
    turns, _ = fc.rope_turns(64)
    t = turns.cuda()
    kw = dict(interleaved=interleaved, mscale=1.5)
    grad = fc.rope(w.cuda(), pos, t, inverse=True, **kw).cpu().double()
    ref, inner = R.rope(w, pos.tolist(), turns, interleaved, 1.5, True)
    R.assert_within(grad, ref, R.rounded_tol(ref, inner, F16), "rope gradient")

    def loss(v):
        return float((fc.rope(v.cuda(), pos, t, **kw).cpu().double() * w.double()).sum())
    step = (loss(x + dx) - loss(x - dx)) / 2
    # every element of the two results and of the gradient is off by half a step of
    # fp16 at most: their sizes are those of the vectors
    u = R.half_step(F16)
    size = 1.5 * float(((x + dx).double().abs() + (x - dx).double().abs()).max()) * 2
    moved = ((x + dx).double() - (x - dx).double()) / 2
    tol = u * (size * float(w.double().abs().sum()) + float((grad.abs() * moved.abs()).sum()) * 2)
    assert abs(step - float((grad * moved).sum())) <= tol


# ---------------------------------------------------------------------- batches
def batch(seed, dtype, lens, new, hq, hkv, d, page, spare=3, fill="values"):
    """Host tensors of a batch whose cache holds random values under random
    scales; what is past a sequence's length is NaN codes."""
    g = gen(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((B, max(max(need), 1)), -7, dtype=torch.int32)    # what is not needed is no page
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]].to(torch.int32)
        at += need[b]
    scales = torch.exp2(torch.randint(-8, -3, (pages, hkv, 2), generator=g).float())
    x = torch.randn((pages, hkv, 2, page // 16, 16 * d), generator=g) / scales[..., None, None] / 2
    codes = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    K, V = R.unpack_k(codes[:, :, 0], d).clone(), R.unpack_v(codes[:, :, 1], d).clone()
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b in range(B):
        for p in range(need[b]):
            used[int(table[b, p]), :min(page, lens[b] - p * page)] = True
    K[~used[:, None].expand(-1, hkv, -1)] = 0x7f
    V[~used[:, None].expand(-1, hkv, -1)] = 0xff
    n16 = page // 16
    codes[:, :, 0] = R.pack_k(K.reshape(pages, hkv, n16, 16, d))
    codes[:, :, 1] = R.pack_v(V.reshape(pages, hkv, n16, 16, d))
    T = sum(new)
    q = (torch.randn((T, hq, d), generator=g) * 2).to(dtype)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(q=q, codes=codes, scales=scales, table=table, cu_q=i32(cu), kv_lens=i32(list(lens)))


def on_gpu(b):
    return {k: v.cuda() for k, v in b.items()}


def attend(fc, b, what, dtype, check_lse=True, **kw):
    """Runs chain_attn and checks out and lse."""
    print("case attn", what, flush=True)
    ref, tol, lse, ltol = R.attention(b["q"], b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"],
                                      **{k: kw[k] for k in ("scale", "causal", "softcap", "window", "slopes") if k in kw})
    dkw = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    out, le = fc.chain_attn(**on_gpu(b), lse=True, **dkw)
    R.assert_within(out, ref, R.rounded_tol(ref, tol, dtype), what)
    if check_lse:
        R.assert_within(le, lse, ltol, what + " lse")
    return out


FORMS = [("rows", 1), ("rows", 3), ("tile", 1), ("tile", 2)]


@pytest.mark.parametrize("variant,splits", FORMS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,new,hq,hkv,d,page", [
    ([1], [1], 1, 1, 64, 16),
    ([0, 5, 64, 65], [0, 1, 1, 1], 8, 2, 64, 16),
    ([17, 300, 33], [1, 1, 1], 6, 2, 128, 32),
    ([130, 129, 1], [3, 0, 1], 4, 4, 128, 64),
    ([200, 77], [5, 40], 10, 2, 192, 16),
    ([513], [7], 3, 1, 256, 128),
    ([260, 40], [70, 40], 8, 2, 64, 256),
    ([150], [150], 2, 1, 128, 32),
])
def test_attn_shapes(fc, variant, splits, dtype, lens, new, hq, hkv, d, page):
    b = batch(sum(lens) + d, dtype, lens, new, hq, hkv, d, page)
    attend(fc, b, "%s/%d %s %s %s" % (variant, splits, lens, new, (hq, hkv, d, page)), dtype, variant=variant,
           splits=splits)


@pytest.mark.parametrize("variant,splits", FORMS)
@pytest.mark.parametrize("kw", [
    dict(causal=False), dict(softcap=5.0), dict(softcap=50.0), dict(window=1), dict(window=16), dict(window=100),
    dict(window=10000), dict(slopes=True), dict(softcap=8.0, slopes=True, window=70), dict(scale=0.5),
    dict(causal=False, slopes=True)], ids=str)
def test_attn_masks(fc, variant, splits, kw):
    kw = dict(kw)
    lens, new = [333, 20, 190], [3, 20, 1]
    b = batch(17, F16, lens, new, 4, 2, 64, 16)
    if kw.get("slopes"):
        kw["slopes"] = torch.tensor([0.5, 0.0, 0.03, -0.02])
    attend(fc, b, "%s/%d %s" % (variant, splits, kw), F16, variant=variant, splits=splits, **kw)


@pytest.mark.parametrize("variant,splits", FORMS)
def test_attn_empty_rows(fc, variant, splits):
    # more queries than keys: the first of them see nothing; a sequence of no keys
    b = batch(3, BF16, [4, 30], [10, 2], 4, 2, 128, 16)
    b["kv_lens"][1] = 0
    out = attend(fc, b, "empty rows", BF16, variant=variant, splits=splits)
    assert out[:6].abs().max() == 0 and out[10:].abs().max() == 0


@pytest.mark.parametrize("variant,splits", FORMS)
def test_attn_masked_places_hold_anything(fc, variant, splits):
    """Pages before the window may be gone (ids that are no page), keys after a
    query may be NaN: nothing of it reaches a row that does not see it."""
    lens, new = [400, 90], [2, 90]
    b = batch(23, F16, lens, new, 4, 2, 64, 16)
    window = 50
    clean, tol, _, _ = R.attention(**b, window=window)
    first = lens[0] - new[0] - window + 1
    b["table"][0, :first // 16] = torch.tensor([2 ** 30, -1] * 50)[:first // 16]      # evicted
    out = fc.chain_attn(**on_gpu(b), window=window, variant=variant, splits=splits)
    R.assert_within(out, clean, R.rounded_tol(clean, tol, F16), "evicted pages")
    # token 60 of the second sequence has a NaN key: rows that see it are NaN
    K = R.unpack_k(b["codes"][:, :, 0], 64)
    page, slot = int(b["table"][1, 60 // 16]), 60 % 16
    K[page, :, slot, 5] = 0x7f
    b["codes"][:, :, 0] = R.pack_k(K.reshape(K.shape[0], 2, 1, 16, 64))
    out = fc.chain_attn(**on_gpu(b), window=window, variant=variant, splits=splits).cpu()
    i = torch.arange(90)
    sees = (i >= 60) & (i - 60 < window)
    assert torch.isnan(out[2:][sees]).all()
    R.assert_within(out[2:][~sees], clean[2:][~sees], R.rounded_tol(clean, tol, F16)[2:][~sees], "NaN key")


@pytest.mark.parametrize("variant,splits", FORMS)
def test_attn_bad_metadata_gives_nan_rows(fc, variant, splits):
    """Ids outside the pool and lengths past the table's row are caught by the
    kernel's own bounds checks: NaN rows for that sequence, no other changes."""
    lens, new = [100, 64, 40], [2, 1, 3]
    b = batch(29, BF16, lens, new, 4, 2, 128, 16)
    good = attend(fc, b, "before", BF16, variant=variant, splits=splits)
    b["table"][0, 3] = b["codes"].shape[0]
    b["kv_lens"][2] = 16 * b["table"].shape[1] + 1
    out, lse = fc.chain_attn(**on_gpu(b), variant=variant, splits=splits, lse=True)
    assert torch.isnan(out[:2]).all() and torch.isnan(out[3:]).all() and torch.isnan(lse[:2]).all()
    assert torch.equal(out[2], good[2])


@pytest.mark.parametrize("variant,splits", FORMS)
def test_attn_hints_only_size_the_launch(fc, variant, splits):
    b = batch(31, F16, [500, 130], [60, 3], 4, 2, 64, 32)
    want = attend(fc, b, "hints", F16, variant=variant, splits=splits)
    for mq, mk in ((1, 1), (0, 0), (2, 40), (60, 500)):
        got = fc.chain_attn(**on_gpu(b), variant=variant, splits=splits, max_q=mq, max_kv=mk).cpu().double()
        ref, tol, _, _ = R.attention(**b)
        R.assert_within(got, ref, R.rounded_tol(ref, tol, F16), "hints %d %d" % (mq, mk))
    assert want.shape == (63, 4, 64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attn_by_rule_strided_lse_out(fc, dtype):
    """The chosen form, q inside a wider row, out and lse of the caller."""
    lens, new = [700, 3, 1200], [1, 1, 1]
    b = batch(37, dtype, lens, new, 8, 2, 128, 64)
    wide = torch.zeros((3, 14, 128), dtype=dtype)
    wide[:, 3:11] = b["q"]
    ref, tol, lse, ltol = R.attention(**b)
    g = on_gpu(b)
    g["q"] = wide.cuda()[:, 3:11]
    out = torch.full((3, 8, 128), float("nan"), dtype=dtype, device="cuda")
    le = torch.full((3, 8), float("nan"), device="cuda")
    o2, l2 = fc.chain_attn(**g, out=out, lse=le, max_q=1, max_kv=1200)
    assert o2 is out and l2 is le
    R.assert_within(out, ref, R.rounded_tol(ref, tol, dtype), "by rule")
    R.assert_within(le, lse, ltol, "by rule lse")
    # the same bits on every run
    for _ in range(3):
        assert torch.equal(fc.chain_attn(**g, max_q=1, max_kv=1200), out)


def test_attn_offsets_past_32_bits(fc):
    """A pool of over 4 GiB whose last pages are in use."""
    print("case attn offsets", flush=True)
    b = batch(41, BF16, [70], [2], 4, 2, 128, 32)
    page_bytes = 2 * 2 * 32 * 128
    pages = (1 << 32) // page_bytes + 50
    codes = torch.zeros((pages, 2, 2, 2, 16 * 128), dtype=torch.uint8, device="cuda")
    scales = torch.ones((pages, 2, 2), device="cuda")
    n = b["codes"].shape[0]
    codes[-n:] = b["codes"].cuda()
    scales[-n:] = b["scales"].cuda()
    ref, tol, _, _ = R.attention(**b)
    g = on_gpu(b)
    g.update(codes=codes, scales=scales, table=torch.where(b["table"] >= 0, b["table"] + (pages - n), 0).to(torch.int32).cuda())
    for variant in ("rows", "tile"):
        out = fc.chain_attn(**g, variant=variant)
        R.assert_within(out, ref, R.rounded_tol(ref, tol, BF16), "offsets " + variant)
    # and the append's
    k, v = torch.randn((2, 2, 128)).to(BF16), torch.randn((2, 2, 128)).to(BF16)
    small = R.append(k, v, b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"])
    fc.kv_append(k.cuda(), v.cuda(), codes, scales, g["table"], g["cu_q"], g["kv_lens"])
    R.assert_appended(codes[-n:], scales[-n:], small, "offsets append")
    assert int(codes[:-n].sum(dtype=torch.int64)) == 0


# -------------------------------------------------------------------- kv_append
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,new,hq,hkv,d,page,rot,interleaved", [
    ([1], [1], 1, 1, 64, 16, 64, False),
    ([5, 16, 17, 0], [1, 1, 1, 0], 4, 2, 64, 16, 32, True),
    ([40, 100, 64], [1, 1, 1], 8, 4, 128, 64, 128, False),
    ([150, 33, 16], [90, 33, 1], 6, 3, 128, 32, 128, True),
    ([100, 7], [61, 5], 2, 2, 192, 16, 48, False),
    ([300, 20], [270, 2], 2, 1, 256, 128, 256, False),
    ([530], [290], 2, 2, 64, 256, 0, False),
])
def test_append(fc, dtype, lens, new, hq, hkv, d, page, rot, interleaved):
    print("case append", dtype, lens, new, hq, hkv, d, page, rot, flush=True)
    b = batch(sum(lens) * 3 + d, dtype, lens, new, hq, hkv, d, page)
    g = gen(sum(new))
    T = sum(new)
    k, v = (torch.randn((T, hkv, d), generator=g) * torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())
            for _ in range(2))
    k, v = k.to(dtype), v.to(dtype)
    turns = fc.rope_turns(rot)[0] if rot else None
    expect = R.append(k, v, b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], turns, interleaved)
    c = on_gpu(b)
    q = b["q"]
    dt = None if turns is None else turns.cuda()
    qo = fc.kv_append(k.cuda(), v.cuda(), c["codes"], c["scales"], c["table"], c["cu_q"], c["kv_lens"], turns=dt,
                      interleaved=interleaved, q=c["q"], max_q=max(new))
    R.assert_appended(c["codes"], c["scales"], expect, "append")
    slots = [s for n, L in zip(new, lens) for s in range(L - n, L)]
    if rot:
        ref, inner = R.rope(q, slots, turns, interleaved)
        R.assert_within(qo, ref, R.rounded_tol(ref, inner, dtype), "append q")
    else:
        assert torch.equal(qo.cpu(), q)
    # the same tokens again: nothing changes
    before = c["codes"].clone(), c["scales"].clone()
    fc.kv_append(k.cuda(), v.cuda(), c["codes"], c["scales"], c["table"], c["cu_q"], c["kv_lens"], turns=dt,
                 interleaved=interleaved)
    assert torch.equal(c["codes"], before[0]) and torch.equal(c["scales"], before[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_special_values(fc, dtype):
    """Zeros, infinities, NaN, subnormals and the type's largest values."""
    print("case append special", dtype, flush=True)
    d, page, hkv = 64, 16, 2
    lens, new = [20, 24, 40, 18, 16, 35], [20, 24, 40, 18, 16, 35]
    b = batch(7, dtype, lens, new, 2, hkv, d, page)
    T = sum(new)
    g = gen(11)
    k, v = torch.randn((T, hkv, d), generator=g).to(dtype), torch.randn((T, hkv, d), generator=g).to(dtype)
    big = torch.finfo(dtype).max
    k[0:20] = 0
    v[0:20] = 0                                        # a page of zeros
    k[21, 0, 3], v[22, 1, 7] = math.inf, -math.inf     # saturate, and do not set the scale
    k[45, 1, 2] = math.nan                             # stays
    v[50, 0, 9] = math.nan                             # marks its key
    k[84:90], v[84:90] = big, -big                     # sequence 3: the largest
    k[102:118] = (torch.randn((16, hkv, d), generator=g) * 1e-7).to(dtype)      # tiny
    v[102:118] = torch.finfo(dtype).smallest_normal / 4
    expect = R.append(k, v, b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"])
    c = on_gpu(b)
    fc.kv_append(k.cuda(), v.cuda(), c["codes"], c["scales"], c["table"], c["cu_q"], c["kv_lens"])
    R.assert_appended(c["codes"], c["scales"], expect, "append special")
    out = fc.chain_attn(c["q"][:, :2], c["codes"], c["scales"], c["table"], c["cu_q"], c["kv_lens"]).cpu()
    # the NaN tokens' own rows and later ones of their sequence and head, and no others
    # (left out: rows 84 - 101, where the largest bf16 keys' scores exceed 32 bits)
    out[84:102] = 0
    nan = torch.isnan(out).all(-1)
    assert not nan[:44].any() and not nan[84:].any()
    assert not nan[44:45].any() and nan[45:84, 1].all()
    assert not nan[44:50, 0].any() and nan[50:84, 0].all()
    assert torch.isfinite(out[~nan].float()).all()


def test_append_step_by_step_equals_reference(fc):
    """Tokens of changing loudness one at a time: pages' scales grow and their
    earlier codes are rounded again."""
    print("case append steps", flush=True)
    d, page, hkv, dtype = 64, 16, 2, F16
    codes, scales = fc.kv_cache(4, hkv, page, d)
    table = i32([[2, 0, 3]])
    turns, _ = fc.rope_turns(64)
    g = gen(13)
    hc, hs = codes.cpu(), scales.cpu()
    for n in range(1, 40):
        k, v = ((torch.randn((1, hkv, d), generator=g) * 2.0 ** ((n * 5) % 7 - 3)).to(dtype) for _ in range(2))
        cu, lens = i32([0, 1]), i32([n])
        expect = R.append(k, v, hc, hs, table, cu, lens, turns)
        fc.kv_append(k.cuda(), v.cuda(), codes, scales, table.cuda(), cu.cuda(), lens.cuda(), turns=turns.cuda(), max_q=1)
        R.assert_appended(codes, scales, expect, "step %d" % n)
        hc, hs = codes.cpu(), scales.cpu()


def test_append_positions_strides_dropped(fc):
    """Positions apart from slots, k and v inside a projection's rows; tokens before
    slot 0, without a page or past the table are not written."""
    print("case append dropped", flush=True)
    d, page, hkv, dtype = 128, 16, 2, BF16
    b = batch(19, dtype, [20, 40, 64], [20, 9, 30], 4, hkv, d, page)
    b["kv_lens"] = i32([12, 40, 70])           # 8 tokens before slot 0; 6 past the table's row of 4 pages
    b["table"][1, 2] = 10 ** 6                  # no page
    T = 59
    g = gen(23)
    rows = torch.randn((T, 4 + 2 * hkv, d), generator=g).to(dtype)
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32)
    turns, mscale = fc.rope_turns(128, scaling="linear", factor=4.0)
    expect = R.append(rows[:, 4:6], rows[:, 6:], b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], turns,
                      False, 1.0, pos)
    c, dr = on_gpu(b), rows.cuda()
    qo = fc.kv_append(dr[:, 4:6], dr[:, 6:], c["codes"], c["scales"], c["table"], c["cu_q"], c["kv_lens"],
                      turns=turns.cuda(), positions=pos.cuda(), q=dr[:, :4])
    R.assert_appended(c["codes"], c["scales"], expect, "append dropped")
    ref, inner = R.rope(rows[:, :4], pos.tolist(), turns)
    R.assert_within(qo, ref, R.rounded_tol(ref, inner, dtype), "append q positions")


def test_empty_calls(fc):
    print("case empty", flush=True)
    codes, scales = fc.kv_cache(2, 2, 16, 64)
    z = torch.zeros((0, 2, 64), dtype=F16, device="cuda")
    meta = i32([[0], [1]]).cuda(), i32([0, 0, 0]).cuda(), i32([0, 5]).cuda()
    assert fc.chain_attn(z, codes, scales, *meta).shape == (0, 2, 64)
    assert fc.kv_append(z, z, codes, scales, *meta, q=z).shape == (0, 2, 64)
    assert fc.rope(z, meta[2][:0], fc.rope_turns(64)[0].cuda()).shape == (0, 2, 64)


# ------------------------------------------------------------ drawn mixtures
@pytest.mark.parametrize("seed", range(24))
def test_attn_drawn(fc, seed):
    """Sizes, heads, pages, masks, forms and splits drawn together."""
    r = random.Random(seed)
    dtype, d, page = DTYPES[seed % 2], (64, 128, 192, 256)[seed // 2 % 4], r.choice([16, 32, 64, 128, 256])
    hkv, G = r.choice([1, 2, 3, 8]), r.choice([1, 2, 3, 4, 7])
    lens = [r.choice([0, 1, 15, 16, 17, r.randrange(1, 900), r.randrange(1, 2500)]) for _ in range(r.randrange(1, 5))]
    new = [min(n, r.choice([0, 1, 1, 2, 5, r.randrange(1, 150)])) for n in lens]
    new[0] = max(new[0], 1)                  # at least one query, of which some see no key where lens[0] = 0
    b = batch(seed + 900, dtype, lens, new, hkv * G, hkv, d, page)
    kw = dict(causal=r.random() < 0.8, softcap=r.choice([0.0, 0.0, 20.0]))
    if kw["causal"]:
        kw["window"] = r.choice([0, 0, 1, 33, 500])
    if r.random() < 0.3:
        kw["slopes"] = torch.tensor([0.25 / (1 + h) for h in range(hkv * G)])
    if r.random() < 0.5:
        kw.update(variant=r.choice(["rows", "tile"]), splits=r.choice([0, 1, 2, 4]))
    if r.random() < 0.5:
        kw.update(max_q=max(new), max_kv=max(lens))
    attend(fc, b, "drawn %d %s %s %s" % (seed, lens, new, (hkv * G, hkv, d, page)), dtype, **kw)


# -------------------------------------------------- streams, graphs, debug build
def test_on_another_stream(fc):
    """Work goes to torch's current stream."""
    print("case stream", flush=True)
    b = batch(43, BF16, [900, 400], [1, 1], 8, 2, 128, 32)
    g = on_gpu(b)
    want = fc.chain_attn(**g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q2 = torch.empty_like(g["q"])
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)
        q2.copy_(g["q"])                       # the call has to wait for this copy
        got = fc.chain_attn(**{**g, "q": q2}, splits=3, variant="rows")
        x = fc.rope(q2, i32([7, 9]).cuda(), fc.rope_turns(128)[0].cuda())
    s.synchronize()
    ref, tol, _, _ = R.attention(**b)
    R.assert_within(got, ref, R.rounded_tol(ref, tol, BF16), "stream")
    assert torch.equal(x, fc.rope(g["q"], i32([7, 9]).cuda(), fc.rope_turns(128)[0].cuda()))
    assert want.shape == got.shape


@pytest.mark.parametrize("new", [1, 40])
def test_step_in_a_graph(fc, new):
    """append (with q turned) and attention captured together, replayed with new
    inputs and growing lengths, against the eager calls on a copy of the pool."""
    print("case graph", new, flush=True)
    lens = [300, 64, 17]
    hq, hkv, d, page = 8, 2, 64, 16
    pages, spare = 90, 12
    g = gen(47)
    codes, scales = fc.kv_cache(pages, hkv, page, d)
    table = torch.randperm(pages, generator=g)[:3 * 30].reshape(3, 30).to(torch.int32).cuda()
    cu = i32([0, new, 2 * new, 3 * new]).cuda()
    kv = i32([n + new for n in lens]).cuda()
    turns = fc.rope_turns(64)[0].cuda()
    rows = torch.empty((3 * new, hq + 2 * hkv, d), dtype=F16, device="cuda")
    rows.normal_()
    out = torch.empty((3 * new, hq, d), dtype=F16, device="cuda")
    qo = torch.empty_like(out)

    def step(c, s, o):
        fc.kv_append(rows[:, hq:hq + hkv], rows[:, hq + hkv:], c, s, table, cu, kv, turns=turns, q=rows[:, :hq], q_out=qo,
                     max_q=new)
        return fc.chain_attn(qo, c, s, table, cu, kv, out=o, max_q=new, max_kv=480)
    step(codes, scales, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(codes, scales, out)
    c2, s2 = codes.clone(), scales.clone()
    o2 = torch.empty_like(out)
    for r in range(4):
        rows.normal_()
        kv.add_(1)
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        step(c2, s2, o2)
        torch.cuda.synchronize()
        assert float(junk) == float(junk)
        assert torch.equal(out, o2) and torch.equal(codes, c2) and torch.equal(scales, s2), "replay %d" % r


@pytest.mark.parametrize("variant,splits", FORMS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_poison_attn(fc, variant, splits, d):
    """The debug build, whose LDS holds NaN codes until a stage's data arrives."""
    print("case poison attn", variant, splits, d, flush=True)
    b = batch(53, BF16, [700, 90, 333], [3, 90, 40], 4, 2, d, 16)
    g = on_gpu(b)
    want = fc.chain_attn(**g, variant=variant, splits=splits)
    torch.cuda.synchronize()
    with fc.poison_build():
        got = fc.chain_attn(**g, variant=variant, splits=splits)
        torch.cuda.synchronize()
    assert torch.isfinite(got.float()).all()
    assert torch.equal(got, want)
