"""Host-only checks of rope_apply, kv_append, chain_attn and kv_check: refusals
(validation runs before any HIP call), the plan, the rotary tables, and the
binding's argument checks with host tensors."""
import ctypes
import math

import pytest

import gemm_conv_chain_amd as fc

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.cpu

OK, E_NULL, E_SHAPE, E_ALIGN, E_UNSUP, E_HIP, E_ARG = range(7)
P = ctypes.c_void_p(0x10000)       # fake, aligned device pointers: validation never reads them
BAD = ctypes.c_void_p(0x10002)
NUL = None


@pytest.fixture(scope="module")
def L():
    return fc.lib()


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rope(L, x=P, y=P, st=(512, 64, 512, 64), pos=P, turns=0x10000, rot=64, table=True, dtype=0, T=4, H=8, D=64):
    r = fc.RopeTable(turns, rot, 0, 1.0) if table else None
    return L.rope_apply(x, y, None if st is None else strides(*st), pos, r, 0, dtype, T, H, D, None)


def test_rope_refusals(L):
    assert rope(L, T=0) == OK and rope(L, H=0) == OK
    assert rope(L, T=0, x=NUL, y=NUL, pos=NUL) == OK
    assert rope(L, x=NUL) == E_NULL and rope(L, y=NUL) == E_NULL and rope(L, pos=NUL) == E_NULL
    assert rope(L, table=False) == E_NULL and rope(L, st=None) == E_NULL
    assert rope(L, turns=None) == E_NULL
    assert rope(L, turns=0x10004) == E_ALIGN
    assert rope(L, x=BAD) == E_ALIGN and rope(L, y=BAD) == E_ALIGN and rope(L, pos=BAD) == E_ALIGN
    assert rope(L, st=(512, 64, 513, 64)) == E_ALIGN
    assert rope(L, T=-1) == E_SHAPE and rope(L, D=72) == E_SHAPE and rope(L, D=0) == E_SHAPE
    assert rope(L, rot=24) == E_SHAPE and rope(L, rot=80) == E_SHAPE and rope(L, rot=-16) == E_SHAPE
    assert b"rot" in L.fc_last_error()
    assert rope(L, D=1040, rot=64) == E_UNSUP
    assert rope(L, dtype=2) == E_ARG


def shape(dtype=0, batch=2, hq=8, hkv=2, d=64, page=16, pages=10, stride=4, tokens=2, max_q=1, max_kv=64):
    return fc.KvShape(dtype, batch, hq, hkv, d, page, pages, stride, tokens, max_q, max_kv)


def append(L, k=P, v=P, q=P, qo=P, st=(1, 8, 1, 8, 1, 8), codes=P, scales=P, table=P, cu=P, lens=P, pos=NUL, rot=64,
           sh=None, no_shape=False, **kw):
    st = strides(*[8 * s for s in st]) if st is not None else None
    r = fc.RopeTable(0x10000, rot, 0, 1.0)
    return L.kv_append(k, v, q, qo, st, codes, scales, table, cu, lens, pos, r,
                       None if no_shape else shape(**kw), None)


def attn(L, q=P, codes=P, scales=P, table=P, cu=P, lens=P, slopes=NUL, out=P, lse=NUL, ws=NUL, wsb=0, scale=0.125, cap=0.0,
         causal=1, window=0, variant=0, splits=1, no_params=False, no_shape=False, st=(512, 64), **kw):
    pa = fc.AttnParams(scale, cap, causal, window, variant, splits)
    return L.chain_attn(q, None if st is None else strides(*st), codes, scales, table, cu, lens, slopes,
                        None if no_params else pa, out, lse, None if no_shape else shape(**kw), ws, wsb, None)


SHAPE_REFUSALS = [
    (dict(dtype=2), E_ARG), (dict(batch=-1), E_SHAPE), (dict(tokens=-1), E_SHAPE), (dict(hq=0), E_SHAPE),
    (dict(hkv=0), E_SHAPE), (dict(hq=7), E_SHAPE), (dict(max_q=-1), E_SHAPE), (dict(max_kv=-1), E_SHAPE),
    (dict(pages=-1), E_SHAPE), (dict(pages=0), E_SHAPE), (dict(stride=0), E_SHAPE), (dict(d=80), E_UNSUP),
    (dict(d=512), E_UNSUP), (dict(page=8), E_UNSUP), (dict(page=48), E_UNSUP), (dict(page=512), E_UNSUP),
    (dict(hq=65536, hkv=1), E_UNSUP), (dict(tokens=2 ** 28), E_UNSUP), (dict(batch=2 ** 20 + 1), E_UNSUP), (dict(stride=2 ** 27), E_UNSUP),
]


@pytest.mark.parametrize("kw,status", SHAPE_REFUSALS, ids=str)
def test_shape_refusals(L, kw, status):
    assert attn(L, **kw) == status
    assert append(L, **kw) == status


def test_append_refusals(L):
    assert append(L, tokens=0, k=NUL, v=NUL, codes=NUL) == OK
    assert append(L, batch=0, k=NUL) == OK
    for name in ("k", "v", "codes", "scales", "table", "cu", "lens"):
        assert append(L, **{name: NUL}) == E_NULL, name
        assert append(L, **{name: BAD}) == E_ALIGN, name
    assert append(L, pos=BAD) == E_ALIGN
    assert append(L, q=NUL) == E_NULL and append(L, qo=NUL) == E_NULL
    assert append(L, st=None) == E_NULL and append(L, no_shape=True) == E_NULL
    assert append(L, rot=80) == E_SHAPE


def test_attn_refusals(L):
    assert attn(L, tokens=0, q=NUL, out=NUL, codes=NUL) == OK
    assert attn(L, batch=0, q=NUL) == OK
    for name in ("q", "codes", "scales", "table", "cu", "lens", "out"):
        assert attn(L, **{name: NUL}) == E_NULL, name
        assert attn(L, **{name: BAD}) == E_ALIGN, name
    assert attn(L, slopes=BAD) == E_ALIGN and attn(L, lse=BAD) == E_ALIGN and attn(L, ws=BAD, splits=2) == E_ALIGN
    assert attn(L, no_params=True) == E_NULL and attn(L, no_shape=True) == E_NULL and attn(L, st=None) == E_NULL
    assert attn(L, st=(512, 60)) == E_ALIGN
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attn(L, scale=s) == E_ARG
    for c in (-1.0, float("nan"), float("inf")):
        assert attn(L, cap=c) == E_ARG
    assert attn(L, window=-1) == E_ARG and attn(L, variant=3) == E_ARG and attn(L, variant=-1) == E_ARG
    assert attn(L, splits=-1) == E_ARG and attn(L, splits=1025) == E_ARG
    assert attn(L, window=5, causal=0) == E_UNSUP
    # a split call needs its workspace, whole
    plan = fc.AttnPlan()
    assert L.chain_attn_plan(shape(), fc.AttnParams(0.125, 0, 1, 0, 0, 3), plan) == OK and plan.workspace > 0
    assert attn(L, splits=3) == E_NULL
    assert attn(L, splits=3, ws=P, wsb=plan.workspace - 1) == E_SHAPE
    assert b"workspace" in L.fc_last_error()


def test_attn_refuses_scales_whose_quotient_leaves_32_bits(L):
    for s in (1e-45, 9e-19, 1.1e18):
        assert attn(L, scale=s) == E_ARG
    for c in (1e-45, 9e-19, 1.1e18):
        assert attn(L, cap=c) == E_ARG


def test_plan_of_tiles():
    def tile(tokens, batch, max_q, max_kv, window=0, hkv=4, d=64):
        p = fc.attn_plan(tokens, batch, 4 * hkv, hkv, d, 64, 512, max_q, max_kv, window=window, variant="tile")
        assert p["splits"] * p["chunk"] >= min(max_kv, window + max_q if window else max_kv)
        assert p["workspace"] == (tokens * 4 * hkv * p["splits"] * (d + 4) * 4 if p["splits"] > 1 else 0)
        return p["splits"]
    assert tile(64, 1, 64, 20000) > 16                        # eight tiles: the keys fill the machine
    assert tile(64, 1, 64, 20000, window=100) == 1            # but a windowed tile sees few of them
    assert tile(4096, 1, 4096, 4096, hkv=32) == 1             # 4096 tiles fill it
    assert tile(1100, 4, 800, 9000) >= tile(3200, 4, 800, 9000)   # a ragged batch has fewer tiles than max_q allows


def test_plan():
    one = fc.attn_plan(1, 1, 8, 2, 64, 16, 40, 1, 513)
    assert one["variant"] == "rows"
    assert fc.attn_plan(4096, 1, 8, 2, 64, 16, 256, 4096, 4096)["variant"] == "tile"
    big = fc.attn_plan(512, 512, 32, 8, 128, 64, 128, 1, 8192)
    assert big["splits"] == 1 and big["workspace"] == 0       # sequences and heads fill the machine
    long = fc.attn_plan(1, 1, 8, 1, 128, 64, 2048, 1, 131072)
    assert long["splits"] > 16 and long["splits"] * long["chunk"] >= 131072
    assert long["workspace"] == 8 * long["splits"] * 132 * 4
    # a window bounds what a split has to cover
    assert fc.attn_plan(1, 1, 8, 1, 128, 64, 2048, 1, 131072, window=512)["splits"] < long["splits"]
    for s in (1, 2, 7, 100):
        p = fc.attn_plan(3, 3, 8, 2, 64, 16, 100, 1, 1600, splits=s)
        assert p["splits"] == s and p["splits"] * p["chunk"] >= 1600
    with pytest.raises(fc.FusedChainError):
        fc.attn_plan(1, 1, 8, 3, 64, 16, 40, 1, 513)


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def test_kv_check():
    table, cu, lens = i32([[0, 1, 2], [3, 4, -1]]), i32([0, 2, 3]), i32([40, 32])
    fc.kv_check(table, cu, lens, pages=5, page=16, writes=True)
    fc.kv_check(i32([[0], [0]]), i32([0, 0, 0]), i32([16, 9]), pages=1, page=16, writes=True)   # a shared prefix
    for change, match in [
        (dict(pages=4), r"table\[1\]\[1\] = 4"), (dict(cu_q=i32([1, 2, 3])), "cu_q"), (dict(cu_q=i32([0, 3, 2])), "cu_q"),
        (dict(kv_lens=i32([1, 32])), "under its"), (dict(kv_lens=i32([40, 33])), r"table\[1\]\[2\] = -1"),
        (dict(kv_lens=i32([49, 32])), "needs 4 pages"), (dict(tokens=2), "exceeds"),
        (dict(kv_lens=i32([-1, 32])), "under its"), (dict(table=i32([[0, 1, 4], [3, 4, -1]])), "named twice")]:
        kw = dict(table=table, cu_q=cu, kv_lens=lens, pages=5, page=16, writes=True)
        kw.update(change)
        with pytest.raises(fc.FusedChainError, match=match):
            fc.kv_check(**kw)
    # a page named twice is no fault where it is only read
    fc.kv_check(i32([[0, 1, 4], [3, 4, -1]]), cu, lens, pages=5, page=16)
    with pytest.raises(TypeError):
        fc.kv_check(table.long(), cu, lens, pages=5, page=16)
    with pytest.raises(ValueError):
        fc.kv_check(table, cu[:2], lens, pages=5, page=16)


def test_rope_turns():
    t, m = fc.rope_turns(64)
    assert t.shape == (32,) and t.dtype == torch.int64 and m == 1.0
    f = [10000.0 ** (-2 * i / 64) for i in range(32)]
    for i in range(32):     # a turn's 2^-64 and the 53 bits of the frequency
        assert abs(int(t[i]) / 2.0 ** 64 - f[i] / (2 * math.pi)) <= f[i] * 2.0 ** -51 + 2.0 ** -64
    lin, _ = fc.rope_turns(64, scaling="linear", factor=4.0)
    assert all(abs(int(a) - 4 * int(b)) <= 4 + abs(int(a)) * 2.0 ** -51 for a, b in zip(t, lin))
    base, _ = fc.rope_turns(64, scaling="base", factor=4.0)
    assert abs(int(base[0]) - int(t[0])) <= 2 ** 12
    assert abs(int(base[31]) * 4 / int(t[31]) - 1) < 1e-9       # the slowest pair is stretched by the factor
    for kind in ("wavelength", "ramp"):
        kw = dict(low=1.0, high=4.0) if kind == "wavelength" else dict(low=1.0, high=32.0)
        s, m = fc.rope_turns(64, scaling=kind, factor=8.0, original=4096, **kw)
        ratio = [int(a) / int(b) for a, b in zip(t, s)]
        assert abs(ratio[0] - 1) < 1e-9 and abs(ratio[-1] - 8) < 1e-6
        assert all(a <= b + 1e-9 for a, b in zip(ratio, ratio[1:]))       # fast pairs stay, slow ones stretch
        assert m == (1.0 if kind == "wavelength" else pytest.approx(0.1 * math.log(8.0) + 1.0))
    for bad in (dict(rot=24), dict(rot=0), dict(rot=64, base=1.0), dict(rot=64, factor=0.5),
                dict(rot=64, scaling="none such"), dict(rot=64, scaling="ramp", factor=2.0)):
        with pytest.raises(ValueError):
            fc.rope_turns(**bad)


def host(dtype=torch.float16, T=3, hq=4, hkv=2, d=64, page=16, pages=5, B=2):
    codes, scales = fc.kv_cache(pages, hkv, page, d, device="cpu")
    return dict(q=torch.zeros((T, hq, d), dtype=dtype), codes=codes, scales=scales,
                table=torch.zeros((B, 2), dtype=torch.int32), cu_q=torch.zeros(B + 1, dtype=torch.int32),
                kv_lens=torch.zeros(B, dtype=torch.int32))


def test_binding_refuses_host_tensors_and_wrong_sizes():
    """Shapes and types first, then that everything is on a device."""
    kw = host()
    with pytest.raises(TypeError, match="device"):
        fc.chain_attn(**kw)
    for change in [dict(codes=kw["codes"][:, :, :, :, :512]), dict(codes=kw["codes"][:, :1]), dict(cu_q=kw["cu_q"][:2]),
                   dict(kv_lens=kw["kv_lens"][:1]), dict(scales=kw["scales"][:4]), dict(table=kw["table"][0]),
                   dict(q=kw["q"][0]), dict(q=kw["q"].transpose(1, 2).contiguous().transpose(1, 2)),
                   dict(slopes=torch.zeros(3)), dict(out=torch.zeros((3, 4, 32), dtype=torch.float16)),
                   dict(lse=torch.zeros((3, 2)))]:
        with pytest.raises(ValueError):
            fc.chain_attn(**{**kw, **change})
    for change in [dict(q=kw["q"].float()), dict(codes=kw["codes"].to(torch.int8)), dict(scales=kw["scales"].half()),
                   dict(table=kw["table"].long()), dict(cu_q=kw["cu_q"].long()), dict(slopes=torch.zeros(4).half()),
                   dict(out=torch.zeros((3, 4, 64), dtype=torch.bfloat16)), dict(lse=torch.zeros((3, 4)).half()),
                   dict(workspace=torch.zeros(4)), dict(q=None)]:
        with pytest.raises(TypeError):
            fc.chain_attn(**{**kw, **change})
    q = kw.pop("q")
    k = torch.zeros((3, 2, 64), dtype=torch.float16)
    ap = dict(k=k, v=k, **kw)
    with pytest.raises(TypeError, match="device"):
        fc.kv_append(**ap)
    for change in [dict(v=k[:2]), dict(q=q[:2]), dict(q_out=q), dict(q=q, q_out=q[:, :2]), dict(k=k[:, :1], v=k[:, :1]),
                   dict(positions=torch.zeros(2, dtype=torch.int32)), dict(turns=torch.zeros((2, 2), dtype=torch.int64))]:
        with pytest.raises(ValueError):
            fc.kv_append(**{**ap, **change})
    for change in [dict(v=k.bfloat16()), dict(q=q.bfloat16()), dict(positions=torch.zeros(3)), dict(turns=torch.zeros(32))]:
        with pytest.raises(TypeError):
            fc.kv_append(**{**ap, **change})
    x, pos, t = q, torch.zeros(3, dtype=torch.int32), fc.rope_turns(64)[0]
    with pytest.raises(TypeError, match="device"):
        fc.rope(x, pos, t)
    for a in [(x[0], pos, t), (x, pos[:2], t), (x, pos, None), (x, pos, t[None])]:
        with pytest.raises(ValueError):
            fc.rope(*a)
    for a in [(x.float(), pos, t), (x, pos.long(), t), (x, pos, t.double())]:
        with pytest.raises(TypeError):
            fc.rope(*a)
    with pytest.raises(ValueError):
        fc.rope(x, pos, t, out=x[:2])
    with pytest.raises(TypeError):
        fc.rope(x, pos, t, out=x.bfloat16())
    with pytest.raises(ValueError):
        fc.kv_cache(4, 2, 24, 64, device="cpu")
