"""Host-only: arguments at the ends of their ranges, of the C entry points and of
the binding."""
import math

import pytest

import gemm_conv_chain_amd as fc

torch = pytest.importorskip("torch")
import test_attn_abi as A  # noqa: E402

pytestmark = pytest.mark.cpu


@pytest.fixture(scope="module")
def L():
    return fc.lib()


@pytest.mark.parametrize("tokens,hq,hkv", [(2 ** 62, 4, 2), (2 ** 61 + 1, 8, 2), (2 ** 63 - 1, 2, 2), (2 ** 30, 1, 1)])
def test_tokens_whose_rows_pass_64_bits(L, tokens, hq, hkv):
    kw = dict(tokens=tokens, hq=hq, hkv=hkv)
    assert A.attn(L, **kw) == A.E_UNSUP and A.append(L, **kw) == A.E_UNSUP
    plan = fc.AttnPlan()
    assert L.chain_attn_plan(A.shape(**kw), fc.AttnParams(0.125, 0, 1, 0, 0, 0), plan) == A.E_UNSUP


def test_windows_past_32_bits():
    """A window that does not fit the C type is no window, not a smaller one."""
    kw = dict(tokens=1, batch=1, hq=8, hkv=1, d=128, page=64, table_stride=2048, max_q=1, max_kv=131072)
    none = fc.attn_plan(**kw)
    assert fc.attn_plan(window=512, **kw) != none
    for w in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 512, 2 ** 63 - 1, 10 ** 30):
        assert fc.attn_plan(window=w, **kw) == none
    for w in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 512, -2 ** 70):
        with pytest.raises(fc.FusedChainError):
            fc.attn_plan(window=w, **kw)


@pytest.mark.parametrize("mscale", [math.nan, math.inf, -math.inf])
def test_factors_that_are_no_numbers(L, mscale):
    r = fc.RopeTable(0x10000, 64, 0, mscale)
    assert L.rope_apply(A.P, A.P, A.strides(512, 64, 512, 64), A.P, r, 0, 0, 4, 8, 64, None) == A.E_ARG
    st = A.strides(*[8] * 6)
    assert L.kv_append(A.P, A.P, None, None, st, A.P, A.P, A.P, A.P, A.P, None, r, A.shape(), None) == A.E_ARG
    assert b"mscale" in L.fc_last_error()


def test_ramp_without_bounds_takes_its_own():
    """The blend by index runs from 32 turns to 1 unless told otherwise, the one by
    wavelength from 4 to 1."""
    kw = dict(rot=64, factor=8.0, original=4096)
    for kind, high in (("ramp", 32.0), ("wavelength", 4.0)):
        t, m = fc.rope_turns(scaling=kind, **kw)
        want, mw = fc.rope_turns(scaling=kind, low=1.0, high=high, **kw)
        assert torch.equal(t, want) and m == mw
        other, _ = fc.rope_turns(scaling=kind, low=1.0, high=36.0 - high, **kw)
        assert not torch.equal(t, other)
    # from the formula: 32 turns within 4096 positions are reached at pair 32 ln(4096 / (64 pi)) / ln 10000
    # = 10.47, one at 22.51: pairs to 10 stay, pairs from 23 on are divided, pair 17 is 7 / 13 of the way
    t, plain = fc.rope_turns(scaling="ramp", **kw)[0], fc.rope_turns(64)[0]
    part = [int(a) / int(b) for a, b in zip(t, plain)]
    assert all(abs(p - 1) < 1e-9 for p in part[:11]) and all(abs(p - 0.125) < 1e-9 for p in part[23:])
    assert abs(part[17] - (1 - 7 / 13 * 0.875)) < 1e-9


def test_table_slices_are_taken():
    """A table that is a slice of a wider one (host tensors: only what is refused
    after it is)."""
    kw = A.host()
    q = kw.pop("q")
    wide = torch.zeros((2, 9), dtype=torch.int32)
    for table in (wide[:, :2], wide[:, 3:5], torch.zeros((2, 2), dtype=torch.int32).t()):
        with pytest.raises(TypeError, match="device"):
            fc.chain_attn(q, **{**kw, "table": table})
        with pytest.raises(TypeError, match="device"):
            fc.kv_append(q[:, :2], q[:, :2], **{**kw, "table": table})
    with pytest.raises(TypeError, match="table"):
        fc.chain_attn(q, **{**kw, "table": wide.long()[:, :2]})
    cu, lens = A.i32([0, 2, 3]), A.i32([40, 32])
    t = A.i32([[9, 0, 1, 2, 9], [9, 3, 4, -1, 9]])
    fc.kv_check(t[:, 1:4], cu, lens, pages=5, page=16, writes=True)
    with pytest.raises(fc.FusedChainError, match=r"table\[1\]\[1\] = 4"):
        fc.kv_check(t[:, 1:4], cu, lens, pages=4, page=16)
