"""Host-only: refusals of the operators around a speculative step, in the C entry
points (validation runs before any HIP call) and in the binding."""
import ctypes

import pytest

import gemm_conv_chain_amd as fc

torch = pytest.importorskip("torch")
import test_attn_abi as A  # noqa: E402

pytestmark = pytest.mark.cpu
OK, E_NULL, E_SHAPE, E_ALIGN, E_UNSUP, E_HIP, E_ARG = range(7)
P, BAD, NUL = A.P, ctypes.c_void_p(0x10001), None


@pytest.fixture(scope="module")
def L():
    return fc.lib()


def tree_attn(L, bits=0x10000, positions=0x10000, words=1, tree=True, causal=1, q=P, st=(512, 64), **kw):
    t = fc.Tree(bits, positions, words) if tree else None
    return L.chain_attn_tree(q, A.strides(*st), P, P, P, P, P, t, NUL, fc.AttnParams(0.125, 0.0, causal, 0, 0, 1), P, NUL,
                             A.shape(**kw), NUL, 0, None)


def test_tree_attention_refusals(L):
    assert tree_attn(L, tokens=0, q=NUL) == OK and tree_attn(L, batch=0) == OK
    assert tree_attn(L, tree=False) == E_NULL
    assert tree_attn(L, bits=None) == E_NULL and tree_attn(L, positions=None) == E_NULL and tree_attn(L, q=NUL) == E_NULL
    assert tree_attn(L, bits=0x10004) == E_ALIGN and tree_attn(L, positions=0x10002) == E_ALIGN
    assert tree_attn(L, words=0) == E_UNSUP and tree_attn(L, words=65) == E_UNSUP and tree_attn(L, words=-1) == E_UNSUP
    assert tree_attn(L, causal=0) == E_ARG and b"causal" in L.fc_last_error()
    for kw, status in A.SHAPE_REFUSALS:
        assert tree_attn(L, **kw) == status


def plan(L, par=P, cu=P, lens=P, batch=2, tokens=9, words=1, bits=P, pos=P):
    return L.tree_plan(par, cu, lens, batch, tokens, words, bits, pos, None)


def test_plan_refusals(L):
    assert plan(L, batch=0, par=NUL) == OK and plan(L, tokens=0, bits=NUL) == OK
    for name in ("par", "cu", "lens", "bits", "pos"):
        assert plan(L, **{name: NUL}) == E_NULL and plan(L, **{name: BAD}) == E_ALIGN, name
    assert plan(L, bits=ctypes.c_void_p(0x10004)) == E_ALIGN
    assert plan(L, batch=-1) == E_SHAPE and plan(L, tokens=-1) == E_SHAPE
    assert plan(L, words=0) == E_UNSUP and plan(L, words=65) == E_UNSUP
    assert plan(L, batch=2 ** 20 + 1) == E_UNSUP and plan(L, tokens=2 ** 30) == E_UNSUP


def acc(L, par=P, dr=P, tg=P, cu=P, lens=P, batch=2, tokens=9, most=4, keep=P, kept=P, nxt=P, after=P):
    return L.tree_accept(par, dr, tg, cu, lens, batch, tokens, most, keep, kept, nxt, after, None)


def test_accept_refusals(L):
    assert acc(L, batch=0, cu=NUL, keep=NUL) == OK
    for name in ("par", "dr", "tg", "cu", "lens", "keep", "kept", "nxt", "after"):
        assert acc(L, **{name: NUL}) == E_NULL and acc(L, **{name: BAD}) == E_ALIGN, name
    assert acc(L, batch=-1) == E_SHAPE and acc(L, tokens=-1) == E_SHAPE
    assert acc(L, most=0) == E_UNSUP and acc(L, most=4097) == E_UNSUP and acc(L, batch=2 ** 20 + 1) == E_UNSUP


def keep(L, codes=P, scales=P, layers=2, table=P, cu=P, lens=P, keep=P, kept=P, most=4, no_shape=False, **kw):
    return L.kv_keep(codes, scales, layers, table, cu, lens, keep, kept, most, None if no_shape else A.shape(**kw), None)


def test_keep_refusals(L):
    assert keep(L, tokens=0, codes=NUL) == OK and keep(L, batch=0, codes=NUL) == OK
    assert keep(L, layers=0, codes=NUL) == OK and keep(L, most=0, keep=NUL) == OK
    for name in ("codes", "scales", "table", "cu", "lens", "keep", "kept"):
        assert keep(L, **{name: NUL}) == E_NULL and keep(L, **{name: BAD}) == E_ALIGN, name
    assert keep(L, no_shape=True) == E_NULL and keep(L, layers=-1) == E_SHAPE and keep(L, most=-1) == E_SHAPE
    assert keep(L, layers=65536) == E_UNSUP and keep(L, most=4097) == E_UNSUP
    for kw, status in A.SHAPE_REFUSALS:
        assert keep(L, **kw) == status


def copy(L, pairs, codes=P, scales=P, layers=1, pages=8, hkv=2, page=16, d=64, n=None):
    flat = [v for p in pairs for v in p]
    arr = (ctypes.c_int32 * max(len(flat), 1))(*flat)
    return L.kv_copy(codes, scales, layers, pages, hkv, page, d, ctypes.addressof(arr), len(pairs) if n is None else n, None)


def test_copy_refusals(L):
    assert copy(L, []) == OK and copy(L, [], codes=NUL) == OK and copy(L, [(0, 1)], layers=0, codes=NUL) == OK
    assert L.kv_copy(P, P, 1, 8, 2, 16, 64, None, 0, None) == OK
    assert L.kv_copy(P, P, 1, 8, 2, 16, 64, None, 1, None) == E_NULL
    assert copy(L, [(0, 1)], codes=NUL) == E_NULL and copy(L, [(0, 1)], scales=NUL) == E_NULL
    assert copy(L, [(0, 1)], codes=BAD) == E_ALIGN and copy(L, [(0, 1)], scales=BAD) == E_ALIGN
    assert copy(L, [(0, 8)]) == E_SHAPE and copy(L, [(8, 0)]) == E_SHAPE and copy(L, [(-1, 0)]) == E_SHAPE
    assert copy(L, [(0, -1)]) == E_SHAPE
    assert copy(L, [(0, 1), (2, 1)]) == E_SHAPE and b"destination of two" in L.fc_last_error()
    assert copy(L, [(0, 1), (1, 2)]) == E_SHAPE and copy(L, [(1, 2), (0, 1)]) == E_SHAPE
    assert copy(L, [(3, 3)]) == E_SHAPE and b"source and a destination" in L.fc_last_error()
    assert copy(L, [(0, 1)], n=-1) == E_SHAPE and copy(L, [(0, 1)] * 9) == E_SHAPE
    assert copy(L, [(0, 1)], hkv=0) == E_SHAPE and copy(L, [(0, 1)], layers=-1) == E_SHAPE
    assert copy(L, [(0, 1)], pages=-1) == E_SHAPE
    assert copy(L, [(0, 1)], d=80) == E_UNSUP and copy(L, [(0, 1)], page=48) == E_UNSUP and copy(L, [(0, 1)], page=8) == E_UNSUP
    assert copy(L, [(0, 1)], layers=65536) == E_UNSUP and copy(L, [(0, 1)], hkv=65536) == E_UNSUP


def sample(L, logits=P, dtype=0, rows=3, vocab=100, stride=100, u=P, out=P, ws=NUL, wsb=0, t=1.0, k=0, p=1.0, m=0.0,
           arrays=(None,) * 4, sampling=True):
    g = fc.Sampling(*arrays, t, k, p, m) if sampling else None
    return L.sample_tokens(logits, dtype, rows, vocab, stride, u, g, out, ws, wsb, None)


def test_sample_refusals(L):
    nan, inf = float("nan"), float("inf")
    assert sample(L, rows=0, logits=NUL, u=NUL, out=NUL) == OK
    assert sample(L, logits=NUL) == E_NULL and sample(L, u=NUL) == E_NULL and sample(L, out=NUL) == E_NULL
    assert sample(L, sampling=False) == E_NULL
    assert sample(L, logits=BAD) == E_ALIGN and sample(L, logits=A.BAD, dtype=2) == E_ALIGN
    assert sample(L, u=BAD) == E_ALIGN and sample(L, out=BAD) == E_ALIGN
    for i in range(4):
        assert sample(L, arrays=tuple(0x10001 if i == j else None for j in range(4))) == E_ALIGN
    assert sample(L, dtype=3) == E_ARG and sample(L, dtype=-1) == E_ARG
    assert sample(L, rows=-1) == E_SHAPE and sample(L, vocab=0) == E_SHAPE and sample(L, stride=-1) == E_SHAPE
    assert sample(L, vocab=2 ** 20 + 1) == E_UNSUP and sample(L, rows=2 ** 31) == E_UNSUP
    for t in (-1.0, nan, inf):
        assert sample(L, t=t) == E_ARG
    assert sample(L, k=-1) == E_ARG
    for v in (-0.1, 1.1, nan):
        assert sample(L, p=v) == E_ARG and sample(L, m=v) == E_ARG
    # the tokens may not be written over what is still read
    assert sample(L, u=0x20000, out=0x20008) == E_ARG and sample(L, u=0x20008, out=0x20000) == E_ARG
    for i in range(4):
        assert sample(L, u=0x30000, out=0x20000, arrays=tuple(0x20000 if i == j else None for j in range(4))) == E_ARG
    # a row's own settings stand in for the value for all
    assert sample(L, rows=0, t=nan, arrays=(0x10000, None, None, None)) == OK
    n = ctypes.c_int64(-1)
    assert L.sample_workspace(0, 3, 100, n) == OK and n.value >= 0
    assert L.sample_workspace(0, 3, 100, None) == E_NULL and L.sample_workspace(0, 3, 0, n) == E_SHAPE


# ---------------------------------------------------------------------- binding
def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_binding_refusals_of_trees():
    par, cu, lens = i32(-1, 0, 0), i32(0, 2, 3), i32(10, 9)
    with pytest.raises(TypeError, match="int32"):
        fc.tree_plan(par.long(), cu, lens)
    with pytest.raises(ValueError, match="cu_q"):
        fc.tree_plan(par, cu[:2], lens)
    with pytest.raises(ValueError, match="4096"):
        fc.tree_plan(par, cu, lens, max_q=5000)
    with pytest.raises(TypeError, match="device"):
        fc.tree_plan(par, cu, lens)
    with pytest.raises(ValueError, match="drafted"):
        fc.tree_accept(par, par[:2], par, cu, lens)
    with pytest.raises(TypeError, match="targets"):
        fc.tree_accept(par, par, par.float(), cu, lens)
    with pytest.raises(TypeError, match="device"):
        fc.tree_accept(par, par, par, cu, lens)


def test_binding_refusals_of_tree_attention():
    kw = A.host()
    q = kw.pop("q")
    T = q.shape[0]
    bits, pos = torch.zeros((T, 1), dtype=torch.int64), torch.zeros(T, dtype=torch.int32)
    with pytest.raises(TypeError, match="pair"):
        fc.chain_attn(q, **kw, tree=bits)
    with pytest.raises(ValueError, match="bits"):
        fc.chain_attn(q, **kw, tree=(bits[:1], pos))
    with pytest.raises(TypeError, match="bits"):
        fc.chain_attn(q, **kw, tree=(bits.int(), pos))
    with pytest.raises(TypeError, match="positions"):
        fc.chain_attn(q, **kw, tree=(bits, pos.long()))
    with pytest.raises(TypeError, match="device"):
        fc.chain_attn(q, **kw, tree=(bits, pos))


def test_binding_refusals_of_the_pool():
    codes, scales = torch.zeros((2, 4, 2, 2, 1, 1024), dtype=torch.uint8), torch.ones((2, 4, 2, 2))
    table, cu, lens = torch.zeros((1, 2), dtype=torch.int32), i32(0, 3), i32(20)
    good = dict(codes=codes, scales=scales, table=table, cu_q=cu, kv_lens=lens, keep=torch.zeros((1, 3), dtype=torch.int32), kept=i32(1))
    for name, v, what in (("codes", codes[0, 0], ValueError), ("codes", codes.int(), TypeError), ("scales", scales[0], ValueError),
                          ("scales", scales.double(), TypeError), ("table", table.long(), TypeError), ("cu_q", i32(0), ValueError),
                          ("kept", i32(1, 1), ValueError), ("keep", i32(0, 1), ValueError), ("kv_lens", lens.long(), TypeError),
                          ("table", None, Exception)):
        with pytest.raises(what):
            fc.kv_keep(**{**good, name: v})
    with pytest.raises(TypeError, match="device"):
        fc.kv_keep(**good)
    with pytest.raises(ValueError, match="two pages"):
        fc.kv_copy(codes, scales, [(1, 2, 3)])
    with pytest.raises(ValueError, match="pairs"):
        fc.kv_copy(codes, scales, torch.zeros((2, 3), dtype=torch.int32))
    with pytest.raises(TypeError, match="pairs"):
        fc.kv_copy(codes, scales, torch.zeros((2, 2)))
    with pytest.raises(TypeError, match="device"):
        fc.kv_copy(codes, scales, [(0, 1)])


def test_binding_refusals_of_sampling():
    x, u = torch.zeros((2, 10)), torch.zeros(2)
    with pytest.raises(TypeError, match="logits"):
        fc.sample_tokens(x.double(), u)
    with pytest.raises(TypeError, match="logits"):
        fc.sample_tokens([1.0], u)
    with pytest.raises(ValueError, match="dims"):
        fc.sample_tokens(x[0], u)
    with pytest.raises(ValueError, match="adjacent"):
        fc.sample_tokens(x.t().contiguous().t(), u)
    with pytest.raises(ValueError, match="u must"):
        fc.sample_tokens(x, torch.zeros(3))
    with pytest.raises(TypeError, match="top_k"):
        fc.sample_tokens(x, u, top_k=torch.zeros(2))
    with pytest.raises(ValueError, match="temperature"):
        fc.sample_tokens(x, u, temperature=torch.zeros(3))
    with pytest.raises(TypeError, match="out"):
        fc.sample_tokens(x, u, out=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError, match="device"):
        fc.sample_tokens(x, u)


def test_plans_of_trees():
    """Few rows take the rows form and whole keys, a batch of wide trees the tile form; what is asked for is kept."""
    few = fc.attn_plan(8, 1, 8, 2, 64, 16, 40, 8, 513, tree=True)
    assert few["variant"] == "rows" and few["splits"] == 1 and few["workspace"] == 0
    long = fc.attn_plan(8, 1, 32, 8, 128, 64, 512, 8, 32768, tree=True)
    assert long["variant"] == "rows" and long["splits"] > 1 and long["workspace"] > 0
    wide = fc.attn_plan(64 * 32, 64, 32, 4, 128, 64, 64, 32, 4000, tree=True)
    assert wide["variant"] == "tile"
    for variant in ("rows", "tile"):
        one = fc.attn_plan(64, 4, 8, 2, 128, 64, 64, 16, 4000, variant=variant, splits=1, tree=True)
        many = fc.attn_plan(64, 4, 8, 2, 128, 64, 64, 16, 4000, variant=variant, splits=7, tree=True)
        assert one["variant"] == many["variant"] == variant
        assert one["workspace"] == 0 and many["workspace"] > 0 and many["splits"] == 7
    # blocks stay within a grid, whatever is asked for
    huge = fc.attn_plan(4096, 4096, 8, 2, 64, 16, 64, 1, 1000, variant="tile", splits=1024, tree=True)
    assert huge["splits"] <= 65535
