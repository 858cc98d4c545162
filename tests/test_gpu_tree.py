"""Trees of drafted tokens on the GPU: the plan and the accepted path, exactly, and
attention over a tree against 64 bits (decode_ref)."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402
import decode_ref as D  # noqa: E402
from test_gpu_attn import BF16, DTYPES, F16, batch, fc, gen, i32, on_gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def grow(rng, n, reach=6):
    return [-1] + [rng.randint(max(0, i - reach), i - 1) for i in range(1, n)] if n else []


def cumulative(new):
    return i32([sum(new[:b]) for b in range(len(new) + 1)])


# ------------------------------------------------------------------ bookkeeping
SIZES = [[1], [8], [3, 0, 1, 64, 65], [5, 128, 129, 0], [300, 2], [0, 0, 7], [33] * 300]


@pytest.mark.parametrize("new", SIZES, ids=lambda v: "x".join(map(str, v[:5])))
def test_plan(fc, new):
    print("case plan", new[:5], flush=True)
    rng = random.Random(sum(new))
    trees = [grow(rng, n) for n in new]
    for t in trees:                       # what names no earlier node is no parent
        for i in range(1, len(t)):
            if rng.random() < 0.15:
                t[i] = rng.choice([-1, i, i + 1, len(t), 2 ** 31 - 1, -2 ** 31])
    lens = [n + rng.randint(0, 5000) for n in new]
    flat = i32(sum(trees, []))
    spare = torch.full((3,), 5, dtype=torch.int32)       # rows of no sequence
    parents = torch.cat((flat, spare)).cuda()
    bits, pos = fc.tree_plan(parents, cumulative(new).cuda(), i32(lens).cuda(), max_q=max(new))
    words = -(-max(max(new), 1) // 64)
    assert bits.shape == (len(flat) + 3, words)
    seen = [D.ancestors(t) for t in trees]
    want = [r for s in seen for r in D.words_of(s, words)]
    assert bits[:len(flat)].tolist() == want
    place = [L - len(t) + len(s) - 1 for t, L, ss in zip(trees, lens, seen) for s in ss]
    assert pos[:len(flat)].tolist() == place


def test_plan_of_the_longest_chain_and_past_it(fc):
    print("case plan 4096", flush=True)
    n = 4096
    parents = torch.arange(-1, n, dtype=torch.int32).cuda()[:n]
    bits, pos = fc.tree_plan(parents, i32([0, n]).cuda(), i32([n + 11]).cuda())
    j = torch.arange(n)
    got = ((bits.cpu()[:, :, None] >> torch.arange(64)) & 1).bool().view(n, n)
    assert torch.equal(got, j <= j[:, None]) and torch.equal(pos.cpu().long(), 11 + j)
    # a sequence of more nodes than its rows have bits sees none
    bits, pos = fc.tree_plan(parents[:70], i32([0, 66, 70]).cuda(), i32([70, 9]).cuda(), max_q=64)
    assert bits[:66].eq(0).all() and pos[:66].eq(4).all() and bits[66:, 0].tolist() == [1, 2, 4, 8]


@pytest.mark.parametrize("reach", [1, 64, 65, 200, 4000])
def test_plan_across_words(fc, reach):
    """Parents in the same 64 nodes, in those before, and far away."""
    print("case plan reach", reach, flush=True)
    rng = random.Random(reach)
    new = [1500, 64, 65, 700]
    trees = [grow(rng, n, reach) for n in new]
    bits, pos = fc.tree_plan(i32(sum(trees, [])).cuda(), cumulative(new).cuda(), i32(new).cuda(), max_q=1500)
    seen = [D.ancestors(t) for t in trees]
    assert bits.tolist() == [r for s in seen for r in D.words_of(s, 24)]
    assert pos.tolist() == [len(s) - 1 for ss in seen for s in ss]


@pytest.mark.parametrize("new", SIZES, ids=lambda v: "x".join(map(str, v[:5])))
@pytest.mark.parametrize("most", [None, 3])
def test_accept(fc, new, most):
    print("case accept", new[:5], most, flush=True)
    rng = random.Random(sum(new) + 1)
    trees = [grow(rng, n, 3) for n in new]
    drafted = [[rng.randint(0, 2) for _ in t] for t in trees]          # many children alike: the lowest is taken
    targets = [[rng.randint(0, 2) for _ in t] for t in trees]
    for t in trees:
        for i in range(2, len(t)):
            if rng.random() < 0.05:
                t[i] = rng.choice([-1, i, i + 1, 2 ** 31 - 1])
    lens = [n + rng.randint(0, 5000) for n in new]
    args = [i32(sum(v, [])).cuda() for v in (trees, drafted, targets)]
    keep, kept, nxt, after = fc.tree_accept(*args, cumulative(new).cuda(), i32(lens).cuda(), max_q=most or max(new))
    most = most or max(max(new), 1)
    assert keep.shape == (len(new), most)
    for b in range(len(new)):
        path, token = D.accept(trees[b], drafted[b], targets[b])
        if len(path) > most:
            path, token = path[:most], targets[b][path[most - 1]]
        assert keep[b].tolist() == path + [-1] * (most - len(path)), b
        assert (int(kept[b]), int(nxt[b]), int(after[b])) == (len(path), token, lens[b] - new[b] + len(path)), b


def test_accept_lengths_in_place_and_long_paths(fc):
    print("case accept chain", flush=True)
    n = 1000
    par, tok = torch.arange(-1, n - 1, dtype=torch.int32).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    tgt = tok + 1
    tgt[700] = 0
    keep, kept, nxt, after = fc.tree_accept(par, tok, tgt, i32([0, n]).cuda(), i32([n + 5]).cuda())
    assert kept.tolist() == [701] and nxt.tolist() == [0] and after.tolist() == [706]
    assert keep[0].tolist() == list(range(701)) + [-1] * 299


def test_bad_offsets_stay_inside(fc):
    """cu_q that falls or passes the tokens is taken inside them."""
    print("case bad cu_q", flush=True)
    par = torch.arange(-1, 9, dtype=torch.int32).cuda()
    guard = torch.full((64,), 77, dtype=torch.int32).cuda()
    for cu in ([0, 40, 10], [5, 2, 10], [-7, 3, 12], [0, 2 ** 31 - 1, -2 ** 31]):
        bits, pos = fc.tree_plan(par, i32(cu).cuda(), i32([20, 20]).cuda())
        keep, kept, nxt, after = fc.tree_accept(par, par, par, i32(cu).cuda(), i32([20, 20]).cuda())
        assert kept.max() <= 10 and guard.eq(77).all()


# -------------------------------------------------------------------- attention
def tree_batch(seed, dtype, lens, new, hq, hkv, d, page, reach=6):
    b = batch(seed, dtype, lens, new, hq, hkv, d, page)
    rng = random.Random(seed)
    trees = [grow(rng, n, reach) for n in new]
    words = -(-max(max(new), 1) // 64)
    seen = [D.ancestors(t) for t in trees]
    bits = torch.tensor([r for s in seen for r in D.words_of(s, words)], dtype=torch.int64).view(-1, words)
    pos = i32([L - len(t) + len(s) - 1 for t, L, ss in zip(trees, lens, seen) for s in ss])
    return b, bits, pos


def check(fc, b, bits, pos, what, **kw):
    g = on_gpu(b)
    ref = D.attention(**b, bits=bits, positions=pos, **{k: v for k, v in kw.items() if k in ("softcap", "window", "slopes", "scale")})
    if kw.get("slopes") is not None:
        kw["slopes"] = kw["slopes"].cuda()
    out, lse = fc.chain_attn(**g, tree=(bits.cuda(), pos.cuda()), lse=True, **kw)
    R.assert_within(out, ref[0], R.rounded_tol(ref[0], ref[1], b["q"].dtype), what)
    R.assert_within(lse, ref[2], ref[3], what + " lse")
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (192, 32), (256, 128)])
@pytest.mark.parametrize("hq,hkv,lens,new", [
    (4, 2, [40, 17, 300], [3, 1, 8]),                  # few rows
    (8, 1, [130, 64, 513], [26, 64, 5]),               # a tile's worth
    (6, 2, [200, 131, 77], [70, 129, 0]),              # more nodes than a word has bits
])
@pytest.mark.parametrize("variant", ["rows", "tile"])
def test_sizes(fc, dtype, d, page, hq, hkv, lens, new, variant):
    print("case tree", dtype, d, page, hq, hkv, lens, new, variant, flush=True)
    b, bits, pos = tree_batch(d + hq, dtype, lens, new, hq, hkv, d, page)
    check(fc, b, bits, pos, "tree", max_q=max(new), max_kv=max(lens), variant=variant)


MASKS = [dict(softcap=20.0), dict(window=5), dict(window=40), dict(window=1), dict(slopes=True), dict(slopes=True, window=3),
         dict(softcap=5.0, slopes=True, window=64), dict(softcap=500.0), dict(softcap=500.0, slopes=True), dict(scale=0.3)]


@pytest.mark.parametrize("kw", MASKS, ids=str)
@pytest.mark.parametrize("variant,dtype,d", [("rows", F16, 64), ("tile", BF16, 128), ("tile", F16, 256), ("rows", BF16, 192)])
def test_masks_and_scores(fc, kw, variant, dtype, d):
    print("case tree masks", kw, variant, dtype, d, flush=True)
    hq, new, lens = 4, [9, 33, 1, 66], [60, 33, 90, 200]      # one whose tree is all it has
    b, bits, pos = tree_batch(3, dtype, lens, new, hq, 2, d, 16, reach=2)
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = torch.tensor([0.5, 0.0, 0.03, 0.25])
    check(fc, b, bits, pos, "tree masks", max_q=max(new), variant=variant, **kw)


@pytest.mark.parametrize("variant", ["rows", "tile"])
@pytest.mark.parametrize("splits", [1, 3, 9])
def test_splits(fc, variant, splits):
    print("case tree splits", variant, splits, flush=True)
    lens, new = [1500, 20, 700], [13, 20, 40]
    b, bits, pos = tree_batch(8, BF16, lens, new, 8, 2, 64, 32)
    check(fc, b, bits, pos, "tree splits", max_q=40, variant=variant, splits=splits, window=900)


@pytest.mark.parametrize("variant", ["rows", "tile", "auto"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_any_bits(fc, variant, dtype):
    """Bits need not be a tree's: rows that see nothing of their own (0 and -inf where
    nothing came before), every node, bits past the last node."""
    print("case any bits", variant, dtype, flush=True)
    lens, new = [12, 31, 70, 5], [12, 7, 70, 5]
    b, _, _ = tree_batch(2, dtype, lens, new, 4, 2, 128, 16)
    g = gen(4)
    T = sum(new)
    bits = torch.randint(-2 ** 63, 2 ** 63 - 1, (T, 2), generator=g)
    bits[0:3] = 0
    bits[3] = -1
    bits[12:15] = 0
    bits[20:24] = 0
    pos = torch.randint(-5, 120, (T,), generator=g, dtype=torch.int32)      # taken into the tree's reach
    out = check(fc, b, bits, pos, "any bits", max_q=70, variant=variant, window=60)
    assert out[0:3].eq(0).all()


@pytest.mark.parametrize("variant", ["rows", "tile"])
@pytest.mark.parametrize("kw", [dict(splits=1), dict(softcap=30.0, splits=1), dict(window=100), {}, dict(splits=4)], ids=str)
def test_a_chain_is_causal(fc, variant, kw):
    """A tree of one branch gives the bits that the causal call gives where both take a
    sequence's keys in the same parts. With a window both are as 64 bits have it: a causal block begins at
    its own first query's window, a tree's at its sequence's. So are calls whose splits the rules of each
    choose, and the tile form's parts, which a tree call cuts by the work of all sequences, a causal one
    by the longest."""
    print("case chain", variant, kw, flush=True)
    lens, new = [300, 64, 1000, 9], [40, 64, 5, 9]
    b = batch(6, BF16, lens, new, 8, 2, 128, 32)
    g = on_gpu(b)
    par = i32([i - 1 for n in new for i in range(n)]).cuda()
    tree = fc.tree_plan(par, g["cu_q"], g["kv_lens"], max_q=64)
    a = fc.chain_attn(**g, max_q=64, variant=variant, **kw)
    t = fc.chain_attn(**g, max_q=64, variant=variant, tree=tree, **kw)
    if kw.get("splits") == 1 or (variant == "rows" and "splits" in kw):
        assert torch.equal(t, a)
        return
    out, tol, _, _ = D.attention(**b, bits=tree[0].cpu(), positions=tree[1].cpu(), window=kw.get("window", 0))
    R.assert_within(a, out, R.rounded_tol(out, tol, BF16), "causal")
    R.assert_within(t, out, R.rounded_tol(out, tol, BF16), "chain")


@pytest.mark.parametrize("variant", ["rows", "tile"])
def test_nan_keys_reach_those_who_see_them(fc, variant):
    print("case tree nan", variant, flush=True)
    lens, new = [100, 50], [20, 30]
    b, bits, pos = tree_batch(12, F16, lens, new, 4, 2, 64, 16)
    K = R.unpack_k(b["codes"][:, :, 0], 64).clone()
    slot = 80 + 3                                                  # node 3 of the first tree
    K[int(b["table"][0, slot // 16]), 1, slot % 16, 7] = 0x7f
    b["codes"][:, :, 0] = R.pack_k(K.reshape(K.shape[0], 2, 1, 16, 64))
    out = check(fc, b, bits, pos, "tree nan", max_q=30, variant=variant)
    sees = torch.tensor([3 in s for s in D.sets_of(bits[:20])])
    bad = torch.isnan(out.cpu()).all(-1)
    assert torch.equal(bad[:20, 2:], sees[:, None].expand(20, 2)) and not bad[:, :2].any() and not bad[20:].any()
    assert sees.any() and not sees.all()


@pytest.mark.parametrize("variant", ["rows", "tile"])
@pytest.mark.parametrize("splits", [1, 3])
def test_bad_metadata_gives_nan(fc, variant, splits):
    """More nodes than the rows have bits, lengths past the table, ids outside the pool."""
    print("case tree bad", variant, splits, flush=True)
    lens, new = [200, 300, 90, 80], [70, 5, 6, 7]
    b, bits, pos = tree_batch(1, BF16, lens, new, 4, 2, 64, 16)
    g = on_gpu(b)
    g["kv_lens"][1] = 16 * b["table"].shape[1] + 1
    g["table"][2, 0] = 10 ** 6
    out, lse = fc.chain_attn(**g, tree=(bits[:, :1].contiguous().cuda(), pos.cuda()), lse=True, max_q=70, max_kv=300,
                             variant=variant, splits=splits)
    assert torch.isnan(out[:81]).all() and torch.isnan(lse[:81]).all() and torch.isfinite(out[81:].float()).all()


def test_strides_streams_and_rows_of_no_sequence(fc):
    print("case tree strides", flush=True)
    lens, new = [500, 130], [9, 14]
    b, bits, pos = tree_batch(5, F16, lens, new, 8, 2, 128, 64)
    ref = D.attention(**b, bits=bits, positions=pos)
    g = on_gpu(b)
    T = sum(new)
    wide = torch.zeros((T + 2, 11, 128), dtype=F16).cuda()
    wide[:T, 1:9] = g["q"]
    g["q"] = wide[:, 1:9]
    out = torch.full((T + 2, 8, 128), 3.0, dtype=F16).cuda()
    tree = (torch.cat((bits, bits[:2])).cuda(), torch.cat((pos, pos[:2])).cuda())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        fc.chain_attn(**g, tree=tree, out=out, max_q=14, variant="tile", splits=1)
    st.synchronize()
    R.assert_within(out[:T], ref[0], R.rounded_tol(ref[0], ref[1], F16), "strided")
    assert out[T:].eq(3.0).all()


def test_split_results_with_poisoned_lds(fc):
    print("case tree poison", flush=True)
    lens, new = [700, 33, 260], [20, 33, 3]
    b, bits, pos = tree_batch(15, BF16, lens, new, 8, 2, 128, 32)
    g = on_gpu(b)
    tree = (bits.cuda(), pos.cuda())
    for variant in ("rows", "tile"):
        for splits in (1, 4):
            a = fc.chain_attn(**g, tree=tree, max_q=33, variant=variant, splits=splits)
            with fc.poison_build():
                p = fc.chain_attn(**g, tree=tree, max_q=33, variant=variant, splits=splits)
            assert torch.equal(a, p), (variant, splits)


@pytest.mark.parametrize("seed", range(24))
def test_drawn_mixtures(fc, seed):
    rng = random.Random(1000 + seed)
    d, page, hkv, G = rng.choice([64, 128, 192, 256]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 3]), rng.choice([1, 2, 4, 5])
    new = [rng.choice([0, 1, 2, 7, 16, 31, 65]) for _ in range(rng.randint(1, 5))]
    if not any(new):
        new[0] = 3
    lens = [n + rng.choice([0, 1, 15, 16, 100, 400]) for n in new]
    kw = dict(max_q=rng.choice([max(new), max(new) + 9]), variant=rng.choice(["rows", "tile", "auto"]), splits=rng.choice([0, 0, 1, 2, 5]))
    if rng.random() < 0.4:
        kw["window"] = rng.choice([1, 5, 33, 200])
    if rng.random() < 0.3:
        kw["softcap"] = rng.choice([5.0, 30.0, 1000.0])
    if rng.random() < 0.3:
        kw["slopes"] = torch.tensor([rng.choice([0.0, 0.01, 0.5]) for _ in range(hkv * G)])
    print("case drawn tree", seed, d, page, hkv, G, new, lens, kw, flush=True)
    b, bits, pos = tree_batch(seed, rng.choice(DTYPES), lens, new, hkv * G, hkv, d, page, rng.choice([1, 6, 70]))
    check(fc, b, bits, pos, "drawn %d" % seed, **kw)
