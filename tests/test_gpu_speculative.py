"""The operators around a speculative step run together, as they are used: the
example's step stage by stage against 64 bits, whole runs against runs of single
tokens, captured and replayed steps, forks over shared pages."""
import os
import random
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402
import decode_ref as D  # noqa: E402
from test_gpu_attn import BF16, DTYPES, F16, batch, fc, gen, i32, on_gpu  # noqa: E402,F401
from test_gpu_tree import check as check_tree, cumulative, grow, tree_batch  # noqa: E402

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex(fc):
    import speculative_decode
    return speculative_decode


def start(ex, lens, seed, steps):
    """(model, batch of each prompt twice, pages): as the example's main does it."""
    g = gen(seed)
    n = len(lens)
    p = ex.make_model(seed)
    room = 2 * sum(-(-(l + ex.NODES * (steps + 1)) // ex.dl.PAGE) for l in lens)
    cache = ex.fc.kv_cache(room, ex.dl.HKV, ex.dl.PAGE, ex.dl.D)
    pages = ex.fc.KvPages(room, ex.dl.PAGE)
    texts = [torch.randint(0, ex.VOCAB, (l,), generator=g) for l in lens]
    first = ex.prompts(p, cache, pages, texts, 0.3, torch.rand(n, generator=g).cuda())
    for i in range(n):
        pages.fork(i, n + i)
    for i in range(2 * n):
        ex.fc.kv_copy(*cache, pages.grow(i, pages.length(i) + ex.NODES * (steps + 1)))
    return p, ex.Batch(cache, pages.table(range(2 * n)).cuda(), lens + lens, first.repeat(2)), pages, g


def test_step_by_stages(ex):
    """Each stage on its own inputs: the tree, attention, the targets, the path, the cache."""
    from test_gpu_decoder_layer import near, product
    p, b, _, g = start(ex, [70, 1, 33], 3, 4)
    T = b.parents.numel()
    for it in range(3):
        print("case speculative stage", it, flush=True)
        b.u.copy_(torch.rand(b.u.shape, generator=g))
        held, last = b.held.tolist(), b.last.tolist()
        codes, scales = b.cache[0].cpu(), b.cache[1].cpu()
        w = ex.step(p, b, 0.3, 200)
        table, cu, kv = b.table.cpu(), b.cu.cpu(), w["kv"].cpu()
        assert kv.tolist() == [h + ex.NODES for h in held] and b.drafted[:, 0].tolist() == last
        bits, pos = (t.cpu() for t in w["tree"])
        sets = D.ancestors(ex.PARENTS)
        assert D.sets_of(bits) == sets * len(held)
        assert pos.tolist() == [h + len(s) - 1 for h in held for s in sets]
        # the cache as the layer left it, then as kv_keep did
        rows = w["qkv"].cpu().view(T, ex.dl.HQ + 2 * ex.dl.HKV, ex.dl.D)
        k, v = rows[:, ex.dl.HQ:ex.dl.HQ + ex.dl.HKV], rows[:, ex.dl.HQ + ex.dl.HKV:]
        turns = p["turns"].cpu()
        q, inner = R.rope(rows[:, :ex.dl.HQ], pos.tolist(), turns)
        near(w["q"], q, inner, "q")
        own = (codes.cuda(), scales.cuda())
        ex.fc.kv_append(k.cuda(), v.cuda(), *own, b.table, b.cu, w["kv"], turns=p["turns"], max_q=ex.NODES,
                        positions=w["tree"][1])
        R.assert_appended(*own, R.append(k, v, codes, scales, table, cu, kv, turns, positions=pos), "cache")
        a, tol, _, _ = D.attention(w["q"].cpu(), own[0].cpu(), own[1].cpu(), table, cu, kv, bits, pos)
        near(w["attn"], a, tol, "attn")
        near(w["logits"], *product(w["y"], p["head"]), "logits")
        # the path, from the step's own targets
        keep = w["keep"].tolist()
        drafted, targets = b.drafted.tolist(), w["targets"].view(-1, ex.NODES).tolist()
        for s in range(len(held)):
            path, nxt = D.accept(ex.PARENTS, drafted[s], targets[s])
            assert keep[s] == path + [-1] * (ex.NODES - len(path))
            assert (b.kept[s], b.last[s], b.held[s]) == (len(path), nxt, held[s] + len(path))
            assert b.path[s].tolist() == [drafted[s][j] for j in path] + [0] * (ex.NODES - len(path))
        want = D.keep_tokens(own[0].cpu(), own[1].cpu(), table, cu, kv, w["keep"].cpu(), b.kept.cpu())
        assert D.same_codes(b.cache[0], want[0]) and torch.equal(b.cache[1].cpu(), want[1])
        # the targets: each where its random number lies, unless it lies on a border
        x, u = w["logits"].cpu().double().numpy(), b.u[1].cpu().double().numpy()
        for i in range(T):
            token, off = D.draw(D.weights_that_stay(x[i], np.float32(0.3), 0, 1.0, 0.0), u[i])
            assert w["targets"][i] == token or off < 1e-6, i


def test_a_captured_step_replays(ex):
    """Two captured steps of two batches, each replayed with other work between, against the
    same steps run eagerly from the same start."""
    def run(graphs):
        sides = [start(ex, lens, 7, 8) for lens in ([33, 100], [257])]
        out = []
        calls = []
        for p, b, _, g in sides:
            def one(p=p, b=b):
                ex.step(p, b, 0.3, 400)
            calls.append(one)
        if graphs:
            state = [[t.clone() for t in (b.held, b.last, *b.cache)] for _, b, _, _ in sides]
            for i, (p, b, _, _) in enumerate(sides):
                calls[i]()
                torch.cuda.synchronize()
                gr = torch.cuda.CUDAGraph()
                with torch.cuda.graph(gr):
                    calls[i]()
                calls[i] = gr.replay
                for t, v in zip((b.held, b.last, *b.cache), state[i]):
                    t.copy_(v)
        for it in range(4):
            for (p, b, _, g), call in zip(sides, calls):
                b.u.copy_(torch.rand(b.u.shape, generator=g))
                call()
                junk = torch.randn(1 << 18, device="cuda").sum()
                torch.cuda.synchronize()
                out.append([t.cpu() for t in (b.held, b.last, b.path, b.kept, *b.cache)])
                assert float(junk) == float(junk)
        return out
    print("case captured steps", flush=True)
    for a, b in zip(run(False), run(True)):
        for i, (x, y) in enumerate(zip(a, b)):
            assert torch.equal(x, y), i


def test_forks_do_not_touch_each_other(ex):
    """What one of two sequences that share a prompt's pages appends leaves the other's rows."""
    print("case forks", flush=True)
    p, b, pages, g = start(ex, [45, 64], 9, 3)
    shared = [set(pages.held(i)) & set(pages.held(2 + i)) for i in range(2)]
    assert [len(s) for s in shared] == [1, 2]                  # the full pages of 45 and 64 tokens
    before = [t[sorted(set.union(*shared))].clone() for t in b.cache]
    for _ in range(3):
        b.u.copy_(torch.rand(b.u.shape, generator=g))
        ex.step(p, b, 0.3, 200)
    assert all(torch.equal(t[sorted(set.union(*shared))], v) for t, v in zip(b.cache, before))
    # both halves saw the same prompt: greedy from the same token, they go on alike
    q, c, _, _ = start(ex, [45, 64], 9, 3)
    for _ in range(3):
        ex.step(q, c, 0.0, 200)
        assert torch.equal(c.held[:2], c.held[2:]) and torch.equal(c.path[:2], c.path[2:])


def test_main_runs(ex, monkeypatch, capsys):
    print("case speculative main", flush=True)
    monkeypatch.setattr(sys, "argv", ["speculative_decode.py", "--steps", "5"])
    ex.main()
    assert "us a step" in capsys.readouterr().out


# ------------------------------------------------------------- each one captured
def replays(step, outs, change):
    """Captures step(), replays it 3 times on changed inputs; outs() must be what an eager
    call gives on them."""
    step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(0)
    for r in range(3):
        change(r)
        junk = torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = outs(step(0))
        torch.cuda.synchronize()
        assert float(junk) == float(junk)
        for a, b in zip(outs(res), want):
            assert torch.equal(a, b), "replay %d" % r


@pytest.mark.parametrize("variant,splits", [("rows", 1), ("rows", 5), ("tile", 1), ("tile", 3), ("auto", 0)])
def test_tree_attention_captured(fc, variant, splits):
    print("case captured attention", variant, splits, flush=True)
    lens, new = [900, 33, 400], [20, 33, 3]
    b, bits, pos = tree_batch(21, BF16, lens, new, 8, 2, 128, 32)
    g = on_gpu(b)
    tree = (bits.cuda(), pos.cuda())
    rnd = gen(1)

    def change(r):
        g["q"].copy_(torch.randn(g["q"].shape, generator=rnd))
        g["kv_lens"].copy_(i32([900 - 100 * r, 33, 400 - r]))
    replays(lambda _: fc.chain_attn(**g, tree=tree, max_q=33, max_kv=900, variant=variant, splits=splits, lse=True),
            lambda o: o, change)


@pytest.mark.parametrize("rows,vocab", [(3, 5), (5, 1000), (2, 60000), (300, 40000)])
def test_sampling_captured(fc, rows, vocab):
    print("case captured sampling", rows, vocab, flush=True)
    rnd = gen(2)
    x, u = torch.randn((rows, vocab)).cuda().bfloat16(), torch.rand(rows).cuda()
    top_p = torch.full((rows,), 0.9).cuda()

    def change(r):
        x.copy_(torch.randn(x.shape, generator=rnd))
        u.copy_(torch.rand(u.shape, generator=rnd))
        top_p.copy_(torch.rand(rows, generator=rnd))
    replays(lambda _: fc.sample_tokens(x, u, 1.1, 0, top_p), lambda o: [o], change)


def test_bookkeeping_captured(fc):
    print("case captured bookkeeping", flush=True)
    rng = random.Random(3)
    new = [33, 1, 8]
    cu, lens = cumulative(new).cuda(), i32([40, 100, 8]).cuda()
    par = i32(sum((grow(rng, n) for n in new), [])).cuda()
    tok, tgt = torch.zeros(42, dtype=torch.int32).cuda(), torch.zeros(42, dtype=torch.int32).cuda()

    def change(r):
        par.copy_(i32(sum((grow(rng, n) for n in new), [])))
        tok.copy_(i32([rng.randint(0, 1) for _ in range(42)]))
        tgt.copy_(i32([rng.randint(0, 1) for _ in range(42)]))
    replays(lambda _: (*fc.tree_plan(par, cu, lens, max_q=33), *fc.tree_accept(par, tok, tgt, cu, lens, max_q=33)),
            lambda o: o, change)


def test_moves_captured(fc):
    print("case captured moves", flush=True)
    b, _, _ = tree_batch(22, BF16, [70, 40], [20, 16], 4, 2, 64, 16)
    g = on_gpu(b)
    start = (g["codes"].clone(), g["scales"].clone())
    keep, kept = torch.full((2, 20), -1, dtype=torch.int32).cuda(), i32([0, 0]).cuda()
    used = set(g["table"].flatten().tolist())
    n = g["codes"].shape[0]
    free = [i for i in range(n) if i not in used]
    pairs = [(int(g["table"][0, 0]), free[0])] if free else []
    rng = random.Random(5)

    def step(_):
        g["codes"].copy_(start[0])
        g["scales"].copy_(start[1])
        fc.kv_copy(g["codes"], g["scales"], pairs)
        fc.kv_keep(g["codes"], g["scales"], g["table"], g["cu_q"], g["kv_lens"], keep, kept)
        return g["codes"].clone(), g["scales"].clone()

    def change(r):
        lists = [sorted(rng.sample(range(m), 5 + r)) for m in (20, 16)]
        keep[:, :5 + r].copy_(i32(lists))
        kept.fill_(5 + r)
    replays(step, lambda o: o, change)


# ---------------------------------------------------- calls at the documents' edges
@pytest.mark.parametrize("variant", ["rows", "tile"])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_a_bound_that_is_too_small_costs_time_only(fc, variant, splits):
    print("case small max_q", variant, splits, flush=True)
    lens, new = [300, 200, 129], [129, 40, 1]
    b, bits, pos = tree_batch(23, BF16, lens, new, 8, 2, 64, 32)
    check_tree(fc, b, bits, pos, "max_q", max_q=2, max_kv=300, variant=variant, splits=splits)
    check_tree(fc, b, bits, pos, "max_kv", max_q=129, max_kv=20, variant=variant, splits=splits)
    check_tree(fc, b, bits, pos, "both", max_q=1, max_kv=1, variant=variant, splits=splits)


@pytest.mark.parametrize("variant", ["rows", "tile"])
@pytest.mark.parametrize("d", [192, 256])
@pytest.mark.parametrize("splits", [2, 5])
def test_wide_heads_split(fc, variant, d, splits):
    print("case wide", variant, d, splits, flush=True)
    lens, new = [333, 60, 190], [30, 60, 2]
    b, bits, pos = tree_batch(24, F16, lens, new, 8, 2, d, 64)
    check_tree(fc, b, bits, pos, "wide", max_q=60, variant=variant, splits=splits)


@pytest.mark.parametrize("splits", [0, 1, 2, 1024])
def test_many_sequences_some_empty(fc, splits):
    """More sequences than a wave has lanes, some without tokens or without new ones."""
    print("case many", splits, flush=True)
    rng = random.Random(7)
    new = [0 if i % 5 == 0 else rng.randint(1, 12) for i in range(150)]
    lens = [0 if i % 10 == 0 else n + rng.randint(0, 90) for i, n in enumerate(new)]
    b, bits, pos = tree_batch(25, BF16, lens, new, 4, 2, 64, 16)
    check_tree(fc, b, bits, pos, "many", max_q=12, variant="tile", splits=splits)


def test_a_workspace_given_or_too_small(fc):
    print("case workspaces", flush=True)
    lens, new = [2000, 33], [20, 33]
    b, bits, pos = tree_batch(26, BF16, lens, new, 8, 2, 128, 32)
    g = on_gpu(b)
    tree = (bits.cuda(), pos.cuda())
    kw = dict(max_q=33, max_kv=2000, variant="tile", splits=3)
    plan = fc.attn_plan(53, 2, 8, 2, 128, 32, g["table"].shape[1], 33, 2000, variant="tile", splits=3, tree=True)
    ref = fc.chain_attn(**g, tree=tree, **kw)
    room = torch.full((plan["workspace"] + 64,), 0xff, dtype=torch.uint8, device="cuda")
    out = fc.chain_attn(**g, tree=tree, workspace=room[:plan["workspace"]], **kw)
    assert torch.equal(out, ref) and room[plan["workspace"]:].eq(0xff).all()
    with pytest.raises(fc.FusedChainError):
        fc.chain_attn(**g, tree=tree, workspace=room[:plan["workspace"] - 16], **kw)
    x, u = torch.randn((7, 50000)).cuda(), torch.rand(7).cuda()
    ref = fc.sample_tokens(x, u, top_p=0.9)
    room = torch.full((1 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    assert torch.equal(fc.sample_tokens(x, u, top_p=0.9, workspace=room), ref)
    with pytest.raises(fc.FusedChainError):
        fc.sample_tokens(x, u, top_p=0.9, workspace=room[:16])


def test_two_streams_at_once(fc):
    """Split attention and sampling of two batches on two streams, workspaces of their own."""
    print("case two streams", flush=True)
    sides = []
    for seed in (31, 32):
        b, bits, pos = tree_batch(seed, BF16, [3000, 200], [26, 9], 8, 2, 128, 32)
        sides.append((on_gpu(b), (bits.cuda(), pos.cuda()), torch.randn((40, 70000), generator=gen(seed)).cuda(),
                      torch.rand(40, generator=gen(seed)).cuda()))

    def call(s):
        return fc.chain_attn(**s[0], tree=s[1], max_q=26, variant="tile", splits=6), fc.sample_tokens(s[2], s[3], top_p=0.95)
    want = [call(s) for s in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(sides):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(s))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])
