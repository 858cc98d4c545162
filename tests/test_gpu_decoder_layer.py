"""The example's layer, prompts and then steps, stage by stage against plain
64-bit forms of each stage on the stage's own inputs."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decoder_layer
    return decoder_layer


def product(a, w, b=None):
    """(result, tolerance before rounding) of a w + b: fp32 sums of exact products."""
    a, w = a.cpu().double(), w.cpu().double()
    r, size = a @ w, a.abs() @ w.abs()
    if b is not None:
        r, size = r + b.cpu().double(), size + b.cpu().double().abs()
    return r, size * (a.shape[1] + 4) * 2.0 ** -24


def near(got, ref, inner, what):
    R.assert_within(got, ref, R.rounded_tol(ref, inner, torch.float16), what)


def check(ex, x, y, mid, p, cache, before, table, cu, kv, what):
    T = x.shape[0]
    near(mid["qkv"], *product(x, p["wqkv"], p["bqkv"]), what + " qkv")
    rows = mid["qkv"].cpu().view(T, ex.HQ + 2 * ex.HKV, ex.D)
    k, v = rows[:, ex.HQ:ex.HQ + ex.HKV], rows[:, ex.HQ + ex.HKV:]
    turns = p["turns"].cpu()
    R.assert_appended(*cache, R.append(k, v, *before, table, cu, kv, turns), what + " cache")
    slots = [s for b in range(len(kv)) for s in range(int(kv[b]) - int(cu[b + 1] - cu[b]), int(kv[b]))]
    q, inner = R.rope(rows[:, :ex.HQ], slots, turns)
    near(mid["q"], q, inner, what + " q")
    a, tol, _, _ = R.attention(mid["q"].cpu(), cache[0].cpu(), cache[1].cpu(), table, cu, kv)
    near(mid["attn"], a, tol, what + " attn")
    r, tol = product(mid["attn"].view(T, -1), p["wo"])
    u = R.half_step(torch.float16)
    near(mid["h"], x.cpu().double() + r, tol + r.abs() * u * 1.01, what + " h")     # the product is rounded, then the sum
    # the hidden layer is rounded once; GELU's slope is at most 1.13
    z, tol0 = product(mid["h"], p["w0"], p["b0"])
    g = torch.nn.functional.gelu(z, approximate="tanh")
    w1 = p["w1"].cpu().double()
    r = g @ w1 + p["b1"].cpu().double()
    tol1 = (1.13 * tol0 + g.abs() * (u + 2.0 ** -20) + 2.0 ** -25) @ w1.abs() + (g.abs() @ w1.abs()) * (ex.FFN + 4) * 2.0 ** -24
    near(mid["mlp"], r, tol1, what + " mlp")
    near(y, mid["h"].cpu().double() + mid["mlp"].cpu().double(), torch.zeros(()), what + " out")


def test_layer(ex):
    fc = ex.fc
    p = ex.make_weights(seed=3)
    lens = [70, 1, 33]
    cache = fc.kv_cache(9, ex.HKV, ex.PAGE, ex.D)
    pages = ex.Pages(9, 3, 4)
    g = torch.Generator()
    g.manual_seed(5)
    new = list(lens)
    for step in range(4):
        print("case layer", step, flush=True)
        x = torch.randn((sum(new), ex.HIDDEN), generator=g).half().cuda()
        cu = torch.tensor([0] + [sum(new[:i + 1]) for i in range(3)], dtype=torch.int32)
        kv = torch.tensor(lens, dtype=torch.int32)
        table = pages.grow(lens).clone()
        before = cache[0].cpu(), cache[1].cpu()
        y, mid = ex.layer(x, p, cache, table.cuda(), cu.cuda(), kv.cuda(), max(new), max(lens))
        check(ex, x, y, mid, p, cache, before, table, cu, kv, "step %d" % step)
        new = [1, 1, 1]
        lens = [n + 1 for n in lens]


def test_main_runs(ex, monkeypatch, capsys):
    print("case example main", flush=True)
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--steps", "6"])
    ex.main()
    assert "us a step" in capsys.readouterr().out
