"""chain_attn split many ways (the join by four waves a row), on the GPU against 64
bits."""
import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402
from test_gpu_attn import DTYPES, batch, fc, on_gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def check(fc, b, what, **kw):  # noqa: F811
    print("case splits", what, kw, flush=True)
    ref, tol, lse, ltol = R.attention(b["q"], b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"])
    out, le = fc.chain_attn(**on_gpu(b), lse=True, **kw)
    R.assert_within(out, ref, R.rounded_tol(ref, tol, b["q"].dtype), what)
    R.assert_within(le, lse, ltol, what + " lse")
    for _ in range(2):      # the same bits on every run
        assert torch.equal(fc.chain_attn(**on_gpu(b), **kw), out)


@pytest.mark.parametrize("splits", [8, 9, 33, 64])
@pytest.mark.parametrize("variant", ["rows", "tile"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_many_splits(fc, splits, variant, dtype, d):  # noqa: F811
    """A short sequence, an empty one and one with fewer keys than queries: most of
    their splits have no keys (of 9 and more, the longest sequence's last too)."""
    lens, new = [701, 33, 1500, 0, 2], [2, 5, 1, 1, 4]
    b = batch(d + splits, dtype, lens, new, 6, 2, d, 32)
    plan = fc.attn_plan(sum(new), len(lens), 6, 2, d, 32, b["table"].shape[1], max(new), max(lens), variant=variant, splits=splits)
    assert plan["splits"] == splits and (splits == 8 or splits * plan["chunk"] > max(lens) + plan["chunk"])
    check(fc, b, "d %d" % d, variant=variant, splits=splits, max_q=max(new), max_kv=max(lens))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,variant", [(1, "rows"), (70, "tile")])
def test_long_context_by_rule(fc, dtype, new, variant):  # noqa: F811
    lens = [70001, 300]
    b = batch(97, dtype, lens, [new, 1], 4, 1, 64, 64)
    plan = fc.attn_plan(new + 1, 2, 4, 1, 64, 64, b["table"].shape[1], new, lens[0], dtype=str(dtype)[6:])
    assert plan["variant"] == variant and plan["splits"] > 8
    check(fc, b, "long", max_q=new, max_kv=lens[0])
