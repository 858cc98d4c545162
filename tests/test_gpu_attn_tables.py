"""Tables that are slices of wider ones, on the GPU."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_attn import F16, batch, fc, gen, on_gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", ["rows", "tile"])
def test_table_slices(fc, variant):  # noqa: F811
    """A table cut out of a wider one: its rows end where the slice ends."""
    print("case table slice", variant, flush=True)
    b = batch(113, F16, [100, 70, 33], [20, 1, 3], 4, 2, 64, 16)
    want = fc.chain_attn(**on_gpu(b), variant=variant)
    n = b["table"].shape[1]
    wide = torch.zeros((3, n + 5), dtype=torch.int32)             # page 0 beside the slice
    wide[:, 2:2 + n] = b["table"]
    g = on_gpu(b)
    for table in (wide.cuda()[:, 2:2 + n], b["table"].t().contiguous().cuda().t()):
        assert not table.is_contiguous()
        assert torch.equal(fc.chain_attn(**{**g, "table": table}, variant=variant), want)
    # a length past the end of the slice is too long, though the wider table could hold it
    long = b["kv_lens"].clone()
    long[0] = n * 16 + 1
    out = fc.chain_attn(**{**g, "table": wide.cuda()[:, 2:2 + n], "kv_lens": long.cuda()}, variant=variant)
    assert torch.isnan(out[:20]).all() and torch.equal(out[20:], want[20:])
    k, v = (torch.randn((24, 2, 64), generator=gen(s)).half().cuda() for s in (1, 2))
    pools = [(g["codes"].clone(), g["scales"].clone()) for _ in range(2)]
    fc.kv_append(k, v, *pools[0], g["table"], g["cu_q"], g["kv_lens"])
    fc.kv_append(k, v, *pools[1], wide.cuda()[:, 2:2 + n], g["cu_q"], g["kv_lens"])
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
