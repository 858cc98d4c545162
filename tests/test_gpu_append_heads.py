"""kv_append with factors that take rotated keys out of 32 bits."""
import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402
from test_gpu_attn import BF16, DTYPES, F16, batch, fc, gen, i32, on_gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new", [1, 20])
def test_rotated_keys_past_32_bits(fc, monkeypatch, interleaved, new):  # noqa: F811
    """A key that its rotation takes past the largest 32-bit number saturates and
    does not set its page's scale."""
    print("case past 32 bits", interleaved, new, flush=True)
    b = batch(107, BF16, [36], [new], 2, 2, 64, 16)
    g = gen(109)
    k, v = (torch.randn((new, 2, 64), generator=g).to(BF16) for _ in range(2))
    k[new - 1, 0, 5] = 2.0 ** 124                   # in head 0 of the last token; times 40 it leaves 32 bits
    turns, rope = fc.rope_turns(64)[0], R.rope

    def rope32(*a):
        y, tol = rope(*a)
        return torch.where(y.abs() > torch.finfo(torch.float32).max, torch.sign(y) * float("inf"), y), tol
    monkeypatch.setattr(R, "rope", rope32)
    mscale = 40.0
    expect = R.append(k, v, b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], turns, interleaved, mscale)
    c = on_gpu(b)
    fc.kv_append(k.cuda(), v.cuda(), c["codes"], c["scales"], c["table"], c["cu_q"], c["kv_lens"], turns=turns.cuda(),
                 interleaved=interleaved, mscale=mscale, max_q=new)
    R.assert_appended(c["codes"], c["scales"], expect, "past 32 bits")
