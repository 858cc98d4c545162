"""kv_append with odd numbers of query heads in prompts (threads that hold two heads
have one left over), and with factors that take rotated keys out of 32 bits."""
import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402
from test_gpu_attn import BF16, DTYPES, F16, batch, fc, gen, i32, on_gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,new,hq,hkv,d,page,rot,interleaved", [
    ([40, 20], [30, 17], 1, 1, 64, 16, 64, False),
    ([90], [70], 3, 1, 128, 32, 128, True),
    ([50, 64], [33, 20], 5, 5, 192, 64, 48, False),
    ([300], [280], 7, 1, 256, 128, 256, False),
])
def test_odd_heads(fc, dtype, lens, new, hq, hkv, d, page, rot, interleaved):  # noqa: F811
    """q in the middle of wider rows, q_out in the middle of a larger buffer: heads
    past the last are neither read into the result nor written."""
    print("case odd heads", dtype, hq, hkv, d, flush=True)
    b = batch(101 + d, dtype, lens, new, hq, hkv, d, page)
    T, g = sum(new), gen(103)
    rows = torch.randn((T, hq + 2 * hkv + 2, d), generator=g).to(dtype)
    q, k, v = rows[:, 1:1 + hq], rows[:, 1 + hq:1 + hq + hkv], rows[:, 1 + hq + hkv:1 + hq + 2 * hkv]
    turns = fc.rope_turns(rot)[0]
    expect = R.append(k, v, b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], turns, interleaved)
    c, dr = on_gpu(b), rows.cuda()
    guard = 2 * hq * d
    whole = torch.full((T * hq * d + 2 * guard,), 7.0, dtype=dtype, device="cuda")
    qo = whole[guard:guard + T * hq * d].view(T, hq, d)
    got = fc.kv_append(dr[:, 1 + hq:1 + hq + hkv], dr[:, 1 + hq + hkv:1 + hq + 2 * hkv], c["codes"], c["scales"], c["table"],
                       c["cu_q"], c["kv_lens"], turns=turns.cuda(), interleaved=interleaved, q=dr[:, 1:1 + hq], q_out=qo,
                       max_q=max(new))
    assert got is qo
    R.assert_appended(c["codes"], c["scales"], expect, "odd heads")
    slots = [s for n, L in zip(new, lens) for s in range(L - n, L)]
    ref, inner = R.rope(q, slots, turns, interleaved)
    R.assert_within(qo, ref, R.rounded_tol(ref, inner, dtype), "odd heads q")
    assert (whole[:guard] == 7).all() and (whole[-guard:] == 7).all()
    assert torch.equal(dr.cpu(), rows)


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
