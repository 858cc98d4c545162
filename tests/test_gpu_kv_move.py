"""kv_keep and kv_copy on the GPU: bytes and scales as decode_ref has them."""
import random

import pytest

torch = pytest.importorskip("torch")
import attn_ref as R  # noqa: E402
import decode_ref as D  # noqa: E402
from test_gpu_attn import BF16, F16, batch, fc, gen, i32, on_gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def lists(rng, new, most=None):
    kept = [rng.randint(0, n) for n in new]
    keep = torch.full((len(new), most or max(new)), -1, dtype=torch.int32)
    for b, (n, k) in enumerate(zip(new, kept)):
        k = kept[b] = min(k, keep.shape[1])
        keep[b, :k] = i32(sorted(rng.sample(range(n), k)))
    return keep, i32(kept)


def run(fc, codes, scales, b, keep, kept):
    c, s = codes.cuda(), scales.cuda()
    fc.kv_keep(c, s, b["table"].cuda(), b["cu_q"].cuda(), b["kv_lens"].cuda(), keep.cuda(), kept.cuda())
    return c, s


@pytest.mark.parametrize("d,page,hkv", [(64, 16, 2), (128, 64, 3), (192, 32, 1), (256, 256, 1), (128, 16, 2)])
@pytest.mark.parametrize("lens,new", [
    ([9], [8]), ([40, 17, 300, 16], [3, 1, 40, 16]), ([130, 64, 513, 33], [26, 64, 0, 17]), ([600, 300], [300, 257])])
def test_keep(fc, d, page, hkv, lens, new):
    print("case keep", d, page, hkv, lens, new, flush=True)
    rng = random.Random(d + sum(new))
    b = batch(d + page, BF16, lens, new, hkv, hkv, d, page)
    keep, kept = lists(rng, new)
    want = D.keep_tokens(b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], keep, kept)
    got = run(fc, b["codes"], b["scales"], b, keep, kept)
    assert torch.equal(got[1].cpu(), want[1])
    assert D.same_codes(got[0], want[0])


def test_keep_every_subset_of_a_small_tree(fc):
    """All lists of six nodes, at every offset of a page."""
    print("case keep subsets", flush=True)
    n, B = 6, 64
    for off in range(0, 17, 4):
        lens, new = [off + n + 3] * B, [n] * B
        b = batch(off, F16, lens, new, 1, 1, 64, 16)
        keep = torch.full((B, n), -1, dtype=torch.int32)
        kept = []
        for m in range(B):
            k = [j for j in range(n) if m >> j & 1]
            keep[m, :len(k)] = i32(k)
            kept.append(len(k))
        kept = i32(kept)
        want = D.keep_tokens(b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], keep, kept)
        got = run(fc, b["codes"], b["scales"], b, keep, kept)
        assert torch.equal(got[1].cpu(), want[1]) and D.same_codes(got[0], want[0]), off


def test_keep_layers_share_a_table(fc):
    print("case keep layers", flush=True)
    lens, new = [100, 31, 64], [20, 31, 3]
    layers = [batch(s, BF16, lens, new, 2, 2, 128, 32) for s in range(3)]
    b = layers[0]
    keep, kept = lists(random.Random(3), new, most=40)
    codes, scales = (torch.stack([x[k] for x in layers]) for k in ("codes", "scales"))
    got = run(fc, codes, scales, b, keep, kept)
    for i in range(3):
        want = D.keep_tokens(codes[i], scales[i], b["table"], b["cu_q"], b["kv_lens"], keep, kept)
        assert torch.equal(got[1][i].cpu(), want[1]) and D.same_codes(got[0][i], want[0])


def test_keep_leaves_what_it_does_not_understand(fc):
    print("case keep bad lists", flush=True)
    lens, new = [60] * 8 + [40, 70], [8] * 8 + [9, 20]
    b = batch(7, F16, lens, new, 2, 2, 64, 16)
    keep = torch.tensor([[0, 2, 4, 6, -1]] * 10, dtype=torch.int32)
    kept = [4] * 10
    keep[0, 1] = 0            # twice the same
    keep[1, :2] = i32([2, 1])  # falling
    keep[2, 3] = 8            # past the new tokens
    keep[3, 0] = -1
    kept[4], kept[5], kept[6] = -1, 9, 6           # no number of tokens; more than there are; more than the list has
    keep[7] = i32([0, 1, 2, 3, 4])                 # nothing moves
    b["table"][8, 1] = 10 ** 7                     # slots 16 .. 31 have no page
    b["kv_lens"][9] = 16 * b["table"].shape[1] + 1
    kept = i32(kept)
    want = D.keep_tokens(b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], keep, kept)
    got = run(fc, b["codes"], b["scales"], b, keep, kept)
    assert torch.equal(got[1].cpu(), want[1]) and D.same_codes(got[0], want[0])
    # only the sequence with a page missing has changed
    pages = [int(p) for p in b["table"][8].tolist() if 0 <= p < b["codes"].shape[0]]
    other = [p for p in range(b["codes"].shape[0]) if p not in pages]
    assert torch.equal(got[0].cpu()[other], b["codes"][other])


def test_keep_tokens_of_a_missing_page(fc):
    """A token that comes from a page outside the pool gets a NaN key, so that who sees it
    turns NaN; one whose own page is outside is not moved."""
    print("case keep missing page", flush=True)
    b = batch(9, F16, [40, 40], [20, 24], 2, 2, 64, 16)     # slots 20 .. 39, 16 .. 39
    keep, kept = i32([[0, 13, 14], [0, 1, 20]]), i32([3, 3])
    b["table"][0, 2] = -1                                    # slots 32 .. 47
    b["table"][1, 1] = 1000
    want = D.keep_tokens(b["codes"], b["scales"], b["table"], b["cu_q"], b["kv_lens"], keep, kept)
    got = run(fc, b["codes"], b["scales"], b, keep, kept)
    assert torch.equal(got[1].cpu(), want[1]) and D.same_codes(got[0], want[0])
    K = R.unpack_k(got[0].cpu()[:, :, 0], 64)[int(b["table"][0, 1])]
    assert K[:, 5:7].eq(0x7f).all() and not K[:, :5].eq(0x7f).any()


def test_keep_past_32_bits(fc):
    """The last pages of a pool of 4.4 GB."""
    print("case keep far", flush=True)
    d, page, H = 256, 256, 4
    P = 2 ** 32 // (H * 2 * page * d) + 40
    codes = torch.zeros((P, H, 2, page // 16, 16 * d), dtype=torch.uint8, device="cuda")
    scales = torch.ones((P, H, 2), device="cuda")
    small = batch(4, BF16, [300], [200], H, H, d, page, spare=0)
    codes[P - 2:], scales[P - 2:] = small["codes"].cuda(), small["scales"].cuda()
    keep, kept = i32([[0, 5, 6, 180, 199]]), i32([5])
    want = D.keep_tokens(small["codes"], small["scales"], small["table"], small["cu_q"], small["kv_lens"], keep, kept)
    fc.kv_keep(codes, scales, (small["table"] + P - 2).cuda(), small["cu_q"].cuda(), small["kv_lens"].cuda(), keep.cuda(), kept.cuda())
    assert torch.equal(scales[P - 2:].cpu(), want[1]) and D.same_codes(codes[P - 2:], want[0])
    fc.kv_copy(codes, scales, [(P - 1, 0), (P - 2, P - 3)])
    assert torch.equal(codes[0], codes[P - 1]) and torch.equal(codes[P - 3], codes[P - 2]) and codes[1:P - 3].eq(0).all()


@pytest.mark.parametrize("pages,hkv,page,d,layers,n", [(2, 1, 16, 64, 1, 1), (9, 2, 32, 128, 3, 4), (1200, 1, 16, 64, 2, 600),
                                                     (7, 3, 256, 256, 1, 3), (40, 5, 16, 192, 2, 20)])
def test_copy(fc, pages, hkv, page, d, layers, n):
    print("case copy", pages, hkv, page, d, layers, n, flush=True)
    g = gen(n)
    codes = torch.randint(0, 256, (layers, pages, hkv, 2, page // 16, 16 * d), generator=g, dtype=torch.uint8)
    scales = torch.rand((layers, pages, hkv, 2), generator=g)
    order = torch.randperm(pages, generator=g).tolist()
    to = order[:n]
    src = [random.Random(i).choice(order[n:]) for i in range(n)]          # a source may serve many
    c, s = codes.cuda(), scales.cuda()
    fc.kv_copy(c, s, list(zip(src, to)))
    codes[:, to], scales[:, to] = codes[:, src], scales[:, src]
    assert torch.equal(c.cpu(), codes) and torch.equal(s.cpu(), scales)
    # one layer's pool, pairs as a tensor
    if n > 1:
        fc.kv_copy(c[0], s[0], torch.tensor([[to[0], src[0]]], dtype=torch.int32))
        codes[0, src[0]], scales[0, src[0]] = codes[0, to[0]], scales[0, to[0]]
        assert torch.equal(c.cpu(), codes) and torch.equal(s.cpu(), scales)


def test_copy_refused_copies_nothing(fc):
    print("case copy refused", flush=True)
    c = torch.randint(0, 256, (6, 1, 2, 1, 1024), dtype=torch.uint8)
    g, s = c.cuda(), torch.rand((6, 1, 2)).cuda()
    for pairs in ([(0, 1), (2, 6)], [(0, 1), (2, 1)], [(0, 1), (1, 2)], [(0, 0)]):
        with pytest.raises(fc.FusedChainError):
            fc.kv_copy(g, s, pairs)
    assert torch.equal(g.cpu(), c)
