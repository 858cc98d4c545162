"""tree_plan and tree_accept write inside their outputs only, whatever cu_q holds: the C
entries on outputs that are slices of larger, filled buffers."""
import random

import pytest

torch = pytest.importorskip("torch")
import decode_ref as D  # noqa: E402
from test_gpu_attn import fc, i32  # noqa: E402,F401
from test_gpu_tree import grow  # noqa: E402

pytestmark = pytest.mark.gpu
MARGIN = 256
FILL = 0x5a5a5a5a


def room(n, dtype=torch.int32):
    """(buffer, its middle n elements)."""
    b = torch.full((n + 2 * MARGIN,), FILL, dtype=dtype, device="cuda")
    return b, b[MARGIN:MARGIN + n]


def margins_are_whole(buffers):
    for b in buffers:
        assert b[:MARGIN].eq(FILL).all() and b[-MARGIN:].eq(FILL).all()


def taken_inside(cu, T):
    """Each sequence's range as the kernels take it: offsets into [0, T], none that falls."""
    out = []
    for a, z in zip(cu, cu[1:]):
        a = min(max(a, 0), T)
        out.append((a, min(max(z, a), T)))
    return out


BIG = 2 ** 31 - 1
OFFSETS = [[0, 40, 10], [5, 2, 10], [-7, 3, 12], [0, BIG, -BIG - 1], [-BIG - 1, BIG, 0], [9, 9, 9], [10, 10, 10], [0, 10, 10],
           [100, 200, 300], [-5, -4, -3], [0, 8, 3, 10], [10, 0, 10, 0, 10], [0, 0, 0, 0, 10, 0]]


@pytest.mark.parametrize("cu", OFFSETS, ids=str)
@pytest.mark.parametrize("T,words", [(10, 1), (10, 3), (70, 1), (70, 2), (300, 4)])
def test_bad_offsets(fc, cu, T, words):
    print("case margins", cu, T, words, flush=True)
    cu = [c * (T // 10) if abs(c) < 1000 else c for c in cu]
    B = len(cu) - 1
    rng = random.Random(T)
    par = grow(rng, T, 5)
    tok, tgt = ([rng.randint(0, 1) for _ in range(T)] for _ in range(2))
    lens = [T + 10 * b for b in range(B)]
    most = 6
    bits_b, bits = room(T * words, torch.int64)
    pos_b, pos = room(T)
    keep_b, keep = room(B * most)
    kept_b, kept = room(B)
    nxt_b, nxt = room(B)
    len_b, after = room(B)
    dev = [i32(v).cuda() for v in (par, tok, tgt, cu, lens)]
    p, k, g, c, n = (t.data_ptr() for t in dev)
    L = fc.lib()
    st = torch.cuda.current_stream().cuda_stream
    assert L.tree_plan(p, c, n, B, T, words, bits.data_ptr(), pos.data_ptr(), st) == 0
    assert L.tree_accept(p, k, g, c, n, B, T, most, keep.data_ptr(), kept.data_ptr(), nxt.data_ptr(), after.data_ptr(), st) == 0
    torch.cuda.synchronize()
    margins_are_whole([bits_b, pos_b, keep_b, kept_b, nxt_b, len_b])
    ranges = taken_inside(cu, T)
    times = [sum(a <= i < z for a, z in ranges) for i in range(T)]
    bits, pos = bits.view(T, words).tolist(), pos.tolist()
    fill = [FILL] * words
    for i in range(T):
        if times[i] == 0:
            assert bits[i] == fill and pos[i] == FILL, i       # rows of no sequence stay as they are
    for b, (a, z) in enumerate(ranges):
        # a tree of its own: parents count from its first token
        seen = D.ancestors(par[a:z])
        if all(t == 1 for t in times[a:z]):                     # (where two sequences meet, either's)
            if z - a > 64 * words:
                assert all(r == [0] * words for r in bits[a:z]) and pos[a:z] == [lens[b] - (z - a)] * (z - a)
            else:
                assert bits[a:z] == D.words_of(seen, words)
                assert pos[a:z] == [lens[b] - (z - a) + len(s) - 1 for s in seen]
        path, token = D.accept(par[a:z], tok[a:z], tgt[a:z])
        if len(path) > most:
            path, token = path[:most], tgt[a:z][path[most - 1]]
        assert keep[b * most:(b + 1) * most].tolist() == path + [-1] * (most - len(path)), b
        assert (int(kept[b]), int(nxt[b]), int(after[b])) == (len(path), token, lens[b] - (z - a) + len(path)), b
