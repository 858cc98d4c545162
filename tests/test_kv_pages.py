"""KvPages: which pages sequences hold, share, copy and free (host only)."""
import random

import pytest

import gemm_conv_chain_amd as fc

pytest.importorskip("torch")
pytestmark = pytest.mark.cpu


def test_grow_cut_free():
    p = fc.KvPages(6, 16)
    p.add("a")
    assert p.grow("a", 0) == [] and p.held("a") == [] and p.available == 6
    assert p.grow("a", 17) == [] and p.held("a") == [0, 1] and p.available == 4
    assert p.grow("a", 32) == [] and p.held("a") == [0, 1]
    p.cut("a", 16)
    assert p.held("a") == [0] and p.available == 5 and p.length("a") == 16
    assert p.grow("a", 33) == [] and p.held("a") == [0, 1, 2]
    p.free("a")
    assert p.available == 6 and p.refs == [0] * 6
    with pytest.raises(KeyError):
        p.held("a")


def test_a_fork_shares_until_someone_writes():
    p = fc.KvPages(8, 16)
    p.add("a")
    p.grow("a", 40)
    p.fork("a", "b")
    p.fork("a", "c")
    assert p.held("b") == [0, 1, 2] and p.refs[:3] == [3, 3, 3] and p.available == 5
    assert p.grow("b", 41) == [(2, 3)] and p.held("b") == [0, 1, 3] and p.refs[:4] == [3, 3, 2, 1]
    assert p.grow("a", 60) == [(2, 4)] and p.held("a") == [0, 1, 4, 5]
    assert p.grow("c", 48) == [] and p.held("c") == [0, 1, 2]      # the last that holds page 2 keeps it
    p.free("a")
    assert p.refs[:6] == [2, 2, 1, 1, 0, 0] and p.available == 4


def test_a_fork_at_a_page_border_copies_nothing():
    p = fc.KvPages(8, 16)
    p.add(1)
    p.grow(1, 32)
    p.fork(1, 2)
    assert p.grow(2, 40) == [] and p.held(2) == [0, 1, 2] and p.grow(1, 33) == [] and p.held(1) == [0, 1, 3]


def test_nothing_to_write_copies_nothing():
    p = fc.KvPages(1, 16)
    p.add("a")
    p.grow("a", 9)
    p.fork("a", "b")
    assert p.grow("b", 9) == [] and p.held("b") == [0] and p.refs == [2]


def test_too_few_pages_change_nothing():
    p = fc.KvPages(3, 16)
    p.add("a")
    p.grow("a", 40)
    p.fork("a", "b")
    for name, n in (("b", 41), ("a", 60)):
        with pytest.raises(MemoryError):
            p.grow(name, n)
    assert p.held("a") == p.held("b") == [0, 1, 2] and p.refs == [2, 2, 2] and p.length("a") == p.length("b") == 40


def test_refusals():
    p = fc.KvPages(3, 16)
    p.add("a")
    p.grow("a", 20)
    with pytest.raises(ValueError):
        p.add("a")
    with pytest.raises(ValueError):
        p.fork("a", "a")
    with pytest.raises(ValueError):
        p.grow("a", 19)
    for n in (-1, 21):
        with pytest.raises(ValueError):
            p.cut("a", n)
    with pytest.raises(ValueError):
        p.table(["a"], width=1)
    for bad in ((-1, 16), (4, 8), (4, 24)):
        with pytest.raises(ValueError):
            fc.KvPages(*bad)
    assert p.table([]).shape == (0, 1) and p.table(["a"], width=4).tolist() == [[0, 1, 0, 0]]


@pytest.mark.parametrize("seed", range(6))
def test_drawn_lives(seed):
    """A host pool of tokens that follows the pairs: every sequence reads its own tokens
    back, whatever is forked, grown, cut, packed and freed; and what is held adds up."""
    rng = random.Random(seed)
    page, P = 16, 24
    p, pool, mine, n = fc.KvPages(P, page), {}, {}, 0

    def run(pairs):
        dst = [b for _, b in pairs]
        assert len(set(dst)) == len(dst) and not set(dst) & {a for a, _ in pairs}
        new = {(b, s): pool[a, s] for a, b in pairs for s in range(page) if (a, s) in pool}
        pool.update(new)
    for _ in range(400):
        names = list(mine)
        act = rng.choice(["add", "fork", "grow", "grow", "grow", "cut", "free", "pack"])
        if act == "add" and len(names) < 6:
            p.add(n)
            mine[n] = []
            n += 1
        elif act == "fork" and names and len(names) < 8:
            a = rng.choice(names)
            p.fork(a, n)
            mine[n] = list(mine[a])
            n += 1
        elif act == "grow" and names:
            a = rng.choice(names)
            to = len(mine[a]) + rng.randint(0, 40)
            try:
                run(p.grow(a, to))
            except MemoryError:
                continue
            for s in range(len(mine[a]), to):
                mine[a].append((a, s, rng.random()))
                pool[p.held(a)[s // page], s % page] = mine[a][-1]
        elif act == "cut" and names:
            a = rng.choice(names)
            to = rng.randint(0, len(mine[a]))
            p.cut(a, to)
            del mine[a][to:]
        elif act == "free" and names:
            a = rng.choice(names)
            p.free(a)
            del mine[a]
        elif act == "pack":
            run(p.pack())
            used = sum(1 for r in p.refs if r)
            assert all(p.refs[:used]) and not any(p.refs[used:]) and p.available == P - used
        for a, toks in mine.items():
            row = p.held(a)
            assert len(row) == -(-len(toks) // page) and p.length(a) == len(toks)
            assert [pool[row[s // page], s % page] for s in range(len(toks))] == toks
        count = [0] * P
        for a in mine:
            for q in p.held(a):
                count[q] += 1
        assert count == p.refs and p.available == count.count(0)
