"""Plain implementations in 64 bits of the operators around a speculative step,
on the host and straight from their definitions (test infrastructure)."""
import math

import numpy as np
import torch

import attn_ref as R


# ------------------------------------------------------------------------ trees
def ancestors(parents):
    """The set of nodes that each node sees: its ancestors and itself."""
    seen = []
    for i, p in enumerate(parents):
        seen.append({i} | (seen[p] if 0 <= p < i else set()))
    return seen


def words_of(seen, words):
    rows = []
    for s in seen:
        v = sum(1 << j for j in s)
        row = [(v >> (64 * w)) & ((1 << 64) - 1) for w in range(words)]
        rows.append([x - (1 << 64) if x >> 63 else x for x in row])
    return rows


def sets_of(bits):
    """[rows, words] int64 -> the set of nodes of each row."""
    out = []
    for row in bits.tolist():
        v = sum((x & ((1 << 64) - 1)) << (64 * w) for w, x in enumerate(row))
        out.append({j for j in range(64 * len(row)) if v >> j & 1})
    return out


def accept(parents, drafted, targets):
    if not parents:
        return [], -1
    path = [0]
    while True:
        now = path[-1]
        nxt = [j for j in range(now + 1, len(parents)) if parents[j] == now and drafted[j] == targets[now]]
        if not nxt:
            return path, targets[now]
        path.append(nxt[0])


def attention(q, codes, scales, table, cu_q, kv_lens, bits, positions, scale=None, softcap=0.0, window=0, slopes=None):
    """(out, tolerance before the output's rounding, lse, lse tolerance); the
    tolerances are attn_ref.attention's, by the same count of roundings, with one more
    of a bias's size for the distance that a node's position puts right."""
    T, hq, d = q.shape
    G = hq // codes.shape[1]
    u = R.half_step(q.dtype)
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros((T, hq, d), dtype=torch.float64)
    tol = torch.zeros((T, hq, d), dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros((T, hq), dtype=torch.float64)
    sets = sets_of(bits)
    for b in range(table.shape[0]):
        a, z = int(cu_q[b]), int(cu_q[b + 1])
        n, L = z - a, int(kv_lens[b])
        if n == 0 or L == 0:
            continue
        s0 = L - n
        K, V = R.gather(codes, scales, table[b], L, d)
        pos = positions[a:z].long().clamp(s0, L - 1)
        place = torch.cat((torch.arange(max(s0, 0)), pos))[-L:]
        gap = pos[:, None] - place
        seen = torch.zeros((n, L), dtype=torch.bool)
        for i in range(n):
            for j in range(L):
                seen[i, j] = j < s0 or (j - s0) in sets[a + i]
        if window:
            seen &= gap < window
        for h in range(hq):
            qq = q[a:z, h].double()
            x = qq @ K[h // G].T * scale
            dx = (d + 4) * 2.0 ** -24 * scale * (qq.abs() @ torch.nan_to_num(K[h // G].abs()).T)
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                dx = dx + softcap * 2.0 ** -21
            if slopes is not None:
                slot = (pos[:, None] - torch.arange(L)).abs()      # the kernels take the slot's distance first
                bias = float(slopes[h]) * gap.abs()
                x = x - bias
                dx = dx + float(slopes[h]) * (gap.abs() + 2 * slot) * 2.0 ** -22
            dx = dx + x.abs() * 2.0 ** -22
            x = x.masked_fill(~seen, -math.inf)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
            l = p.sum(-1, keepdim=True)
            w = p / torch.where(l == 0, 1.0, l)
            vv = torch.where(seen.any(0)[:, None], V[h // G], 0.0)
            out[a:z, h] = w @ vv
            err = torch.where(seen, dx, 0.0).amax(-1, keepdim=True) + 2.0 ** -20
            tol[a:z, h] = w @ vv.abs() * (u + 2 * err) + R.TINY[q.dtype] * (seen.double() @ vv.abs())
            lse[a:z, h] = torch.where(seen.any(-1), (m + torch.log(l))[:, 0], -math.inf)
            ltol[a:z, h] = err[:, 0] + 2.0 ** -22 * lse[a:z, h].abs().nan_to_num(0, 0, 0)
    return out, tol, lse, ltol


# --------------------------------------------------------------- drawing tokens
def weights_that_stay(x, temperature, top_k, top_p, min_p):
    """float64 [V]: the weights of the tokens that stay, 0 elsewhere.  x float64."""
    order = np.lexsort((np.arange(len(x)), -x))
    if not temperature > 0:
        w = np.zeros(len(x))
        w[order[0]] = 1.0
        return w
    with np.errstate(under="ignore", invalid="ignore"):
        e = np.exp((x[order] - x[order[0]]) / temperature)
    e[x[order] == -np.inf] = 0.0
    if top_k > 0:
        e[int(top_k):] = 0.0
    before = np.concatenate(([0.0], np.cumsum(e)[:-1]))
    if top_p < 1:
        stays = before < top_p * e.sum()
        stays[0] = True
        e = np.where(stays, e, 0.0)
    lead = e[0]
    e = np.where(e >= min(min_p, 1.0), e, 0.0)
    e[0] = lead
    w = np.zeros(len(x))
    w[order] = e
    return w


def draw(w, u):
    """(token, distance of u from the nearest border of the token's share)."""
    upto = np.cumsum(w)
    total = upto[-1]
    token = int(np.argmax(upto > u * total))
    lo = upto[token] - w[token]
    return token, min(abs(u - lo / total), abs(upto[token] / total - u))


def middles(w, count, rng):
    """Random numbers inside the shares of some tokens, as 32-bit floats: the widest, the
    first and the last that stay, and others; shares under 1e-6 are too narrow for one."""
    upto = np.cumsum(w)
    total = upto[-1]
    some = np.nonzero(w / total > 1e-6)[0]
    pick = [int(np.argmax(w)), int(some[0]), int(some[-1])] + [int(rng.choice(some)) for _ in range(count)]
    pick = pick[:count]
    return pick, [float(np.float32((upto[t] - w[t] / 2) / total)) for t in pick]


# ------------------------------------------------------------------- the cache
def keep_tokens(codes, scales, table, cu_q, kv_lens, keep, kept):
    """One layer's pool after kv_keep (codes, scales)."""
    d = codes.shape[4] // 16
    page = codes.shape[3] * 16
    P, H = codes.shape[:2]
    codes, scales = codes.clone(), scales.clone()
    sides = [R.unpack_k(codes[:, :, 0], d).clone(), R.unpack_v(codes[:, :, 1], d).clone()]   # [P, H, page, d]
    for b in range(table.shape[0]):
        n, L, m = int(cu_q[b + 1] - cu_q[b]), int(kv_lens[b]), int(kept[b])
        ks = keep[b, :max(m, 0)].tolist()
        start = L - n
        if m <= 0 or m > n or m > keep.shape[1] or start < 0 or L > page * table.shape[1]:
            continue
        if any(k <= (ks[i - 1] if i else -1) or k >= n for i, k in enumerate(ks)) or ks == list(range(m)):
            continue

        def page_of(slot):
            i = int(table[b, slot // page])
            return i if 0 <= i < P else -1
        was, had = [s.clone() for s in sides], scales.clone()
        for p in range(start // page, (start + m - 1) // page + 1):
            to = page_of(p * page)
            if to < 0:
                continue
            here = [i for i in range(m) if (start + i) // page == p]
            for h in range(H):
                for side in range(2):
                    new = max([float(had[to, h, side])] + [float(had[page_of(start + ks[i]), h, side]) for i in here
                                                           if page_of(start + ks[i]) >= 0])
                    by = float(had[to, h, side]) / new
                    first = max(0, start - p * page)
                    if by < 1 and first:
                        old = was[side][to, h, :first].contiguous().view(torch.float8_e4m3fn).double()
                        sides[side][to, h, :first] = R.encode(old * by)
                    for i in here:
                        src, at = page_of(start + ks[i]), (start + i) % page
                        if src < 0:
                            sides[side][to, h, at] = 0x7f if side == 0 else 0
                            continue
                        row = was[side][src, h, (start + ks[i]) % page]
                        by = float(had[src, h, side]) / new
                        if by < 1:
                            row = R.encode(row.contiguous().view(torch.float8_e4m3fn).double() * by)
                        sides[side][to, h, at] = row
                    scales[to, h, side] = new
    n16 = page // 16
    codes[:, :, 0] = R.pack_k(sides[0].reshape(P, H, n16, 16, d))
    codes[:, :, 1] = R.pack_v(sides[1].reshape(P, H, n16, 16, d))
    return codes, scales


def same_codes(got, want):
    """Bytes are equal, but for which NaN it is."""
    g, w = got.cpu(), want.cpu()
    nan = ((g & 0x7f) == 0x7f) & ((w & 0x7f) == 0x7f)
    return bool(((g == w) | nan).all())
