"""Plain implementations in 64 bits of rope, kv_append and chain_attn, on the
host and straight from their definitions, with the tolerance each result is due
(test infrastructure)."""
import math

import numpy as np
import torch

E_RANGE = {torch.float16: (-15, 7), torch.bfloat16: (-100, 119)}
# subnormal spacing: below it a rounding is absolute
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ the cache
def pack_k(k):
    """[.., n, 16 tokens, d] -> [.., n, 16 * d] in a block's order."""
    *lead, n, t, d = k.shape
    return k.reshape(*lead, n, 16, d // 16, 16).transpose(-3, -2).reshape(*lead, n, 16 * d)


def unpack_k(c, d):
    *lead, n, _ = c.shape
    return c.reshape(*lead, n, d // 16, 16, 16).transpose(-3, -2).reshape(*lead, n * 16, d)


def pack_v(v):
    *lead, n, t, d = v.shape
    return v.transpose(-1, -2).reshape(*lead, n, 16 * d)


def unpack_v(c, d):
    *lead, n, _ = c.shape
    return c.reshape(*lead, n, d, 16).transpose(-1, -2).reshape(*lead, n * 16, d)


def values(codes):
    """uint8 codes -> the numbers they are (NaN codes included), float64."""
    return codes.contiguous().view(torch.float8_e4m3fn).to(torch.float64)


def page_values(codes, scales, d):
    """(K, V) [pages, hkv, page, d] in float64, scales applied."""
    K = unpack_k(values(codes[:, :, 0]), d) * scales[:, :, 0, None, None].double()
    V = unpack_v(values(codes[:, :, 1]), d) * scales[:, :, 1, None, None].double()
    return K, V


def gather(codes, scales, row, n, d):
    """Keys and values [hkv, n, d] of a sequence whose table row is `row`."""
    page = codes.shape[3] * 16
    ids = row[:-(-n // page)].long()
    K, V = page_values(codes[ids], scales[ids], d)
    return [x.permute(1, 0, 2, 3).reshape(codes.shape[1], -1, d)[:, :n] for x in (K, V)]


# ------------------------------------------------------------------------ rope
def frequencies(turns):
    return turns.double() / 2.0 ** 64   # turns a position


def rope(x, positions, turns, interleaved=False, mscale=1.0, inverse=False):
    """(result, tolerance before the output's own rounding) in float64.  The
    product position * turns is taken exactly, in integers."""
    rot = 2 * turns.numel()
    t = [int(v) for v in turns]
    frac = np.array([[(int(p) * f) % (1 << 64) for f in t] for p in positions], dtype=object)
    ang = torch.from_numpy((frac / (1 << 64)).astype(np.float64)) * (2 * math.pi)
    ang = ang.reshape(len(positions), rot // 2)
    c, s = (ang.cos() * mscale)[:, None], (ang.sin() * mscale * (-1 if inverse else 1))[:, None]
    y = x.double().clone()
    if interleaved:
        a, b = x[..., 0:rot:2].double(), x[..., 1:rot:2].double()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2].double(), x[..., rot // 2:rot].double()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    # sine and cosine are good to 1.3e-7 + the fraction's 2^-24 turn (as a 32-bit
    # float) * 2 pi, products and their sum to 3 roundings of 2^-24
    size = torch.zeros_like(y)
    m = (a.abs() + b.abs()) * abs(mscale)
    if interleaved:
        size[..., 0:rot:2], size[..., 1:rot:2] = m, m
    else:
        size[..., :rot // 2], size[..., rot // 2:rot] = m, m
    return y, size * (1.3e-7 + 2 * math.pi * 2.0 ** -25 + 3 * 2.0 ** -24)


def assert_within(got, ref, tol, what):
    g, r = got.detach().cpu().double(), ref
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), "%s: NaN in other places" % what
    inf = torch.isinf(r) | torch.isinf(g)
    assert torch.equal(g[inf], r[inf]), "%s: infinities differ" % what
    ok = ~(torch.isnan(r) | inf)
    off = (g - r).abs()[ok] - tol.expand_as(r)[ok]
    if off.numel():
        k = int(off.argmax())
        assert off.max() <= 0, "%s: off by %.3g, allowed %.3g, at a value %.4g" % (
            what, float((g - r).abs()[ok][k]), float(tol.expand_as(r)[ok][k]), float(r[ok][k]))


def rounded_tol(ref, inner, dtype):
    """The inner error, then one rounding to dtype."""
    return inner + (ref.abs() + inner) * half_step(dtype) + TINY[dtype]


# -------------------------------------------------------------------- kv_append
def need_exponent(amax, dtype):
    lo, hi = E_RANGE[dtype]
    if amax == 0:
        return lo
    m, e = math.frexp(amax / 448.0) if amax / 448.0 * 448.0 == amax else math.frexp(amax / 448.0)
    e = e - 1 if m == 0.5 else e
    while amax > 448.0 * 2.0 ** e:
        e += 1
    while amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return min(max(e, lo), hi)


def encode(x):
    """Values over their scale -> codes; saturated, NaN kept."""
    return x.clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)


def code_half_step(y):
    """Half the spacing of e4m3 at |y| (subnormal spacing 2^-9)."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    return 2.0 ** (e - 4)


def append(k, v, codes, scales, table, cu_q, kv_lens, turns=None, interleaved=False, mscale=1.0, positions=None):
    """The pool after the append, as lists of what to expect: (codes, scales,
    exact, loose) where `exact` marks bytes that have to be equal and loose =
    (value over scale, allowed distance) at the others (rotated keys)."""
    dtype, d = k.dtype, k.shape[2]
    codes, scales = codes.clone(), scales.clone()
    page = codes.shape[3] * 16
    P, H = codes.shape[:2]
    K, V = unpack_k(codes[:, :, 0], d).clone(), unpack_v(codes[:, :, 1], d).clone()   # uint8
    want = torch.zeros(K.shape, dtype=torch.float64)
    room = torch.full(K.shape, -1.0, dtype=torch.float64)      # < 0: the byte has to be equal
    for b in range(table.shape[0]):
        a, z = int(cu_q[b]), int(cu_q[b + 1])
        n = z - a
        start = int(kv_lens[b]) - n
        if n == 0:
            continue
        slots = torch.arange(start, start + n)
        pos = slots if positions is None else positions[a:z]
        if turns is None:
            kr, tol = k[a:z].double(), torch.zeros(k[a:z].shape, dtype=torch.float64)
        else:
            kr, tol = rope(k[a:z], pos.tolist(), turns, interleaved, mscale)
        for p in range(max(start, 0) // page, (start + n - 1) // page + 1):
            if p >= table.shape[1] or not 0 <= int(table[b, p]) < P:
                continue
            pid = int(table[b, p])
            here = (slots >= p * page) & (slots < (p + 1) * page) & (slots >= 0)
            first = int(slots[here][0]) - p * page
            ts = slots[here] - p * page
            for h in range(H):
                for side, rows in ((0, kr[here][:, h]), (1, v[a:z][here][:, h].double())):
                    fin = rows[torch.isfinite(rows)].abs()
                    amax = float(fin.max()) if fin.numel() else 0.0
                    e = need_exponent(amax, dtype)
                    old = float(scales[pid, h, side])
                    if first > 0 and 2.0 ** e < old:
                        e = int(round(math.log2(old)))
                    s = 2.0 ** e
                    side_codes = K if side == 0 else V
                    if first > 0 and s > old:
                        kept = side_codes[pid, h, :first].contiguous().view(torch.float8_e4m3fn).double() * (old / s)
                        side_codes[pid, h, :first] = encode(kept)
                    scales[pid, h, side] = s
                    y = rows / s
                    if side == 1:
                        y = torch.where(torch.isnan(y), 0.0, y)
                    K_nan = torch.isnan(v[a:z][here][:, h]).any(-1)
                    if side == 0:
                        y[K_nan, 0] = math.nan
                    side_codes[pid, h, ts] = encode(y)
                    if side == 0 and turns is not None:
                        want[pid, h, ts] = y.clamp(-448, 448)
                        room[pid, h, ts] = torch.where(torch.isfinite(y), code_half_step(y) * (1 + 2.0 ** -20) +
                                                       tol[here][:, h] / s, -1.0)
    n = page // 16
    codes[:, :, 0] = pack_k(K.reshape(P, H, n, 16, d))
    codes[:, :, 1] = pack_v(V.reshape(P, H, n, 16, d))
    return codes, scales, want, room


def assert_appended(got_codes, got_scales, expect, what):
    codes, scales, want, room = expect
    d = want.shape[-1]
    gc, gs = got_codes.cpu(), got_scales.cpu()
    assert torch.equal(gs, scales), "%s: scales differ at %s" % (what, (gs != scales).nonzero()[:4].tolist())
    assert torch.equal(gc[:, :, 1], codes[:, :, 1]), "%s: V codes differ" % what
    g, e = unpack_k(gc[:, :, 0], d), unpack_k(codes[:, :, 0], d)
    strict = room < 0
    nan = ((g & 0x7f) == 0x7f) & ((e & 0x7f) == 0x7f)
    bad = (g != e) & strict & ~nan
    assert not bad.any(), "%s: %d K codes differ, first at %s" % (what, int(bad.sum()), bad.nonzero()[0].tolist())
    off = (values(g) - want).abs() - room
    assert not (off[~strict] > 0).any(), "%s: a K code is %.3g further from its value than a rounding" % (
        what, float(off[~strict].max()))


# ------------------------------------------------------------------- chain_attn
def attention(q, codes, scales, table, cu_q, kv_lens, scale=None, causal=True, softcap=0.0, window=0, slopes=None):
    """(out, tolerance before the output's rounding, lse, lse tolerance)."""
    T, hq, d = q.shape
    hkv = codes.shape[1]
    G = hq // hkv
    u = half_step(q.dtype)
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros((T, hq, d), dtype=torch.float64)
    tol = torch.zeros((T, hq, d), dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros((T, hq), dtype=torch.float64)
    for b in range(table.shape[0]):
        a, z = int(cu_q[b]), int(cu_q[b + 1])
        n, L = z - a, int(kv_lens[b])
        if n == 0 or L == 0:
            continue
        K, V = gather(codes, scales, table[b], L, d)
        j = torch.arange(L)
        pos = torch.arange(L - n, L)
        gap = pos[:, None] - j
        seen = torch.ones((n, L), dtype=torch.bool)
        if causal:
            seen = gap >= 0
        if window:
            seen = seen & (gap < window)
        for h in range(hq):
            qq = q[a:z, h].double()
            x = qq @ K[h // G].T * scale
            # fp32 accumulation of d exact products, and the scale's own roundings
            dx = (d + 4) * 2.0 ** -24 * scale * (qq.abs() @ torch.nan_to_num(K[h // G].abs()).T)
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                dx = dx + softcap * 2.0 ** -21
            if slopes is not None:
                bias = float(slopes[h]) * gap.abs()
                x = x - bias
                dx = dx + bias * 2.0 ** -22
            dx = dx + x.abs() * 2.0 ** -22       # to units of log 2, and the exponential's argument
            x = x.masked_fill(~seen, -math.inf)
            m = x.amax(-1, keepdim=True)
            some = seen.any(-1)
            p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
            l = p.sum(-1, keepdim=True)
            w = p / torch.where(l == 0, 1.0, l)
            vv = torch.where(seen.any(0)[:, None], V[h // G], 0.0)
            out[a:z, h] = w @ vv
            err = torch.where(seen, dx, 0.0).amax(-1, keepdim=True) + 2.0 ** -20
            A = w @ vv.abs()
            tol[a:z, h] = A * (u + 2 * err) + TINY[q.dtype] * (seen.double() @ vv.abs())
            lse[a:z, h] = torch.where(some, (m + torch.log(l))[:, 0], -math.inf)
            ltol[a:z, h] = err[:, 0] + 2.0 ** -22 * lse[a:z, h].abs().nan_to_num(0, 0, 0)
    return out, tol, lse, ltol
