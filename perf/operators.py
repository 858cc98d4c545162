"""What is measured of the attention-serving operators: rotary positions, appending to a paged 8-bit cache, and attention
over that cache.  `run` computes them in elementary torch operations, or with this repository's kernels where `own` is set.

The cache: codes [pages, kv heads, 2 (K, V), page / 16, 16 * d] in e4m3, held in blocks of 16 tokens; a block of K is
[d / 16][16 tokens][16 dims], a block of V is [d][16 tokens].  scales [pages, kv heads, 2] are powers of two, one for each
page, head and side.  A sequence's token s lives in page table[b, s // page], slot s % page.
"""
import math
import random

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E_RANGE = {"fp16": (-15, 7), "bf16": (-100, 119)}   # scale exponents: code * scale is exactly a value of the type


def listed():
    return [
        # the rotation of one step's queries for a handful of sequences: nothing but the latency of a call
        dict(name="rope_step", op="rope", dtype="fp16", tokens=8, heads=32, d=128, rot=128, interleaved=False,
             inverse=False, far=4000, scaling=1.0),
        # a long prompt's queries and keys, rotated inside the joint projection's rows (strided), positions far out
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=16385, heads=40, d=128, rot=128, interleaved=False,
             inverse=False, far=1000000, scaling=8.0),
        # the gradient's direction, interleaved pairs, a third of the head rotated
        dict(name="rope_partial_inverse", op="rope", dtype="fp16", tokens=4099, heads=12, d=192, rot=64,
             interleaved=True, inverse=True, far=30000, scaling=1.0),
        # one token of one conversation
        dict(name="append_one", op="append", dtype="fp16", batch=1, new=1, kv=1000, hq=8, hkv=2, d=64, page=16,
             rot=64, interleaved=True, ragged=False),
        # one token each of a full batch
        dict(name="append_step", op="append", dtype="bf16", batch=128, new=1, kv=2048, hq=32, hkv=8, d=128, page=64,
             rot=128, interleaved=False, ragged=True),
        # prompts of several lengths, some of them continued inside a page
        dict(name="append_prompt", op="append", dtype="bf16", batch=6, new=5000, kv=7000, hq=32, hkv=8, d=128, page=32,
             rot=128, interleaved=False, ragged=True),
        # one short conversation: latency
        dict(name="attn_one", op="attn", dtype="fp16", batch=1, new=1, kv=513, hq=8, hkv=2, d=64, page=16, cap=0.0,
             window=0, bias=False, ragged=False),
        # a serving batch with grouped heads, lengths spread
        dict(name="attn_step", op="attn", dtype="bf16", batch=64, new=1, kv=8192, hq=32, hkv=8, d=128, page=64, cap=0.0,
             window=0, bias=False, ragged=True),
        # two very long contexts: few rows, a long axis
        dict(name="attn_step_long", op="attn", dtype="bf16", batch=2, new=1, kv=131071, hq=32, hkv=4, d=128, page=128,
             cap=0.0, window=0, bias=False, ragged=False),
        # a head for every key head, capped scores, a sliding window, three speculated tokens
        dict(name="attn_step_window", op="attn", dtype="fp16", batch=24, new=3, kv=9000, hq=16, hkv=16, d=256, page=32,
             cap=30.0, window=4096, bias=False, ragged=True),
        # whole prompts
        dict(name="attn_prompt", op="attn", dtype="bf16", batch=2, new=4096, kv=4096, hq=32, hkv=8, d=128, page=64,
             cap=0.0, window=0, bias=False, ragged=False),
        # a chunk of each prompt on what the cache holds of it, scores biased by distance
        dict(name="attn_chunk", op="attn", dtype="fp16", batch=4, new=515, kv=12001, hq=16, hkv=4, d=64, page=16, cap=0.0,
             window=0, bias=True, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    dtype = rng.choice(["fp16", "bf16"])
    d = rng.choice([64, 128, 192, 256])
    rot = d if rng.random() < 0.6 else 16 * rng.randint(1, d // 16)
    if op == "rope":
        heads = _log(rng, 1, 40)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, min(16385, 16385 * 40 * 128 // (heads * d))), heads=heads, d=d,
                    rot=rot, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, far=_log(rng, 100, 1000000),
                    scaling=rng.choice([1.0, 4.0, 8.0]))
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([1, 2, 4, 5, 8])
    hq = hkv * group
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.7
    if op == "append":
        most = 0.7 * 6 * 5000 * 8 * 128 // (max(hkv, hq / 4) * d)
        batch = _log(rng, 1, 128)
        new = _log(rng, 1, max(1, min(5000, int(most / batch))))
        return dict(op=op, dtype=dtype, batch=batch, new=new, kv=new + _log(rng, 1, 4000), hq=hq, hkv=hkv, d=d, page=page,
                    rot=rot, interleaved=rng.random() < 0.5, ragged=ragged)
    bias = rng.random() < 0.25
    cap = rng.choice([0.0, 0.0, 20.0, 50.0])
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    if rng.random() < 0.6:     # a few tokens a sequence: the keys' bytes are the work
        new = rng.choice([1, 1, 1, 2, 5])
        batch = _log(rng, 1, 64)
        kv = _log(rng, 16, max(16, min(131071, 64 * 5700 * 8 * 128 // (batch * hkv * d), 2 ** 27 // (batch * hq * new))))
    else:                      # prompts: the products are the work
        batch = _log(rng, 1, 4)
        most = 4096 * 4096 * 32 * 128 / (batch * hq * d)     # pairs of a query and a key
        new = _log(rng, 16, max(16, min(4096, int(math.sqrt(most)))))
        kv = min(_log(rng, new, 32768), max(new, int(most / new)))
    return dict(op=op, dtype=dtype, batch=batch, new=new, kv=max(kv, new), hq=hq, hkv=hkv, d=d, page=page, cap=cap,
                window=window, bias=bias, ragged=ragged)


def _lengths(c):
    """(new tokens, length with them) of each sequence: all alike, or spread between about a third of the size and all of it."""
    rng = random.Random(c["batch"] * 1000003 + c["kv"] * 31 + c["new"])
    new, kv = [], []
    for b in range(c["batch"]):
        n = c["new"] if not c["ragged"] or c["new"] < 8 or b == 0 else rng.randint(c["new"] // 3, c["new"])
        before = c["kv"] - c["new"]
        k = n + (before if not c["ragged"] or b == 0 else rng.randint(before // 3, before))
        new.append(n)
        kv.append(k)
    return new, kv


def _frequencies(rot, scaling):
    """Radians a position, in 64 bits: base 10000, every wavelength stretched by `scaling`."""
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / scaling


def _turns(freq):
    """The same as 64-bit fractions of a turn, as the kernels take them."""
    return torch.round(freq / (2 * math.pi) * 2.0 ** 64).to(torch.int64)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T = DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    s = dict(case=c)
    if c["op"] == "rope":
        # the heads sit in rows of the joint projection, which also holds values that are not rotated
        rows = normal(c["tokens"], c["heads"] + 1, c["d"]).to(T)
        s["x"] = rows[:, :c["heads"]]
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device=dev, dtype=torch.int32)
        s["freq"] = _frequencies(c["rot"], c["scaling"]).to(dev)
        s["turns"] = _turns(s["freq"].cpu()).to(dev)
        s["mscale"] = 1.0 if c["scaling"] == 1.0 else 0.1 * math.log(c["scaling"]) + 1.0
        return s
    new, kv = _lengths(c)
    page, d, hkv, hq, B = c["page"], c["d"], c["hkv"], c["hq"], c["batch"]
    need = [-(-k // page) for k in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.zeros((B, max(need)), dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"] = table.to(dev)
    s["cu_q"] = torch.tensor([0] + [sum(new[:b + 1]) for b in range(B)], dtype=torch.int32).to(dev)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32).to(dev)
    s["max_q"], s["max_kv"] = max(new), max(kv)
    tokens = sum(new)
    # pages as they are in use: values of about unit variance under scales of a few neighbouring powers of two
    e = torch.randint(-7, -4, (pages, hkv, 2), generator=g, device=dev)
    s["scales"] = torch.exp2(e.float())
    codes = torch.empty((pages, hkv, 2, page // 16, 16 * d), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (hkv * 2 * page * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        codes[p:p + n] = (normal(n, hkv, 2, page // 16, 16 * d) / s["scales"][p:p + n, :, :, None, None]).clamp(
            -448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["codes"] = codes
    rows = normal(tokens, hq + 2 * hkv, d).to(T)      # the joint projection's rows: q, k, v heads
    s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    if c["op"] == "append":
        s["freq"] = _frequencies(c["rot"], 1.0).to(dev)
        s["turns"] = _turns(s["freq"].cpu()).to(dev)
        # some tokens are louder, so that pages in use have to take a larger scale
        loud = torch.rand((tokens, 1, 1), generator=g, device=dev) < 0.1
        rows *= torch.where(loud, 4.0, 1.0).to(T)
    else:
        rows *= 2.0                                   # scores spread over a few units
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=dev, dtype=torch.float32) / hq) if c["bias"] else None
    return s


# ---------------------------------------------------------------- plain forms
def _rotated(x, positions, freq, interleaved, inverse, mscale):
    """x [tokens, heads, d] in 32 bits, its first 2 * len(freq) dims rotated."""
    rot = 2 * freq.numel()
    angle = positions.double()[:, None] * freq[None]
    cos = (angle.cos() * mscale).float()[:, None]
    sin = (angle.sin() * (-mscale if inverse else mscale)).float()[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _tokens_of(s, tokens):
    """Each token's sequence and its place among the sequence's new ones."""
    at = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(s["cu_q"], at.to(torch.int32), right=True) - 1
    return b, at - s["cu_q"].long()[b]


def _plain_rope(s):
    c = s["case"]
    return _rotated(s["x"].float(), s["positions"], s["freq"], c["interleaved"], c["inverse"], s["mscale"]).to(s["x"].dtype)


def _views(codes, d):
    """K as [pages, heads, blocks, d / 16, 16 tokens, 16 dims] and V as [pages, heads, blocks, d, 16 tokens]."""
    P, H, _, n, _ = codes.shape
    return codes[:, :, 0].view(P, H, n, d // 16, 16, 16), codes[:, :, 1].view(P, H, n, d, 16)


def _plain_append(s):
    c = s["case"]
    page, d, codes, scales = c["page"], c["d"], s["codes"], s["scales"]
    tokens = s["k"].shape[0]
    b, i = _tokens_of(s, tokens)
    n_new = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    before = s["kv_lens"].long() - n_new
    slot = before[b] + i
    q = _rotated(s["q"].float(), slot, s["freq"], c["interleaved"], False, 1.0).to(s["q"].dtype)
    kv = torch.stack((_rotated(s["k"].float(), slot, s["freq"], c["interleaved"], False, 1.0), s["v"].float()), 2)
    of = s["table"].long()[b, slot // page]
    # the scale each page needs for its new tokens, and keeps of its earlier ones
    most = torch.zeros_like(scales).index_reduce_(0, of, kv.abs().amax(-1), "amax")
    lo, hi = E_RANGE[c["dtype"]]
    m, e = torch.frexp(most / 448.0)                   # most / 448 = m * 2^e, 0.5 <= m < 1
    e = torch.where(m == 0.5, e - 1, e)
    need = torch.exp2(torch.where(most > 0, e, lo).clamp(lo, hi).float())
    held = s["table"].long().gather(1, (before // page).clamp_max(s["table"].shape[1] - 1)[:, None])[:, 0]
    keeps = (before % page > 0) & (n_new > 0)
    held = torch.where(keeps, held, s["table"].long()[:, 0])
    old = scales[held].clone()
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, of, True)
    scales.copy_(torch.where(touched[:, None, None], need, scales))
    scales[held] = torch.where(keeps[:, None, None], torch.maximum(scales[held], old), scales[held])
    # earlier tokens of a page whose scale grew are rounded again
    ratio = torch.where(keeps[:, None, None], old / scales[held], 1.0)
    K, V = _views(codes, d)
    kept = (torch.arange(page, device="cuda") < (before % page)[:, None]) & keeps[:, None]
    kept = kept.view(-1, 1, page // 16, 1, 16)
    oldK, oldV = K[held], V[held]
    newK = (oldK.view(torch.float8_e4m3fn).float() * ratio[:, :, 0, None, None, None, None]).to(torch.float8_e4m3fn)
    newV = (oldV.view(torch.float8_e4m3fn).float() * ratio[:, :, 1, None, None, None]).to(torch.float8_e4m3fn)
    K[held] = torch.where(kept[..., None], newK.view(torch.uint8), oldK)
    V[held] = torch.where(kept, newV.view(torch.uint8), oldV)
    # the new ones
    new = (kv / scales[of][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    blk, tok = slot % page // 16, slot % 16
    K[of, :, blk, :, tok] = new[:, :, 0].reshape(tokens, c["hkv"], d // 16, 16)
    V[of, :, blk, :, tok] = new[:, :, 1]
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales, "q": q}


def _plain_attn(s):
    c = s["case"]
    page, d, hkv, B = c["page"], c["d"], c["hkv"], c["batch"]
    G, N = c["hq"] // hkv, s["max_q"]
    n = -(-s["max_kv"] // page)
    ids = s["table"].long()[:, :n]
    K, V = _views(s["codes"][ids.reshape(-1)], d)
    sc = s["scales"][ids.reshape(-1)]
    K = K.view(torch.float8_e4m3fn).float() * sc[:, :, 0, None, None, None, None]
    V = V.view(torch.float8_e4m3fn).float() * sc[:, :, 1, None, None, None]
    L = n * page
    K = K.view(B, n, hkv, page // 16, d // 16, 16, 16).permute(0, 2, 4, 6, 1, 3, 5).reshape(B * hkv, d, L)   # transposed
    V = V.view(B, n, hkv, page // 16, d, 16).permute(0, 2, 1, 3, 5, 4).reshape(B, hkv, L, d)
    j = torch.arange(L, device="cuda")
    V = torch.where((j < s["kv_lens"][:, None])[:, None, :, None], V, 0.0).view(B * hkv, L, d)
    n_new = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(N, device="cuda")
    at = (s["cu_q"][:-1].long()[:, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][at].float().view(B, N, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B * hkv, G * N, d)
    x = torch.bmm(q, K).mul_(1.0 / math.sqrt(d)).view(B, hkv, G, N, L)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    pos = (s["kv_lens"].long() - n_new)[:, None] + i                       # [B, N]
    gap = pos[:, :, None] - j                                              # [B, N, L]
    if s["slopes"] is not None:
        x = x.sub_(s["slopes"].view(1, hkv, G, 1, 1) * gap[:, None, None].float())
    seen = (gap >= 0) & (j < s["kv_lens"][:, None, None])
    if c["window"]:
        seen &= gap < c["window"]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B * hkv, G * N, L), V).view(B, hkv, G, N, d) / torch.where(l > 0, l, 1.0)
    b, i = _tokens_of(s, s["q"].shape[0])
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, c["hq"], d)[b, i].to(s["q"].dtype)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[c["op"]](s)
    import gemm_conv_chain_amd as fc
    if c["op"] == "rope":
        return fc.rope(s["x"], s["positions"], s["turns"], interleaved=c["interleaved"], inverse=c["inverse"],
                       mscale=s["mscale"])
    if c["op"] == "append":
        q = fc.kv_append(s["k"], s["v"], s["codes"], s["scales"], s["table"], s["cu_q"], s["kv_lens"], turns=s["turns"],
                         interleaved=c["interleaved"], q=s["q"], max_q=s["max_q"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"], "q": q}
    return fc.chain_attn(s["q"], s["codes"], s["scales"], s["table"], s["cu_q"], s["kv_lens"], causal=True,
                         softcap=c["cap"], window=c["window"], slopes=s["slopes"], max_q=s["max_q"], max_kv=s["max_kv"])


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["d"]
        return {"bytes": 4 * n + 4 * c["tokens"] + 4 * c["rot"],
                "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    new, kv = _lengths(c)
    tokens = sum(new)
    if c["op"] == "append":
        n = tokens * c["hkv"] * c["d"]
        return {"bytes": 2 * n * (2 + 1) + tokens * c["hq"] * c["d"] * 4 + sum(-(-a // c["page"]) for a in new) * c["hkv"] * 16,
                "flops": tokens * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    pairs = keys = 0
    for n, k in zip(new, kv):
        w = c["window"] or k + 1
        first = k - n                       # a query at pos sees min(pos + 1, w) keys
        short = max(0, min(n, w - 1 - first))
        pairs += short * (first + 1) + short * (short - 1) // 2 + (n - short) * w if c["window"] else n * (first + 1) + n * (n - 1) // 2
        keys += min(k, n + w - 1)
    return {"bytes": 4 * tokens * c["hq"] * c["d"] + 2 * keys * c["hkv"] * c["d"] + 8 * -(-keys // c["page"]) * c["hkv"],
            "flops": 4 * c["hq"] * c["d"] * pairs}


# ------------------------------------------------- from the definition, 64 bits
def _turn64(x, positions, freq, interleaved, sign, mscale):
    """The rotation as a product of complex numbers; x [tokens, heads, d]."""
    x, rot = x.double().clone(), 2 * freq.numel()
    part = x[..., :rot].unflatten(-1, (-1, 2) if interleaved else (2, -1))
    z = torch.complex(part[..., 0], part[..., 1]) if interleaved else torch.complex(part[..., 0, :], part[..., 1, :])
    z = z * torch.polar(torch.full_like(freq, mscale)[None], sign * positions.double()[:, None] * freq)[:, None]
    x[..., :rot] = torch.stack((z.real, z.imag), -1 if interleaved else -2).flatten(-2)
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return _turn64(s["x"], s["positions"], s["freq"], c["interleaved"], -1 if c["inverse"] else 1, s["mscale"])
    new, kv = _lengths(c)
    page, d, hkv, G = c["page"], c["d"], c["hkv"], c["hq"] // c["hkv"]
    table, at = s["table"].tolist(), 0
    if c["op"] == "append":
        lo, hi = E_RANGE[c["dtype"]]
        # codes are given as the values before their rounding to 8 bits
        codes = s["codes"].view(torch.float8_e4m3fn).double()
        scales = s["scales"].double()
        K, V = _views(codes, d)
        qs = []
        for b, (n, k) in enumerate(zip(new, kv)):
            first = k - n
            pos = torch.arange(first, k, device="cuda")
            qs.append(_turn64(s["q"][at:at + n], pos, s["freq"], c["interleaved"], 1, 1.0))
            rows = torch.stack((_turn64(s["k"][at:at + n], pos, s["freq"], c["interleaved"], 1, 1.0),
                                s["v"][at:at + n].double()))               # [2, n, hkv, d]
            at += n
            for p in range(first // page, -(-k // page)):
                a, z = max(first, p * page), min(k, (p + 1) * page)
                x, page_id = rows[:, a - first:z - first], table[b][p]
                most = x.abs().amax((1, 3)).T                              # [hkv, 2]
                e = torch.ceil(torch.log2(most / 448.0))
                e = torch.where(most > 448.0 * torch.exp2(e), e + 1, torch.where(most <= 448.0 * torch.exp2(e - 1), e - 1, e))
                scale = torch.exp2(torch.where(most > 0, e, float(lo)).clamp(lo, hi))
                if a > p * page:
                    scale = torch.maximum(scale, scales[page_id])
                    ratio = scales[page_id] / scale
                    for t in range(a - p * page):
                        K[page_id, :, t // 16, :, t % 16] *= ratio[:, 0, None, None]
                        V[page_id, :, t // 16, :, t % 16] *= ratio[:, 1, None]
                scales[page_id] = scale
                x = (x / scale.T[:, None, :, None]).clamp(-448, 448)
                slot = torch.arange(a, z, device="cuda") % page
                K[page_id, :, slot // 16, :, slot % 16] = x[0].unflatten(-1, (-1, 16))
                V[page_id, :, slot // 16, :, slot % 16] = x[1]
        return {"codes": codes, "scales": scales, "q": torch.cat(qs)}
    out = torch.zeros((sum(new), c["hq"], d), dtype=torch.float64, device="cuda")
    for b, (n, k) in enumerate(zip(new, kv)):
        ids = torch.tensor(table[b][:-(-k // page)], device="cuda")
        K, V = _views(s["codes"][ids], d)
        sc = s["scales"][ids].double()
        first = k - n
        for h in range(hkv):
            key = K[:, h].view(torch.float8_e4m3fn).double() * sc[:, h, 0, None, None, None, None]
            key = key.transpose(2, 3).reshape(-1, d)[:k]
            val = V[:, h].view(torch.float8_e4m3fn).double() * sc[:, h, 1, None, None, None]
            val = val.transpose(2, 3).reshape(-1, d)[:k]
            for i in range(0, n, 1024):
                q = s["q"][at + i:at + min(n, i + 1024), h * G:(h + 1) * G].double()
                gap = (first + i + torch.arange(q.shape[0], device="cuda"))[:, None] - torch.arange(k, device="cuda")
                x = (q.reshape(-1, d) @ key.T).unflatten(0, (-1, G)) / math.sqrt(d)
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"].double()[h * G:(h + 1) * G, None] * gap[:, None].double()
                hidden = (gap < 0) | (gap >= c["window"]) if c["window"] else gap < 0
                p = torch.softmax(x.masked_fill(hidden[:, None], -math.inf), -1)
                out[at + i:at + i + q.shape[0], h * G:(h + 1) * G] = (p.flatten(0, 1) @ val).unflatten(0, (-1, G))
        at += n
    return out
