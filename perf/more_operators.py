"""What is measured of the speculative-decoding operators over the paged 8-bit cache: attention of a tree of drafted tokens,
drawing tokens from logits, the tree's bookkeeping, keeping the accepted tokens of a draft, and copying pages.  `run`
computes them in elementary torch operations, or with this repository's kernels where `own` is set.

The cache: codes [layers, pages, kv heads, 2 (K, V), page / 16, 16 * d] in e4m3, held in blocks of 16 tokens; a block of K is
[d / 16][16 tokens][16 dims], a block of V is [d][16 tokens].  scales [layers, pages, kv heads, 2] are powers of two, one for
each page, head and side.  A sequence's token s lives in page table[b, s // page], slot s % page; the last cu_q[b + 1] -
cu_q[b] of its kv_lens[b] tokens are the step's new ones, the nodes of its tree.  A node's parent is an earlier node of the
same sequence, or -1.
"""
import math
import random

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one conversation with a handful of drafted tokens: latency
        dict(name="tree_attn_one", op="attn", dtype="fp16", batch=1, nodes=8, kv=513, hq=8, hkv=2, d=64, page=16, cap=0.0,
             window=0, bias=False, ragged=False),
        # a serving batch with grouped heads, lengths and trees spread
        dict(name="tree_attn_step", op="attn", dtype="bf16", batch=32, nodes=26, kv=8192, hq=32, hkv=8, d=128, page=64,
             cap=0.0, window=0, bias=False, ragged=True),
        # two long contexts with wide trees
        dict(name="tree_attn_long", op="attn", dtype="fp16", batch=2, nodes=60, kv=100001, hq=32, hkv=4, d=128, page=128,
             cap=0.0, window=0, bias=False, ragged=False),
        # the next token of one conversation
        dict(name="sample_one", op="sample", dtype="fp16", rows=1, vocab=32000, temperature=0.8, top_k=0, top_p=0.95,
             min_p=0.0, mixed=False, masked=0.0),
        # a full batch over a large vocabulary, the whole distribution
        dict(name="sample_step", op="sample", dtype="bf16", rows=128, vocab=131072, temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, mixed=False, masked=0.0),
        # every node of a batch of trees, each request with its own settings, an odd vocabulary with tokens shut out
        dict(name="sample_tree", op="sample", dtype="fp32", rows=832, vocab=100003, temperature=0.7, top_k=50, top_p=0.9,
             min_p=0.05, mixed=True, masked=0.1),
        # the bookkeeping around a step: of one small tree, and of a large batch of wide ones
        dict(name="tree_one", op="tree", batch=1, nodes=8, ragged=False),
        dict(name="tree_batch", op="tree", batch=512, nodes=64, ragged=True),
        # the accepted tokens of one conversation, one layer
        dict(name="keep_one", op="keep", dtype="fp16", batch=1, nodes=8, kv=200, hkv=2, d=64, page=16, layers=1,
             ragged=False),
        # a batch, all layers of a model in one call
        dict(name="keep_layers", op="keep", dtype="bf16", batch=32, nodes=26, kv=300, hkv=8, d=128, page=32, layers=8,
             ragged=True),
        # a conversation forked: its last, partly filled page
        dict(name="copy_fork", op="copy", dtype="fp16", pairs=1, pages=40, hkv=2, d=64, page=16, layers=1),
        # a pool packed together: many pages of all layers
        dict(name="copy_pack", op="copy", dtype="bf16", pairs=401, pages=1000, hkv=8, d=128, page=64, layers=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "sample", "sample", "tree", "keep", "copy"])
    dtype = rng.choice(["fp16", "bf16"])
    d = rng.choice([64, 128, 192, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.7
    if op == "attn":
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        batch, nodes = _log(rng, 1, 32), _log(rng, 1, 128)
        most = min(2 * 100001 * 4 * 128 // (batch * hkv * d), 2 * 60 * 100001 * 32 * 128 // (batch * nodes * hq * d))
        kv = nodes + _log(rng, 1, max(1, min(100001, most) - nodes))
        return dict(op=op, dtype=dtype, batch=batch, nodes=nodes, kv=kv, hq=hq, hkv=hkv, d=d, page=page,
                    cap=rng.choice([0.0, 0.0, 0.0, 30.0]), window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
                    bias=rng.random() < 0.2, ragged=ragged)
    if op == "sample":
        dtype = rng.choice(["fp16", "bf16", "fp32"])
        vocab = _log(rng, 100, 262144)
        rows = _log(rng, 1, max(1, min(832, 832 * 100003 // vocab // 2)))
        return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, temperature=rng.choice([0.0, 0.5, 0.8, 1.0, 1.3]),
                    top_k=rng.choice([0, 0, _log(rng, 1, 1000)]), top_p=rng.choice([1.0, 0.5, 0.9, 0.99]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.4,
                    masked=rng.choice([0.0, 0.0, 0.3]))
    if op == "tree":
        batch = _log(rng, 1, 512)
        return dict(op=op, batch=batch, nodes=_log(rng, 1, max(1, min(128, 512 * 64 // batch))), ragged=ragged)
    if op == "keep":
        batch, nodes, layers = _log(rng, 1, 32), _log(rng, 1, 64), rng.randint(1, 8)
        kv = nodes + _log(rng, 1, 300)
        while layers * batch * (kv + page) * hkv * d > 8 * 32 * 332 * 8 * 128 and layers * batch > 1:
            layers, batch = (layers - 1, batch) if layers > 1 else (1, batch - 1)
        return dict(op=op, dtype=dtype, batch=batch, nodes=nodes, kv=kv, hkv=hkv, d=d, page=page, layers=layers, ragged=ragged)
    layers = rng.randint(1, 8)
    pairs = _log(rng, 1, max(1, min(401, 401 * 8 * 8 * 128 * 64 // (layers * hkv * d * page))))
    return dict(op=op, dtype=dtype, pairs=pairs, pages=2 * pairs + rng.randint(1, 40), hkv=hkv, d=d, page=page, layers=layers)


def _lengths(c):
    """(nodes, length with them) of each sequence: all alike, or spread between about a third of the size and all of it."""
    rng = random.Random(c["batch"] * 1000003 + c["nodes"] * 31 + c.get("kv", 0))
    before = c.get("kv", 900) - c["nodes"]
    new, kv = [], []
    for b in range(c["batch"]):
        n = c["nodes"] if not c["ragged"] or b == 0 else rng.randint(-(-c["nodes"] // 3), c["nodes"])
        new.append(n)
        kv.append(n + (before if not c["ragged"] or b == 0 else rng.randint(before // 3, before)))
    return new, kv


def _parents(rng, n):
    """A tree as drafters grow them: each new node under one of the latest few, or anywhere."""
    return [-1] + [rng.randint(max(0, i - 6), i - 1) if rng.random() < 0.6 else rng.randint(0, i - 1) for i in range(1, n)]


def _path_lengths(c):
    """How many nodes of each sequence are kept: a few, as drafts fare."""
    rng = random.Random(c["batch"] * 7 + c["nodes"])
    return [min(n, 1 + rng.randint(0, 5)) for n in _lengths(c)[0]]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32)

    s = dict(case=c)
    if c["op"] == "sample":
        R, V = c["rows"], c["vocab"]
        x = normal(R, V).mul_(2.0)
        # a few dozen tokens stand out of each row, some of them far
        at = torch.randint(0, V, (R, 40), generator=g, device=dev)
        x.scatter_add_(1, at, 4.0 - 2.5 * torch.log(uniform(R, 40).clamp_min(1e-6)))
        if c["masked"]:
            x[uniform(R, V) < c["masked"]] = -math.inf
            x[:, 0] = 0.0
        s["logits"], s["u"] = x.to(DT[c["dtype"]]), uniform(R)
        s["set"] = {k: c[k] for k in ("temperature", "top_k", "top_p", "min_p")}
        if c["mixed"]:
            def some(values, dtype):
                return torch.tensor([rng.choice(values) for _ in range(R)], dtype=dtype).to(dev)
            s["set"] = dict(temperature=some([0.0, c["temperature"], c["temperature"], 1.0, 1.2], torch.float32),
                            top_k=some([0, c["top_k"], c["top_k"], 20], torch.int32),
                            top_p=some([1.0, c["top_p"], 0.8], torch.float32),
                            min_p=some([0.0, 0.0, c["min_p"]], torch.float32))
        return s
    if c["op"] == "copy":
        new = kv = need = []
        pages = c["pages"]
        order = torch.randperm(pages, generator=g, device=dev).tolist()
        s["pairs"] = [(order[2 * i], order[2 * i + 1]) for i in range(c["pairs"])]
    else:
        new, kv = _lengths(c)
        s["cu_q"], s["kv_lens"] = _i32([sum(new[:b]) for b in range(len(new) + 1)]), _i32(kv)
        s["max_q"], s["max_kv"] = max(new), max(kv)
    tokens = sum(new)
    if c["op"] == "tree" or c["op"] == "attn":
        trees = [_parents(rng, n) for n in new]
        s["parents"] = _i32(sum(trees, []))
    if c["op"] == "tree":
        drafted, targets = [], []
        for p in trees:
            t = [rng.randint(0, 50000) for _ in p]
            first = {}
            for i, a in enumerate(p):
                first.setdefault(a, i)
            # the model agrees with a drafted child, or goes elsewhere
            targets += [t[first[i]] if i in first and rng.random() < 0.8 else rng.randint(0, 50000) for i in range(len(p))]
            drafted += t
        s["drafted"], s["targets"] = _i32(drafted), _i32(targets)
        return s
    page, d, hkv, L = c["page"], c["d"], c["hkv"], c.get("layers", 1)
    if c["op"] != "copy":
        need = [-(-k // page) for k in kv]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
        table = torch.zeros((len(kv), max(need)), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table.to(dev)
    # pages as they are in use: values of about unit variance under scales of a few neighbouring powers of two
    s["scales"] = torch.exp2(torch.randint(-7, -4, (L, pages, hkv, 2), generator=g, device=dev).float())
    codes = torch.empty((L, pages, hkv, 2, page // 16, 16 * d), dtype=torch.uint8, device=dev)
    flat, scale = codes.view(L * pages, hkv, 2, page // 16, 16 * d), s["scales"].view(L * pages, hkv, 2)
    step = max(1, (1 << 26) // (hkv * 2 * page * d))
    for p in range(0, L * pages, step):
        n = min(step, L * pages - p)
        flat[p:p + n] = (normal(n, hkv, 2, page // 16, 16 * d) / scale[p:p + n, :, :, None, None]).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
    s["codes"] = codes
    if c["op"] == "keep":
        keep = torch.full((len(new), max(new)), -1, dtype=torch.int32)
        kept = _path_lengths(c)
        for b, (n, k) in enumerate(zip(new, kept)):
            keep[b, :k] = torch.tensor([0] + sorted(rng.sample(range(1, n), k - 1)), dtype=torch.int32)
        s["keep"], s["kept"] = keep.to(dev), _i32(kept)
    if c["op"] == "attn":
        rows = normal(tokens, c["hq"] + 2 * hkv, d) * 2.0     # the joint projection's rows; scores spread over a few units
        s["q"] = rows.to(DT[c["dtype"]])[:, :c["hq"]]
        # what a program makes once a step of its trees, for the attention of all its layers: the nodes that each sees, a
        # bit each (its ancestors and itself), and each one's position (its depth past what came before)
        seen = torch.zeros((tokens, 64 * -(-max(new) // 64)), dtype=torch.int64)
        place, at = [], 0
        for p, k in zip(trees, kv):
            depth = []
            for i, a in enumerate(p):
                if a >= 0:
                    seen[at + i] = seen[at + a]
                seen[at + i, i] = 1
                depth.append(0 if a < 0 else depth[a] + 1)
            place += [k - len(p) + x for x in depth]
            at += len(p)
        weights = torch.tensor([1 << i if i < 63 else -(1 << 63) for i in range(64)])
        s["tree"] = ((seen.view(tokens, -1, 64) * weights).sum(-1).cuda(), _i32(place))
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["hq"] + 1, device=dev, dtype=torch.float32) / c["hq"]) if c["bias"] else None
    return s


# ---------------------------------------------------------------- plain forms
def _views(codes, d):
    """K as [.., pages, heads, blocks, d / 16, 16 tokens, 16 dims] and V as [.., pages, heads, blocks, d, 16 tokens]."""
    lead, n = codes.shape[:-3], codes.shape[-2]
    return codes[..., 0, :, :].view(*lead, n, d // 16, 16, 16), codes[..., 1, :, :].view(*lead, n, d, 16)


def _seen(s):
    """Which of its sequence's nodes each node sees, as truth values [tokens, 64 * words]."""
    bits = s["tree"][0]
    return ((bits[..., None] >> torch.arange(64, device="cuda")) & 1).bool().flatten(1)


def _plain_attn(s):
    c = s["case"]
    page, d, hkv, B = c["page"], c["d"], c["hkv"], c["batch"]
    G, N = c["hq"] // hkv, s["max_q"]
    n = -(-s["max_kv"] // page)
    ids = s["table"].long()[:, :n]
    K, V = _views(s["codes"][0, ids.reshape(-1)], d)
    sc = s["scales"][0, ids.reshape(-1)]
    K = K.view(torch.float8_e4m3fn).float() * sc[:, :, 0, None, None, None, None]
    V = V.view(torch.float8_e4m3fn).float() * sc[:, :, 1, None, None, None]
    L = n * page
    K = K.view(B, n, hkv, page // 16, d // 16, 16, 16).permute(0, 2, 4, 6, 1, 3, 5).reshape(B * hkv, d, L)   # transposed
    V = V.view(B, n, hkv, page // 16, d, 16).permute(0, 2, 1, 3, 5, 4).reshape(B, hkv, L, d)
    j = torch.arange(L, device="cuda")
    V = torch.where((j < s["kv_lens"][:, None])[:, None, :, None], V, 0.0).view(B * hkv, L, d)
    n_new = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    start = s["kv_lens"].long() - n_new
    at = (s["cu_q"][:-1].long()[:, None] + torch.arange(N, device="cuda")).clamp_max(s["q"].shape[0] - 1)      # [B, N]
    q = s["q"][at].float().view(B, N, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B * hkv, G * N, d)
    x = torch.bmm(q, K).mul_(1.0 / math.sqrt(d)).view(B, hkv, G, N, L)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    # a slot before the tree is at its own position and seen, one of the tree where and if the tree says
    node = j - start[:, None]                                              # [B, L]
    inside = (node >= 0) & (j < s["kv_lens"][:, None])
    which = node.clamp(0, N - 1)
    place = s["tree"][1].long()[at]                                        # [B, N]
    key = torch.where(inside, place.gather(1, which), j)
    gap = place[:, :, None] - key[:, None]                                 # [B, N, L]
    if s["slopes"] is not None:
        x = x.sub_(s["slopes"].view(1, hkv, G, 1, 1) * gap[:, None, None].float().abs())
    seen = _seen(s)[at].gather(2, which[:, None].expand(B, N, L)) & inside[:, None] | (node < 0)[:, None]
    if c["window"]:
        seen &= gap < c["window"]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B * hkv, G * N, L), V).view(B, hkv, G, N, d) / torch.where(l > 0, l, 1.0)
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"], t.to(torch.int32), right=True) - 1
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, c["hq"], d)[b, t - s["cu_q"].long()[b]].to(s["q"].dtype)


def _settings(s):
    """temperature, top_k, top_p, min_p as [rows, 1]; the fractions as the 32-bit numbers that they are, in 64 bits."""
    R = s["case"]["rows"]

    def column(v, dtype):
        v = v if isinstance(v, torch.Tensor) else torch.full((R,), v, dtype=dtype, device="cuda")
        return v[:, None]
    p = s["set"]
    return (column(p["temperature"], torch.float32).double(), column(p["top_k"], torch.int32).long(),
            column(p["top_p"], torch.float32).double(), column(p["min_p"], torch.float32).double())


def _plain_sample(s):
    """In 64 bits: a sum of 100000 weights next to the border that the random number draws."""
    T, k, top_p, min_p = _settings(s)
    x, order = s["logits"].double().sort(dim=1, descending=True, stable=True)
    w = ((x - x[:, :1]) / torch.where(T > 0, T, 1.0)).exp_()
    rank = torch.arange(x.shape[1], device="cuda")
    w = torch.where((rank < k) | (k <= 0), w, 0.0)
    total = w.cumsum(1)
    stays = (total - w < top_p * total[:, -1:]) | (top_p >= 1.0) | (rank == 0)
    w = torch.where(stays & (w >= min_p), w, 0.0)
    total = torch.zeros_like(w).scatter_(1, order, w).cumsum_(1)
    token = (total <= s["u"].double()[:, None] * total[:, -1:]).sum(1)
    return torch.where(T[:, 0] > 0, token, order[:, 0]).int()


def _plain_tree(s):
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    B, N, T = len(new), s["max_q"], s["parents"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["cu_q"], t.int(), right=True) - 1
    node = (t - s["cu_q"][b]).long()
    # all nodes step from parent to parent together
    seen = torch.zeros((T, 64 * -(-N // 64)), dtype=torch.bool, device="cuda")
    depth = torch.zeros_like(t)
    up = node
    for _ in range(N):
        live = up >= 0
        at = up.clamp_min(0)
        seen.scatter_(1, at[:, None], (seen.gather(1, at[:, None])[:, 0] | live)[:, None])
        up = torch.where(live, s["parents"].long()[s["cu_q"].long()[b] + at], -1)
        depth += up >= 0
    one = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(64, device="cuda")
    bits = (seen.view(T, -1, 64) * one).sum(-1)
    start = s["kv_lens"] - new
    positions = (start[b] + depth).int()
    # and all sequences from accepted node to accepted node
    keep = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    kept = torch.zeros(B, dtype=torch.int64, device="cuda")
    now = torch.zeros(B, dtype=torch.int64, device="cuda")
    going = new > 0
    first = s["cu_q"][:-1].long()
    for i in range(N):
        keep[:, i] = torch.where(going, now.int(), -1)
        kept += going
        want = s["targets"][(first + now).clamp_max(T - 1)]
        fits = (s["parents"] == now[b]) & (s["drafted"] == want[b]) & going[b]
        nxt = torch.full((B,), N, dtype=torch.int64, device="cuda").scatter_reduce_(0, b, torch.where(fits, node, N), "amin")
        going = going & (nxt < N)
        now = torch.where(going, nxt, now)
    token = torch.where(new > 0, s["targets"][(first + now).clamp_max(T - 1)], -1)
    return dict(bits=bits, positions=positions, keep=keep, kept=kept.int(), next=token.int(), lens=(start + kept).int())


def _plain_keep(s):
    c = s["case"]
    page, d, codes, scales = c["page"], c["d"], s["codes"], s["scales"]
    K, V = _views(codes, d)
    B, N = s["keep"].shape
    start = s["kv_lens"].long() - (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(N, device="cuda")
    b = torch.arange(B, device="cuda")[:, None].expand(B, N)
    live = i < s["kept"][:, None]
    b, to, src = b[live], (start[:, None] + i)[live], (start[:, None] + s["keep"].long())[live]
    page_to, page_from = s["table"].long()[b, to // page], s["table"].long()[b, src // page]
    old = scales.clone()
    scales.index_reduce_(1, page_to, old[:, page_from], "amax")
    # what came before in a page whose scale grew is rounded again
    ratio = old / scales
    first = torch.full((codes.shape[1],), page, dtype=torch.int64, device="cuda")
    first = torch.zeros_like(first).scatter_reduce_(0, page_to, (start[b] - to // page * page).clamp(0, page), "amax")
    touched = first.nonzero()[:, 0]
    before = (torch.arange(page, device="cuda") < first[touched][:, None]).view(-1, 1, page // 16, 1, 16)
    rk, rv = ratio[:, touched, :, 0, None, None, None, None], ratio[:, touched, :, 1, None, None, None]
    oldK, oldV = K[:, touched], V[:, touched]
    newK = (oldK.view(torch.float8_e4m3fn).float() * rk).to(torch.float8_e4m3fn).view(torch.uint8)
    newV = (oldV.view(torch.float8_e4m3fn).float() * rv).to(torch.float8_e4m3fn).view(torch.uint8)
    # (all sources are read before anything is written)
    blk, tok = src % page // 16, src % 16
    by = (old[:, page_from] / scales[:, page_to])
    moveK = K[:, page_from, :, blk, :, tok].view(torch.float8_e4m3fn).float()        # [tokens, layers, heads, d / 16, 16]
    moveV = V[:, page_from, :, blk, :, tok].view(torch.float8_e4m3fn).float()        # [tokens, layers, heads, d]
    by = by.transpose(0, 1)
    moveK = (moveK * by[..., 0, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    moveV = (moveV * by[..., 1, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    K[:, touched] = torch.where(before[..., None], newK, oldK)
    V[:, touched] = torch.where(before, newV, oldV)
    blk, tok = to % page // 16, to % 16
    K[:, page_to, :, blk, :, tok] = moveK
    V[:, page_to, :, blk, :, tok] = moveV
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}


def _plain_copy(s):
    src, to = torch.tensor(s["pairs"]).cuda().T
    s["codes"][:, to] = s["codes"][:, src]
    s["scales"][:, to] = s["scales"][:, src]
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"attn": _plain_attn, "sample": _plain_sample, "tree": _plain_tree, "keep": _plain_keep,
                "copy": _plain_copy}[c["op"]](s)
    import gemm_conv_chain_amd as fc
    if c["op"] == "attn":
        return fc.chain_attn(s["q"], s["codes"][0], s["scales"][0], s["table"], s["cu_q"], s["kv_lens"], tree=s["tree"],
                             softcap=c["cap"], window=c["window"], slopes=s["slopes"], max_q=s["max_q"], max_kv=s["max_kv"])
    if c["op"] == "sample":
        return fc.sample_tokens(s["logits"], s["u"], **s["set"])
    if c["op"] == "tree":     # the call before a step's layers and the one behind them
        bits, positions = fc.tree_plan(s["parents"], s["cu_q"], s["kv_lens"], max_q=s["max_q"])
        keep, kept, token, lens = fc.tree_accept(s["parents"], s["drafted"], s["targets"], s["cu_q"], s["kv_lens"],
                                                 max_q=s["max_q"])
        return dict(bits=bits, positions=positions, keep=keep, kept=kept, next=token, lens=lens)
    if c["op"] == "keep":
        fc.kv_keep(s["codes"], s["scales"], s["table"], s["cu_q"], s["kv_lens"], s["keep"], s["kept"])
    else:
        fc.kv_copy(s["codes"], s["scales"], s["pairs"])
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def work(case):
    c = case
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * DT[c["dtype"]].itemsize + 8 * c["rows"] + (16 * c["rows"] if c["mixed"] else 0), "flops": 3 * n}
    if c["op"] == "copy":
        return {"bytes": 2 * c["pairs"] * c["layers"] * c["hkv"] * 2 * (c["page"] * c["d"] + 4), "flops": 0}
    new, kv = _lengths(c)
    tokens = sum(new)
    if c["op"] == "tree":
        words = -(-max(new) // 64)
        return {"bytes": tokens * (4 + 8 * words + 4) + tokens * 12 + c["batch"] * (8 + 4 * max(new) + 12), "flops": 0}
    if c["op"] == "keep":
        moved = sum(k - 1 for k in _path_lengths(c)) * c["layers"] * c["hkv"] * 2     # (node 0 stays where it is)
        return {"bytes": 2 * moved * c["d"] + sum(_path_lengths(c)) * 4 + 12 * c["batch"], "flops": moved * c["d"]}
    before = [min(k - n, c["window"] or k) for n, k in zip(new, kv)]
    keys = sum(before) + tokens
    pairs = sum(n * a for n, a in zip(new, before)) + 2 * tokens     # a node sees itself and its root at least
    return {"bytes": 4 * tokens * c["hq"] * c["d"] + 2 * keys * c["hkv"] * c["d"] + 8 * -(-keys // c["page"]) * c["hkv"] +
            tokens * (4 + 8 * -(-max(new) // 64)), "flops": 4 * c["hq"] * c["d"] * pairs}


# ------------------------------------------------- from the definition, 64 bits
def _exact_sample(s):
    """Row by row: the tokens that stay are those over a value, and of those at it the first few."""
    T, k, top_p, min_p = (v[:, 0].tolist() for v in _settings(s))
    out = []
    for r, u in enumerate(s["u"].tolist()):
        x = s["logits"][r].double()
        if T[r] <= 0:
            out.append(int((x == x.max()).nonzero()[0, 0]))
            continue
        w = torch.exp((x - x.max()) / T[r])
        if 0 < k[r] < len(x):
            least = torch.topk(x, k[r]).values[-1]
            over, at = x > least, (x == least).nonzero()[:, 0]
            over[at[:k[r] - int(over.sum())]] = True
            w = torch.where(over, w, 0.0)
        if top_p[r] < 1.0:
            value, many = torch.unique(x[w > 0], return_counts=True)
            value, many = value.flip(0), many.flip(0)
            mass = torch.exp((value - x.max()) / T[r])
            goal = top_p[r] * float((mass * many).sum())
            upto = torch.cumsum(mass * many, 0)
            i = min(int((upto < goal).sum()), len(value) - 1)
            ahead = float(upto[i - 1]) if i else 0.0
            n = min(max(math.ceil((goal - ahead) / float(mass[i])), 1 if i == 0 else 0), int(many[i]))
            at = ((x == value[i]) & (w > 0)).nonzero()[:, 0]
            stay = (x > value[i]) & (w > 0)
            stay[at[:n]] = True
            w = torch.where(stay, w, 0.0)
        w = torch.where(w >= min_p[r], w, 0.0)
        where = (w > 0).nonzero()[:, 0]
        upto = torch.cumsum(w[where], 0)
        out.append(int(where[min(int((upto <= u * float(upto[-1])).sum()), len(where) - 1)]))
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _exact_tree(s):
    cu, lens = s["cu_q"].tolist(), s["kv_lens"].tolist()
    parents, drafted, targets = s["parents"].tolist(), s["drafted"].tolist(), s["targets"].tolist()
    words = -(-s["max_q"] // 64)
    bits, place, keep, kept, token, after = [], [], [], [], [], []
    for b, n in enumerate(lens):
        p, dr, tg = (v[cu[b]:cu[b + 1]] for v in (parents, drafted, targets))
        sets, child = [], {}
        for i, a in enumerate(p):
            sets.append((sets[a] if a >= 0 else 0) | 1 << i)
            child.setdefault((a, dr[i]), i)
            place.append(n - len(p) + bin(sets[i]).count("1") - 1)
            word = [sets[i] >> 64 * w & (1 << 64) - 1 for w in range(words)]
            bits.append([v - (1 << 64) if v >> 63 else v for v in word])
        path = [0] if p else []
        while path and (path[-1], tg[path[-1]]) in child:
            path.append(child[path[-1], tg[path[-1]]])
        keep.append(path + [-1] * (s["max_q"] - len(path)))
        kept.append(len(path))
        token.append(tg[path[-1]] if p else -1)
        after.append(n - len(p) + len(path))
    return dict(bits=torch.tensor(bits).cuda(), positions=_i32(place), keep=_i32(keep), kept=_i32(kept), next=_i32(token),
                lens=_i32(after))


def _exact_keep(s):
    """Codes are given as the values before their rounding to 8 bits."""
    c = s["case"]
    page, d = c["page"], c["d"]
    codes, scales = s["codes"].view(torch.float8_e4m3fn).double(), s["scales"].double()
    was, had = codes.clone(), scales.clone()
    K, V = _views(codes, d)
    wasK, wasV = _views(was, d)
    cu, lens, keep, kept, table = (s[k].tolist() for k in ("cu_q", "kv_lens", "keep", "kept", "table"))
    for b, n in enumerate(lens):
        start = n - (cu[b + 1] - cu[b])
        moves = [(start + i, start + keep[b][i]) for i in range(kept[b])]
        for p in sorted({to // page for to, _ in moves}):
            here = [(to, src) for to, src in moves if to // page == p]
            pid = table[b][p]
            new = had[:, pid]
            for _, src in here:
                new = torch.maximum(new, had[:, table[b][src // page]])
            scales[:, pid] = new
            old = torch.arange(max(0, min(page, start - p * page)), device="cuda")
            if len(old):
                by = (had[:, pid] / new)[None]
                K[:, pid, :, old // 16, :, old % 16] = wasK[:, pid, :, old // 16, :, old % 16] * by[..., 0, None, None]
                V[:, pid, :, old // 16, :, old % 16] = wasV[:, pid, :, old // 16, :, old % 16] * by[..., 1, None]
            for to, src in here:
                sid, x, y = table[b][src // page], src % page, to % page
                by = had[:, sid] / new
                K[:, pid, :, y // 16, :, y % 16] = wasK[:, sid, :, x // 16, :, x % 16] * by[:, :, 0, None, None]
                V[:, pid, :, y // 16, :, y % 16] = wasV[:, sid, :, x // 16, :, x % 16] * by[:, :, 1, None]
    return {"codes": codes, "scales": scales}


def _exact_copy(s):
    codes, scales = s["codes"].view(torch.float8_e4m3fn).double(), s["scales"].double()
    for a, b in s["pairs"]:
        codes[:, b] = s["codes"][:, a].view(torch.float8_e4m3fn).double()
        scales[:, b] = s["scales"][:, a].double()
    return {"codes": codes, "scales": scales}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] != "attn":
        return {"sample": _exact_sample, "tree": _exact_tree, "keep": _exact_keep, "copy": _exact_copy}[c["op"]](s)
    new, kv = _lengths(c)
    page, d, hkv, G = c["page"], c["d"], c["hkv"], c["hq"] // c["hkv"]
    table, at = s["table"].tolist(), 0
    parents, place = s["parents"].tolist(), s["tree"][1].tolist()
    out = torch.zeros((sum(new), c["hq"], d), dtype=torch.float64, device="cuda")
    for b, (n, k) in enumerate(zip(new, kv)):
        ids = torch.tensor(table[b][:-(-k // page)], device="cuda")
        K, V = _views(s["codes"][0, ids], d)
        sc = s["scales"][0, ids].double()
        hidden = torch.ones((n, k), dtype=torch.bool)
        hidden[:, :k - n] = False
        for i in range(n):
            a = i
            while a >= 0:
                hidden[i, k - n + a] = False
                a = parents[at + a]
        where = torch.tensor(place[at:at + n])
        gap = where[:, None] - torch.cat((torch.arange(k - n), where))
        if c["window"]:
            hidden |= gap >= c["window"]
        hidden, gap = hidden.cuda(), gap.cuda().double().abs()
        for h in range(hkv):
            key = K[:, h].view(torch.float8_e4m3fn).double() * sc[:, h, 0, None, None, None, None]
            key = key.transpose(2, 3).reshape(-1, d)[:k]
            val = V[:, h].view(torch.float8_e4m3fn).double() * sc[:, h, 1, None, None, None]
            val = val.transpose(2, 3).reshape(-1, d)[:k]
            q = s["q"][at:at + n, h * G:(h + 1) * G].double()
            x = (q.reshape(-1, d) @ key.T).unflatten(0, (-1, G)) / math.sqrt(d)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if s["slopes"] is not None:
                x = x - s["slopes"].double()[h * G:(h + 1) * G, None] * gap[:, None]
            p = torch.softmax(x.masked_fill(hidden[:, None], -math.inf), -1)
            out[at:at + n, h * G:(h + 1) * G] = (p.flatten(0, 1) @ val).unflatten(0, (-1, G))
        at += n
    return out
