"""The windowed attention and the drafted tokens' operators as measured: attention with a sliding window and
visible first tokens (training: forward, and with its backward; serving: over the FP8 key/value cache), the
masks and positions of a tree of drafted tokens, its attention over the cache, and keeping the tokens that
were accepted.  ``run`` computes them in plain torch, or, with ``own`` set, through the package."""

import math

import torch

own = False

TILE = 64          # keys that share one scale of P
FP8_MAX = 448.0
BLOCK = 128        # query rows that the plain window attention takes together


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a short fine-tuning sequence, odd in every size, small heads: latency of a training pass
        dict(name="window_small", op="window", B=1, H=5, N=1531, D=64, W=100, S=5, quant=1, train=True),
        # the causal training workload with a window of an eighth of its length and four sinks
        dict(name="window_train", op="window", B=4, H=32, N=8192, D=128, W=1024, S=4, quant=1, train=True),
        # scoring a long document: the forward pass alone
        dict(name="window_long", op="window", B=1, H=8, N=32768, D=128, W=4096, S=64, quant=1, train=False),
        # a serving batch of ragged lengths, some shorter than the window
        dict(name="steps_batch", op="steps", B=64, T=1, Hq=32, Hkv=8, D=128, page=64, lo=129, hi=8192,
             W=1024, S=4, quant=1),
        # two very long contexts of which little is seen, an odd number of query heads a key head
        dict(name="steps_long", op="steps", B=2, T=1, Hq=40, Hkv=8, D=128, page=128, lo=250001, hi=262144,
             W=4096, S=130, quant=1),
        # one user, a short conversation, a small tree: latency
        dict(name="tree_one", op="tree", B=1, T=8, Hq=32, Hkv=8, D=128, page=64, lo=1537, hi=1537, W=0, S=0,
             quant=1),
        # a serving batch that drafts 32 tokens, long contexts
        dict(name="tree_batch", op="tree", B=16, T=32, Hq=32, Hkv=8, D=128, page=64, lo=2001, hi=16384, W=0,
             S=0, quant=1),
        # many sequences with the widest trees, eight query heads a key head
        dict(name="tree_wide", op="tree", B=64, T=64, Hq=64, Hkv=8, D=128, page=32, lo=129, hi=4096, W=0,
             S=0, quant=1),
        # masks and positions of one user's tree, and of a large batch's
        dict(name="draft_one", op="draft", B=1, T=16),
        dict(name="draft_batch", op="draft", B=256, T=64),
        # the accepted paths of a serving batch, and of a large one with the longest paths
        dict(name="keep_batch", op="keep", B=16, T=32, L=6, Hkv=8, D=128, page=64, lo=2001, hi=16384),
        dict(name="keep_large", op="keep", B=256, T=64, L=24, Hkv=8, D=128, page=32, lo=129, hi=2048),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "steps", "steps", "tree", "tree", "tree", "draft", "keep"])
    D = rng.choice([64, 128, 128])
    if op == "window":
        train = rng.random() < 0.6
        W = _spread(rng, 1, 8192)
        heads = _spread(rng, 1, 128)
        H = rng.choice([h for h in (1, 3, 5, 8, 24, 32, 40) if h <= heads])
        B = max(1, min(4, heads // H))
        most = min(65536, (1 << 30) // (B * H * (min(W, 4096) + 192)))
        return dict(op=op, B=B, H=H, N=_spread(rng, 17, max(64, most)), D=D, W=W,
                    S=rng.choice([0, 1, 4, 17, 64, 130]), quant=rng.choice([0, 1, 1]), train=train)
    if op == "draft":
        return dict(op=op, B=_spread(rng, 1, 512), T=rng.randint(1, 64))
    Hkv = rng.choice([1, 2, 4, 5, 8, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    G = rng.choice([1, 3, 4, 5, 8])
    B = _spread(rng, 1, 64)
    if op == "steps":
        T = rng.choice([1, 1, 1, 2, 5, 16])
        hi = _spread(rng, 17, max(64, min(262144, 4000000 // (B * Hkv))))
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, lo=rng.randint(1, hi), hi=hi,
                    W=_spread(rng, 1, 8192), S=rng.choice([0, 1, 4, 64, 130]), quant=rng.choice([0, 1, 1]))
    T = rng.randint(1, 64)
    if op == "keep":
        hi = _spread(rng, T, max(T, min(16384, 2000000 // (B * Hkv))))
        return dict(op=op, B=B, T=T, L=rng.randint(1, T), Hkv=Hkv, D=D, page=page,
                    lo=rng.randint(T // 2, hi), hi=hi)
    most = min(4000000 // (B * Hkv), 500000000 // (B * Hkv * G * T), 131072)
    hi = _spread(rng, T, max(64, most))
    W = rng.choice([0, 0, _spread(rng, T, 8192)])
    return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, lo=rng.randint(T // 2, hi), hi=hi, W=W,
                S=rng.choice([0, 4, 130]) if W else 0, quant=rng.choice([0, 1, 1]))


def _lens(case):
    """The sequences' lengths: evenly spread, so that a case's work is the same for every seed."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def work(case):
    op = case["op"]
    if op == "window":
        N, W, S = case["N"], case["W"], case["S"]
        inside = min(N, W)
        pairs = inside * (inside + 1) // 2 + (N - inside) * inside  # of the windows
        behind = max(0, N - W)                                    # rows that have left key 0 behind
        ramp = min(behind, S)
        pairs += ramp * (ramp + 1) // 2 + (behind - ramp) * S
        heads = case["B"] * case["H"]
        return {"bytes": heads * N * case["D"] * 2 * (8 if case["train"] else 4),
                "flops": heads * pairs * case["D"] * (16 if case["train"] else 4)}
    if op == "draft":
        return {"bytes": case["B"] * (16 * case["T"] + 4), "flops": case["B"] * case["T"] * 6}
    D = case["D"]
    if op == "keep":
        rows = case["B"] * case["L"]
        return {"bytes": rows * case["Hkv"] * 4 * (D + 4) + 4 * rows + 12 * case["B"], "flops": 0}
    T, W, S = case["T"], case["W"], case["S"]
    seen = sum(n if not W else min(n, min(S, n) + W + T - 1) for n in _lens(case))
    new = case["B"] * T * case["Hq"]
    return {"bytes": seen * case["Hkv"] * 2 * (D + 4) + new * (4 * D + 4) + (8 * case["B"] * T if op == "tree" else 0),
            "flops": seen * T * case["Hq"] * 4 * D}


# ------------------------------------------------------------------------------------------ inputs

def _pages(case, lens, g):
    """A page table whose pages lie scattered over the cache."""
    per = max(1, -(-max(max(lens), 1) // case["page"]))
    n = case["B"] * per
    order = torch.randperm(n, generator=g, device="cuda", dtype=torch.int32)
    return order.view(case["B"], per).contiguous(), n


def _parents(case, g):
    """Trees as drafting makes them: each token continues one of the eight before it, some the text itself."""
    B, T = case["B"], case["T"]
    t = torch.arange(T, device="cuda")
    back = 1 + torch.randint(0, 8, (B, T), generator=g, device="cuda")
    return (t - back).clamp(min=-1).to(torch.int32)


def _ancestors(parents):
    """Whether token t is s or descends from it: [B, T, T], truth values."""
    B, T = parents.shape
    t = torch.arange(T, device="cuda")
    reach = ((parents[..., None] == t) | (t[:, None] == t)).float()
    for _ in range(6):  # paths of up to 64 steps
        reach = (reach @ reach).clamp(max=1.0)
    return reach > 0


def _packed(seen):
    """Truth values [B, T, T] as the bits of int64 [B, T]."""
    t = torch.arange(seen.shape[-1], device="cuda")
    return (seen.long() << t).sum(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    op, B = case["op"], case["B"]
    s = {"case": case}
    if op == "window":
        shape = (B, case["H"], case["N"], case["D"])
        # scores of spread 1.5, keys with an offset in each channel as trained keys have
        s["q"] = normal(*shape, dtype=torch.bfloat16) * 1.5
        s["k"] = normal(*shape, dtype=torch.bfloat16) + 0.5 * normal(case["D"], dtype=torch.bfloat16)
        s["v"] = normal(*shape, dtype=torch.bfloat16)
        if case["train"]:
            s["do"] = normal(*shape, dtype=torch.bfloat16)
        return s
    if op == "draft":
        s["parents"] = _parents(case, g)
        s["lens"] = (case["T"] + torch.randint(0, 100000, (B,), generator=g, device="cuda")).to(torch.int32)
        return s

    D, Hkv, T = case["D"], case["Hkv"], case["T"]
    lens = _lens(case)
    s["table"], n = _pages(case, lens, g)
    order = torch.randperm(B, generator=g, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[order]
    # what a cache holds: codes spread as those of normal keys and values, scales that vary by token
    shape = (n, Hkv, case["page"])
    for x in "kv":
        code = torch.empty(*shape, D, dtype=torch.float8_e4m3fn, device="cuda")
        for i in range(0, n, 1024):
            code[i:i + 1024] = (normal(*code[i:i + 1024].shape, dtype=torch.bfloat16) * 150).clamp(
                -FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        s[x] = code
        s[x + "_scale"] = (0.4 + torch.rand(*shape, generator=g, device="cuda")) / 150
    if op == "keep":
        # paths as verification returns them: ascending places, as many as each sequence accepted
        places = torch.rand(B, T, generator=g, device="cuda").argsort(-1)[:, :case["L"]]
        s["path"] = places.sort(-1).values.to(torch.int32).contiguous()
        s["path_lens"] = torch.randint(0, case["L"] + 1, (B,), generator=g, device="cuda").to(torch.int32)
        s["path_lens"][0] = case["L"]
    else:
        s["q"] = normal(B, case["Hq"], T, D, dtype=torch.bfloat16) * 2  # scores of spread 2
    if op == "tree":
        s["tree"] = _packed(_ancestors(_parents(case, g)))
    if own:
        from quantization_aware_attention_gb300 import KVCache
        s["cache"] = KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _fake_quant(p):
    """P by the rule of the attention: tiles of 64 keys, whose largest value becomes 448."""
    tiles = torch.nn.functional.pad(p, (0, -p.shape[-1] % TILE)).unflatten(-1, (-1, TILE))
    amax = tiles.amax(-1, keepdim=True)
    code = (tiles * torch.where(amax > 0, FP8_MAX / amax, 0.0)).to(torch.float8_e4m3fn).float()
    return (code * (amax / FP8_MAX)).flatten(-2)[..., :p.shape[-1]]


def _plain_window(s):
    """Blocks of 128 query rows against the keys that any of them sees: the sinks' tiles, then the windows'."""
    case = s["case"]
    N, D, W, S = (case[n] for n in ("N", "D", "W", "S"))
    blocks = -(-N // BLOCK)
    back = -(-(min(W, N) - 1) // TILE) * TILE
    ahead = -(-S // TILE) * TILE
    first = BLOCK * torch.arange(blocks, device="cuda")[:, None]
    band = first - back + torch.arange(back + BLOCK, device="cuda")
    sink = torch.arange(ahead, device="cuda").expand(blocks, -1)
    key = torch.cat((sink, band), -1)                                              # [blocks, C]
    there = torch.cat((sink >= 0, band >= ahead), -1) & (key < N)
    at = key.clamp(0, N - 1)
    row = first + torch.arange(BLOCK, device="cuda")                               # [blocks, 128]
    key_, row_ = key[:, None], row[..., None]
    seen = there[:, None] & (key_ <= row_) & ((key_ > row_ - W) | (key_ < S))

    def by_rows(x):
        return torch.nn.functional.pad(x.float(), (0, 0, 0, blocks * BLOCK - N)).unflatten(2, (blocks, BLOCK))

    scale = D ** -0.5
    q, k, v = by_rows(s["q"]), s["k"].float()[:, :, at], s["v"].float()[:, :, at]
    p = (q @ k.transpose(-1, -2) * scale).masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (_fake_quant(p) if case["quant"] else p) @ v / total

    def back_to(x):
        return x.flatten(2, 3)[:, :, :N].to(torch.bfloat16)

    if not case["train"]:
        return [back_to(o)]
    p /= total
    do = by_rows(s["do"])
    delta = (do * (p @ v)).sum(-1, keepdim=True)

    def over_keys(x):  # sums of the blocks' keys
        out = torch.zeros(s["k"].shape, device="cuda")
        return out.index_add_(2, at.flatten(), x.flatten(2, 3)).to(torch.bfloat16)

    dv = over_keys(p.transpose(-1, -2) @ do)
    ds = (do @ v.transpose(-1, -2)).sub_(delta).mul_(p)
    return [back_to(o), back_to(ds @ k * scale), over_keys(ds.transpose(-1, -2) @ q * scale), dv]


def _plain_cached(s):
    """Attention of each sequence's last T tokens over the keys that any of them may see."""
    case = s["case"]
    B, T, Hq, Hkv, D, W, S = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "W", "S"))
    lens = s["lens"].long()[:, None]
    t = torch.arange(T, device="cuda")
    if W:
        ahead, back = -(-S // TILE) * TILE, (-(-(W + T) // TILE) + 1) * TILE
        first = (lens - T - W + 1).clamp(min=0) // TILE * TILE
        band = first + torch.arange(back, device="cuda")
        sink = torch.arange(ahead, device="cuda").expand(B, -1)
        key = torch.cat((sink, band), -1)
        there = torch.cat((sink < lens, (band >= ahead) & (band < lens)), -1)
    else:
        key = torch.arange(s["table"].shape[1] * case["page"], device="cuda").expand(B, -1)
        there = key < lens
    key, there = key[:, None], there[:, None]                                      # [B, 1, C]
    base = (lens - T)[:, None]
    if case["op"] == "tree":
        place = key - base
        bits = (s["tree"][..., None] >> place.clamp(0, 63)) & 1
        seen = there & ((place < 0) | (bits == 1))
        depth = ((s["tree"][..., None] >> torch.arange(64, device="cuda")) & 1).sum(-1)
        if W:
            pos = base + depth[..., None] - 1
            seen &= (place >= 0) | (key > pos - W) | (key < S)
    else:
        pos = base + t[:, None]
        seen = there & (key <= pos)
        if W:
            seen &= (key > pos - W) | (key < S)
    at = torch.where(there, key, 0)[:, 0]
    pages, slots = s["table"].long().gather(1, at // case["page"]), at % case["page"]

    def rows(x):  # [B, Hkv, C, D] in 32 bits, zeros where nothing is
        code = s[x].view(torch.uint8)[pages, :, slots].view(torch.float8_e4m3fn).float()
        y = code * s[x + "_scale"][pages, :, slots][..., None]
        return torch.where(there[:, 0, :, None, None], y, 0.0).transpose(1, 2)

    k, v = rows("k"), rows("v")
    q = s["q"].float().view(B, Hkv, -1, D)
    p = (q @ k.transpose(-1, -2) * (D ** -0.5)).view(B, Hq, T, -1)
    p = p.masked_fill_(~seen[:, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()) / math.log(2.0)
    if case["quant"]:
        p = _fake_quant(p)
    o = (p.view(B, Hkv, -1, p.shape[-1]) @ v).view(B, Hq, T, D)
    return [torch.where(total > 0, o / total, 0.0).to(torch.bfloat16), lse[..., 0]]


def _plain_draft(s):
    seen = _ancestors(s["parents"])
    pos = s["lens"][:, None] - s["case"]["T"] + seen.sum(-1) - 1
    return [_packed(seen), pos.to(torch.int32)]


def _plain_keep(s):
    case = s["case"]
    T, L, page = case["T"], case["L"], case["page"]
    base = s["lens"].long() - T
    i = torch.arange(L, device="cuda")
    b, i = ((i < s["path_lens"][:, None]) & (base[:, None] + i >= 0) & (
        base[:, None] + s["path"] >= 0)).nonzero(as_tuple=True)
    old, new = base[b] + s["path"][b, i], base[b] + i
    table = s["table"].long()
    for x in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["k_scale"], s["v_scale"]):
        x[table[b, new // page], :, new % page] = x[table[b, old // page], :, old % page]
    lens = (base + s["path_lens"]).clamp(min=0).to(torch.int32)
    return [s["k"], s["v"], s["k_scale"], s["v_scale"], lens]


# ------------------------------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"window": _plain_window, "steps": _plain_cached, "tree": _plain_cached, "draft": _plain_draft,
                "keep": _plain_keep}[op](state)
    import quantization_aware_attention_gb300 as qat
    if op == "window":
        q, k, v = (state[n] for n in "qkv")
        how = dict(causal=True, quant_mode=case["quant"], window=case["W"], sinks=case["S"])
        if not case["train"]:
            return [qat.attention(q, k, v, **how)]
        leaves = [t.detach().requires_grad_(True) for t in (q, k, v)]
        o = qat.attention(*leaves, **how)
        return [o.detach()] + list(torch.autograd.grad(o, leaves, state["do"]))
    if op == "draft":
        return qat.qat_draft_tree(state["parents"], state["lens"])
    cache, table, lens = state["cache"], state["table"], state["lens"]
    if op == "keep":
        lens = cache.keep(table, lens, case["T"], state["path"], state["path_lens"])
        return [cache.k, cache.v, cache.k_scale, cache.v_scale, lens]
    how = dict(quant_mode=case["quant"], return_lse=True)
    if case["W"]:
        how.update(window=case["W"], sinks=case["S"])
    if op == "tree":
        return qat.qat_attention_tree(state["q"], cache, table, lens, state["tree"], **how)
    return qat.qat_attention_decode(state["q"], cache, table, lens, **how)


# ------------------------------------------------------------------------------------------ in 64 bits

def _e4m3(x):
    """x rounded to the nearest E4M3 value, ties to even, |x| <= 448: three bits of fraction, steps of
    2^-9 below 2^-6."""
    exponent = torch.frexp(x)[1] - 1
    step = torch.ldexp(torch.ones_like(x), exponent.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _softmax(score, quant):
    """Weights and their fake-quantized form, tiles of 64 from column 0 on; logarithm of the sum."""
    norm = torch.logsumexp(score, -1, keepdim=True)
    weight = torch.where(norm == -math.inf, 0.0, (score - norm).exp())
    if not quant:
        return weight, weight, norm[..., 0]
    n = score.shape[-1]
    tile = torch.zeros(*score.shape[:-1], -(-n // TILE) * TILE, dtype=torch.float64, device="cuda")
    tile[..., :n] = weight
    tile = tile.unflatten(-1, (-1, TILE))
    unit = tile.max(-1, keepdim=True).values / FP8_MAX
    unit = torch.where(unit > 0, unit, 1.0)
    return weight, (_e4m3(tile / unit) * unit).flatten(-2)[..., :n], norm[..., 0]


def _exact_window(s):
    """512 query rows at a time against columns that are the whole tiles before the last row's end."""
    case = s["case"]
    N, D, W, S = (case[n] for n in ("N", "D", "W", "S"))
    q, k, v = (s[n].double() for n in "qkv")
    do = s["do"].double() if case["train"] else None
    o, dq, dk, dv = (torch.zeros_like(q) for _ in range(4))
    for i in range(0, N, 512):
        e = min(i + 512, N)
        rows = slice(i, e)
        begin = max(0, i - W + 1) // TILE * TILE
        cols = torch.arange(begin, e, device="cuda")
        ahead = min(-(-S // TILE) * TILE, begin)  # sinks' tiles before the window's
        cols = torch.cat((torch.arange(ahead, device="cuda"), cols))
        r = torch.arange(i, e, device="cuda")[:, None]
        hidden = (cols > r) | ((cols <= r - W) & (cols >= S))
        kc, vc = k[:, :, cols], v[:, :, cols]
        score = torch.einsum("bhid,bhjd->bhij", q[:, :, rows], kc) / math.sqrt(D)
        weight, rounded, _ = _softmax(score.masked_fill(hidden, -math.inf), case["quant"])
        del score
        o[:, :, rows] = torch.einsum("bhij,bhjd->bhid", rounded, vc)
        if not case["train"]:
            continue
        g = do[:, :, rows]
        dv[:, :, cols] += torch.einsum("bhij,bhid->bhjd", weight, g)
        dp = torch.einsum("bhid,bhjd->bhij", g, vc)
        ds = weight * (dp - (weight * dp).sum(-1, keepdim=True)) / math.sqrt(D)
        dq[:, :, rows] = torch.einsum("bhij,bhjd->bhid", ds, kc)
        dk[:, :, cols] += torch.einsum("bhij,bhid->bhjd", ds, q[:, :, rows])
    return [o, dq, dk, dv] if case["train"] else [o]


def _exact_rows(s, x, b, n):
    """The first n cached rows of sequence b: [Hkv, n, D]."""
    pages = s["table"][b].long()[: -(-n // s["case"]["page"])]
    code = s[x].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
    scale = s[x + "_scale"][pages].double()
    return (code * scale[..., None]).transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_cached(s):
    case = s["case"]
    T, Hq, Hkv, D, W, S = (case[n] for n in ("T", "Hq", "Hkv", "D", "W", "S"))
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    tree = s["tree"].tolist() if case["op"] == "tree" else None
    for b, n in enumerate(s["lens"].tolist()):
        k, v = _exact_rows(s, "k", b, n), _exact_rows(s, "v", b, n)
        seen = torch.zeros(T, n, dtype=torch.bool)
        for t in range(T):
            prefix = max(0, n - T)
            if tree is None:
                pos = n - T + t
                seen[t, :max(0, pos + 1)] = True
            else:
                pos = n - T + bin(tree[b][t] & (2 ** 64 - 1)).count("1") - 1
                seen[t, :prefix] = True
            if W:
                seen[t, min(S, n):max(0, min(S, n), pos - W + 1)] = False
            if tree is not None:
                seen[t, prefix:] = torch.tensor([bool(tree[b][t] >> (j - (n - T)) & 1) for j in range(prefix, n)],
                                                dtype=torch.bool)
        q = s["q"][b].double().view(Hkv, Hq // Hkv, T, D)
        score = torch.einsum("hgtd,hnd->hgtn", q, k) / math.sqrt(D)
        _, weight, norm = _softmax(score.masked_fill(~seen.cuda(), -math.inf), case["quant"])
        o[b] = torch.einsum("hgtn,hnd->hgtd", weight, v).reshape(Hq, T, D)
        lse[b] = norm.reshape(Hq, T) / math.log(2.0)
    return [o, lse]


def _exact_keep(s):
    """Codes and scales after the move: each accepted row in its new place, every other slot as it was."""
    case = s["case"]
    page = case["page"]
    out = [s["k"].double(), s["v"].double(), s["k_scale"].double(), s["v_scale"].double()]
    old = [x.clone() for x in out]
    table, path = s["table"].tolist(), s["path"].tolist()
    to, of = [], []
    for b, (n, kept) in enumerate(zip(s["lens"].tolist(), s["path_lens"].tolist())):
        base = n - case["T"]
        for i in range(kept):
            at, was = base + i, base + path[b][i]
            if at >= 0 and was >= 0:
                to.append((table[b][at // page], at % page))
                of.append((table[b][was // page], was % page))
    if to:
        (p, i), (q, j) = (torch.tensor(x, device="cuda").T for x in (to, of))
        for x, y in zip(out, old):
            x[p, :, i] = y[q, :, j]
    return out + [None]


def exact(case, seed):
    if case["op"] == "draft":
        return None
    return {"window": _exact_window, "steps": _exact_cached, "tree": _exact_cached,
            "keep": _exact_keep}[case["op"]](prepare(case, seed))
