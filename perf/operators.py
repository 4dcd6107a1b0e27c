"""The serving and positions operators as measured: query/key norm with rotary positions (forward, and
with its backward), the FP8 key/value cache (append, read back) and the attention of a few new tokens
over that cache.  ``run`` computes them in plain torch, or, with ``own`` set, through the package."""

import math

import torch

own = False

TILE = 64          # keys that share one scale of P
FP8_MAX = 448.0
TINY = 2.0 ** -110  # rows of smaller magnitude are stored as zeros
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's queries and keys of 16 sequences, far into a context stretched 8 times
        dict(name="rope_step", op="rope", B=16, N=1, Hq=32, Hkv=8, D=128, R=128, layout="half",
             scaling="yarn", factor=8.0, base=10000.0, start=60000, train=False),
        # queries and keys of the long video self-attention workload, a whole forward
        dict(name="rope_video", op="rope", B=1, N=32768, Hq=40, Hkv=40, D=128, R=128,
             layout="interleaved", scaling="none", factor=1.0, base=10000.0, start=0, train=False),
        # a training step's share of the causal workload: forward, gradients of q, k and both weights
        dict(name="rope_train", op="rope", B=4, N=8192, Hq=32, Hkv=32, D=128, R=128, layout="half",
             scaling="none", factor=1.0, base=500000.0, start=0, train=True),
        # small heads of which half is rotated, an odd length, training
        dict(name="rope_train_odd", op="rope", B=3, N=1531, Hq=24, Hkv=8, D=64, R=32, layout="half",
             scaling="linear", factor=4.0, base=10000.0, start=7, train=True),
        # one decode step's new keys and values of 64 sequences
        dict(name="append_step", op="append", B=64, N=1, Hkv=8, D=128, page=16, lo=1, hi=1,
             past=255),
        # prompts of different lengths, padded to the longest
        dict(name="append_prompts", op="append", B=8, N=8192, Hkv=8, D=128, page=64, lo=1000, hi=8192,
             past=0),
        # one sequence of the image workload read back
        dict(name="read_one", op="read", B=1, N=4608, Hkv=24, D=128, page=64, lo=4608, hi=4608),
        # cached prefixes of different lengths read back for the next chunks of their prompts
        dict(name="read_prefixes", op="read", B=6, N=32768, Hkv=8, D=128, page=32, lo=9000, hi=32768),
        # one user, a short conversation: latency
        dict(name="decode_one", op="decode", B=1, T=1, Hq=32, Hkv=8, D=128, page=64, lo=1537, hi=1537,
             quant=1),
        # a serving batch of ragged lengths
        dict(name="decode_batch", op="decode", B=64, T=1, Hq=32, Hkv=8, D=128, page=64, lo=129, hi=8192,
             quant=1),
        # two very long contexts, an odd number of query heads a key head
        dict(name="decode_long", op="decode", B=2, T=1, Hq=40, Hkv=8, D=128, page=128, lo=250001,
             hi=262144, quant=1),
        # small heads without sharing, four tokens checked at once, P not quantized
        dict(name="decode_draft", op="decode", B=12, T=4, Hq=16, Hkv=16, D=64, page=16, lo=33, hi=4099,
             quant=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "read", "decode", "decode"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        train = rng.random() < 0.5
        rows = _spread(rng, 64, 1 << 20)
        Hq = Hkv * rng.choice([1, 1, 3, 4])
        tokens = max(1, rows // (Hq + Hkv))
        B = min(rng.choice([1, 2, 3, 8]), tokens)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, B=B, N=max(1, tokens // B), Hq=Hq, Hkv=Hkv, D=D,
                    R=rng.choice([D, D, D // 2, D // 4]), layout=rng.choice(["half", "interleaved"]),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    base=rng.choice([10000.0, 500000.0]), start=rng.randrange(0, 1000000), train=train)
    if op == "decode":
        T = rng.choice([1, 1, 1, 2, 3, 5])
        G = rng.choice([1, 3, 4, 8])
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 17, max(64, min(131072, 4000000 // (B * Hkv))))
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, lo=rng.randint(1, hi), hi=hi,
                    quant=rng.choice([0, 1, 1]))
    B = _spread(rng, 1, 64)
    hi = _spread(rng, 1, max(4, 524288 // (B * Hkv)))
    c = dict(op=op, B=B, N=hi, Hkv=Hkv, D=D, page=page, lo=rng.randint(0, hi), hi=hi)
    if op == "append":
        c["past"] = rng.randint(0, 200)
    return c


def _lens(case):
    """The sequences' lengths: evenly spread, so that a case's work is the same for every seed."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        rows = case["B"] * case["N"] * (case["Hq"] + case["Hkv"])
        return {"bytes": rows * D * 2 * (5 if case["train"] else 2) + 4 * case["B"] * case["N"],
                "flops": rows * D * (30 if case["train"] else 9)}
    tokens = sum(_lens(case))
    rows = tokens * case["Hkv"]
    if case["op"] == "append":
        return {"bytes": rows * 2 * (2 * D + D + 4), "flops": rows * 2 * 4 * D}
    if case["op"] == "read":  # the rows behind a sequence's end are written too, as zeros
        out = case["B"] * case["N"] * case["Hkv"]
        return {"bytes": rows * 2 * (D + 4) + out * 2 * 2 * D, "flops": rows * 2 * D}
    new = case["B"] * case["T"] * case["Hq"]
    return {"bytes": rows * 2 * (D + 4) + new * (4 * D + 4), "flops": tokens * case["T"] * case["Hq"] * 4 * D}


# ------------------------------------------------------------------------------------------ inputs

def _frequencies(case):
    """Radians a position of each pair, and the amplitude of the rotated channels."""
    R, base, factor = case["R"], case["base"], case["factor"]
    if case["scaling"] == "ntk":
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    if case["scaling"] != "yarn":
        return f, 1.0

    def pair_of(turns):  # the pair that makes so many turns in the original context
        return R * math.log(8192 / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), R - 1)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(R // 2)]
    return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def _pages(case, lens, g):
    """A page table whose pages lie scattered over the cache."""
    per = max(1, -(-max(max(lens), 1) // case["page"]))
    n = case["B"] * per
    order = torch.randperm(n, generator=g, device="cuda", dtype=torch.int32)
    return order.view(case["B"], per).contiguous(), n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    s = {"case": case}
    if case["op"] == "rope":  # q and k are parts of one projection's output, heads innermost
        N, Hq = case["N"], case["Hq"]
        x = normal(B, N, Hq + 2 * Hkv, D, dtype=torch.bfloat16) * (0.5 + 2.0 * torch.rand(
            D, generator=g, device="cuda")).to(torch.bfloat16)
        s["q"], s["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["wq"], s["wk"] = (1.0 + 0.2 * normal(D) for _ in range(2))
        first = case["start"] + torch.randint(0, 1 + case["start"] // 8, (B, 1), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(N, device="cuda")).to(torch.int32)
        f, s["amplitude"] = _frequencies(case)
        s["f"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        if case["train"]:
            s["dq"], s["dk"] = (normal(B, h, N, D, dtype=torch.bfloat16) for h in (Hq, Hkv))
        if own:
            from quantization_aware_attention_gb300 import RopePlan
            more = {} if case["scaling"] != "yarn" else {"original_len": 8192}
            s["rope"] = RopePlan(case["R"], base=case["base"], layout=case["layout"],
                                 scaling=case["scaling"], factor=case["factor"], device="cuda", **more)
        return s

    lens = _lens(case)
    past = case.get("past", 0)
    s["table"], n = _pages(case, [x + past for x in lens], g)
    order = torch.randperm(B, generator=g, device="cuda")
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")[order]
    s["lens"] = lens + past
    shape = (n, Hkv, case["page"])
    # what a cache holds: codes spread as those of normal keys and values, scales that vary by token
    for x in "kv":
        code = torch.empty(*shape, D, dtype=torch.float8_e4m3fn, device="cuda")
        for i in range(0, n, 1024):
            code[i:i + 1024] = (normal(*code[i:i + 1024].shape, dtype=torch.bfloat16) * 150).clamp(
                -FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        s[x] = code
        s[x + "_scale"] = (0.4 + torch.rand(*shape, generator=g, device="cuda")) / 150
    if case["op"] == "append":
        new = normal(B, case["N"], 2 * Hkv, D, dtype=torch.bfloat16) * (0.5 + torch.rand(
            B, case["N"], 2 * Hkv, 1, generator=g, device="cuda")).to(torch.bfloat16)
        # the keys have been made by the norm and rotation, the values come from the projection
        s["new_k"] = new[:, :, :Hkv].transpose(1, 2).contiguous()
        s["new_v"] = new[:, :, Hkv:].transpose(1, 2)
        s["new_lens"] = lens
    if case["op"] == "decode":
        s["q"] = normal(B, case["Hq"], case["T"], D, dtype=torch.bfloat16) * 2  # scores of spread 2
    if own:
        from quantization_aware_attention_gb300 import KVCache
        s["cache"] = KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _pairs(z, case):
    """The two halves of the rotated pairs."""
    R = case["R"]
    if case["layout"] == "half":
        return z[..., :R // 2], z[..., R // 2:R]
    return z[..., 0:R:2], z[..., 1:R:2]


def _unpairs(a, b, z, case):
    R = case["R"]
    rotated = torch.cat((a, b), -1) if case["layout"] == "half" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((rotated, z[..., R:]), -1)


def _cos_sin(s):
    angle = s["positions"].double()[:, None, :, None] * s["f"]
    return (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()


def _norm_rope(x, w, cos, sin, case):
    x = x.float()
    z = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    a, b = _pairs(z, case)
    return _unpairs(a * cos - b * sin, a * sin + b * cos, z, case).to(torch.bfloat16)


def _norm_rope_back(x, w, dy, cos, sin, case):
    x, dy = x.float(), dy.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    a, b = _pairs(dy, case)
    dz = _unpairs(a * cos + b * sin, b * cos - a * sin, dy, case)
    n = x * r
    dn = dz * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dz * n).double().sum((0, 1, 2)).float()


def _plain_rope(s):
    case = s["case"]
    cos, sin = _cos_sin(s)
    out = [_norm_rope(s["q"], s["wq"], cos, sin, case), _norm_rope(s["k"], s["wk"], cos, sin, case)]
    if case["train"]:
        dq, dwq = _norm_rope_back(s["q"], s["wq"], s["dq"], cos, sin, case)
        dk, dwk = _norm_rope_back(s["k"], s["wk"], s["dk"], cos, sin, case)
        out += [dq, dk, dwq, dwk]
    return out


def _plain_append(s):
    page = s["case"]["page"]
    n = torch.arange(s["case"]["N"], device="cuda")
    b, i = (n < s["new_lens"][:, None]).nonzero(as_tuple=True)
    at = (s["lens"] - s["new_lens"])[b] + i
    where = s["table"][b, at // page].long()
    for x in "kv":
        rows = s["new_" + x].transpose(1, 2)[b, i].float()
        amax = rows.abs().amax(-1)
        amax = torch.where(amax < TINY, 0.0, amax)
        inv = torch.where(amax > 0, FP8_MAX / amax, 0.0)
        code = (rows * inv[..., None]).to(torch.float8_e4m3fn)
        s[x].view(torch.uint8)[where, :, at % page] = code.view(torch.uint8)
        s[x + "_scale"][where, :, at % page] = amax / FP8_MAX
    return [s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _gathered(s, x):
    """The cached rows in the sequences' order, in 32 bits: [B, Hkv, pages * page, D]."""
    table = s["table"].long()
    code = s[x].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    v = code * s[x + "_scale"][table][..., None]
    return v.transpose(1, 2).flatten(2, 3)


def _plain_read(s):
    N = s["case"]["N"]
    seen = (torch.arange(N, device="cuda") < s["lens"][:, None])[:, None, :, None]
    return [torch.where(seen, _gathered(s, x)[:, :, :N], 0.0).to(torch.bfloat16) for x in "kv"]


def _plain_decode(s):
    case = s["case"]
    B, T, Hq, Hkv, D = (case[n] for n in ("B", "T", "Hq", "Hkv", "D"))
    k, v = _gathered(s, "k"), _gathered(s, "v")
    q = s["q"].float().view(B, Hkv, -1, D)
    scores = q @ k.transpose(-1, -2) * (D ** -0.5)
    key = torch.arange(k.shape[2], device="cuda")
    last = s["lens"][:, None] - T + torch.arange(T, device="cuda")  # the newest key a token sees
    hidden = (key > last[..., None])[:, None, None]
    scores = scores.view(B, Hkv, Hq // Hkv, T, -1).masked_fill(hidden, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(m == -math.inf, 0.0, m)).exp()
    total = p.sum(-1, keepdim=True)
    if case["quant"]:
        tiles = torch.nn.functional.pad(p, (0, -p.shape[-1] % TILE)).unflatten(-1, (-1, TILE))
        amax = tiles.amax(-1, keepdim=True)
        code = (tiles * torch.where(amax > 0, FP8_MAX / amax, 0.0)).to(torch.float8_e4m3fn).float()
        p = (code * (amax / FP8_MAX)).flatten(-2)[..., :p.shape[-1]]
    o = p.reshape(B, Hkv, -1, k.shape[2]) @ torch.where(
        (key < s["lens"][:, None])[:, None, :, None], v, 0.0)
    o = torch.where(total.view(B, Hkv, -1, 1) > 0, o / total.view(B, Hkv, -1, 1), 0.0)
    lse = (m + total.log()) / math.log(2.0)
    return [o.view(B, Hq, T, D).to(torch.bfloat16), lse.view(B, Hq, T)]


# ------------------------------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read,
                "decode": _plain_decode}[op](state)
    import quantization_aware_attention_gb300 as qat
    if op == "rope":
        q, k, wq, wk = (state[n] for n in ("q", "k", "wq", "wk"))
        if not case["train"]:
            return qat.qat_qk_norm_rope(q, k, state["positions"], state["rope"], wq, wk, eps=EPS)
        leaves = [t.detach().requires_grad_(True) for t in (q, k, wq, wk)]
        out = qat.qat_qk_norm_rope(leaves[0], leaves[1], state["positions"], state["rope"], leaves[2],
                                   leaves[3], eps=EPS)
        grads = torch.autograd.grad(out, leaves, (state["dq"], state["dk"]))
        return [t.detach() for t in out] + list(grads)
    cache = state["cache"]
    if op == "append":
        cache.append(state["new_k"], state["new_v"], state["table"], state["lens"], state["new_lens"])
        return [cache.k, cache.v, cache.k_scale, cache.v_scale]
    if op == "read":
        return cache.read(state["table"], state["lens"], length=case["N"])
    return qat.qat_attention_decode(state["q"], cache, state["table"], state["lens"],
                                    quant_mode=case["quant"], return_lse=True)


# ------------------------------------------------------------------------------------------ in 64 bits

def _e4m3(x):
    """x rounded to the nearest E4M3 value, ties to even, |x| <= 448: three bits of fraction, steps of
    2^-9 below 2^-6."""
    exponent = torch.frexp(x)[1] - 1
    step = torch.ldexp(torch.ones_like(x), exponent.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_rope(s):
    case = s["case"]
    R = case["R"]
    f = torch.tensor(_frequencies(case)[0], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(f, s["amplitude"]), torch.zeros_like(f)) * torch.exp(
        1j * s["positions"].to(torch.float64)[:, None, :, None] * f)

    def planes(x):  # the rotated channels as complex numbers
        if case["layout"] == "half":
            return torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous())
        return torch.view_as_complex(x[..., :R].unflatten(-1, (-1, 2)).contiguous())

    def turned(x, by):
        c = planes(x) * by
        part = (torch.cat((c.real, c.imag), -1) if case["layout"] == "half"
                else torch.view_as_real(c).flatten(-2))
        return torch.cat((part, x[..., R:]), -1)

    outs, grads, weights = [], [], []
    for x, w, dy in (("q", "wq", "dq"), ("k", "wk", "dk")):
        x, w = s[x].double(), s[w].double()
        rms = (x.square().sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
        unit = x / rms
        outs.append(turned(unit * w, turn))
        if case["train"]:
            dz = turned(s[dy].double(), turn.conj())
            weights.append((dz * unit).sum((0, 1, 2)))
            g = dz * w
            grads.append((g - unit * ((g * unit).sum(-1, keepdim=True) / case["D"])) / rms)
    return outs + grads + weights


def _exact_append(s):
    """Codes and scales after the append: each new row's own, every other slot as it was.  (A value
    halfway between two codes goes to the even one here; the rule's 32-bit reciprocal may miss that.)"""
    page = s["case"]["page"]
    out = []
    lens, new_lens, table = (s[n].tolist() for n in ("lens", "new_lens", "table"))
    for x in "kv":
        code, scale = s[x].double(), s[x + "_scale"].double()
        for b in range(s["case"]["B"]):
            n = new_lens[b]
            if n == 0:
                continue
            rows = s["new_" + x][b, :, :n].double()
            largest = rows.abs().max(-1).values
            unit = largest / FP8_MAX
            flat = torch.arange(lens[b] - n, lens[b])
            where = torch.tensor(table[b])[flat // page].cuda()
            off = (flat % page).cuda()
            value = torch.where(largest[..., None] < TINY, 0.0, _e4m3(rows * FP8_MAX / largest[..., None]))
            code[where, :, off] = value.transpose(0, 1)
            scale[where, :, off] = torch.where(largest < TINY, 0.0, unit).transpose(0, 1)
        out.append((code, scale))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def _exact_rows(s, x, b, n):
    """The first n cached rows of sequence b: [Hkv, n, D]."""
    pages = s["table"][b].long()[: -(-n // s["case"]["page"])]
    code = torch.stack([s[x][i] for i in pages.tolist()], 1).double()
    scale = s[x + "_scale"][pages].double().transpose(0, 1)
    return (code * scale.unsqueeze(-1)).reshape(code.shape[0], -1, code.shape[-1])[:, :n]


def _exact_read(s):
    case = s["case"]
    out = []
    for x in "kv":
        y = torch.zeros(case["B"], case["Hkv"], case["N"], case["D"], dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            if n:
                y[b, :, :n] = _exact_rows(s, x, b, n)
        out.append(y)
    return out


def _exact_decode(s):
    case = s["case"]
    T, Hq, Hkv, D = (case[n] for n in ("T", "Hq", "Hkv", "D"))
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        k, v = _exact_rows(s, "k", b, n), _exact_rows(s, "v", b, n)
        for t in range(T):
            seen = n - T + t + 1
            if seen <= 0:
                continue
            q = s["q"][b, :, t].double().view(Hkv, Hq // Hkv, D)
            score = torch.einsum("hgd,hnd->hgn", q, k[:, :seen]) / math.sqrt(D)
            norm = torch.logsumexp(score, -1)
            weight = (score - norm[..., None]).exp()
            if case["quant"]:
                whole = -(-seen // TILE) * TILE
                tile = torch.zeros(*weight.shape[:2], whole, dtype=torch.float64, device="cuda")
                tile[..., :seen] = weight
                tile = tile.view(*weight.shape[:2], -1, TILE)
                unit = tile.max(-1, keepdim=True).values / FP8_MAX
                unit = torch.where(unit > 0, unit, 1.0)
                weight = (_e4m3(tile / unit) * unit).flatten(-2)[..., :seen]
            o[b, :, t] = torch.einsum("hgn,hnd->hgd", weight, v[:, :seen]).reshape(Hq, D)
            lse[b, :, t] = norm.reshape(Hq) / math.log(2.0)
    return [o, lse]


def exact(case, seed):
    return {"rope": _exact_rope, "append": _exact_append, "read": _exact_read,
            "decode": _exact_decode}[case["op"]](prepare(case, seed))
