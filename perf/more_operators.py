"""The attention block of a decoder layer over a paged cache: what is measured, and its plain forms.

Three operators between a layer's query/key/value projection and its output projection:

* ``rope``    norms of the query and key heads and the rotation of their positions,
* ``append``  the same, the keys and values going into the slots of a paged cache,
* ``attend``  softmax attention of each sequence's new tokens over its pages.

Query, key and value heads are slices of one row a token, as the projection
leaves them.  A cache is [pages, page size, key heads, D] (or that shape over
another order in memory), either bf16 or e4m3 codes with one e8m0 scale byte
2^(b - 127) for each token and head.  Rotary pairs are (i, i + R/2) ("half") or
(2i, 2i + 1) ("interleaved") of the first R of D dimensions; frequencies are
theta^(-2i/R), or for long contexts blended by their wave length between those
and the ones divided by a factor.

A query is the last of its sequence's length or so many tokens before it, sees
the keys up to itself and, with a window, only so many.  Cases are dicts of
plain values; the lengths of a ragged batch follow from them.
"""

import math

import torch

own = False

EPS = 1e-6
THETA = 1e6
BETA_FAST, BETA_SLOW = 32.0, 1.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, T, Hq, Hk, D, R, layout, norm, factor=1.0, start=0):
    c = {"op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "layout": layout, "norm": norm, "factor": factor,
         "start": start}
    return dict(c, name=name) if name else c


def _append(name, T, Hq, Hk, D, R, layout, norm, kind, page, order, factor=1.0, start=0):
    c = {"op": "append", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "layout": layout, "norm": norm, "kind": kind,
         "page": page, "order": order, "factor": factor, "start": start}
    return dict(c, name=name) if name else c


def _attend(name, B, new, kv, ragged, Hq, Hk, D, kind, page, order, window=0, behind=0):
    c = {"op": "attend", "B": B, "new": new, "kv": kv, "ragged": ragged, "Hq": Hq, "Hk": Hk, "D": D, "kind": kind,
         "page": page, "order": order, "window": window, "behind": behind}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token's heads: latency
        _rope("rope 1x32+8x128", 1, 32, 8, 128, 128, "half", True, 1.0, 4097),
        # an odd prompt, a quarter of a wide head rotated in the other layout, far positions of a scaled context
        _rope("rope 517x16+2x256 part", 517, 16, 2, 256, 64, "interleaved", False, 16.0, 250000),
        # a long prompt: bandwidth
        _rope("rope 8192x32+8x128", 8192, 32, 8, 128, 128, "half", True),
        # a decode batch, each token into its own sequence's page, 8 bits
        _append("append 32x32+8x128 e4m3", 32, 32, 8, 128, 128, "half", True, "e4m3", 16, "slots", 1.0, 1500),
        # a long prompt into large pages that keep each head's rows together
        _append("append 8192x40+8x128 bf16", 8192, 40, 8, 128, 64, "interleaved", True, "bf16", 64, "heads"),
        # one token of one short sequence: latency
        _attend("attend 1x1 of 777 bf16", 1, 1, 777, False, 32, 8, 128, "bf16", 16, "slots"),
        # one token over a long context: the cache is split over the machine
        _attend("attend 1x1 of 131072 bf16", 1, 1, 131072, False, 64, 8, 128, "bf16", 64, "heads"),
        # an ordinary decode batch of mixed lengths, 8 bits: bandwidth
        _attend("attend 48x1 of 8192 e4m3", 48, 1, 8192, True, 32, 8, 128, "e4m3", 16, "slots", 0, 3),
        # four drafted tokens a sequence, wide heads
        _attend("attend 16x4 of 3001 e4m3 256", 16, 4, 3001, True, 16, 2, 256, "e4m3", 32, "heads"),
        # a ragged batch of prompts in a window, five query heads a key head, small heads
        _attend("attend 5x700 of 4500 window", 5, 700, 4500, True, 40, 8, 64, "e4m3", 16, "slots", 1024),
        # a chunk of a prompt on wide heads
        _attend("attend 1x1024 of 6000 256", 1, 1024, 6000, False, 16, 2, 256, "bf16", 16, "slots"),
        # a long chunk of a long prompt: matrix products
        _attend("attend 1x4096 of 16384 bf16", 1, 4096, 16384, False, 32, 8, 128, "bf16", 64, "slots"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend", "attend"))
    D = rng.choice((64, 128, 128, 256))
    Hk = rng.choice((1, 2, 4, 8))
    Hq = Hk * rng.choice((1, 4, 5, 8))
    kind, page, order = rng.choice(("bf16", "e4m3")), rng.choice((16, 32, 64)), rng.choice(("slots", "heads"))
    if op != "attend":
        R = rng.choice((D, D // 2, D // 4))
        args = (_spread(rng, 1, 8192), Hq, Hk, D, R, rng.choice(("half", "interleaved")), rng.random() < 0.7)
        tail = (rng.choice((1.0, 1.0, 8.0)), _spread(rng, 1, 200000))
        return _rope(None, *args, *tail) if op == "rope" else _append(None, *args, kind, page, order, *tail)
    window = rng.choice((0, 0, 0, 512, 1000))
    form = rng.choice(("decode", "decode", "drafts", "chunk"))
    if form == "chunk":
        new = _spread(rng, 17, 2048)
        B = rng.choice((1, 1, 2, 3)) if new < 1024 else 1
        kv = new + _spread(rng, 1, 6000)
        return _attend(None, B, new, kv, rng.random() < 0.5, Hq, Hk, D, kind, page, order, window)
    B = _spread(rng, 1, 48)
    kv = _spread(rng, 20, min(32768, 400000 // B))
    new = 1 if form == "decode" else rng.randint(2, 8)
    return _attend(None, B, new, kv, rng.random() < 0.7, Hq, Hk, D, kind, page, order, window, rng.choice((0, 0, 5)))


def _lengths(c):
    """(new tokens, length) of each sequence of a batch: the longest first where ragged."""
    n = []
    for b in range(c["B"]):
        cut = b / c["B"] * 0.9 if c["ragged"] else 0.0
        new = max(1, c["new"] - int(cut * c["new"] * 0.8))
        n.append((new, max(new, c["kv"] - int(cut * c["kv"]))))
    return n


def _visible(new, kv, window):
    """How many keys the queries of a sequence see together."""
    first = kv - new + 1
    if not window:
        return (first + kv) * new // 2
    full = sum(1 for _ in range(max(first, window), kv + 1))
    part = new - full
    return full * window + (first + first + part - 1) * part // 2


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _heads(g, T, Hq, Hk, D, device):
    """Query, key and value heads, slices of one row a token: bf16 values whose
    heads differ in size and whose channels include a few large ones."""
    H = Hq + 2 * Hk
    v = torch.randn((T, H, D), generator=g, device=device)
    v = v * torch.exp(0.3 * torch.randn((1, H, 1), generator=g, device=device))
    v = v * torch.where(torch.rand((1, H, D), generator=g, device=device) < 0.01, 8.0, 1.0)
    v = v.to(torch.bfloat16)
    return v[:, :Hq], v[:, Hq:Hq + Hk], v[:, Hq + Hk:]


def _cache(c, pages, device):
    """An empty cache's tensors in the case's order, all of logical shape
    [pages, page, Hk, D] (scales without D)."""
    shape = (pages, c["page"], c["Hk"], c["D"])

    def make(dtype, n):
        if c["order"] == "heads":
            s = (shape[0], shape[2], shape[1], shape[3])[:n]
            return torch.zeros(s, dtype=dtype, device=device).transpose(1, 2)
        return torch.zeros(shape[:n], dtype=dtype, device=device)

    if c["kind"] == "bf16":
        return {"k": make(torch.bfloat16, 4), "v": make(torch.bfloat16, 4), "ks": None, "vs": None}
    return {"k": make(torch.uint8, 4), "v": make(torch.uint8, 4), "ks": make(torch.uint8, 3), "vs": make(torch.uint8, 3)}


def prepare(case, seed):
    device = torch.device("cuda")
    g = _generator(seed, device)
    c = dict(case, kept={})  # kept: the handles and scratch that a program makes at its first call
    if c["op"] == "attend":
        lengths = _lengths(c)
        T = sum(n for n, _ in lengths) + c["behind"]
        # as after the norms of queries and keys
        c["q"] = torch.randn((T, c["Hq"], c["D"]), generator=g, device=device).to(torch.bfloat16)
        need = [-(-kv // c["page"]) for _, kv in lengths]
        pages = sum(need) + 3
        c["cache"] = _cache(c, pages, device)
        for name, scale in (("k", "ks"), ("v", "vs")):
            step = max(1, (1 << 26) // (c["page"] * c["Hk"] * c["D"]))
            for p in range(0, pages, step):
                v = torch.randn(c["cache"][name][p:p + step].shape, generator=g, device=device)
                if c["kind"] == "bf16":
                    c["cache"][name][p:p + step] = v.to(torch.bfloat16)
                else:
                    c["cache"][name][p:p + step], c["cache"][scale][p:p + step] = _quantised(v)
        ids = torch.randperm(pages, generator=g, device=device).to(torch.int32)
        table = torch.zeros((c["B"], max(need) + 1), dtype=torch.int32, device=device)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        c["table"] = table
        cu, total = [0], 0
        for n, _ in lengths:
            total += n
            cu.append(total)
        c["cu"] = torch.tensor(cu, dtype=torch.int32, device=device)
        c["lens"] = torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=device)
        c["most"] = max(n for n, _ in lengths)
        c["longest"] = max(kv for _, kv in lengths)
        c["o"] = torch.zeros((T, c["Hq"], c["D"]), dtype=torch.bfloat16, device=device)
        return c
    T, D = c["T"], c["D"]
    c["q"], c["k"], c["v"] = _heads(g, T, c["Hq"], c["Hk"], D, device)
    c["positions"] = c["start"] + torch.arange(T, device=device)
    c["gq"], c["gk"] = ((1.0 + 0.25 * torch.randn(D, generator=g, device=device)).to(torch.bfloat16) for _ in range(2))
    c["q_out"] = torch.zeros((T, c["Hq"], D), dtype=torch.bfloat16, device=device)
    if c["op"] == "rope":
        c["k_out"] = torch.zeros((T, c["Hk"], D), dtype=torch.bfloat16, device=device)
    else:
        pages = -(-T // c["page"]) + 1
        c["cache"] = _cache(c, pages, device)
        # tokens in order through pages in no order
        ids = torch.randperm(pages, generator=g, device=device)
        t = torch.arange(T, device=device)
        c["slots"] = ids[t // c["page"]] * c["page"] + t % c["page"]
    return c


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _quantised(v):
    """(codes, scale bytes) of float32 [..., D]: the smallest power of two that keeps a row within 448."""
    m, e = torch.frexp(v.abs().amax(-1) / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    codes = torch.ldexp(v, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, scales):
    """float32 [..., D] that the codes and scales stand for, or bf16 keys and values as they are."""
    if scales is None:
        return codes.float()
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), scales.int().unsqueeze(-1) - 127)


def _frequencies(c, device):
    """float64 [R/2] angle a position, and the factor of the rotated values."""
    R = c["R"]
    f = THETA ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    if c["factor"] == 1.0:
        return f, 1.0
    # by the turns that a pair makes in the original context: many keep their frequency, few have it divided
    at = [R * math.log(_original(c) / (b * 2 * math.pi)) / (2 * math.log(THETA)) for b in (BETA_FAST, BETA_SLOW)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
    ramp = ((torch.arange(R // 2, dtype=torch.float64, device=device) - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / c["factor"] * ramp, 0.1 * math.log(c["factor"]) + 1.0


def _original(c):
    return 32768


def _rotated(x, gamma, c):
    """float32 [T, H, D]: the heads' norm and rotation."""
    x = x.float()
    if c["norm"]:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
    f, size = _frequencies(c, x.device)
    a = c["positions"].double().unsqueeze(1) * f
    cos, sin = ((t * size).float().unsqueeze(1) for t in (torch.cos(a), torch.sin(a)))
    R = c["R"]
    if c["layout"] == "half":
        u, w = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat((u * cos - w * sin, w * cos + u * sin, x[..., R:]), -1)
    u, w = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat((torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2), x[..., R:]), -1)


def _plain_rope(s):
    return [_rotated(s["q"], s["gq"], s).to(torch.bfloat16), _rotated(s["k"], s["gk"], s).to(torch.bfloat16)]


def _plain_append(s):
    s["q_out"].copy_(_rotated(s["q"], s["gq"], s))
    page, slot = s["slots"] // s["page"], s["slots"] % s["page"]
    k, v, cache = _rotated(s["k"], s["gk"], s), s["v"].float(), s["cache"]
    if s["kind"] == "bf16":
        cache["k"][page, slot], cache["v"][page, slot] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    else:
        cache["k"][page, slot], cache["ks"][page, slot] = _quantised(k)
        cache["v"][page, slot], cache["vs"][page, slot] = _quantised(v)
    return _appended(s)


def _appended(s):
    """The queries and the cache; its codes and scale bytes as the numbers that they stand for."""
    cache = s["cache"]
    if s["kind"] == "bf16":
        return [s["q_out"], cache["k"], cache["v"]]
    return [s["q_out"], cache["k"].view(torch.float8_e4m3fn), cache["v"].view(torch.float8_e4m3fn),
            cache["ks"].view(torch.float8_e8m0fnu), cache["vs"].view(torch.float8_e8m0fnu)]


def _plain_attend(s):
    B, D, Hq, Hk = s["B"], s["D"], s["Hq"], s["Hk"]
    G, cache = Hq // Hk, s["cache"]
    at = torch.arange(s["longest"], device=s["q"].device)
    page, slot = s["table"][:, at // s["page"]].long(), (at % s["page"]).expand(B, -1)
    k = _values(cache["k"][page, slot], cache["ks"][page, slot] if cache["ks"] is not None else None)
    v = _values(cache["v"][page, slot], cache["vs"][page, slot] if cache["vs"] is not None else None)
    k, v = k.transpose(1, 2), v.transpose(1, 2)  # [B, Hk, kv, D]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(s["most"], device=at.device)
    there = i < new.unsqueeze(1)  # [B, new]
    rows = torch.where(there, s["cu"][:-1].long().unsqueeze(1) + i, 0)
    q = s["q"][rows].float().view(B, s["most"], Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * s["most"], D)
    p = q @ k.transpose(2, 3) / math.sqrt(D)
    p = p.view(B, Hk, G, s["most"], -1)
    where = (s["lens"].long() - new).unsqueeze(1) + i  # each query's place
    seen = at <= where.unsqueeze(2)
    if s["window"]:
        seen &= at > where.unsqueeze(2) - s["window"]
    p.masked_fill_(~seen[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, Hk, G * s["most"], -1) @ v
    o = torch.where(total > 0, o.view(B, Hk, G, s["most"], D) / total, 0.0)
    s["o"][rows[there]] = o.permute(0, 3, 1, 2, 4).reshape(B, s["most"], Hq, D)[there].to(torch.bfloat16)
    return s["o"]


def run(state):
    s = state
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    import fp8_block_scale_x128_gb300 as fb
    kept = s["kept"]
    if "cache" in s and "cache" not in kept:
        kept["cache"] = fb.KvCache(s["cache"]["k"], s["cache"]["v"], s["cache"]["ks"], s["cache"]["vs"])
    if s["op"] == "attend":
        if "workspace" not in kept:
            kept["workspace"] = fb.new_attn_workspace(s["D"])
        return fb.fp8bs_attn_paged(s["q"], kept["cache"], s["table"], s["cu"], s["lens"], window=s["window"], o=s["o"],
                                   workspace=kept["workspace"])
    if "rope" not in kept:
        long = {} if s["factor"] == 1.0 else {"scaling": fb.FP8BS_ROPE_BY_PARTS, "factor": s["factor"],
                                              "original_length": _original(s), "beta_fast": BETA_FAST, "beta_slow": BETA_SLOW}
        kept["rope"] = fb.Rope(s["R"], THETA, fb.FP8BS_ROPE_HALF if s["layout"] == "half" else fb.FP8BS_ROPE_INTERLEAVED,
                               **long)
    gq, gk = (s["gq"], s["gk"]) if s["norm"] else (None, None)
    if s["op"] == "rope":
        return list(fb.fp8bs_qk_norm_rope(s["q"], s["k"], s["positions"], kept["rope"], gq, gk, EPS, q_out=s["q_out"],
                                          k_out=s["k_out"]))
    fb.fp8bs_qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], kept["rope"], kept["cache"], gq, gk,
                                 EPS, q_out=s["q_out"])
    return _appended(s)


# ---------------------------------------------------------------------------
# the work of a pass, and its answer in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    row = 2 * D if c.get("kind", "bf16") == "bf16" else D + 1  # a key or value of the cache
    if c["op"] == "attend":
        lengths = _lengths(c)
        pairs = sum(_visible(n, kv, c["window"]) for n, kv in lengths)
        keys = sum(min(kv, c["window"] + n - 1) if c["window"] else kv for n, kv in lengths)
        return {"bytes": 4.0 * Hq * D * sum(n for n, _ in lengths) + 2.0 * keys * Hk * row, "flops": 4.0 * pairs * Hq * D}
    T = c["T"]
    if c["op"] == "rope":
        return {"bytes": 4.0 * T * (Hq + Hk) * D + 8 * T, "flops": 8.0 * T * (Hq + Hk) * D}
    return {"bytes": 4.0 * T * Hq * D + T * Hk * (4.0 * D + 2 * row) + 16 * T, "flops": 8.0 * T * (Hq + Hk) * D}


def _exact_heads(c, x, gamma):
    """float64 [T, H, D] of heads, pair by pair as a product of complex numbers."""
    x = x.double()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / c["D"] + EPS) * gamma.double()
    R, i = c["R"], torch.arange(c["R"] // 2, dtype=torch.float64, device=x.device)
    f, size = torch.exp(-2.0 * i / R * math.log(THETA)), 1.0
    if c["factor"] != 1.0:
        def index(turns):
            return R / 2 * math.log(_original(c) / (2 * math.pi * turns), THETA)
        low, high = max(0, math.floor(index(BETA_FAST))), min(R - 1, math.ceil(index(BETA_SLOW)))
        share = torch.clamp((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        f, size = f * (1.0 - share + share / c["factor"]), 1.0 + 0.1 * math.log(c["factor"])
    turn = torch.polar(torch.full_like(f, size).expand(c["T"], -1), torch.outer(c["positions"].double(), f))
    y = x.clone()
    if c["layout"] == "half":
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn[:, None]
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:R:2].contiguous(), x[..., 1:R:2].contiguous()) * turn[:, None]
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    return y


def _exact_cache(c, k, v):
    """The cache's outputs with the rows in their slots, empty ones as they were."""
    out = []
    flat = c["slots"]
    for x in (k, v):
        pages = c["cache"]["k"].shape[0]
        to = torch.zeros((pages * c["page"], c["Hk"], c["D"]), dtype=torch.float64, device=x.device)
        if c["kind"] == "bf16":
            to[flat] = x
            out.append((to.view(pages, c["page"], c["Hk"], c["D"]), None))
            continue
        most = x.abs().amax(-1)
        power = torch.exp2(torch.ceil(torch.log2(most / 448.0)))
        power = torch.where(power * 224.0 >= most, power / 2, power)  # where the logarithm passed a whole number
        to[flat] = x / power.unsqueeze(-1)
        scale = torch.full((pages * c["page"], c["Hk"]), 2.0 ** -127, dtype=torch.float64, device=x.device)
        scale[flat] = power
        out.append((to.view(pages, c["page"], c["Hk"], c["D"]), scale.view(pages, c["page"], c["Hk"])))
    return [t for t, _ in out] + [t for _, t in out if t is not None]


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] != "attend":
        q, k = _exact_heads(c, c["q"], c["gq"]), _exact_heads(c, c["k"], c["gk"])
        return [q, k] if c["op"] == "rope" else [q] + _exact_cache(c, k, c["v"].double())
    out = torch.zeros(c["o"].shape, dtype=torch.float64, device=c["o"].device)
    G, first = c["Hq"] // c["Hk"], 0
    for b, (new, kv) in enumerate(_lengths(c)):
        pages = c["table"][b, :-(-kv // c["page"])].long()
        place = torch.arange(kv - new, kv, device=out.device).unsqueeze(1)
        key = torch.arange(kv, device=out.device)
        hidden = key > place
        if c["window"]:
            hidden |= key <= place - c["window"]
        for h in range(c["Hk"]):
            k, v = (_exact_rows(c, n, pages, h)[:kv] for n in ("k", "v"))
            for j in range(h * G, (h + 1) * G):
                for r in range(0, new, 1024):
                    q = c["q"][first + r:first + min(new, r + 1024), j].double()
                    s = torch.einsum("qd,kd->qk", q, k) * c["D"] ** -0.5
                    w = torch.softmax(s.masked_fill(hidden[r:r + 1024], -math.inf), 1)
                    out[first + r:first + min(new, r + 1024), j] = torch.einsum("qk,kd->qd", w, v)
        first += new
    return out


def _exact_rows(c, name, pages, h):
    """float64 [tokens, D] of one head's keys or values, e4m3 codes from their bits."""
    x = c["cache"][name][pages, :, h].flatten(0, 1)
    if c["kind"] == "bf16":
        return x.double()
    n = x.long()
    e, f = (n >> 3) & 15, (n & 7).double()
    size = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e.double() - 7))
    scale = c["cache"][name + "s"][pages, :, h].flatten().double()
    return torch.where(n >= 128, -size, size) * (2.0 ** (scale - 127)).unsqueeze(1)
