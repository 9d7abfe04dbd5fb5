"""The 4-bit-weight decode operators: what is measured, and their plain forms.

Three operators of a decode step on 4-bit weights:

* ``gemv``   y[M, N] = bf16(x . W^T) for a few bf16 tokens and a 4-bit weight,
* ``route``  the mixture-of-experts router: expert logits, softmax, top-k,
* ``moe``    the routed experts on 4-bit weights (gate/up, silu, down, combine).

Two weight formats, both as [N, K/2] bytes (the even k in the low nibble) and
one scale per 1xG group along K:

* ``mxfp4``  e2m1 codes, e8m0 scale bytes 2^(b - 127), G = 32,
* ``int4``   codes q = 0..15 for the value q - 8, bf16 scales, G = 32, 64 or 128.

Cases are dicts of plain values.  Projection and expert sizes are those of
this repository's benchmark (5120x4096, 4096x2048, 16384x8192; hidden 4096,
513 experts of 256 or 128, 10 routed slots and a shared one) or odd ones.
"""

import math

import numpy as np
import torch

own = False

OUTLIER_FRACTION, OUTLIER_SCALE, WEIGHT_STD = 0.01, 20.0, 0.02
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _gemv(name, M, N, K, fmt, group, pad=0):
    c = {"op": "gemv", "M": M, "N": N, "K": K, "fmt": fmt, "group": group, "pad": pad}
    return dict(c, name=name) if name else c


def _route(name, M, E, H, k, renorm=True, shared="one"):
    c = {"op": "route", "M": M, "E": E, "H": H, "k": k, "renorm": renorm, "shared": shared}
    return dict(c, name=name) if name else c


def _moe(name, M, E, H, I, k, shared, fmt, group):
    c = {"op": "moe", "M": M, "E": E, "H": H, "I": I, "k": k, "shared": shared, "fmt": fmt, "group": group}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through the smallest projection of the benchmark: latency
        _gemv("gemv 1x4096x2048 mxfp4", 1, 4096, 2048, "mxfp4", 32),
        # one token through an ordinary projection, the usual int4 group
        _gemv("gemv 1x5120x4096 int4", 1, 5120, 4096, "int4", 128),
        # a small batch, an odd number of rows, rows of x inside a wider buffer
        _gemv("gemv 5x4999x7168 int4 g32", 5, 4999, 7168, "int4", 32, 64),
        # the largest decode batch on the largest weight: bandwidth
        _gemv("gemv 16x16384x8192 mxfp4", 16, 16384, 8192, "mxfp4", 32),
        # one token's routing: latency
        _route("route 1 of 512", 1, 512, 4096, 10),
        # a batch with an odd expert count, weights not renormalised, gated shared expert
        _route("route 21 of 161", 21, 161, 7168, 6, False, "gate"),
        # a full decode batch
        _route("route 64 of 512", 64, 512, 4096, 10),
        # one token through the whole set of experts (10 routed + 1 shared)
        _moe("moe 1 of 513x256 mxfp4", 1, 513, 4096, 256, 10, True, "mxfp4", 32),
        # a small batch on the narrower experts of a wider split, int4
        _moe("moe 8 of 513x128 int4", 8, 513, 4096, 128, 10, True, "int4", 128),
        # few experts, each with several tokens, an odd batch, no shared expert
        _moe("moe 19 of 24x512 int4 g64", 19, 24, 2048, 512, 4, False, "int4", 64),
        # a decode batch that reads most of the experts: bandwidth
        _moe("moe 32 of 513x256 mxfp4", 32, 513, 4096, 256, 10, True, "mxfp4", 32),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _format(rng):
    return ("mxfp4", 32) if rng.random() < 0.5 else ("int4", rng.choice((32, 64, 128)))


def draw(rng):
    op = rng.choice(("gemv", "gemv", "route", "moe"))
    if op == "gemv":
        fmt, group = _format(rng)
        return _gemv(None, _spread(rng, 1, 16), _spread(rng, 200, 16384), 128 * _spread(rng, 4, 64), fmt, group,
                     rng.choice((0, 0, 8, 256)))
    if op == "route":
        k = rng.randint(1, 12)
        return _route(None, _spread(rng, 1, 64), _spread(rng, 16, 512), 128 * _spread(rng, 4, 56), k,
                      rng.random() < 0.5, rng.choice(("none", "one", "gate")))
    fmt, group = _format(rng)
    shared = rng.random() < 0.5
    k = rng.randint(1, 10)
    return _moe(None, _spread(rng, 1, 32), _spread(rng, 16, 480), 128 * _spread(rng, 4, 32),
                rng.choice((128, 256)), k, shared, fmt, group)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _activations(g, M, K, pad, device):
    """bf16 N(0, 1) with 1% of the entries 20 times as large."""
    v = torch.randn((M, K + pad), generator=g, device=device)
    v = torch.where(torch.rand((M, K + pad), generator=g, device=device) < OUTLIER_FRACTION, v * OUTLIER_SCALE, v)
    return v.to(torch.bfloat16)[:, :K]


def _weights(g, rows, K, fmt, group, device):
    """(codes uint8 [rows, K/2], scales [rows, K/group]) of N(0, 0.02) weights,
    rounded to their 4-bit format a block of rows at a time."""
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((rows, K // group), dtype=torch.uint8 if fmt == "mxfp4" else torch.bfloat16, device=device)
    edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=device)
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        w = torch.randn((n, K // group, group), generator=g, device=device) * WEIGHT_STD
        amax = w.abs().amax(-1)
        if fmt == "mxfp4":  # the smallest power of two that keeps the group within 6
            m, e = torch.frexp(amax / 6.0)
            e = torch.where(m > 0.5, e, e - 1)
            scales[r:r + n] = (e + 127).to(torch.uint8)
            v = torch.ldexp(w, -e.unsqueeze(-1))
            c = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        else:
            s = (amax / 7.0).to(torch.bfloat16)
            scales[r:r + n] = s
            c = (torch.round(w / s.float().unsqueeze(-1)).clamp(-8, 7) + 8).to(torch.uint8)
        c = c.view(n, K // 2, 2)
        codes[r:r + n] = c[..., 0] | (c[..., 1] << 4)
    return codes, scales


def _routing(g, M, E, k, shared, device):
    """(ids int32 [M, S], weights float32 [M, S]): k distinct experts a token,
    weights that sum to 1, and the last expert with weight 1 where shared."""
    n = E - 1 if shared else E
    ids = torch.rand((M, n), generator=g, device=device).argsort(1)[:, :k]
    w = torch.softmax(torch.randn((M, k), generator=g, device=device), 1)
    if shared:
        ids = torch.cat((ids, torch.full((M, 1), E - 1, device=device)), 1)
        w = torch.cat((w, torch.ones((M, 1), device=device)), 1)
    return ids.to(torch.int32).contiguous(), w.contiguous()


def prepare(case, seed):
    device = torch.device("cuda")
    g = _generator(seed, device)
    c = dict(case)
    if c["op"] == "gemv":
        c["x"] = _activations(g, c["M"], c["K"], c["pad"], device)
        c["codes"], c["scales"] = _weights(g, c["N"], c["K"], c["fmt"], c["group"], device)
        c["y"] = torch.empty((c["M"], c["N"]), dtype=torch.bfloat16, device=device)
    elif c["op"] == "route":
        rows = c["E"] + (1 if c["shared"] == "gate" else 0)
        c["x"] = _activations(g, c["M"], c["H"], 0, device)
        c["w"] = (torch.randn((rows, c["H"]), generator=g, device=device) * WEIGHT_STD).to(torch.bfloat16)
        S = c["k"] + (0 if c["shared"] == "none" else 1)
        c["ids"] = torch.empty((c["M"], S), dtype=torch.int32, device=device)
        c["weights"] = torch.empty((c["M"], S), dtype=torch.float32, device=device)
    else:
        M, E, H, I = c["M"], c["E"], c["H"], c["I"]
        c["x"] = _activations(g, M, H, 0, device)
        c["ids"], c["weights"] = _routing(g, M, E, c["k"], c["shared"], device)
        codes, scales = _weights(g, E * 2 * I, H, c["fmt"], c["group"], device)
        c["w13"], c["s13"] = codes.view(E, 2 * I, H // 2), scales.view(E, 2 * I, -1)
        codes, scales = _weights(g, E * H, I, c["fmt"], c["group"], device)
        c["w2"], c["s2"] = codes.view(E, H, I // 2), scales.view(E, H, -1)
        c["y"] = torch.empty((M, H), dtype=torch.bfloat16, device=device)
    c["workspace"] = None  # a program's own scratch, kept from its first call on
    return c


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _dequantised(codes, scales, fmt, group):
    """float32 [..., K] of codes [..., K/2] and scales [..., K/group]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    if fmt == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        v = table[c.int()]
        s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    else:
        v = c.float() - 8.0
        s = scales.float()
    return (v.unflatten(-1, (-1, group)) * s.unsqueeze(-1)).flatten(-2)


def _plain_gemv(s):
    w = _dequantised(s["codes"], s["scales"], s["fmt"], s["group"])
    return (s["x"].float() @ w.t()).to(torch.bfloat16)


def _plain_route(s):
    # in 64 bits: the order of two nearly equal logits decides whole numbers
    E, k = s["E"], s["k"]
    logits = s["x"].double() @ s["w"].double().t()
    p = torch.exp(logits[:, :E] - logits[:, :E].amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    ids = torch.sort(logits[:, :E], dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if s["shared"] != "none":
        ids = torch.cat((ids, torch.full_like(ids[:, :1], E)), 1)
        w = torch.cat((w, 1.0 / (1.0 + torch.exp(-logits[:, E:])) if s["shared"] == "gate" else torch.ones_like(w[:, :1])), 1)
    return [ids.to(torch.int32), w.float()]


def _plain_moe(s):
    ids, M, S = s["ids"].long(), s["M"], s["ids"].shape[1]
    flat = ids.flatten()
    x = s["x"].float().repeat_interleave(S, 0)
    w13 = _dequantised(s["w13"][flat], s["s13"][flat], s["fmt"], s["group"])
    h = torch.bmm(w13, x.unsqueeze(-1)).squeeze(-1)
    del w13
    gate, up = h[:, :s["I"]], h[:, s["I"]:]
    a = gate / (1.0 + torch.exp(-gate)) * up
    w2 = _dequantised(s["w2"][flat], s["s2"][flat], s["fmt"], s["group"])
    o = torch.bmm(w2, a.unsqueeze(-1)).view(M, S, -1)
    return (o * s["weights"].unsqueeze(-1)).sum(1).to(torch.bfloat16)


def run(state):
    s = state
    if not own:
        return {"gemv": _plain_gemv, "route": _plain_route, "moe": _plain_moe}[s["op"]](s)
    import fp8_block_scale_x128_gb300 as fb
    if s["op"] == "gemv":
        return fb.fp8bs_gemv_w4a16(s["x"], s["codes"], s["scales"], _FORMAT[s["fmt"]], s["group"], y=s["y"])
    if s["op"] == "route":
        if s["workspace"] is None:
            s["workspace"] = fb.new_moe_route_workspace(s["M"], s["E"], s["H"])
        return list(fb.fp8bs_moe_route(s["x"], s["w"], s["k"], renorm=s["renorm"], shared=s["shared"], ids=s["ids"],
                                       weights=s["weights"], workspace=s["workspace"]))
    if s["workspace"] is None:
        s["workspace"] = fb.new_moe_w4_workspace(s["M"], s["ids"].shape[1], s["I"])
    return fb.fp8bs_moe_w4a16(s["x"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"],
                              _FORMAT[s["fmt"]], s["group"], y=s["y"], workspace=s["workspace"])


_FORMAT = {"mxfp4": 0, "int4": 1}  # the library's FP8BS_W4_MXFP4 and FP8BS_W4_INT4


# ---------------------------------------------------------------------------
# the work of a pass, and its answer in 64 bits
# ---------------------------------------------------------------------------

def _scale_bytes(fmt):
    return 1 if fmt == "mxfp4" else 2


def work(case):
    c = case
    if c["op"] == "gemv":
        M, N, K = c["M"], c["N"], c["K"]
        weight = N * K / 2 + N * (K // c["group"]) * _scale_bytes(c["fmt"])
        return {"bytes": weight + 2 * M * K + 2 * M * N, "flops": 2.0 * M * N * K}
    if c["op"] == "route":
        rows = c["E"] + (1 if c["shared"] == "gate" else 0)
        S = c["k"] + (0 if c["shared"] == "none" else 1)
        return {"bytes": 2.0 * rows * c["H"] + 2 * c["M"] * c["H"] + 8 * c["M"] * S,
                "flops": 2.0 * c["M"] * rows * c["H"]}
    M, E, H, I, k = c["M"], c["E"], c["H"], c["I"], c["k"]
    S = k + (1 if c["shared"] else 0)
    routed = E - 1 if c["shared"] else E
    # distinct experts that M draws of k out of the routed ones reach on average
    active = routed * (1.0 - (1.0 - min(k, routed) / routed) ** M) + (1 if c["shared"] else 0)
    expert = 3.0 * I * H * (0.5 + _scale_bytes(c["fmt"]) / c["group"])
    return {"bytes": active * expert + 4 * M * H + 8 * M * S, "flops": 6.0 * M * S * I * H}


def _value64(codes, scales, fmt, group):
    """float64 [rows, K], from the formats' definition: sign, exponent and
    fraction bits of e2m1, or the offset integer."""
    c = codes.to(torch.int64)
    v = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        n = (c >> (4 * half)) & 15
        if fmt == "mxfp4":
            exponent, fraction = (n >> 1) & 3, (n & 1).double()
            size = torch.where(exponent == 0, 0.5 * fraction, (1.0 + 0.5 * fraction) * 2.0 ** (exponent.double() - 1.0))
            v[:, half::2] = torch.where(n >= 8, -size, size)
        else:
            v[:, half::2] = n.double() - 8.0
    s = 2.0 ** (scales.double() - 127.0) if fmt == "mxfp4" else scales.double()
    return v * s.repeat_interleave(group, 1)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if s["op"] == "gemv":
        y = torch.empty((s["M"], s["N"]), dtype=torch.float64, device=x.device)
        for r in range(0, s["N"], 2048):
            w = _value64(s["codes"][r:r + 2048], s["scales"][r:r + 2048], s["fmt"], s["group"])
            y[:, r:r + 2048] = torch.einsum("mk,nk->mn", x, w)
        return y
    if s["op"] == "route":
        xs, ws = x.cpu().numpy(), s["w"].double().cpu().numpy()
        out = np.empty((s["M"], s["ids"].shape[1]))
        for m in range(s["M"]):
            logits = ws @ xs[m]
            top = np.lexsort((np.arange(s["E"]), -logits[:s["E"]]))[:s["k"]]
            z = np.exp(logits[:s["E"]] - logits[:s["E"]].max())
            out[m, :s["k"]] = z[top] / (z[top].sum() if s["renorm"] else z.sum())
            if s["shared"] != "none":
                out[m, s["k"]] = 1.0 / (1.0 + np.exp(-logits[s["E"]])) if s["shared"] == "gate" else 1.0
        return [None, torch.from_numpy(out)]
    ids, weights = s["ids"].cpu().numpy(), s["weights"].double()
    y = torch.zeros((s["M"], s["H"]), dtype=torch.float64, device=x.device)
    for e in np.unique(ids):
        token, slot = (torch.from_numpy(v).to(x.device) for v in np.nonzero(ids == e))
        h = x[token] @ _value64(s["w13"][e], s["s13"][e], s["fmt"], s["group"]).t()
        gate, up = h.split(s["I"], 1)
        o = (gate * torch.sigmoid(gate) * up) @ _value64(s["w2"][e], s["s2"][e], s["fmt"], s["group"]).t()
        y.index_add_(0, token, o * weights[token, slot].unsqueeze(1))
    return y
