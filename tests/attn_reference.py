"""A plain implementation, in 64 bits on the CPU, of the attention block's operators,
and the bounds of what fp32 arithmetic and one rounding may differ from it by.

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value, to e4m3 by 2^-4 of it
or 2^-10 below the normal numbers.  fp32 steps count 2^-24 each, twice that where a
matrix unit may cut off instead of rounding.

* Heads: the norm's sum of at most 256 squares over lanes (13 steps), its root and
  three products; an angle's fraction of a turn rounded to fp32 (below pi 2^-25), the
  sine and cosine (2 steps each) and the rotation's two products and sum: below 32 steps
  of the pair's magnitude times the amplitude.
* Attention: a score's D products are summed in D/16 steps of 16: with Q = scale sum
  |q k|, off by Q 2^-23 (D/16 + 16); its multiplication by log2(e) and the difference
  from the maximum by 3 steps of |score| and |maximum|; exp2 by 2^-21.  A weight in the
  product is off by `weight` more of itself.  A sum of n weighted values is off by n/16
  + 16 steps of the sum of magnitudes.  Numerator and denominator may each be off so far.
* Attention over codes, whose products are in fp16 (steps of 2^-24 below 2^-14): a
  weight times its value's scale, or that of its neighbours, of which 2^7 stands for the
  largest weight times the largest scale (the maximum may lag, never lead), is off by
  half a step there, 2^-25 2^-7 of those, and multiplies the value's code; q's largest magnitude is brought to 2^14 at least, and q is
  off by 2^-25 2^-14 of it; a key or a value, multiplied by its scale over the largest of
  up to 128 neighbours (here: of all), by 2^-25 of that scale.
"""

import math

import torch

from tests.w4_reference import bf16  # noqa: F401

STEP = 2.0 ** -24


def frequencies(R, theta, scaling=0, factor=1.0, original=0.0, fast=32.0, slow=1.0):
    """float64 [R/2] angle a position, and the amplitude."""
    f = [theta ** (-2 * i / R) for i in range(R // 2)]
    if scaling == 1:
        f = [x / factor for x in f]
    if scaling == 2:
        def pair(turns):
            return R * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))
        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
        s = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(R // 2)]
        f = [x * (1 - a) + x / factor * a for x, a in zip(f, s)]
    return torch.tensor(f, dtype=torch.float64), (0.1 * math.log(factor) + 1.0 if scaling == 2 else 1.0)


def heads(x, positions, f, amplitude, half, gamma, eps):
    """(float64 [T, H, D], bound of the fp32 error before the last rounding)."""
    x = x.double().cpu()
    if gamma is not None:
        ms = (x * x).mean(-1, keepdim=True) + eps
        x = torch.where(ms > 0, x * torch.where(ms > 0, ms, 1.0) ** -0.5, 0.0) * gamma.double().cpu()
    y, size = x.clone(), x.abs()
    R = 2 * len(f)
    if R:
        # (the table's own rounding: 2^-52 of a turn's angle a position)
        a = torch.outer(positions.double().cpu(), f)
        c, s = (amplitude * t.unsqueeze(1) for t in (torch.cos(a), torch.sin(a)))
        i, j = (slice(0, R // 2), slice(R // 2, R)) if half else (slice(0, R, 2), slice(1, R, 2))
        u, w = x[..., i], x[..., j]
        y[..., i], y[..., j] = u * c - w * s, w * c + u * s
        size[..., i] = size[..., j] = amplitude * (u.abs() + w.abs())
        far = a.abs().unsqueeze(1) * 2.0 ** -51
    bound = 32 * STEP * size
    if R:
        bound[..., i] += far * size[..., i]
        bound[..., j] += far * size[..., j]
    return y, bound


def e4m3_values(codes, scale):
    """float64 values of codes [..., D] and scale bytes [...] from their bits."""
    n = codes.cpu().long()
    e, f = (n >> 3) & 15, (n & 7).double()
    v = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e.double() - 7))
    v = torch.where(n & 0x7F == 0x7F, math.nan, v)
    s = scale.cpu().double()
    s = torch.where(s == 255, math.nan, 2.0 ** (s - 127))
    return torch.where(n >= 128, -v, v) * s.unsqueeze(-1)


def rows_of(cache, table, n):
    """float64 k and v [n, heads, D] of a sequence from a cache's tensors (k, v[, k_scale, v_scale])."""
    page = cache[0].shape[1]
    j = torch.arange(n)
    p, s = table.cpu().long()[j // page], j % page
    out = []
    for i in range(2):
        x = cache[i].cpu()[p, s]
        out.append(e4m3_values(x, cache[2 + i].cpu()[p, s]) if len(cache) == 4 else x.double())
    return out


def attend(q, k, v, kv, scale, window, weight, codes=None):
    """One sequence: q [n, Hq, D] (the newest of kv tokens), k and v [kv, Hk, D].
    Returns float64 o [n, Hq, D] and its bound; `weight`: the rounding of a weight;
    `codes`: scales [kv, Hk] of the keys and of the values, where they are codes."""
    q = q.double().cpu()
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, bound = torch.zeros_like(q), torch.zeros_like(q)
    place = torch.arange(kv - n, kv).unsqueeze(1)
    key = torch.arange(kv)
    seen = key <= place
    if window:
        seen &= key > place - window
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = q[:, h] @ kh.t() * scale
        size = q[:, h].abs() @ kh.abs().t() * scale
        s = torch.where(seen, s, -math.inf)
        most = s.amax(1, keepdim=True) if kv else torch.full((n, 1), -math.inf, dtype=torch.float64)
        none = ~seen.any(1, keepdim=True)
        w = torch.where(seen, torch.exp(s - torch.where(none, 0.0, most)), 0.0)
        if codes:
            qh = q[:, h].abs()
            more = 2.0 ** -25 * codes[0][:, h // G].max() * qh.sum(1, keepdim=True) + 2.0 ** -39 * qh.amax(1, keepdim=True) * kh.abs().sum(1)
        else:
            more = torch.zeros_like(s)
        off = scale * more + 2.0 ** -23 * (D / 16 + 16) * size + 3 * STEP * 1.5 * (torch.where(seen, s, 0.0).abs() + torch.where(none, 0.0, most).abs()) + 2.0 ** -21
        off = torch.where(seen, torch.expm1(torch.nan_to_num(off, nan=0.0, posinf=0.0)), 0.0) + weight
        total = torch.where(none, 1.0, w.sum(1, keepdim=True))
        vs = torch.where(torch.isfinite(vh), vh, 0.0)
        o[:, h] = w @ vs / total
        bad = torch.where(torch.isfinite(vh), 0.0, vh)
        for j in torch.nonzero((bad != 0).any(1)).flatten().tolist():  # only the rows that see such a value have it
            rows = seen[:, j]
            o[rows, h] += bad[j]
        steps = 2 * STEP * (kv / 16 + 16)
        least = 0.0
        if codes:
            unit = codes[1][:, h // G]
            least = 2.0 ** -32 * w.amax(1, keepdim=True) * unit.max() * (vs.abs() / unit.unsqueeze(1)).sum(0) / total + 2.0 ** -25 * unit.max()
        bound[:, h] = (w * (off + steps)) @ vs.abs() / total + (w * (off + steps)).sum(1, keepdim=True) / total * (w @ vs.abs() / total) + least
    return o, bound


def near(y, ref, bound, bits=2.0 ** -8):
    """Whether y is within `bound` and one rounding (of `bits`) of ref, and not finite where ref is not."""
    y = y.double().cpu()
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(y)), "infinities or NaNs elsewhere"
    d = (y - ref).abs()[fine]
    allowed = (bound + bits * (ref.abs() + bound))[fine]
    worst = float((d - allowed).max()) if d.numel() else 0.0
    assert bool((d <= allowed + 1e-38).all()), f"off by {worst:.3g} more than allowed, {int((d > allowed).sum())} of {d.numel()}"
