"""Plain 64-bit numpy implementation of the 4-bit-weight operators, and the
error bounds their kernels are held to.

Bounds.  Outputs are rounded once to bf16: half a step, 2^-8 of the value.
Before that a sum of K products goes through at most ROUNDINGS(K) fp32
roundings on any path: 8 chained matrix instructions of a 128-wide chunk, each
counted as two (their internal alignment may truncate), one addition per scale
group, one per slice of K, and a few constants.  Each is at most 2^-23 of the
sum of absolute products (2^-24 for a rounding, twice that for a truncation).
An activation is carried with 11 significant bits in fp16: bf16 values are
exact down to 2^-31 of their slice's largest magnitude and off by at most
2^-39 of it below (half of the smallest step, 2^-25, of at least 2^14).
"""

from __future__ import annotations

import numpy as np

import synth

MXFP4, INT4 = 0, 1
FORMATS = [(MXFP4, 32), (INT4, 32), (INT4, 64), (INT4, 128)]
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
HALF_BF16 = 2.0 ** -8


def roundings(K: int) -> int:
    return 16 + K // 32 + 16


def bf16(v) -> np.ndarray:
    """bf16 bit patterns (nearest even) of finite float64 values that fp32 holds."""
    return synth.f32_to_bf16_bits(np.asarray(v, dtype=np.float32))


def value(codes: np.ndarray, scales: np.ndarray, fmt: int, group: int) -> np.ndarray:
    """float64 [..., K] of codes uint8 [..., K/2] and scales (uint8 e8m0 or uint16 bf16)."""
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    if fmt == MXFP4:
        v = np.where(n >= 8, -1.0, 1.0) * E2M1[n & 7]
        s = 2.0 ** (scales.astype(np.float64) - 127)
    else:
        v = n.astype(np.float64) - 8
        s = synth.bf16_bits_to_f32(scales).astype(np.float64)
    return v * np.repeat(s, group, -1)


def quant(w: np.ndarray, fmt: int, group: int):
    """fp32 w [N, K] -> (codes, scales): the definition, in fp32 where it says so."""
    N, K = w.shape
    g = w.reshape(N, K // group, group)
    amax = np.abs(g).max(-1).astype(np.float32)
    if fmt == MXFP4:
        m, e = np.frexp((amax / np.float32(6)).astype(np.float64))
        byte = np.clip(np.where(m == 0.5, e - 1, e) + 127, 0, 254)
        byte = np.where(amax == 0, 0, byte).astype(np.uint8)
        v = np.abs(g.astype(np.float64)) / (2.0 ** (byte.astype(np.float64) - 127))[..., None]
        d = np.abs(v[..., None] - E2M1)
        best = d.min(-1, keepdims=True)
        # of two equally near values the one with an even code
        near = d == best
        code = np.where(near.sum(-1) > 1, np.where(near & (np.arange(8) % 2 == 0), np.arange(8), 0).max(-1), near.argmax(-1))
        n = code | (np.signbit(g).astype(np.int64) << 3)
        scales = byte
    else:
        scales = bf16(amax / np.float32(7))
        s = synth.bf16_bits_to_f32(scales)[..., None]
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.rint((g / s).astype(np.float32))
        n = (np.clip(np.where(s > 0, q, 0), -8, 7) + 8).astype(np.int64)
    n = n.reshape(N, K)
    return (n[:, 0::2] | (n[:, 1::2] << 4)).astype(np.uint8), scales.reshape(N, K // group)


def weight(rows: int, K: int, fmt: int, group: int, seed: int):
    return quant(synth.w_f32(rows, K, seed=seed), fmt, group)


def gemv(x: np.ndarray, w: np.ndarray):
    """(y, bound) float64: x bf16 bits [M, K], w float64 [N, K]."""
    xf = synth.bf16_bits_to_f32(x).astype(np.float64)
    y = xf @ w.T
    total = np.abs(xf) @ np.abs(w).T
    flush = 2.0 ** -39 * np.abs(xf).max(1, keepdims=True) * np.abs(w).sum(1)
    err = roundings(x.shape[1]) * 2.0 ** -23 * total + flush
    return y, HALF_BF16 * np.abs(y) + (1 + HALF_BF16) * err


def moe(x, ids, tw, w13, w2):
    """(y, bound) float64; w13 [E, 2I, H] and w2 [E, H, I] float64; ids outside
    [0, E) contribute nothing."""
    xf = synth.bf16_bits_to_f32(x).astype(np.float64)
    M, H = xf.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    y, err = np.zeros((M, H)), np.zeros((M, H))
    for m in range(M):
        for s in range(ids.shape[1]):
            e, t = int(ids[m, s]), float(tw[m, s])
            if not 0 <= e < E:
                continue
            h = w13[e] @ xf[m]
            dh = roundings(H) * 2.0 ** -23 * (np.abs(w13[e]) @ np.abs(xf[m])) + 2.0 ** -39 * np.abs(xf[m]).max() * np.abs(w13[e]).sum(1)
            g, u = h[:I], h[I:]
            silu = g / (1 + np.exp(-g))
            a = silu * u
            # |silu'| <= 1.1; exp within 2 units, division and products a few roundings
            da = 1.1 * dh[:I] * (np.abs(u) + dh[I:]) + np.abs(silu) * dh[I:] + 2.0 ** -20 * np.abs(a)
            da = da + 2.0 ** -11 * (np.abs(a) + da) + 2.0 ** -39 * np.abs(a).max()
            o = w2[e] @ a
            do = np.abs(w2[e]) @ da + roundings(I) * 2.0 ** -23 * (np.abs(w2[e]) @ (np.abs(a) + da))
            y[m] += t * o
            err[m] += abs(t) * (do + (ids.shape[1] + 1) * 2.0 ** -24 * np.abs(o))
    return y, HALF_BF16 * np.abs(y) + (1 + HALF_BF16) * err


def route(x, w, E, k, renorm, shared):
    """(ids, weights, relative bound of the weights), w bf16 bits [E or E + 1, H]."""
    xf, wf = (synth.bf16_bits_to_f32(v).astype(np.float64) for v in (x, w))
    logits = xf @ wf.T
    err = roundings(x.shape[1]) * 2.0 ** -23 * (np.abs(xf) @ np.abs(wf).T).max(1, keepdims=True)
    l = logits[:, :E]
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    p = np.exp(l - l.max(1, keepdims=True))
    p = p / p.sum(1, keepdims=True)
    wt = np.take_along_axis(p, order, 1)
    if renorm:
        wt = wt / wt.sum(1, keepdims=True)
    if shared != "none":
        order = np.concatenate((order, np.full_like(order[:, :1], E)), 1)
        last = 1 / (1 + np.exp(-logits[:, E:])) if shared == "gate" else np.ones_like(wt[:, :1])
        wt = np.concatenate((wt, last), 1)
    # numerator, denominator, and exp's own error relative to its argument
    rel = 2 * err + 2.0 ** -19
    return order.astype(np.int32), wt, rel * np.ones_like(wt)
