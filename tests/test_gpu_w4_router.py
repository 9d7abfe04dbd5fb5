"""The router's order where fp32 sums do not decide it.

The order is that of the exact logits.  Each case asserts on the host that
plain fp32 sums, taken in two usual orders, put some token's experts wrong, so
that it does not become empty."""

import numpy as np
import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
import synth
from tests import w4_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fb.build()
    fb.lib()
    return torch.device("cuda", 0)


def bf16_dev(bits, dev):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(dev).view(torch.bfloat16)


def rounded(v):
    """float64 values of the nearest bf16 numbers."""
    return synth.bf16_bits_to_f32(R.bf16(v)).astype(np.float64)


def fp32_logits(x, w, run):
    """x . w^T in fp32: sums of `run` neighbours, then those in order."""
    p = (x[:, None, :] * w[None]).astype(np.float32).reshape(x.shape[0], w.shape[0], -1, run)
    part = np.zeros(p.shape[:-1], np.float32)
    for i in range(run):
        part = part + p[..., i]
    total = np.zeros(part.shape[:-1], np.float32)
    for i in range(part.shape[-1]):
        total = total + part[..., i]
    return total


def check(dev, x, w, k, M):
    """Route all of x, M tokens a call."""
    logits = x @ w.T
    order = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    for run in (16, 128):
        plain = np.argsort(-fp32_logits(x[:12], w, run), axis=1, kind="stable")[:, :k]
        assert np.any(plain != order[:12]), "fp32 sums are enough for this case"
    outs = [fb.fp8bs_moe_route(bf16_dev(R.bf16(x[m:m + M]), dev), bf16_dev(R.bf16(w), dev), k)
            for m in range(0, len(x), M)]
    ids, wt = (torch.cat(t).cpu().numpy() for t in zip(*outs))
    wrong = np.any(ids != order, axis=1)
    assert not np.any(wrong), f"{wrong.sum()} of {len(x)} tokens"
    # a chosen logit's fp32 sum is off by roundings(H) 2^-23 of the sum of magnitudes, in
    # the numerator and in the denominator; exp and the division by 2^-19
    z = np.exp(logits - logits.max(1, keepdims=True))
    ref = np.take_along_axis(z, order, 1)
    ref = ref / ref.sum(1, keepdims=True)
    err = R.roundings(x.shape[1]) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T).max(1, keepdims=True)
    assert np.all(np.abs(wt - ref) <= (np.expm1(2 * err) + 2.0 ** -19) * ref)


@pytest.mark.parametrize("M", [1, 8, 9, 40, 70])
@pytest.mark.parametrize("size", [40.0, 100.0, 400.0])
@pytest.mark.parametrize("E,k", [(64, 6), (512, 10), (700, 8)])
def test_route_cancelling_channels(dev, M, size, E, k):
    # two channels of x whose products cancel in every expert, at another size in
    # each; pairs of experts that differ by a few 2^-21 besides
    Hd = 2048
    rng = np.random.default_rng(int(size) + E + M)
    x = rounded(rng.standard_normal((max(M, 12), Hd)))
    w = rounded(np.repeat(rng.standard_normal((E // 2, Hd)) * 0.05, 2, 0))
    x[:, 130], x[:, 1900] = 64.0, 64.0
    q = rounded(rng.uniform(0.5, 1.0, E) * size / 64.0)
    w[:, 130], w[:, 1900] = q, -q
    x[:, 77], w[:, 77] = 2.0 ** -14, 0.0
    w[1::2, 77] = rng.choice([-1.0, 1.0], E // 2) * 2.0 ** -7 * rng.integers(1, 4, E // 2)
    check(dev, x, w, k, M)


@pytest.mark.parametrize("M", [3, 24])
def test_route_the_same_terms_in_another_order(dev, M):
    # x repeats with period 64, rows are rolled by multiples of 64: the same
    # products in another order, and a correcting element that decides
    Hd, E, k = 4096, 48, 6
    rng = np.random.default_rng(5)
    x = np.tile(rounded(rng.standard_normal((24, 64)) * 8), (1, Hd // 64))
    base = rounded(rng.standard_normal((6, Hd)))
    base[:, 9::64] = 0.0
    w = np.stack([np.roll(base[e // 8], 64 * (7 * e % 64)) for e in range(E)])
    w[:, 9] = (rng.permutation(E) - E // 2) * 2.0 ** -9
    x[:, 9::64] = 2.0 ** -9
    check(dev, x, w, k, M)


@pytest.mark.parametrize("M", [2, 12])
def test_route_many_experts_within_rounding(dev, M):
    # every expert within fp32's rounding of every other: the correcting
    # elements alone decide, over more than 64 candidates
    Hd, E, k = 1024, 200, 8
    rng = np.random.default_rng(11)
    x = np.tile(rounded(rng.standard_normal((12, 64)) * 8), (1, Hd // 64))
    base = rounded(rng.standard_normal(Hd))
    base[9::64] = 0.0
    w = np.stack([np.roll(base, 64 * (e % 16)) for e in range(E)])
    w[:, 9] = (rng.permutation(E) - E // 2) * 2.0 ** -10
    x[:, 9::64] = 2.0 ** -12
    check(dev, x, w, k, M)
