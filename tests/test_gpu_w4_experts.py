"""The 4-bit expert layer where its kept activations decide the result."""

import numpy as np
import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
import synth
from tests import w4_reference as R

pytestmark = pytest.mark.gpu

MXFP4, INT4 = R.MXFP4, R.INT4


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fb.build()
    fb.lib()
    return torch.device("cuda", 0)


def to_dev(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def bf16_dev(bits, dev):
    return to_dev(np.ascontiguousarray(bits).view(np.int16), dev).view(torch.bfloat16)


def scales_dev(scales, fmt, dev):
    return to_dev(scales, dev) if fmt == MXFP4 else bf16_dev(scales, dev)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def encoded(values, fmt, group):
    """(codes, scales of 1) of float64 values [..., K] that the format's codes hold."""
    if fmt == MXFP4:
        n = np.abs(np.abs(values)[..., None] - R.E2M1).argmin(-1) + 8 * (values < 0)
        scales = np.full((*values.shape[:-1], values.shape[-1] // group), 127, np.uint8)
    else:
        n = (values + 8).astype(np.int64)
        scales = np.full((*values.shape[:-1], values.shape[-1] // group), 0x3F80, np.uint16)
    codes = (n[..., 0::2] | n[..., 1::2] << 4).astype(np.uint8)
    assert np.array_equal(R.value(codes, scales, fmt, group), values)
    return codes, scales


@pytest.mark.parametrize("fmt,group", R.FORMATS)
@pytest.mark.parametrize("M", [1, 3, 5, 9, 18])
def test_moe_differences_of_nearly_equal_activations(dev, fmt, group, M):
    # Rows of w2 subtract activations silu(g) (1 + c / 512) from one another, so
    # that an output is a few 512ths of them.  An activation is the product of
    # an exact fp32 sum and one silu common to its token: off by 2^-24 of itself
    # and silu's 2^-20, which the differences share.  Kept as the sum of two
    # fp16 numbers it is off by 2^-22 more, and 2^-39 of the largest.
    Hd, I, E = 512, 256, 2
    levels = np.arange(-6, 7) if fmt == INT4 else np.array([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6])
    x = np.zeros((M, Hd))
    x[:, 3], x[:, 40], x[:, 300] = 1.0, 2.0 ** -9, 1.0 + np.arange(M) / 16.0
    w13 = np.zeros((E, 2 * I, Hd))
    w13[:, :I, 300] = 1.0
    w13[:, I:, 3] = 1.0
    w13[:, I:, 40] = levels[np.arange(I) % len(levels)]
    w2 = np.zeros((E, Hd, I))
    row = np.arange(Hd)
    w2[:, row, row % I] = 1.0
    w2[:, row, (5 * row + 7) % I] -= 1.0
    c13, s13 = encoded(w13, fmt, group)
    c2, s2 = encoded(w2, fmt, group)
    ids, tw = np.full((M, 1), 1, np.int32), np.ones((M, 1), np.float32)
    y = f64(fb.fp8bs_moe_w4a16(bf16_dev(R.bf16(x), dev), to_dev(ids, dev), to_dev(tw, dev), to_dev(c13, dev),
                               scales_dev(s13, fmt, dev), to_dev(c2, dev), scales_dev(s2, fmt, dev), fmt, group))
    h = x @ w13[1].T
    g, u = h[:, :I], h[:, I:]
    a = g / (1 + np.exp(-g)) * u
    ref, total = a @ w2[1].T, np.abs(a) @ np.abs(w2[1]).T
    err = (2.0 ** -24 + 2.0 ** -22 + 2.0 ** -39 + R.roundings(I) * 2.0 ** -23) * total + 2.0 ** -20 * np.abs(ref)
    bound = R.HALF_BF16 * np.abs(ref) + (1 + R.HALF_BF16) * err
    assert np.all(np.abs(y - ref) <= bound), np.max(np.abs(y - ref) / bound)
