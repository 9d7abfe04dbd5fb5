"""4-bit weights whose scales lie far apart: a weight is its code's value times
its group's scale, whatever stands in the rows and groups beside it."""

import numpy as np
import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
import synth
from tests import w4_reference as R
from tests.test_gpu_w4_experts import bf16_dev, dev, f64, scales_dev, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu

MXFP4, INT4 = R.MXFP4, R.INT4


def power_scales(exponents, fmt):
    """Scales 2^e."""
    if fmt == MXFP4:
        return (exponents + 127).astype(np.uint8)
    return R.bf16(2.0 ** exponents.astype(np.float64))


@pytest.mark.parametrize("fmt,group", R.FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (3, 16, 1024), (8, 5000, 512), (12, 70, 2048)])
def test_gemv_large_scales_beside_tiny_ones(dev, fmt, group, M, N, K):  # noqa: F811
    # rows in turn large (2^97 and more) and tiny (down to 2^-120), so that no
    # output leaves bf16's range: x about 2^10, at most 2^16
    rng = np.random.default_rng(M + N)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    e = np.where((np.arange(N) % 3 == 0)[:, None], rng.integers(97, 102, (N, K // group)),
                 rng.integers(-120, -60, (N, K // group)))
    scales = power_scales(e, fmt)
    x = R.bf16(synth.bf16_bits_to_f32(synth.x_bf16(M, K, seed=N)).astype(np.float64) * 2.0 ** 10)
    y = f64(fb.fp8bs_gemv_w4a16(bf16_dev(x, dev), to_dev(codes, dev), scales_dev(scales, fmt, dev), fmt, group))
    ref, bound = R.gemv(x, R.value(codes, scales, fmt, group))
    assert np.all(np.isfinite(y)) and np.all(np.abs(y - ref) <= bound), np.max(np.abs(y - ref) / bound)


@pytest.mark.parametrize("fmt,group", R.FORMATS)
def test_gemv_large_scales_of_empty_groups(dev, fmt, group):  # noqa: F811
    # in every row the groups with a large scale hold zeros: the others decide
    M, N, K = 4, 48, 1024
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 256, (N, K // group, group // 2)).astype(np.uint8)
    e = rng.integers(-118, -80, (N, K // group))
    large = rng.random((N, K // group)) < 0.5
    e[large] = 120
    codes[large] = 0x88 if fmt == INT4 else 0x00
    codes, scales = codes.reshape(N, K // 2), power_scales(e, fmt)
    x = R.bf16(synth.bf16_bits_to_f32(synth.x_bf16(M, K, seed=9)).astype(np.float64) * 2.0 ** 12)
    y = f64(fb.fp8bs_gemv_w4a16(bf16_dev(x, dev), to_dev(codes, dev), scales_dev(scales, fmt, dev), fmt, group))
    w = R.value(codes, scales, fmt, group)
    ref, bound = R.gemv(x, w)
    assert np.all(np.abs(y - ref) <= bound), np.max(np.abs(y - ref) / bound)


@pytest.mark.parametrize("fmt,group", R.FORMATS)
def test_moe_large_scales_beside_tiny_ones(dev, fmt, group):  # noqa: F811
    M, S, E, Hd, I = 5, 2, 3, 256, 256
    rng = np.random.default_rng(17)
    c13, c2 = (rng.integers(0, 256, s).astype(np.uint8) for s in ((E, 2 * I, Hd // 2), (E, Hd, I // 2)))
    # up rows in turn 2^97 and more and 2^-100, gates about 1; rows of w2 the same
    e13 = np.zeros((E, 2 * I, Hd // group), np.int64) - 4
    e13[:, I:] = np.where(np.arange(I) % 2, 97, -100)[None, :, None]
    e2 = np.broadcast_to(np.where(np.arange(Hd) % 2, -40, -110)[None, :, None], (E, Hd, I // group)).copy()
    e2[:, 5] = 98
    # row 5 takes no activation of a large row
    v = c2.reshape(E, Hd, I // 2)
    zero = 0x8 if fmt == INT4 else 0x0
    v[:, 5] = (v[:, 5] & 0x0F) | zero << 4
    s13, s2 = power_scales(e13, fmt), power_scales(e2, fmt)
    x = synth.x_bf16(M, Hd, seed=18)
    ids, tw = synth.moe_routing(M, S, E, seed=19)
    y = f64(fb.fp8bs_moe_w4a16(bf16_dev(x, dev), to_dev(ids, dev), to_dev(tw, dev), to_dev(c13, dev),
                               scales_dev(s13, fmt, dev), to_dev(c2, dev), scales_dev(s2, fmt, dev), fmt, group))
    ref, bound = R.moe(x, ids, tw, R.value(c13, s13, fmt, group), R.value(c2, s2, fmt, group))
    keep = np.arange(Hd) != 5  # (there the small activations are below 2^-39 of the largest)
    assert np.all(np.abs(y - ref)[:, keep] <= bound[:, keep])


@pytest.mark.parametrize("fmt,group", R.FORMATS)
def test_quantiser_keeps_infinities_and_nan_in_sight(dev, fmt, group):  # noqa: F811
    # no code stands for them: their group becomes NaN, the others stay what they are
    N, K = 9, 512
    w = synth.w_f32(N, K, seed=23)
    clean_c, clean_s = R.quant(w, fmt, group)
    bad = w.copy()
    bad[1, 5], bad[2, 500], bad[3, 130], bad[8, 256] = np.inf, -np.inf, np.nan, np.nan
    bad[3, 131] = np.inf
    codes, scales = fb.fp8bs_quant_weight_w4(to_dev(bad, dev), fmt, group)
    x = R.bf16(np.ones((1, K)))
    y = f64(fb.fp8bs_gemv_w4a16(bf16_dev(x, dev), codes, scales, fmt, group))[0]
    assert np.array_equal(np.isnan(y), np.isin(np.arange(N), (1, 2, 3, 8)))
    codes = codes.cpu().numpy()
    scales = scales.cpu().numpy() if fmt == MXFP4 else scales.view(torch.int16).cpu().numpy().view(np.uint16)
    hit = np.zeros((N, K // group), bool)
    for r, c in ((1, 5), (2, 500), (3, 130), (8, 256)):
        hit[r, c // group] = True
    assert np.array_equal(scales[~hit], clean_s[~hit])
    assert np.all(scales[hit] == (255 if fmt == MXFP4 else 0x7FC0))
    half = np.repeat(hit, group // 2, 1)
    assert np.array_equal(codes[~half], clean_c[~half])
    assert np.all(codes[half] == (0 if fmt == MXFP4 else 0x88))
