"""Each variant of the 4-bit kernels that the sizes choose between: the GEMV's
tiles a stage, ring depths and staging of the activations, over more than one
group of tiles a warp, and the down projection's tiles, warps and stages."""

import numpy as np
import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
import synth
from tests import w4_reference as R
from tests.test_gpu_w4_experts import bf16_dev, dev, f64, scales_dev, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu

MXFP4, INT4 = R.MXFP4, R.INT4


def random_weight(shape, fmt, group, seed):
    """Any codes, scales within a factor of eight of 2^-6."""
    rng = np.random.default_rng(seed)
    *rows, K = shape
    codes = rng.integers(0, 256, (*rows, K // 2)).astype(np.uint8)
    if fmt == MXFP4:
        return codes, rng.integers(119, 124, (*rows, K // group)).astype(np.uint8)
    return codes, R.bf16(rng.uniform(2.0 ** -8, 2.0 ** -5, (*rows, K // group)))


def value_dev(codes, scales, fmt, group, dev):  # noqa: F811
    """float64 [N, K] on the device."""
    c = to_dev(codes, dev)
    n = torch.stack((c & 15, c >> 4), -1).flatten(-2).int()
    if fmt == MXFP4:
        v = torch.tensor(np.concatenate((R.E2M1, -R.E2M1)), device=dev)[n]
    else:
        v = n.double() - 8
    s = to_dev(scales, dev).double()
    s = 2.0 ** (s - 127) if fmt == MXFP4 else scales_dev(scales, fmt, dev).double()
    return v * s.repeat_interleave(group, -1)


@pytest.mark.parametrize("fmt,group", R.FORMATS)
@pytest.mark.parametrize("M,K", [
    (3, 2048),   # two tiles a stage, x kept
    (1, 8192),   # the same, a slice in two stages
    (4, 2048),   # two tiles a stage, x kept or (four groups a chunk) not
    (8, 2048),   # two tiles a stage, x staged for four tiles
    (3, 5120),   # one tile, three stages in flight, x kept
    (5, 5120),   # one tile, two stages in flight, x kept
    (8, 5120),   # one tile, x staged for four tiles a stage at a time
    (2, 40960),  # the same, many stages a slice
    (9, 2048), (16, 5120), (13, 384),
])
def test_gemv_variants_over_several_groups_of_tiles(dev, fmt, group, M, K):  # noqa: F811
    # nine tiles a warp (five of the smaller weights): two groups of four and one more
    N = 19997 if K <= 8192 else 10003
    x = synth.x_bf16(M, K, seed=M + K)
    codes, scales = random_weight((N, K), fmt, group, M + K + 1)
    y = fb.fp8bs_gemv_w4a16(bf16_dev(x, dev), to_dev(codes, dev), scales_dev(scales, fmt, dev), fmt, group)
    w, xd = value_dev(codes, scales, fmt, group, dev), bf16_dev(x, dev).double()
    ref, total = xd @ w.t(), xd.abs() @ w.abs().t()
    # the bound of w4_reference.gemv
    err = R.roundings(K) * 2.0 ** -23 * total + 2.0 ** -39 * xd.abs().amax(1, keepdim=True) * w.abs().sum(1)
    bound = R.HALF_BF16 * ref.abs() + (1 + R.HALF_BF16) * err
    off = (y.double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("fmt,group", R.FORMATS)
@pytest.mark.parametrize("M,S,E,Hd,I", [
    (3, 2, 5, 2560, 128),    # two tiles a stage, all of I in it
    (3, 2, 5, 2560, 384),    # two tiles a stage, I in two stages, the second half filled
    (9, 8, 6, 4096, 768),    # two tiles a stage, several entries an expert
    (20, 9, 7, 2560, 256),   # two tiles, two or three pairs an entry
    (20, 9, 7, 2560, 640),   # the same, I in three stages
    (40, 9, 7, 2560, 256),   # more pairs than two tiles leave room for: 8 warps
    (40, 9, 7, 2560, 640),   # the same, I in three stages
    (88, 3, 9, 512, 128),    # no more tiles than multiprocessors: 16 warps
    (88, 3, 9, 512, 384),    # the same, I in two stages
    (100, 10, 9, 512, 128),  # more pairs than 16 warps leave room for: 8
    (100, 10, 9, 512, 384),  # the same, I in two stages
    (7, 5, 4, 640, 1536),    # few pairs, I in six stages
])
def test_moe_variants(dev, fmt, group, M, S, E, Hd, I):  # noqa: F811
    x = synth.x_bf16(M, Hd, seed=M + I)
    rng = np.random.default_rng(M * S + I)
    ids = rng.integers(0, E, (M, S)).astype(np.int32)
    tw = rng.standard_normal((M, S)).astype(np.float32)
    c13, s13 = random_weight((E, 2 * I, Hd), fmt, group, 7)
    c2, s2 = random_weight((E, Hd, I), fmt, group, 8)
    ws = fb.new_moe_w4_workspace(M, S, I, dev)
    y = fb.fp8bs_moe_w4a16(bf16_dev(x, dev), to_dev(ids, dev), to_dev(tw, dev), to_dev(c13, dev),
                           scales_dev(s13, fmt, dev), to_dev(c2, dev), scales_dev(s2, fmt, dev), fmt, group, workspace=ws)
    assert fb.fp8bs_check_error(ws) == 0
    ref, bound = R.moe(x, ids, tw, R.value(c13, s13, fmt, group), R.value(c2, s2, fmt, group))
    off = np.abs(f64(y) - ref)
    assert np.all(off <= bound), np.max(off / bound)
