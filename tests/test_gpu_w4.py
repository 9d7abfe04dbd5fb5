"""The 4-bit-weight decode operators (quantiser, GEMV, router, expert layer)
against their plain 64-bit implementation.  Bounds are derived in
w4_reference.py, none is measured."""

import numpy as np
import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
import synth
from tests import helpers as H
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


def check(got, ref, bound, what):
    d = np.abs(f64(got) - ref)
    assert np.all(np.isfinite(f64(got))), what
    assert np.all(d <= bound), f"{what}: {np.max(d / np.maximum(bound, 1e-300))} of the bound"


def run_gemv(dev, M, N, K, fmt, group, seed, x=None, **kw):
    x = synth.x_bf16(M, K, seed=seed) if x is None else x
    codes, scales = R.weight(N, K, fmt, group, seed + 1)
    y = fb.fp8bs_gemv_w4a16(bf16_dev(x, dev), to_dev(codes, dev), scales_dev(scales, fmt, dev), fmt, group, **kw)
    return y, x, R.value(codes, scales, fmt, group)


# ---- quantiser -----------------------------------------------------------------

def special_weights(N, K, seed):
    w = synth.w_f32(N, K, seed=seed)
    w[0, :] = 0.0
    w[0, 1] = -0.0
    w[1, :K // 2] *= np.float32(1e-30)
    w[1, K // 2:] *= np.float32(1e30)
    w[2, :] = 6.0
    w[3, :] = np.tile(np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25],
                               np.float32), K // 16)  # every tie of e2m1
    w[4, :] = np.tile(np.array([7, 6.5, 5.5, 0.5, 1.5, -7, -0.5, -1.5], np.float32), K // 8)  # ties of the integers
    w[5, ::128] = 1e-42  # subnormal amax
    w[5, 1:] *= np.float32(1e-42)
    return w


@pytest.mark.parametrize("fmt,group", R.FORMATS)
@pytest.mark.parametrize("N,K", [(7, 128), (33, 640), (129, 2048)])
def test_quant_weight_codes_and_scales(dev, fmt, group, N, K):
    w = special_weights(N, K, seed=N + K)
    wide = torch.zeros((N, K + 64), device=dev)
    wide[:, :K] = to_dev(w, dev)
    codes, scales = fb.fp8bs_quant_weight_w4(wide[:, :K], fmt, group)
    ref_c, ref_s = R.quant(w, fmt, group)
    got_s = scales.cpu().numpy() if fmt == MXFP4 else H.torch_u16_to_np(scales)
    assert np.array_equal(got_s, ref_s)
    assert np.array_equal(codes.cpu().numpy(), ref_c)


# ---- GEMV ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,group", R.FORMATS)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 128),      # one row, one chunk: seven idle row tiles
    (1, 17, 256),     # two slices of K
    (2, 250, 384),    # a chunk count that is no power of two
    (3, 1031, 1152),  # 9 chunks over 8 slices: one slice of none
    (7, 96, 5120),    # a slice in two stages, the second partly filled
    (8, 513, 2048),
    (9, 40, 1024),    # two tiles of token columns
    (16, 130, 4096),
    (16, 35, 16384),  # the activations do not all fit in shared memory
])
def test_gemv_matches_64_bits(dev, fmt, group, M, N, K):
    y, x, w = run_gemv(dev, M, N, K, fmt, group, seed=10 * M + N)
    check(y, *R.gemv(x, w), f"gemv {M}x{N}x{K}")


@pytest.mark.parametrize("M", range(1, 17))
def test_gemv_every_token_count(dev, M):
    y, x, w = run_gemv(dev, M, 64, 1024, MXFP4, 32, seed=900 + M)
    check(y, *R.gemv(x, w), f"gemv M={M}")


def test_gemv_more_tiles_than_blocks(dev):
    y, x, w = run_gemv(dev, 4, 12000, 512, INT4, 128, seed=77)
    check(y, *R.gemv(x, w), "gemv persistent grid")


@pytest.mark.parametrize("fmt,group", R.FORMATS)
def test_gemv_strided_operands_and_output(dev, fmt, group):
    M, N, K = 5, 70, 1024
    x = synth.x_bf16(M, K, seed=5)
    codes, scales = R.weight(N, K, fmt, group, 6)
    xw = torch.full((M, K + 40), float("nan"), dtype=torch.bfloat16, device=dev)
    xw[:, 8:8 + K] = bf16_dev(x, dev)
    cw = torch.full((N, K // 2 + 64), 0x77, dtype=torch.uint8, device=dev)
    cw[:, 16:16 + K // 2] = to_dev(codes, dev)
    s = scales_dev(scales, fmt, dev)
    sw = torch.zeros((N, K // group + 32), dtype=s.dtype, device=dev)
    sw[:, 8:8 + K // group] = s
    yw = torch.full((M, N + 3), 7.0, dtype=torch.bfloat16, device=dev)
    fb.fp8bs_gemv_w4a16(xw[:, 8:8 + K], cw[:, 16:16 + K // 2], sw[:, 8:8 + K // group], fmt, group, y=yw[:, 1:1 + N])
    check(yw[:, 1:1 + N], *R.gemv(x, R.value(codes, scales, fmt, group)), "strided")
    assert bool((yw[:, 0] == 7).all()) and bool((yw[:, 1 + N:] == 7).all())


def test_gemv_every_code_and_scale_byte(dev):
    # x picks single columns, so each output is one weight: exact
    K, N = 128, 16 * 8
    codes = np.tile(np.arange(256, dtype=np.uint8)[:64], (N, 1))
    codes = (codes + 16 * np.arange(N, dtype=np.uint8)[:, None]).astype(np.uint8)
    scales = np.broadcast_to((np.arange(N, dtype=np.uint8) + 60)[:, None], (N, K // 32)).copy()
    w = R.value(codes, scales, MXFP4, 32)
    for k0 in range(0, K, 16):
        x = np.zeros((16, K), np.float32)
        x[np.arange(16), k0 + np.arange(16)] = 1.0
        y = fb.fp8bs_gemv_w4a16(bf16_dev(R.bf16(x), dev), to_dev(codes, dev), to_dev(scales, dev), MXFP4, 32)
        assert np.array_equal(f64(y), w[:, k0:k0 + 16].T)


def test_gemv_all_scale_exponents(dev):
    # every e8m0 byte but 255, against an activation that keeps the product in range
    N, K = 255, 128
    codes = np.full((N, K // 2), 0x22, np.uint8)  # 1.0
    scales = np.repeat(np.arange(N, dtype=np.uint8)[:, None], K // 32, 1)
    for e in (-20, 0, 20):
        x = np.zeros((1, K), np.float32)
        x[0, 5] = 2.0 ** e
        y = f64(fb.fp8bs_gemv_w4a16(bf16_dev(R.bf16(x), dev), to_dev(codes, dev), to_dev(scales, dev), MXFP4, 32))[0]
        want = 2.0 ** (np.arange(N) - 127.0 + e)
        ok = (want < 2.0 ** 128) & (want >= 2.0 ** -126)
        assert np.array_equal(y[ok], want[ok])
        assert np.all(np.isinf(y[want >= 2.0 ** 128]))


@pytest.mark.parametrize("factor", [2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 2.0 ** 110])
def test_gemv_activation_range(dev, factor):
    x = R.bf16(synth.bf16_bits_to_f32(synth.x_bf16(3, 1024, seed=31)).astype(np.float64) * factor)
    y, x, w = run_gemv(dev, 3, 64, 1024, INT4, 64, seed=32, x=x)
    ref, bound = R.gemv(x, w)
    check(y, ref, bound + 2.0 ** -133, "range")


def test_gemv_wide_activation_range_keeps_small_values(dev):
    # a slice whose large values meet zero weights: the small ones decide
    M, N, K = 1, 16, 1024
    x = np.full((M, K), 2.0 ** -20, np.float32)
    x[:, ::2] = 1024.0
    codes = np.full((N, K // 2), 0x20, np.uint8)  # even k: 0, odd k: 1.0
    scales = np.full((N, K // 32), 127, np.uint8)
    y = fb.fp8bs_gemv_w4a16(bf16_dev(R.bf16(x), dev), to_dev(codes, dev), to_dev(scales, dev), MXFP4, 32)
    assert np.array_equal(f64(y), np.full((M, N), K / 2 * 2.0 ** -20))


@pytest.mark.parametrize("fmt,group", [(MXFP4, 32), (INT4, 128)])
def test_gemv_infinities_and_nan_stay_in_their_token(dev, fmt, group):
    M, N, K = 6, 40, 1024
    x = synth.x_bf16(M, K, seed=41)
    x[1, 100] = 0x7F80   # inf
    x[2, 7] = 0xFF80     # -inf
    x[3, 900] = 0x7FC0   # NaN
    x[4, :] = 0
    y, x, w = run_gemv(dev, M, N, K, fmt, group, seed=41, x=x)
    xf = synth.bf16_bits_to_f32(x).astype(np.float64)
    got = f64(y)
    clean = [0, 4, 5]
    ref, bound = R.gemv(x[clean], w)
    assert np.all(np.abs(got[clean] - ref) <= bound)
    assert np.all(got[4] == 0)
    with np.errstate(invalid="ignore"):
        for m in (1, 2, 3):
            want = (xf[m] * w).sum(1)
            assert np.array_equal(np.isnan(got[m]), np.isnan(want))
            fine = ~np.isnan(want)
            assert np.array_equal(got[m][fine], want[fine])


def test_gemv_repeats_bit_for_bit_on_another_stream_pdl_and_graph(dev):
    M, N, K, fmt, group = 4, 1000, 2048, MXFP4, 32
    x = bf16_dev(synth.x_bf16(M, K, seed=51), dev)
    codes, scales = R.weight(N, K, fmt, group, 52)
    codes, scales = to_dev(codes, dev), scales_dev(scales, fmt, dev)
    first = fb.fp8bs_gemv_w4a16(x, codes, scales, fmt, group)
    outs = [torch.zeros_like(first) for _ in range(5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fb.fp8bs_gemv_w4a16(x, codes, scales, fmt, group, y=outs[0], stream=side)
    with torch.cuda.stream(side):
        for i in (1, 2, 3):
            fb.fp8bs_gemv_w4a16(x, codes, scales, fmt, group, y=outs[i], pdl=i > 1)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.fp8bs_gemv_w4a16(x, codes, scales, fmt, group, y=outs[4])
    graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), first.view(torch.int16))


def test_gemv_codes_beyond_32_bit_offsets(dev):
    # 5.4 GB of codes; only the first and the last rows are not zero
    M, N, K, fmt, group = 2, (1 << 20) + 5, 10240, INT4, 128
    x = synth.x_bf16(M, K, seed=71)
    c, s = R.weight(64, K, fmt, group, 72)
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device=dev)  # the value 0
    scales = torch.ones((N, K // group), dtype=torch.bfloat16, device=dev)
    for rows in (slice(0, 32), slice(N - 32, N)):
        part = slice(0, 32) if rows.start == 0 else slice(32, 64)
        codes[rows] = to_dev(c[part], dev)
        scales[rows] = scales_dev(s[part], fmt, dev)
    y = fb.fp8bs_gemv_w4a16(bf16_dev(x, dev), codes, scales, fmt, group)
    ref, bound = R.gemv(x, R.value(c, s, fmt, group))
    check(torch.cat((y[:, :32], y[:, N - 32:]), 1), ref, bound, "large offsets")
    assert bool((y[:, 32:N - 32] == 0).all())


def test_gemv_empty_batch(dev):
    y = torch.full((0, 64), 1.0, dtype=torch.bfloat16, device=dev)
    codes, scales = R.weight(64, 256, MXFP4, 32, 1)
    out = fb.fp8bs_gemv_w4a16(torch.empty((0, 256), dtype=torch.bfloat16, device=dev), to_dev(codes, dev),
                              to_dev(scales, dev), y=y)
    assert out.shape == (0, 64)


# ---- router ------------------------------------------------------------------------

def run_route(dev, x, w, k, renorm, shared, calls=1):
    E = w.shape[0] - (1 if shared == "gate" else 0)
    ws = fb.new_moe_route_workspace(x.shape[0], E, x.shape[1], dev)
    for _ in range(calls):
        ids, wt = fb.fp8bs_moe_route(bf16_dev(x, dev), bf16_dev(w, dev), k, renorm=renorm, shared=shared, workspace=ws)
    assert int(ws[:4].view(torch.int32).item()) == 0  # ready for the next call
    ref_ids, ref_w, rel = R.route(x, w, E, k, renorm, shared)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    got = f64(wt)
    assert np.all(np.abs(got - ref_w) <= rel * ref_w), np.max(np.abs(got - ref_w) / (rel * ref_w))
    return ids, wt


@pytest.mark.parametrize("renorm,shared", [(True, "one"), (False, "none"), (True, "gate")])
@pytest.mark.parametrize("M,E,Hd,k", [
    (1, 1, 128, 1), (1, 16, 256, 16), (2, 33, 1024, 32), (1, 512, 4096, 10), (31, 160, 640, 6), (32, 257, 512, 8),
    (33, 512, 1024, 10), (70, 1024, 384, 3), (64, 128, 7168, 8),
])
def test_route_matches_64_bits(dev, M, E, Hd, k, renorm, shared):
    x = synth.x_bf16(M, Hd, seed=M + E)
    w = R.bf16(synth.w_f32(E + (shared == "gate"), Hd, seed=M + E + 1))
    run_route(dev, x, w, k, renorm, shared, calls=2)


def test_route_ties_go_to_the_lowest_index(dev):
    Hd, E = 512, 300
    x = synth.x_bf16(5, Hd, seed=61)
    x[4] = 0  # every logit 0
    row = synth.w_f32(3, Hd, seed=62)
    w = R.bf16(row[np.arange(E) % 3])  # three values, each a hundred times
    w[150:] = R.bf16(synth.w_f32(E - 150, Hd, seed=63) * np.float32(0.01))
    ids, _ = run_route(dev, x, w, 8, True, "none")
    assert np.array_equal(ids[4].cpu().numpy(), np.arange(8))


def test_route_near_ties_follow_the_exact_logits(dev):
    # pairs of experts whose logits differ by less than fp32 sums resolve
    Hd, E, k = 4096, 64, 6
    rng = np.random.default_rng(7)
    base = synth.w_f32(E // 2, Hd, seed=64)
    w = np.repeat(base, 2, 0)
    x = synth.bf16_bits_to_f32(synth.x_bf16(16, Hd, seed=65)).copy()
    col = rng.integers(0, Hd, E // 2)
    wb = synth.bf16_bits_to_f32(R.bf16(w)).copy()
    x[:, col] = (rng.choice([-1.0, 1.0], (16, E // 2)) * 2.0 ** -18).astype(np.float32)
    wb[1::2][np.arange(E // 2), col] = 0.5  # logit off by about 2^-19
    run_route(dev, R.bf16(x), R.bf16(wb), k, True, "none")


def test_route_nan_and_infinite_logits(dev):
    Hd, E, k = 256, 40, 4
    x = synth.x_bf16(4, Hd, seed=66, outliers=False)
    w = R.bf16(synth.w_f32(E, Hd, seed=67))
    x[1, 3] = 0x7FC0  # every logit NaN
    w2 = w.copy()
    w2[9, 0] = 0x7FC0  # one expert's logit NaN for every token
    ids, wt = fb.fp8bs_moe_route(bf16_dev(x, dev), bf16_dev(w2, dev), k, shared="one")
    ids, wt = ids.cpu().numpy(), f64(wt)
    assert np.all(np.isnan(wt[:, :k])) and np.all(wt[:, k] == 1)
    for m in range(4):
        assert len(set(ids[m, :k])) == k and ids[m, k] == E and np.all((ids[m, :k] >= 0) & (ids[m, :k] < E))
    ref, _, _ = R.route(x[:1], w, E, E, True, "none")
    assert np.array_equal(ids[0, :k], [e for e in ref[0] if e != 9][:k])


# ---- expert layer --------------------------------------------------------------------

def experts(E, Hd, I, fmt, group, seed):
    c13, s13 = R.weight(E * 2 * I, Hd, fmt, group, seed)
    c2, s2 = R.weight(E * Hd, I, fmt, group, seed + 1)
    return (c13.reshape(E, 2 * I, -1), s13.reshape(E, 2 * I, -1), c2.reshape(E, Hd, -1), s2.reshape(E, Hd, -1))


def run_moe(dev, M, S, E, Hd, I, fmt, group, seed, ids=None, tw=None, calls=1):
    x = synth.x_bf16(M, Hd, seed=seed)
    if ids is None:
        ids, tw = synth.moe_routing(M, S, E, seed=seed + 1)
    c13, s13, c2, s2 = experts(E, Hd, I, fmt, group, seed + 2)
    ws = fb.new_moe_w4_workspace(M, S, I, dev)
    outs = []
    for _ in range(calls):
        outs.append(fb.fp8bs_moe_w4a16(bf16_dev(x, dev), to_dev(ids, dev), to_dev(tw, dev), to_dev(c13, dev),
                                       scales_dev(s13, fmt, dev), to_dev(c2, dev), scales_dev(s2, fmt, dev), fmt, group,
                                       workspace=ws))
    status = fb.fp8bs_check_error(ws)
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    ref, bound = R.moe(x, ids, tw, R.value(c13, s13, fmt, group), R.value(c2, s2, fmt, group))
    check(outs[0], ref, bound, f"moe M={M} S={S} E={E} H={Hd} I={I}")
    return status


@pytest.mark.parametrize("fmt,group", R.FORMATS)
@pytest.mark.parametrize("M,S,E,Hd,I", [
    (1, 1, 2, 128, 128), (1, 4, 9, 512, 256), (3, 3, 7, 1152, 128), (8, 4, 16, 1024, 384), (20, 4, 9, 640, 512),
    (5, 2, 5, 256, 640),
])
def test_moe_matches_64_bits(dev, fmt, group, M, S, E, Hd, I):
    assert run_moe(dev, M, S, E, Hd, I, fmt, group, seed=100 + M + I) == 0


def test_moe_many_experts_and_repeats(dev):
    assert run_moe(dev, 16, 11, 513, 512, 128, MXFP4, 32, seed=300, calls=3) == 0


def test_moe_wide_hidden_size(dev):
    # 5 chunks of H a warp: the second stage of a slice is partly filled
    assert run_moe(dev, 4, 5, 12, 5120, 128, INT4, 64, seed=310) == 0


def test_moe_largest_hidden_size(dev):
    assert run_moe(dev, 2, 2, 2, 32768, 128, MXFP4, 32, seed=320) == 0


def test_moe_experts_with_many_pairs(dev):
    M, S, E = 40, 3, 5
    ids = np.tile(np.array([[0, 1, 4]], np.int32), (M, 1))
    tw = np.tile(np.array([[0.5, 0.25, 1.0]], np.float32), (M, 1))
    assert run_moe(dev, M, S, E, 512, 256, INT4, 128, seed=400, ids=ids, tw=tw) == 0


def test_moe_most_pairs(dev):
    assert run_moe(dev, 128, 8, 20, 256, 128, MXFP4, 32, seed=410) == 0


def test_moe_one_expert_in_several_slots(dev):
    ids = np.array([[2, 2, 2], [0, 2, 0]], np.int32)
    tw = np.array([[0.5, 0.25, -1.0], [0.0, 1.0, 2.0]], np.float32)
    assert run_moe(dev, 2, 3, 3, 256, 128, MXFP4, 32, seed=420, ids=ids, tw=tw) == 0


def test_moe_invalid_ids_are_reported_and_contribute_nothing(dev):
    M, S, E = 3, 4, 6
    ids, tw = synth.moe_routing(M, S, E, seed=501)
    ids[1, 2], ids[2, 0] = E + 7, -3
    tw[2, 0] = np.nan
    assert run_moe(dev, M, S, E, 256, 128, INT4, 32, seed=502, ids=ids, tw=tw) == fb.FP8BS_ERR_DEVICE


def test_moe_only_invalid_ids_give_zeros(dev):
    ids = np.full((2, 2), -1, np.int32)
    tw = np.ones((2, 2), np.float32)
    assert run_moe(dev, 2, 2, 3, 256, 128, MXFP4, 32, seed=510, ids=ids, tw=tw) == fb.FP8BS_ERR_DEVICE


def test_moe_weights_beyond_32_bit_offsets(dev):
    # 4.3 GB of gate/up codes: the experts used are the first and the last
    E, Hd, I, fmt, group, M = 4096, 4096, 256, MXFP4, 32, 3
    c13, s13, c2, s2 = experts(2, Hd, I, fmt, group, 520)
    big = [torch.zeros((E, *v.shape[1:]), dtype=torch.uint8, device=dev) for v in (c13, s13, c2, s2)]
    for b, v in zip(big, (c13, s13, c2, s2)):
        b[0], b[E - 1] = to_dev(v[0], dev), to_dev(v[1], dev)
    x = synth.x_bf16(M, Hd, seed=521)
    small = np.array([[0, 1], [1, 0], [1, 1]], np.int32)
    tw = np.array([[0.5, 0.5], [1.0, -0.25], [0.75, 0.5]], np.float32)
    ws = fb.new_moe_w4_workspace(M, 2, I, dev)
    y = fb.fp8bs_moe_w4a16(bf16_dev(x, dev), to_dev(small * (E - 1), dev), to_dev(tw, dev), *big, fmt, group, workspace=ws)
    assert fb.fp8bs_check_error(ws) == 0
    check(y, *R.moe(x, small, tw, R.value(c13, s13, fmt, group), R.value(c2, s2, fmt, group)), "large offsets")


@pytest.mark.parametrize("fmt,group", [(MXFP4, 32), (INT4, 64)])
def test_moe_infinities_and_nan_stay_in_their_token(dev, fmt, group):
    M, S, E, Hd, I = 5, 3, 4, 512, 256
    x = synth.x_bf16(M, Hd, seed=530)
    x[1, 3], x[3, 400] = 0x7F80, 0x7FC0  # inf, NaN
    ids, tw = synth.moe_routing(M, S, E, seed=531)
    c13, s13, c2, s2 = experts(E, Hd, I, fmt, group, 532)
    y = f64(fb.fp8bs_moe_w4a16(bf16_dev(x, dev), to_dev(ids, dev), to_dev(tw, dev), to_dev(c13, dev),
                               scales_dev(s13, fmt, dev), to_dev(c2, dev), scales_dev(s2, fmt, dev), fmt, group))
    clean = [0, 2, 4]
    ref, bound = R.moe(x[clean], ids[clean], tw[clean], R.value(c13, s13, fmt, group), R.value(c2, s2, fmt, group))
    assert np.all(np.abs(y[clean] - ref) <= bound)
    assert not np.any(np.isfinite(y[[1, 3]]))


@pytest.mark.parametrize("Hd,I,M", [(4096, 128, 8), (4096, 256, 3), (2560, 128, 8), (8192, 128, 2)])
def test_moe_tile_and_warp_choices_of_the_down_projection(dev, Hd, I, M):
    # one and two tiles a stage, 8 and 16 warps, more tiles than blocks
    assert run_moe(dev, M, 4, 12, Hd, I, INT4, 128, seed=540 + M) == 0


def test_layer_routed_and_captured(dev):
    # router, experts and an output projection in one graph, on new tokens
    M, E, Hd, I, k, fmt, group = 6, 12, 512, 128, 3, MXFP4, 32
    c13, s13, c2, s2 = experts(E + 1, Hd, I, fmt, group, 601)
    co, so = R.weight(384, Hd, fmt, group, 603)
    wr = R.bf16(synth.w_f32(E, Hd, seed=604))
    args = [to_dev(v, dev) for v in (c13, s13, c2, s2)]
    cod, sod, wrd = to_dev(co, dev), to_dev(so, dev), bf16_dev(wr, dev)
    x = torch.zeros((M, Hd), dtype=torch.bfloat16, device=dev)
    wsr, wsm = fb.new_moe_route_workspace(M, E, Hd, dev), fb.new_moe_w4_workspace(M, k + 1, I, dev)

    def layer():
        ids, tw = fb.fp8bs_moe_route(x, wrd, k, shared="one", workspace=wsr)
        y = fb.fp8bs_moe_w4a16(x, ids, tw, *args, fmt, group, workspace=wsm)
        return ids, tw, y, fb.fp8bs_gemv_w4a16(y, cod, sod, fmt, group, pdl=True)

    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, tw, y, out = layer()
    for seed in (610, 611):
        xb = synth.x_bf16(M, Hd, seed=seed)
        x.copy_(bf16_dev(xb, dev))
        graph.replay()
        torch.cuda.synchronize()
        ref_ids, ref_w, rel = R.route(xb, wr, E, k, True, "one")
        assert np.array_equal(ids.cpu().numpy(), ref_ids)
        ref, bound = R.moe(xb, ref_ids, tw.cpu().numpy(), R.value(c13, s13, fmt, group), R.value(c2, s2, fmt, group))
        check(y, ref, bound, "layer experts")
        check(out, *R.gemv(H.torch_u16_to_np(y), R.value(co, so, fmt, group)), "layer projection")
    assert fb.fp8bs_check_error(wsm) == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
def test_example_decode_step(dev, fmt):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_w4.py")
    spec = importlib.util.spec_from_file_location("decode_w4", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    # two bf16 roundings on the way (y and the output), half a step each, and
    # fp32 sums far below them
    assert mod.main(["--format", fmt, "--tokens", "5", "--steps", "2"]) <= 2 * R.HALF_BF16
