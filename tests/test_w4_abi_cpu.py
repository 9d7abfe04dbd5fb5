"""Host checks of the 4-bit-weight entry points and the binding's own refusals:
no device pointer is dereferenced on these paths, nothing is launched."""

import numpy as np
import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
from tests import w4_reference as R

OK, ARG, SHAPE, ALIGN, WS = 0, -1, -2, -3, -5
P = 0x10000000  # a fake, well-aligned device address: refused before any launch

pytestmark = pytest.mark.skipif(
    torch.cuda.is_available(),
    reason="fake device pointers: host-check tests run only where no GPU is visible")


@pytest.fixture(scope="module")
def L():
    fb.build()
    return fb.lib()


def gemv(L, x=P, M=4, ldx=4096, codes=P, ldc=2048, scales=P, lds=128, N=5120, K=4096, fmt=0, group=32, y=P, ldy=5120,
         flags=0):
    return L.fp8bs_gemv_w4a16(x, M, ldx, codes, ldc, scales, lds, N, K, fmt, group, y, ldy, flags, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), ARG), (dict(group=64), ARG), (dict(fmt=1, group=16), ARG), (dict(fmt=1, group=0), ARG),
    (dict(flags=2), ARG), (dict(M=17), SHAPE), (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=4000), SHAPE),
    (dict(K=0), SHAPE), (dict(N=(1 << 24) + 1), SHAPE), (dict(x=None), ARG), (dict(codes=None), ARG),
    (dict(scales=None), ARG), (dict(y=None), ARG), (dict(ldx=4088), ARG), (dict(ldc=2032), ARG), (dict(ldc=(1 << 28) + 16), ARG), (dict(lds=127), ARG),
    (dict(ldy=5119), ARG), (dict(x=P + 8), ALIGN), (dict(ldx=4100), ALIGN), (dict(codes=P + 8), ALIGN),
    (dict(ldc=2056), ALIGN), (dict(scales=P + 2), ALIGN), (dict(lds=130), ALIGN), (dict(y=P + 1), ALIGN),
    (dict(fmt=1, scales=P + 4), ALIGN), (dict(fmt=1, lds=130), ALIGN), (dict(fmt=1, group=128, lds=33, scales=P + 1), ALIGN),
    (dict(M=0, x=None, y=None), OK),
])
def test_gemv_host_checks(L, kw, status):
    assert gemv(L, **kw) == status


def test_quant_weight_w4_host_checks(L):
    q = L.fp8bs_quant_weight_w4
    assert q(P, 64, 256, 256, 0, 64, P, P, None) == ARG
    assert q(P, 64, 256, 256, 3, 32, P, P, None) == ARG
    assert q(P, 0, 256, 256, 0, 32, P, P, None) == SHAPE
    assert q(P, 64, 200, 256, 0, 32, P, P, None) == SHAPE
    assert q(None, 64, 256, 256, 0, 32, P, P, None) == ARG
    assert q(P, 64, 256, 128, 0, 32, P, P, None) == ARG
    assert q(P + 4, 64, 256, 256, 0, 32, P, P, None) == ALIGN
    assert q(P, 64, 256, 258, 0, 32, P, P, None) == ALIGN
    assert q(P, 64, 256, 256, 0, 32, P + 2, P, None) == ALIGN
    assert q(P, 64, 256, 256, 1, 32, P, P + 1, None) == ALIGN


def route(L, x=P, M=4, H=4096, ldx=4096, w=P, E=512, k=10, renorm=1, shared=1, ids=P, wt=P, ws=P, n=None):
    n = L.fp8bs_moe_route_workspace_bytes(4, 512, 4096) if n is None else n
    return L.fp8bs_moe_route(x, M, H, ldx, w, E, k, renorm, shared, ids, wt, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(shared=3), ARG), (dict(shared=-1), ARG), (dict(M=-1), SHAPE), (dict(M=1025), SHAPE), (dict(E=1025), SHAPE),
    (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(E=8, k=9), SHAPE), (dict(k=33), SHAPE), (dict(H=4000), SHAPE),
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(ids=None), ARG), (dict(wt=None), ARG), (dict(ws=None), ARG),
    (dict(ldx=4000), ARG), (dict(x=P + 8), ALIGN), (dict(ldx=4100), ALIGN), (dict(w=P + 8), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(wt=P + 2), ALIGN), (dict(ws=P + 128), ALIGN), (dict(n=256), WS),
    (dict(M=0, x=None, ids=None), OK),
])
def test_route_host_checks(L, kw, status):
    assert route(L, **kw) == status


def test_route_workspace_bytes(L):
    wsb = L.fp8bs_moe_route_workspace_bytes
    assert wsb(0, 512, 4096) >= 256 and wsb(64, 512, 4096) > wsb(1, 512, 4096)
    # the shared expert's gate row is always provided for
    assert wsb(1, 16, 128) == 256 + 1 * 32 * 4
    assert wsb(1, 0, 128) == wsb(1, 1025, 128) == wsb(1, 16, 100) == wsb(-1, 16, 128) == wsb(1025, 16, 128) == 0


def moe(L, x=P, M=4, H=4096, ldx=4096, ids=P, tw=P, S=11, w13=P, s13=P, w2=P, s2=P, E=513, I=256, fmt=0, group=32, y=P,
        ws=P, n=None):
    n = L.fp8bs_moe_w4a16_workspace_bytes(4, 11, 256) if n is None else n
    return L.fp8bs_moe_w4a16(x, M, H, ldx, ids, tw, S, w13, s13, w2, s2, E, I, fmt, group, y, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=5), ARG), (dict(group=128), ARG), (dict(M=-1), SHAPE), (dict(S=0), SHAPE), (dict(M=94), SHAPE),
    (dict(M=1 << 40, S=1 << 40), SHAPE), (dict(E=0), SHAPE), (dict(E=4097), SHAPE), (dict(I=200), SHAPE),
    (dict(I=8320), SHAPE), (dict(H=4000), SHAPE), (dict(H=32896, ldx=32896), SHAPE), (dict(x=None), ARG), (dict(ids=None), ARG), (dict(tw=None), ARG),
    (dict(w13=None), ARG), (dict(s13=None), ARG), (dict(w2=None), ARG), (dict(s2=None), ARG), (dict(y=None), ARG),
    (dict(ws=None), ARG), (dict(ldx=4088), ARG), (dict(x=P + 8), ALIGN), (dict(ldx=4100), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(w13=P + 8), ALIGN), (dict(s13=P + 4), ALIGN), (dict(w2=P + 8), ALIGN),
    (dict(s2=P + 4), ALIGN), (dict(y=P + 1), ALIGN), (dict(ws=P + 128), ALIGN), (dict(n=256 + 4 * 11 * 256 * 4 - 1), WS),
    (dict(M=0, x=None, y=None), OK),
])
def test_moe_host_checks(L, kw, status):
    assert moe(L, **kw) == status


def test_moe_workspace_bytes(L):
    wsb = L.fp8bs_moe_w4a16_workspace_bytes
    assert wsb(16, 11, 256) == 256 + 16 * 11 * 256 * 4
    assert wsb(100, 11, 256) == wsb(1, 11, 200) == wsb(1, 0, 256) == 0


def test_binding_refuses_formats_and_cpu_tensors(L):
    x = torch.zeros((1, 256), dtype=torch.bfloat16)
    c, s = torch.zeros((8, 128), dtype=torch.uint8), torch.zeros((8, 8), dtype=torch.uint8)
    with pytest.raises(ValueError):
        fb.fp8bs_gemv_w4a16(x, c, s)
    with pytest.raises(fb.Fp8bsError) as e:
        fb._w4_scale_dtype(fb.FP8BS_W4_MXFP4, 64, "fp8bs_gemv_w4a16")
    assert e.value.status == ARG


# ---- the plain implementation the GPU tests compare with ---------------------------

def test_reference_formats_by_hand():
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] + [0] * 56], np.uint8)
    scales = np.array([[128, 127, 127, 127]], np.uint8)
    v = R.value(codes, scales, R.MXFP4, 32)
    want = [0, 1, 2, 3, 4, 6, 8, 12]
    assert np.array_equal(v[0, :16], want + [-t for t in want]) and np.all(v[0, 16:] == 0)
    v = R.value(codes, np.array([[0x4000]], np.uint16), R.INT4, 128)
    assert np.array_equal(v[0, :16], 2.0 * (np.arange(16) - 8))


@pytest.mark.parametrize("fmt,group", R.FORMATS)
def test_reference_quantiser_is_nearest(fmt, group):
    rng = np.random.default_rng(3)
    w = rng.standard_normal((6, 256)).astype(np.float32)
    codes, scales = R.quant(w, fmt, group)
    v = R.value(codes, scales, fmt, group)
    # no other code of the group's scale is nearer
    for n in range(16):
        other = R.value(np.full_like(codes, n | n << 4), scales, fmt, group)
        assert np.all(np.abs(v - w) <= np.abs(other - w) + 1e-6)


def test_reference_experts_against_a_dense_product():
    rng = np.random.default_rng(5)
    x = R.bf16(rng.standard_normal((2, 128)))
    w13, w2 = rng.standard_normal((3, 8, 128)), rng.standard_normal((3, 128, 4))
    ids, tw = np.array([[0, 2], [1, -1]], np.int32), np.array([[0.5, 2.0], [1.0, 3.0]], np.float32)
    y, bound = R.moe(x, ids, tw, w13, w2)
    xt, a = torch.from_numpy(R.synth.bf16_bits_to_f32(x)).double(), []
    for e in range(3):
        h = xt @ torch.from_numpy(w13[e]).T
        a.append((torch.nn.functional.silu(h[:, :4]) * h[:, 4:]) @ torch.from_numpy(w2[e]).T)
    want = torch.stack((0.5 * a[0][0] + 2.0 * a[2][0], a[1][1]))
    assert np.allclose(y, want.numpy(), rtol=1e-12) and np.all(bound > 0)
