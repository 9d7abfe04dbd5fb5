"""Norms and rotation of heads, and appending to a paged cache, against 64 bits."""

import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
from tests import attn_reference as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    fb.build()
    return torch.device("cuda", 0)


def qkv(T, Hq, Hk, D, seed, dev, pad=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((T, Hq + 2 * Hk, D), generator=g, device=dev) * 3
    x = torch.where(torch.rand(x.shape, generator=g, device=dev) < 0.01, x * 20, x).to(torch.bfloat16)
    buf = torch.zeros((T, (Hq + 2 * Hk) * D + pad), dtype=torch.bfloat16, device=dev)
    buf[:, :(Hq + 2 * Hk) * D] = x.flatten(1)
    x = buf[:, :(Hq + 2 * Hk) * D].view(T, -1, D)
    gam = [(1 + 0.25 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2)]
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], gam


CASES = [  # T, Hq, Hk, D, R, layout, norm, pad
    (1, 32, 8, 128, 128, 0, True, 0), (3, 5, 1, 64, 64, 1, True, 8), (7, 16, 2, 256, 64, 0, True, 0),
    (2, 1, 1, 256, 256, 1, True, 24), (5, 3, 3, 128, 32, 0, False, 0), (9, 4, 2, 64, 6, 1, True, 0),
    (1, 1, 0, 64, 0, 0, True, 0), (4, 0, 5, 128, 128, 0, True, 0), (700, 7, 1, 128, 96, 0, True, 0),
    (1300, 9, 3, 64, 16, 0, False, 8), (2, 33, 7, 128, 0, 1, False, 0),
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,layout,norm,pad", CASES)
@pytest.mark.parametrize("start", [0, 10_000_019])
def test_heads(dev, T, Hq, Hk, D, R, layout, norm, pad, start):
    q, k, _, gam = qkv(T, Hq, Hk, D, T + R, dev, pad)
    rope = fb.Rope(R, 1e6 if R != 6 else 1e4, layout, fb.FP8BS_ROPE_BY_PARTS if R == 96 else fb.FP8BS_ROPE_PLAIN, 8.0, 4096.0)
    f, amp = A.frequencies(R, 1e6 if R != 6 else 1e4, 2 if R == 96 else 0, 8.0, 4096.0) if R else (torch.zeros(0, dtype=torch.float64), 1.0)
    assert abs(rope.amplitude - amp) <= 2.0 ** -24 * amp
    pos = start + torch.randperm(T, device=dev) * 3 - (5 if start == 0 else 0)  # negative ones too
    gq, gk = gam if norm else (None, None)
    qo, ko = fb.fp8bs_qk_norm_rope(q, k, pos, rope, gq, gk, 1e-6)
    for x, y, gm in ((q, qo, gq), (k, ko, gk)):
        A.near(y, *A.heads(x, pos, f, amp, layout == 0, gm, 1e-6))


def test_in_place_strided_and_untouched(dev):
    T, Hq, Hk, D = 6, 4, 2, 128
    q, k, v, (gq, gk) = qkv(T, Hq, Hk, D, 1, dev, 8)
    rope = fb.Rope(64, 1e4)
    pos = torch.arange(T, device=dev)
    want = fb.fp8bs_qk_norm_rope(q, k, pos, rope, gq, gk)
    # into every second head of a larger buffer, the others left as they were
    wide = torch.full((T, 2 * Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
    keys = torch.empty((T, Hk, D), dtype=torch.bfloat16, device=dev)
    fb.fp8bs_qk_norm_rope(q, k, pos, rope, gq, gk, q_out=wide[:, ::2], k_out=keys)
    assert torch.equal(wide[:, ::2], want[0]) and torch.equal(keys, want[1]) and bool((wide[:, 1::2] == 7).all())
    before = v.clone()
    fb.fp8bs_qk_norm_rope(q, k, pos, rope, gq, gk, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)


def test_special_rows(dev):
    D = 128
    x = torch.zeros((1, 4, D), dtype=torch.bfloat16, device=dev)
    x[0, 1, 5] = float("nan")
    x[0, 2, 6] = float("inf")
    x[0, 3] = 1e-30
    gam = torch.ones(D, dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(1, dtype=torch.int64, device=dev)
    rope = fb.Rope(D)
    q, _ = fb.fp8bs_qk_norm_rope(x, x[:, :1], pos, rope, gam, gam, 0.0)
    assert bool((q[0, 0] == 0).all())                      # zeros stay
    assert bool(torch.isnan(q[0, 1]).all())                # as x / sqrt(NaN)
    assert bool(torch.isnan(q[0, 2, [6, 70]]).all()) and int(torch.isnan(q[0, 2]).sum()) == 2
    # its neighbours in a warp are not touched
    assert bool((fb.fp8bs_qk_norm_rope(x[:, 3:], x[:, :1], pos, rope, gam, gam, 1e-6)[0].abs() < 1e-20).all())


def cache_tensors(pages, page, Hk, D, codes, order, dev):
    def make(dtype, n, fill):
        s = (pages, page, Hk, D)[:n]
        if order == "heads":
            return torch.full((s[0], s[2], s[1], *s[3:]), fill, dtype=dtype, device=dev).transpose(1, 2)
        return torch.full(s, fill, dtype=dtype, device=dev)
    if codes:
        return [make(torch.uint8, n, 9) for n in (4, 4, 3, 3)]
    return [make(torch.bfloat16, 4, 9.0) for _ in range(2)]


@pytest.mark.parametrize("T,Hq,Hk,D,R,layout,norm,page,order", [
    (1, 32, 8, 128, 128, 0, True, 16, "slots"), (37, 5, 1, 64, 64, 1, True, 8, "heads"), (9, 16, 2, 256, 64, 0, True, 1, "slots"),
    (50, 0, 3, 128, 0, 0, False, 64, "heads"), (1100, 4, 4, 128, 128, 0, True, 32, "slots"), (3, 40, 8, 64, 32, 1, False, 1024, "slots")])
@pytest.mark.parametrize("codes", [False, True])
def test_append(dev, T, Hq, Hk, D, R, layout, norm, page, order, codes):
    q, k, v, gam = qkv(T, Hq, Hk, D, T, dev, 8)
    pages = -(-T // page) + 2
    tensors = cache_tensors(pages, page, Hk, D, codes, order, dev)
    cache = fb.KvCache(*tensors)
    slots = torch.randperm(pages * page, generator=torch.Generator(device=dev).manual_seed(3), device=dev)[:T].contiguous()
    if T > 2:
        slots[T // 2] = -1  # a padded token
    rope = fb.Rope(R, 1e4, layout)
    f, amp = A.frequencies(R, 1e4) if R else (torch.zeros(0, dtype=torch.float64), 1.0)
    pos = torch.arange(T, device=dev) + 1000
    gq, gk = gam if norm else (None, None)
    qo = fb.fp8bs_qk_norm_rope_append(q, k, v, pos, slots, rope, cache, gq, gk)
    if Hq:
        assert torch.equal(qo, fb.fp8bs_qk_norm_rope(q, k, pos, rope, gq, gk)[0])
    there = slots >= 0
    page_of, at = slots[there] // page, slots[there] % page
    ref, bound = A.heads(k, pos, f, amp, layout == 0, gk, 1e-6)
    ref, bound = ref[there.cpu()], bound[there.cpu()]
    if codes:
        got, scale = tensors[0][page_of, at], tensors[2][page_of, at]
        most = ref.abs().amax(-1)
        byte = torch.ceil(torch.log2(most / 448) - 1e-12) + 127
        s = scale.cpu().double()
        # the largest may be rounded over a power of two
        edge = ((torch.log2(most / 448) - torch.round(torch.log2(most / 448))).abs() < 1e-4)
        assert bool(((s == byte) | (edge & ((s - byte).abs() == 1))).all())
        unit = 2.0 ** (s - 127).unsqueeze(-1)
        y = A.e4m3_values(got, scale)
        assert bool(((y - ref).abs() <= bound + torch.maximum(2.0 ** -4 * (ref.abs() + bound), 2.0 ** -10 * unit)).all())
        # values: the library's own rule, bit for bit
        vr = v[there].contiguous()
        if D == 128:
            xq, xs = fb.fp8bs_quant(vr.view(-1, D), fb.FP8BS_SCALE_UE8M0)
            assert torch.equal(tensors[1][page_of, at].reshape(-1, D), xq)
            assert torch.equal(tensors[3][page_of, at].reshape(-1), xs.flatten())
        vv = A.e4m3_values(tensors[1][page_of, at], tensors[3][page_of, at])
        vs = 2.0 ** (tensors[3][page_of, at].cpu().double() - 127).unsqueeze(-1)
        vd = vr.double().cpu()
        assert bool(((vv - vd).abs() <= torch.maximum(2.0 ** -4 * vd.abs(), 2.0 ** -10 * vs)).all())
    else:
        A.near(tensors[0][page_of, at], ref, bound)
        assert torch.equal(tensors[1][page_of, at], v[there])
    # nothing else is written
    free = torch.ones(pages * page, dtype=torch.bool, device=dev)
    free[slots[there]] = False
    for t in tensors:
        assert bool((t.reshape(pages * page, *t.shape[2:])[free] == 9).all())


def test_append_special_rows_and_bad_slots(dev):
    T, Hk, D = 5, 2, 128
    k = torch.randn((T, Hk, D), device=dev).to(torch.bfloat16)
    v = torch.randn((T, Hk, D), device=dev).to(torch.bfloat16)
    k[0, 0, 3], v[1, 1, 4], v[2, 0] = float("inf"), float("nan"), 0.0
    tensors = cache_tensors(2, 4, Hk, D, True, "slots", dev)
    error = torch.zeros(256, dtype=torch.uint8, device=dev)
    slots = torch.tensor([0, 1, 2, -7, 8], device=dev)
    fb.fp8bs_qk_norm_rope_append(k[:, :0], k, v, torch.arange(T, device=dev), slots, fb.Rope(0), fb.KvCache(*tensors), error=error)
    assert fb.fp8bs_check_error(error) == fb.FP8BS_ERR_DEVICE and fb.fp8bs_check_error(error) == 0
    kk, vv, ks, vs = (t.reshape(8, *t.shape[2:]) for t in tensors)
    assert int(ks[0, 0]) == 255 and int(vs[1, 1]) == 255 and int(vs[2, 0]) == 0 and bool((vv[2, 0] == 0).all())
    assert int(ks[0, 1]) != 255 and int(vs[1, 0]) != 255
    for t in (kk, vv, ks, vs):
        assert bool((t[3:] == 9).all())
