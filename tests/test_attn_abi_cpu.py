"""Host checks of the attention block's entry points, the frequency table, and the
binding's own refusals: no device pointer is dereferenced, nothing is launched."""

import ctypes
import math

import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
from tests import attn_reference as A
from tests.test_streams_cpu import BF16, I32, SIDE, U8, Tensor, box  # noqa: F401

OK, ARG, SHAPE, ALIGN, WS = 0, -1, -2, -3, -5
P = 0x10000000  # a fake, well-aligned device address: refused before any launch
I64 = torch.int64

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device pointers: host-check tests run only where no GPU is visible")


@pytest.fixture(scope="module")
def L():
    fb.build()
    return fb.lib()


def test_the_new_limits_match_the_header():
    with open(fb.HEADER_PATH) as f:
        text = f.read()
    for name in ("FP8BS_ATTN_MAX_SEQS",):
        assert f"#define {name} {getattr(fb, name)} " in text
    for name in ("FP8BS_ROPE_HALF", "FP8BS_ROPE_INTERLEAVED", "FP8BS_ROPE_PLAIN", "FP8BS_ROPE_LINEAR",
                 "FP8BS_ROPE_BY_PARTS", "FP8BS_KV_BF16", "FP8BS_KV_E4M3"):
        assert f"{name} = {getattr(fb, name)}," in text
    assert ctypes.sizeof(fb._KvCacheStruct) == 4 * 8 + 4 * 4 + 7 * 8


# ---- frequencies -------------------------------------------------------------------

@pytest.mark.parametrize("R,theta,kw", [
    (128, 10000.0, {}), (2, 1.5, {}), (256, 1e7, {}), (6, 500000.0, {}), (64, 1e4, dict(scaling=1, factor=4.0)),
    (128, 1e6, dict(scaling=2, factor=16.0, original=32768.0)), (64, 1e4, dict(scaling=2, factor=1.0, original=4096.0)),
    (128, 1e4, dict(scaling=2, factor=40.0, original=4096.0, fast=32.0, slow=1.0)), (4, 1e4, dict(scaling=2, factor=8.0, original=100.0)),
])
def test_frequencies(L, R, theta, kw):
    f, amplitude = A.frequencies(R, theta, **kw)
    got, amp = (ctypes.c_uint64 * (R // 2))(), ctypes.c_float()
    rc = L.fp8bs_rope_freqs(R, theta, kw.get("scaling", 0), kw.get("factor", 0.0), kw.get("original", 0.0),
                            kw.get("fast", 32.0), kw.get("slow", 1.0), got, ctypes.byref(amp))
    assert rc == OK and abs(amp.value - amplitude) <= 2.0 ** -24 * amplitude
    for i in range(R // 2):
        # both take a power in 64 bits: a few steps of 2^-53; the table is whole in units of 2^-64
        assert abs(got[i] / 2.0 ** 64 - float(f[i]) / (2 * math.pi)) <= float(f[i]) * 2.0 ** -49 + 2.0 ** -65
    assert L.fp8bs_rope_freqs(R, theta, 0, 0.0, 0.0, 0.0, 0.0, got, None) == OK


@pytest.mark.parametrize("args,status", [
    ((0, 1e4, 0, 1, 1, 32, 1), SHAPE), ((258, 1e4, 0, 1, 1, 32, 1), SHAPE), ((7, 1e4, 0, 1, 1, 32, 1), SHAPE),
    ((-2, 1e4, 0, 1, 1, 32, 1), SHAPE), ((64, 1.0, 0, 1, 1, 32, 1), ARG), ((64, math.nan, 0, 1, 1, 32, 1), ARG),
    ((64, math.inf, 0, 1, 1, 32, 1), ARG), ((64, 1e4, 3, 1, 1, 32, 1), ARG), ((64, 1e4, -1, 1, 1, 32, 1), ARG),
    ((64, 1e4, 1, 0.5, 1, 32, 1), ARG), ((64, 1e4, 1, math.nan, 1, 32, 1), ARG), ((64, 1e4, 2, 4, 0, 32, 1), ARG),
    ((64, 1e4, 2, 4, 4096, 1, 1), ARG), ((64, 1e4, 2, 4, 4096, 32, 0), ARG), ((64, 1e4, 2, 4, 4096, math.inf, 1), ARG),
])
def test_frequency_refusals(L, args, status):
    got = (ctypes.c_uint64 * 128)()
    assert L.fp8bs_rope_freqs(*args, got, None) == status
    assert L.fp8bs_rope_freqs(64, 1e4, 0, 1, 1, 32, 1, None, None) == ARG


# ---- norm and rotation -------------------------------------------------------------

def rope(L, q=P, ldq=6144, hsq=128, k=P, ldk=6144, hsk=128, T=4, Hq=32, Hk=8, D=128, pos=P, freqs=P, R=128, layout=0, amp=1.0,
         gq=P, gk=P, eps=1e-6, qo=P, ldqo=4096, hsqo=128, ko=P, ldko=1024, hsko=128):
    return L.fp8bs_qk_norm_rope(q, ldq, hsq, k, ldk, hsk, T, Hq, Hk, D, pos, freqs, R, layout, amp, gq, gk, eps, qo, ldqo,
                                hsqo, ko, ldko, hsko, None)


@no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(layout=2), ARG), (dict(amp=math.inf), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(T=-1), SHAPE),
    (dict(T=(1 << 24) + 1), SHAPE), (dict(Hq=1025), SHAPE), (dict(Hq=-1), SHAPE), (dict(Hk=1 << 40), SHAPE), (dict(Hq=0, Hk=0), SHAPE),
    (dict(D=96), SHAPE), (dict(D=512), SHAPE), (dict(R=130), SHAPE), (dict(R=24), SHAPE), (dict(R=7, layout=1), SHAPE),
    (dict(R=-2, layout=1), SHAPE), (dict(q=None), ARG), (dict(k=None), ARG), (dict(qo=None), ARG), (dict(ko=None), ARG),
    (dict(pos=None), ARG), (dict(freqs=None), ARG), (dict(ldqo=64), ARG), (dict(hsqo=64), ARG), (dict(hsko=0), ARG),
    (dict(ldq=-8), ARG), (dict(hsk=1 << 41), ARG), (dict(q=P + 8), ALIGN), (dict(ldq=6148), ALIGN), (dict(hsk=132), ALIGN),
    (dict(qo=P + 2), ALIGN), (dict(ldko=1028), ALIGN), (dict(pos=P + 4), ALIGN), (dict(freqs=P + 4), ALIGN), (dict(gq=P + 8), ALIGN),
    (dict(gk=P + 2), ALIGN), (dict(T=0, q=None, qo=None), OK),
])
def test_rope_host_checks(L, kw, status):
    assert rope(L, **kw) == status


def cache(**kw):
    s = fb._KvCacheStruct()
    base = dict(k=P, v=P, k_scale=P, v_scale=P, kind=1, head_dim=128, kv_heads=8, page_size=16, pages=100)
    for name, value in {**base, **{n: v for n, v in kw.items() if n not in ("strides", "scale_strides")}}.items():
        setattr(s, name, value)
    s.strides[:] = kw.get("strides", (16 * 8 * 128, 8 * 128, 128))
    s.scale_strides[:] = kw.get("scale_strides", (16 * 8, 8, 1))
    return s


BAD_CACHES = [
    (dict(kind=2), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=None), ARG),
    (dict(strides=(-16, 1024, 128)), ARG), (dict(strides=(16384, 1024, 1 << 41)), ARG), (dict(scale_strides=(-1, 8, 1)), ARG),
    (dict(head_dim=80), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE), (dict(page_size=0), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=1 << 17), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(strides=(64, 1024, 128)), ARG), (dict(strides=(16384, 0, 128)), ARG), (dict(strides=(16384, 1024, 64)), ARG),
    (dict(scale_strides=(128, 0, 1)), ARG), (dict(k=P + 8), ALIGN), (dict(v=P + 1), ALIGN), (dict(strides=(16392, 1024, 128)), ALIGN),
    (dict(strides=(16384, 1032, 128)), ALIGN), (dict(kind=0, strides=(16384, 1028, 128)), ALIGN),
]


def append(L, c=None, q=P, ldq=6144, hsq=128, k=P, v=P, ldv=6144, T=4, Hq=32, pos=P, slots=P, freqs=P, R=128, qo=P, err=None, **kw):
    c = cache(**kw) if c is None else c
    return L.fp8bs_qk_norm_rope_append(q, ldq, hsq, k, 6144, 128, v, ldv, 128, T, Hq, pos, slots, freqs, R, 0, 1.0, None, None, 1e-6,
                                       qo, 4096, 128, ctypes.addressof(c) if c else None, err, None)


@no_gpu
@pytest.mark.parametrize("kw,status", BAD_CACHES + [
    (dict(c=False), ARG), (dict(v=None), ARG), (dict(slots=None), ARG), (dict(slots=P + 4), ALIGN), (dict(err=P + 64), ALIGN),
    (dict(ldv=6148), ALIGN), (dict(Hq=1025), SHAPE), (dict(T=0), OK), (dict(ldv=-8), ARG)])
def test_append_host_checks(L, kw, status):
    assert append(L, **kw) == status


def attn(L, c=None, q=P, ldq=4096, hsq=128, T=4, Hq=32, table=P, stride=64, cols=64, B=4, cu=P, lens=P, scale=0.1, window=0, o=P,
         ldo=4096, hso=128, ws=P, n=1 << 40, **kw):
    c = cache(**kw) if c is None else c
    return L.fp8bs_attn_paged(q, ldq, hsq, T, Hq, ctypes.addressof(c) if c else None, table, stride, cols, B, cu, lens, scale, window,
                              o, ldo, hso, ws, n, None)


@no_gpu
@pytest.mark.parametrize("kw,status", BAD_CACHES + [
    (dict(c=False), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=math.nan), ARG), (dict(scale=1e6), ARG),
    (dict(window=-1), ARG), (dict(T=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=30), SHAPE), (dict(Hq=2048), SHAPE), (dict(B=-1), SHAPE),
    (dict(B=1025), SHAPE), (dict(cols=-1), SHAPE), (dict(T=1 << 23), SHAPE), (dict(q=None), ARG), (dict(o=None), ARG),
    (dict(table=None), ARG), (dict(cu=None), ARG), (dict(lens=None), ARG), (dict(ws=None), ARG), (dict(stride=63), ARG),
    (dict(ldo=64), ARG), (dict(hso=64), ARG), (dict(ldq=-8), ARG), (dict(q=P + 8), ALIGN), (dict(ldq=4100), ALIGN), (dict(o=P + 2), ALIGN),
    (dict(table=P + 2), ALIGN), (dict(cu=P + 1), ALIGN), (dict(lens=P + 2), ALIGN), (dict(ws=P + 128), ALIGN), (dict(T=0, q=None), OK),
    (dict(B=0, table=None), OK)])
def test_attn_host_checks(L, kw, status):
    assert attn(L, **kw) == status


def test_attn_workspace_bytes(L):
    wsb = L.fp8bs_attn_paged_workspace_bytes
    assert wsb(128, 152) > wsb(64, 152) > 0 and wsb(128, 152) > wsb(128, 100)
    assert wsb(96, 152) == wsb(0, 152) == wsb(128, 1 << 20) == 0


# ---- the binding, with stand-ins for tensors and the library -------------------------

class Strided(Tensor):
    def __init__(self, shape, dtype, device=0, made_on="before the call"):
        super().__init__(shape, dtype, device, made_on)


def given(name, device=0):
    rope_of = fb.Rope.__new__(fb.Rope)
    rope_of.rotary_dim, rope_of.layout, rope_of.amplitude, rope_of.freqs = 64, 0, 1.0, Tensor((32,), I64)
    kv = fb.KvCache(*(Tensor((4, 16, 2, 128), BF16) for _ in range(2)))
    q, k = Tensor((3, 4, 128), BF16), Tensor((3, 2, 128), BF16)
    pos = Tensor((3,), I64)
    return {
        "fp8bs_qk_norm_rope": dict(q=q, k=k, positions=pos, rope=rope_of),
        "fp8bs_qk_norm_rope_append": dict(q=q, k=k, v=Tensor((3, 2, 128), BF16), positions=pos, slots=Tensor((3,), I64), rope=rope_of,
                                          cache=kv),
        "fp8bs_attn_paged": dict(q=q, cache=kv, block_table=Tensor((2, 5), I32), cu_q=Tensor((3,), I32), kv_len=Tensor((2,), I32)),
    }[name]


MADE = {"fp8bs_qk_norm_rope": dict(q_out=((3, 4, 128), BF16), k_out=((3, 2, 128), BF16)),
        "fp8bs_qk_norm_rope_append": dict(q_out=((3, 4, 128), BF16)),
        "fp8bs_attn_paged": dict(o=((3, 4, 128), BF16), workspace=((1024,), U8))}
GIVEN = {"fp8bs_qk_norm_rope": ("q", "k", "positions"), "fp8bs_qk_norm_rope_append": ("q", "k", "v", "positions", "slots"),
         "fp8bs_attn_paged": ("q", "block_table", "cu_q", "kv_len")}


@pytest.mark.parametrize("name", MADE)
def test_buffers_belong_to_the_calls_stream(box, name):  # noqa: F811
    library, made = box
    getattr(fb, name)(**given(name), stream=SIDE)
    assert len(made) == len(MADE[name]) and all(t.made_on == SIDE for t in made)
    assert len(library.calls) == 1 and library.calls[0][1][-1] == SIDE
    made.clear()
    getattr(fb, name)(**given(name))
    assert all(t.made_on == "the current stream" for t in made) and library.calls[1][1][-1] == 0x77


@pytest.mark.parametrize("device", [-1, 1])
@pytest.mark.parametrize("name,which", [(n, w) for n in MADE for w in (*GIVEN[n], *MADE[n], "gamma_k", "cache", "error")])
def test_a_tensor_elsewhere_is_refused(box, name, which, device):  # noqa: F811
    library, _ = box
    a = given(name)
    if which in ("gamma_k", "error", "cache") and (which == "gamma_k") == (name == "fp8bs_attn_paged"):
        return
    if which == "error" and name != "fp8bs_qk_norm_rope_append" or which == "cache" and "cache" not in a:
        return
    if which == "cache":
        a["cache"].device_index = device
        a["cache"].tensors[0].index = device
    else:
        t = a.get(which)
        shape, dtype = (t.shape, t.dtype) if t is not None else MADE[name].get(which, ((128,), BF16 if which == "gamma_k" else U8))
        a[which] = Tensor(shape, dtype, device=device)
    with pytest.raises(ValueError):
        getattr(fb, name)(**a)
    assert not library.calls


@pytest.mark.parametrize("name", MADE)
def test_another_current_device_is_refused(box, monkeypatch, name):  # noqa: F811
    library, _ = box
    a = given(name)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        getattr(fb, name)(**a)
    assert not library.calls


def test_caches_that_do_not_fit_together_are_refused(box):  # noqa: F811
    k, z = Tensor((4, 16, 2, 128), U8), Tensor((4, 16, 2), U8)
    with pytest.raises(ValueError):
        fb.KvCache(Tensor((4, 16, 2, 128), BF16, device=-1), Tensor((4, 16, 2, 128), BF16, device=-1))
    with pytest.raises(ValueError):
        fb.KvCache(k, k, z, None)
    for bad in [(k, k), (Tensor((4, 16, 2, 128), BF16), k), (k, k, z, Tensor((4, 16, 3), U8)), (k, Tensor((5, 16, 2, 128), U8), z, z)]:
        with pytest.raises(AssertionError):
            fb.KvCache(*bad)
    with pytest.raises(fb.Fp8bsError):
        fb.new_kv_cache(2, 16, 2, 128, 7, torch.device("cuda", 0))


def test_a_table_whose_rows_overlap_is_refused(box, monkeypatch):  # noqa: F811
    library, _ = box
    a = given("fp8bs_attn_paged")
    for strides in ((0, 1), (4, 1), (10, 2)):  # one row for all, rows into one another, every second entry
        monkeypatch.setattr(a["block_table"], "stride", lambda s=strides: s, raising=False)
        with pytest.raises(AssertionError):
            fb.fp8bs_attn_paged(**a)
    assert not library.calls
    monkeypatch.setattr(a["block_table"], "stride", lambda: (9, 1), raising=False)
    fb.fp8bs_attn_paged(**a)
    assert library.calls[0][1][7] == 9 and library.calls[0][1][8] == 5
