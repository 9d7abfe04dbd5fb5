"""The binding's buffers, streams and devices, without a GPU: tensors and the
library are stand-ins that record what they are asked for."""

import contextlib

import pytest
import torch

import fp8_block_scale_x128_gb300 as fb

SIDE = 0x5150  # a raw stream


class Tensor:
    def __init__(self, shape, dtype, device=0, made_on="before the call"):
        self.shape, self.dtype, self.index, self.made_on = torch.Size(shape), dtype, device, made_on
        self.device = torch.device("cuda", max(device, 0))

    is_cuda = property(lambda self: self.index >= 0)

    def get_device(self):
        return self.index

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


class Library:
    """Every call succeeds and is kept; sizes are small and positive."""

    def __init__(self):
        self.calls = []

    def fp8bs_status_string(self, status):
        return b""

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 1024
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def box(monkeypatch):
    """(library, list of the tensors made inside a call); current device 0."""
    made, now = [], ["the current stream"]

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s
        yield
        now[0] = before

    def new(shape, dtype=None, device=None):
        made.append(Tensor(shape if isinstance(shape, (tuple, list)) else (shape,), dtype, made_on=now[0]))
        return made[-1]

    library = Library()
    monkeypatch.setattr(fb, "_lib", library)
    monkeypatch.setattr(torch, "empty", new)
    monkeypatch.setattr(torch, "zeros", new)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: raw)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0x77, raising=False)
    return library, made


BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


def operands(name):
    """The tensors that a call has to be given, by its parameters' names."""
    return {
        "fp8bs_quant_weight_w4": dict(w=Tensor((64, 256), F32)),
        "fp8bs_gemv_w4a16": dict(x=Tensor((2, 256), BF16), codes=Tensor((64, 128), U8), scales=Tensor((64, 8), U8)),
        "fp8bs_moe_route": dict(x=Tensor((2, 256), BF16), w=Tensor((16, 256), BF16)),
        "fp8bs_moe_w4a16": dict(x=Tensor((2, 256), BF16), topk_ids=Tensor((2, 3), I32), topk_w=Tensor((2, 3), F32),
                                w13=Tensor((4, 256, 128), U8), s13=Tensor((4, 256, 8), U8),
                                w2=Tensor((4, 256, 64), U8), s2=Tensor((4, 256, 4), U8)),
    }[name]


# the 8-bit calls: their tensors and how many they make themselves
EIGHT_BIT = {
    "fp8bs_encode_e4m3": (dict(v=Tensor((256,), F32)), 1),
    "fp8bs_quant": (dict(x=Tensor((2, 256), BF16)), 2),
    "fp8bs_rmsnorm_quant": (dict(x=Tensor((2, 256), BF16), gamma=Tensor((256,), BF16), want_y=True), 3),
    "fp8bs_moe_w8a16": (dict(x=Tensor((2, 512), BF16), topk_ids=Tensor((2, 3), I32), topk_w=Tensor((2, 3), F32),
                             w13=Tensor((4, 256, 512), U8), s13=Tensor((4, 2, 4), F32), w2=Tensor((4, 512, 128), U8),
                             s2=Tensor((4, 4, 1), F32)), 2),
    "fp8bs_quant_weight": (dict(w=Tensor((128, 256), F32)), 2),
    "fp8bs_prepack_weight": (dict(wq=Tensor((128, 256), U8), ws=Tensor((1, 2), F32)), 1),
    "fp8bs_gemm_fused": (dict(x=Tensor((2, 256), BF16), packed=Tensor((1024,), U8), N=128, K=256), 2),
    "fp8bs_gemm_prequant": (dict(xq=Tensor((2, 256), U8), xs=Tensor((2, 2), F32), packed=Tensor((1024,), U8), N=128, K=256), 2),
    "fp8bs_gemm_fused_static": (dict(x=Tensor((2, 256), BF16), packed=Tensor((1024,), U8), N=128, K=256), 1),
    "new_workspace": (dict(N=128, K=256, device=torch.device("cuda", 0)), 1),
}


# what each call makes itself where it is not given it
MADE = {
    "fp8bs_quant_weight_w4": dict(codes=((64, 128), U8), scales=((64, 8), U8)),
    "fp8bs_gemv_w4a16": dict(y=((2, 64), BF16)),
    "fp8bs_moe_route": dict(ids=((2, 4), I32), weights=((2, 4), F32), workspace=((1024,), U8)),
    "fp8bs_moe_w4a16": dict(y=((2, 256), BF16), workspace=((1024,), U8)),
}
EXTRA = {"fp8bs_moe_route": dict(k=4)}


def call(name, **kw):
    return getattr(fb, name)(**{**operands(name), **EXTRA.get(name, {}), **kw})


@pytest.mark.parametrize("name", MADE)
def test_buffers_a_call_makes_belong_to_its_stream(box, name):
    library, made = box
    call(name, stream=SIDE)
    assert len(made) == len(MADE[name]) and all(t.made_on == SIDE for t in made)
    assert len(library.calls) == 1 and library.calls[0][1][-1] == SIDE


@pytest.mark.parametrize("name", MADE)
def test_buffers_without_a_stream_are_the_current_ones(box, name):
    library, made = box
    call(name)
    assert all(t.made_on == "the current stream" for t in made) and library.calls[0][1][-1] == 0x77


@pytest.mark.parametrize("device", [-1, 1])
@pytest.mark.parametrize("name,which", [(n, w) for n in MADE for w in (*operands(n), *MADE[n])])
def test_a_tensor_elsewhere_is_refused(box, name, which, device):
    library, _ = box
    t = operands(name).get(which)
    shape, dtype = (t.shape, t.dtype) if t is not None else MADE[name][which]
    with pytest.raises(ValueError):
        call(name, **{which: Tensor(shape, dtype, device=device)})
    assert not library.calls


@pytest.mark.parametrize("name", MADE)
def test_another_current_device_is_refused(box, monkeypatch, name):
    library, _ = box
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        call(name)
    assert not library.calls


@pytest.mark.parametrize("name", ["fp8bs_moe_route", "fp8bs_moe_w4a16"])
def test_a_workspace_that_is_not_one_piece_is_refused(box, name):
    library, _ = box
    ws = Tensor((1 << 20,), U8)
    ws.is_contiguous = lambda: False
    with pytest.raises(AssertionError):
        call(name, workspace=ws)
    assert not library.calls


@pytest.mark.parametrize("kw,status", [(dict(shared="both"), fb.FP8BS_ERR_ARG), (dict(shared=None), fb.FP8BS_ERR_ARG),
                                       (dict(k=0), fb.FP8BS_ERR_SHAPE), (dict(k=-3), fb.FP8BS_ERR_SHAPE),
                                       (dict(k=17), fb.FP8BS_ERR_SHAPE), (dict(k=16, shared="gate"), fb.FP8BS_ERR_SHAPE)])
def test_router_refusals_are_the_librarys(box, kw, status):
    library, made = box
    with pytest.raises(fb.Fp8bsError) as e:
        call("fp8bs_moe_route", **kw)
    assert e.value.status == status and not library.calls and not made


@pytest.mark.parametrize("name", EIGHT_BIT)
def test_buffers_an_8_bit_call_makes_belong_to_its_stream(box, name):
    library, made = box
    given, count = EIGHT_BIT[name]
    getattr(fb, name)(**given, stream=SIDE)
    assert len(made) == count and all(t.made_on == SIDE for t in made)
    assert all(args[-1].value == SIDE for _, args in library.calls)


def test_early_reads_are_documented_for_the_whole_stream():
    # quant and the fused GEMM let their successor start before they wait for
    # their own predecessor: "the work just before" is not far enough back
    with open(fb.HEADER_PATH) as f:
        header = " ".join(f.read().replace("*", " ").split())
    for text in (fb.fp8bs_gemm_fused.__doc__, fb.fp8bs_gemv_w4a16.__doc__):
        text = " ".join(text.split())
        assert "no unfinished work on the stream" in text and "just before" not in text
    assert header.count("no unfinished work on the stream") == 2
    assert "work just before this call" not in header
