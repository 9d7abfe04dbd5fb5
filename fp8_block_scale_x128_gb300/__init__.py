"""Python binding of libfp8bs (small-M W8A8 FP8 block-scale linear for GB300).

Argument marshalling only: every function here turns torch tensors into the
device pointers, sizes and the cudaStream_t of the C ABI declared in
``include/fp8bs.h`` and calls it; all arithmetic runs in the library's CUDA
kernels.  There is no fallback: if the compiled library is missing, or a call
returns an error status, an exception is raised.

A call given a `stream` (a torch.cuda.Stream or a raw cudaStream_t) runs there
and not on the current one: its inputs have to be ready on it, and what the call
allocates itself (outputs, workspaces) belongs to it, as under
``torch.cuda.stream(stream)``.

The names match the C entry points.  Layout and rounding rules are documented
in the header; the method is the one of "[AMD] Small-M FP8 block-scale GEMM
with fused activation quant for gfx950 (Qwen3.5)", "Modifications", with the
power-of-two variant of "[Perf] [AMD] dsv4: optional e8m0 mxscale GEMM for
dense 128x128 fp8 linears (6/8)".
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import re
import threading

import torch

FP8BS_SCALE_F32 = 0
FP8BS_SCALE_UE8M0 = 1
FP8BS_MAX_M = 64
FP8BS_FLAG_PDL = 1
FP8BS_STATIC_MAX_K = 16384
FP8BS_STATIC_MAX_SMS = 160
FP8BS_W4_MXFP4 = 0
FP8BS_W4_INT4 = 1
FP8BS_W4_MAX_M = 16
FP8BS_ROUTE_MAX_E = 1024
FP8BS_ROUTE_MAX_K = 32
FP8BS_ROUTE_MAX_M = 1024
FP8BS_MOE_W4_MAX_I = 8192
FP8BS_MOE_W4_MAX_H = 32768

STATUS = {
    0: "FP8BS_OK", -1: "FP8BS_ERR_ARG", -2: "FP8BS_ERR_SHAPE", -3: "FP8BS_ERR_ALIGN",
    -4: "FP8BS_ERR_SCALE_KIND", -5: "FP8BS_ERR_WORKSPACE", -6: "FP8BS_ERR_CUDA",
    -7: "FP8BS_ERR_TIMEOUT", -8: "FP8BS_ERR_DEVICE", -9: "FP8BS_ERR_RESIDENCY",
}
globals().update({name: code for code, name in STATUS.items()})

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfp8bs.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "fp8bs.h")

_lock = threading.Lock()
_lib = None


class Fp8bsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({fp8bs_status_string(status)})")


def build(force: bool = False) -> str:
    """Compile the CUDA library in-tree (nvcc, sm_103a)."""
    from . import native_build as _b
    return _b.build(force=force)


def use_trace_library() -> str:
    """Build the traced variant of the library (the fused kernel stamps its
    phase boundaries, read back with fp8bs_trace_read) and make lib() load it.
    Must be called before the first lib() call of the process."""
    global LIB_PATH
    from . import native_build as _b
    with _lock:
        if _lib is not None:
            raise RuntimeError("the library is already loaded")
        LIB_PATH = _b.build(trace=True)
    return LIB_PATH


def declared_functions() -> list[str]:
    """Names of the functions include/fp8bs.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fp8bs_[a-z0-9_]+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfp8bs.so is not built ({LIB_PATH}); call "
                               "fp8_block_scale_x128_gb300.build() first")
        L = ctypes.CDLL(LIB_PATH)
        c = ctypes
        vp, i64, sz, ci = c.c_void_p, c.c_int64, c.c_size_t, c.c_int
        sig = {
            "fp8bs_status_string": ([ci], c.c_char_p),
            "fp8bs_version": ([], ci),
            "fp8bs_encode_e4m3": ([vp, i64, vp, vp], ci),
            "fp8bs_quant": ([vp, i64, i64, i64, ci, vp, vp, vp], ci),
            "fp8bs_rmsnorm_quant": ([vp, i64, i64, i64, vp, ctypes.c_float, ci, vp, vp, vp, i64, vp], ci),
            "fp8bs_moe_workspace_bytes": ([i64, i64, i64, i64], ctypes.c_size_t),
            "fp8bs_moe_w8a16": ([vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, i64, i64, vp, vp,
                                 ctypes.c_size_t, vp], ci),
            "fp8bs_quant_weight_w4": ([vp, i64, i64, i64, ci, ci, vp, vp, vp], ci),
            "fp8bs_gemv_w4a16": ([vp, i64, i64, vp, i64, vp, i64, i64, i64, ci, ci, vp, i64, c.c_uint, vp], ci),
            "fp8bs_moe_route_workspace_bytes": ([i64, i64, i64], sz),
            "fp8bs_moe_route": ([vp, i64, i64, i64, vp, i64, i64, ci, ci, vp, vp, vp, sz, vp], ci),
            "fp8bs_moe_w4a16_workspace_bytes": ([i64, i64, i64], sz),
            "fp8bs_moe_w4a16": ([vp, i64, i64, i64, vp, vp, i64, vp, vp, vp, vp, i64, i64, ci, ci, vp, vp, sz, vp],
                                ci),
            "fp8bs_quant_weight": ([vp, i64, i64, i64, ci, vp, vp, vp], ci),
            "fp8bs_packed_weight_bytes": ([i64, i64, ci], sz),
            "fp8bs_prepack_weight": ([vp, i64, vp, i64, i64, ci, vp, sz, vp], ci),
            "fp8bs_workspace_bytes": ([i64, i64, ci], sz),
            "fp8bs_workspace_init": ([vp, sz, vp], ci),
            "fp8bs_gemm_fused": ([vp, i64, i64, vp, sz, i64, i64, ci, vp, i64, vp, sz, vp, vp,
                                  c.c_uint, vp], ci),
            "fp8bs_check_error": ([vp, vp], ci),
            "fp8bs_gemm_prequant": ([vp, i64, i64, vp, vp, sz, i64, i64, ci, vp, i64, vp, sz, c.c_uint, vp],
                                    ci),
            "fp8bs_gemm_fused_static": ([vp, i64, i64, vp, sz, i64, i64, ci, vp, i64, vp, vp, vp,
                                         c.c_uint, vp], ci),
            "fp8bs_trace_read": ([vp, sz], ci),
            "fp8bs_debug_config": ([ctypes.c_longlong, ci], ci),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return L


def fp8bs_status_string(status: int) -> str:
    try:
        return lib().fp8bs_status_string(int(status)).decode()
    except RuntimeError:
        return STATUS.get(status, "unknown")


def fp8bs_version() -> int:
    return int(lib().fp8bs_version())


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise Fp8bsError(rc, where)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _raw_stream(stream, device_index: int) -> int:
    """The cudaStream_t as an integer: the given stream, else the device's
    current one (looked up without building a torch.cuda.Stream)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device_index)
    if not isinstance(stream, torch.cuda.Stream):
        return int(stream)
    if stream.device_index != device_index:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, the tensors are on cuda:{device_index}")
    return stream.cuda_stream


def _on_stream(stream, device_index: int):
    """A context in which new tensors belong to `stream`: set up by it, and their
    memory not used again before what it has been given is done."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(stream)
        stream = torch.cuda.ExternalStream(raw, device=device_index) if raw else torch.cuda.default_stream(device_index)
    return torch.cuda.stream(stream)


def _wrong_device(*ts):
    """The library launches on the current device: refuse tensors elsewhere."""
    where = sorted({t.get_device() for t in ts})
    if where[0] < 0:
        raise ValueError("fp8bs tensors must live on a CUDA device")
    raise ValueError("fp8bs tensors must live on the current CUDA device: they are on "
                     f"{', '.join(f'cuda:{i}' for i in where)}, it is cuda:{torch._C._cuda_getDevice()}")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _scale_dtype(kind: int):
    return torch.uint8 if kind == FP8BS_SCALE_UE8M0 else torch.float32


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("fp8bs tensors must live on a CUDA device")


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def fp8bs_encode_e4m3(v: torch.Tensor, codes: torch.Tensor | None = None, stream=None):
    """fp32 v [n] (n % 4 == 0) -> uint8 e4m3fn codes [n] (RNE, satfinite)."""
    _require_cuda(v)
    assert v.dtype == torch.float32 and v.is_contiguous()
    with _on_stream(stream, v.get_device()):
        if codes is None:
            codes = torch.empty(v.numel(), dtype=torch.uint8, device=v.device)
    rc = lib().fp8bs_encode_e4m3(_ptr(v), v.numel(), _ptr(codes), _stream(stream))
    _check(rc, "fp8bs_encode_e4m3")
    return codes


def fp8bs_quant(x: torch.Tensor, scale_kind: int = FP8BS_SCALE_F32, xq: torch.Tensor | None = None,
                xs: torch.Tensor | None = None, stream=None):
    """bf16 x [M, K] (row stride x.stride(0)) -> (xq uint8 [M, K], xs [M, K/128])."""
    _require_cuda(x)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    with _on_stream(stream, x.get_device()):
        if xq is None:
            xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        if xs is None:
            xs = torch.empty((M, K // 128), dtype=_scale_dtype(scale_kind), device=x.device)
    rc = lib().fp8bs_quant(_ptr(x), M, K, x.stride(0), int(scale_kind), _ptr(xq), _ptr(xs),
                           _stream(stream))
    _check(rc, "fp8bs_quant")
    return xq, xs


def fp8bs_rmsnorm_quant(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                        scale_kind: int = FP8BS_SCALE_F32, xq: torch.Tensor | None = None,
                        xs: torch.Tensor | None = None, y: torch.Tensor | None = None,
                        want_y: bool = False, stream=None):
    """RMSNorm of bf16 x [M, K] with bf16 weight gamma [K], then the 1x128 quant.

    Returns (xq uint8 [M, K], xs [M, K/128], y bf16 [M, K] or None); y is
    written when given or when want_y."""
    _require_cuda(x, gamma)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert gamma.dtype == torch.bfloat16 and gamma.dim() == 1 and gamma.is_contiguous()
    M, K = x.shape
    with _on_stream(stream, x.get_device()):
        if xq is None:
            xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        if xs is None:
            xs = torch.empty((M, K // 128), dtype=_scale_dtype(scale_kind), device=x.device)
        if y is None and want_y:
            y = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
    if y is not None:
        assert y.dtype == torch.bfloat16 and y.dim() == 2 and y.stride(1) == 1
    rc = lib().fp8bs_rmsnorm_quant(_ptr(x), M, K, x.stride(0), _ptr(gamma), float(eps),
                                   int(scale_kind), _ptr(xq), _ptr(xs),
                                   _ptr(y) if y is not None else None,
                                   y.stride(0) if y is not None else 0, _stream(stream))
    _check(rc, "fp8bs_rmsnorm_quant")
    return xq, xs, y


def fp8bs_moe_workspace_bytes(M: int, S: int, H: int, I: int) -> int:
    return int(lib().fp8bs_moe_workspace_bytes(int(M), int(S), int(H), int(I)))


def new_moe_workspace(M: int, S: int, H: int, I: int, device=None) -> torch.Tensor:
    """Allocate (with torch) a zeroed MoE workspace for up to M tokens x S slots."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    n = fp8bs_moe_workspace_bytes(M, S, H, I)
    if n == 0:
        raise Fp8bsError(FP8BS_ERR_SHAPE, "fp8bs_moe_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def fp8bs_moe_w8a16(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                    w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor,
                    y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """One small-M MoE layer: bf16 x [M, H]; int32 topk_ids and fp32 topk_w
    [M, S]; e4m3 (uint8) w13 [E, 2I, H] with fp32 s13 [E, 2I/128, H/128]; w2
    [E, H, I] with s2 [E, H/128, I/128].  Returns bf16 y [M, H]."""
    _require_cuda(x, topk_ids, topk_w, w13, s13, w2, s2, y, workspace)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_contiguous()
    assert topk_ids.dtype == torch.int32 and topk_w.dtype == torch.float32
    assert topk_ids.is_contiguous() and topk_w.is_contiguous() and topk_ids.shape == topk_w.shape
    for t in (w13, s13, w2, s2):
        assert t.is_contiguous()
    assert w13.dtype == torch.uint8 and w2.dtype == torch.uint8
    assert s13.dtype == torch.float32 and s2.dtype == torch.float32
    M, H = x.shape
    S = topk_ids.shape[1]
    E, I2, _ = w13.shape
    I = I2 // 2
    with _on_stream(stream, x.get_device()):
        if y is None:
            y = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            workspace = new_moe_workspace(M, S, H, I, x.device)
    rc = lib().fp8bs_moe_w8a16(_ptr(x), M, H, _ptr(topk_ids), _ptr(topk_w), S, _ptr(w13), _ptr(s13),
                               _ptr(w2), _ptr(s2), E, I, _ptr(y), _ptr(workspace),
                               workspace.numel(), _stream(stream))
    _check(rc, "fp8bs_moe_w8a16")
    return y


_W4_FORMATS = {(FP8BS_W4_MXFP4, 32): torch.uint8, (FP8BS_W4_INT4, 32): torch.bfloat16,
               (FP8BS_W4_INT4, 64): torch.bfloat16, (FP8BS_W4_INT4, 128): torch.bfloat16}


def _w4_scale_dtype(fmt: int, group: int, where: str):
    dtype = _W4_FORMATS.get((fmt, group))
    if dtype is None:
        raise Fp8bsError(FP8BS_ERR_ARG, where)  # not a 4-bit format, or not one of its group sizes
    return dtype


def fp8bs_quant_weight_w4(w: torch.Tensor, fmt: int = FP8BS_W4_MXFP4, group: int = 32,
                          codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """fp32 w [N, K] -> (codes uint8 [N, K/2], scales [N, K/group]) in a 4-bit
    format: FP8BS_W4_MXFP4 (group 32, uint8 e8m0 scales) or FP8BS_W4_INT4
    (group 32, 64 or 128, bf16 scales)."""
    _require_cuda(w, codes, scales)
    device = w.get_device()
    if device != torch._C._cuda_getDevice():
        _wrong_device(w)
    scale_dtype = _w4_scale_dtype(fmt, group, "fp8bs_quant_weight_w4")
    assert w.dtype == torch.float32 and w.dim() == 2 and w.stride(1) == 1
    N, K = w.shape
    if codes is None or scales is None:
        with _on_stream(stream, device):
            if codes is None:
                codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
            if scales is None:
                scales = torch.empty((N, K // group), dtype=scale_dtype, device=w.device)
    if not device == codes.get_device() == scales.get_device():
        _wrong_device(w, codes, scales)
    assert codes.dtype == torch.uint8 and codes.is_contiguous() and codes.shape == (N, K // 2)
    assert scales.dtype == scale_dtype and scales.is_contiguous() and scales.shape == (N, K // group)
    rc = lib().fp8bs_quant_weight_w4(_ptr(w), N, K, w.stride(0), int(fmt), int(group), _ptr(codes), _ptr(scales),
                                     _raw_stream(stream, device))
    _check(rc, "fp8bs_quant_weight_w4")
    return codes, scales


def fp8bs_gemv_w4a16(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, fmt: int = FP8BS_W4_MXFP4,
                     group: int = 32, y: torch.Tensor | None = None, pdl: bool = False,
                     stream=None) -> torch.Tensor:
    """Y = bf16(x . W^T) for bf16 x [M <= 16, K] and a 4-bit weight: codes uint8
    [N, K/2], scales [N, K/group] (rows may be strided).  pdl=True launches with
    programmatic dependent launch; use it only when no unfinished work on the
    stream, however far back, writes the weight."""
    device = x.get_device()
    if device < 0 or not device == codes.get_device() == scales.get_device() == torch._C._cuda_getDevice():
        _wrong_device(x, codes, scales)
    scale_dtype = _w4_scale_dtype(fmt, group, "fp8bs_gemv_w4a16")
    M, K = x.shape
    N, half = codes.shape
    ldx, x1 = x.stride()
    ldc, c1 = codes.stride()
    lds, s1 = scales.stride()
    assert x.dtype is torch.bfloat16 and codes.dtype is torch.uint8 and scales.dtype is scale_dtype
    assert x1 == c1 == s1 == 1 and 2 * half == K and scales.shape == (N, K // group)
    if y is None:
        with _on_stream(stream, device):
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    elif y.get_device() != device:
        _wrong_device(x, y)
    ldy, y1 = y.stride()
    assert y.dtype is torch.bfloat16 and y1 == 1 and y.shape == (M, N)
    rc = (_lib or lib()).fp8bs_gemv_w4a16(x.data_ptr(), M, ldx, codes.data_ptr(), ldc, scales.data_ptr(), lds, N, K,
                                          fmt, group, y.data_ptr(), ldy, FP8BS_FLAG_PDL if pdl else 0,
                                          torch._C._cuda_getCurrentRawStream(device) if stream is None else
                                          _raw_stream(stream, device))
    if rc:
        raise Fp8bsError(rc, "fp8bs_gemv_w4a16")
    return y


_ROUTE_SHARED = {"none": 0, "one": 1, "gate": 2}


def fp8bs_moe_route_workspace_bytes(M: int, E: int, H: int) -> int:
    return int(lib().fp8bs_moe_route_workspace_bytes(int(M), int(E), int(H)))


def new_moe_route_workspace(M: int, E: int, H: int, device=None) -> torch.Tensor:
    """Allocate (with torch, zeroed by the current stream) a router workspace for up to M tokens."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    n = fp8bs_moe_route_workspace_bytes(M, E, H)
    if n == 0:
        raise Fp8bsError(FP8BS_ERR_SHAPE, "fp8bs_moe_route_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def fp8bs_moe_route(x: torch.Tensor, w: torch.Tensor, k: int, renorm: bool = True, shared: str = "none",
                    ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None):
    """Router: bf16 x [M, H] and w [E, H] -> (int32 ids, fp32 weights) [M, S],
    the k experts with the largest logits per token, softmax weights
    (renormalised over them or not).  shared="one" appends expert E with
    weight 1, shared="gate" with weight sigmoid(x . w[E]) (w then has E + 1
    rows)."""
    device = x.get_device()
    if device < 0 or not device == w.get_device() == torch._C._cuda_getDevice():
        _wrong_device(x, w)
    M, H = x.shape
    rows, Hw = w.shape
    ldx, x1 = x.stride()
    code = _ROUTE_SHARED.get(shared, -1)
    E = rows - 1 if code == 2 else rows
    if code < 0 or not 0 < k <= E:
        raise Fp8bsError(FP8BS_ERR_ARG if code < 0 else FP8BS_ERR_SHAPE, "fp8bs_moe_route")
    S = k + 1 if code else k
    assert x.dtype is torch.bfloat16 and x1 == 1
    assert w.dtype is torch.bfloat16 and Hw == H and w.is_contiguous()
    if ids is None or weights is None or workspace is None:
        with _on_stream(stream, device):
            if ids is None:
                ids = torch.empty((M, S), dtype=torch.int32, device=x.device)
            if weights is None:
                weights = torch.empty((M, S), dtype=torch.float32, device=x.device)
            if workspace is None:
                workspace = new_moe_route_workspace(M, E, H, x.device)
    if not device == ids.get_device() == weights.get_device() == workspace.get_device():
        _wrong_device(x, ids, weights, workspace)
    assert ids.dtype is torch.int32 and ids.is_contiguous() and ids.shape == (M, S)
    assert weights.dtype is torch.float32 and weights.is_contiguous() and weights.shape == (M, S)
    assert workspace.dtype is torch.uint8 and workspace.is_contiguous()
    rc = (_lib or lib()).fp8bs_moe_route(x.data_ptr(), M, H, ldx, w.data_ptr(), E, k, 1 if renorm else 0, code,
                                         ids.data_ptr(), weights.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                         torch._C._cuda_getCurrentRawStream(device) if stream is None else
                                         _raw_stream(stream, device))
    if rc:
        raise Fp8bsError(rc, "fp8bs_moe_route")
    return ids, weights


def fp8bs_moe_w4a16_workspace_bytes(M: int, S: int, I: int) -> int:
    return int(lib().fp8bs_moe_w4a16_workspace_bytes(int(M), int(S), int(I)))


def new_moe_w4_workspace(M: int, S: int, I: int, device=None) -> torch.Tensor:
    """Allocate (with torch, zeroed by the current stream) a 4-bit MoE workspace for up to M tokens x S slots."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    n = fp8bs_moe_w4a16_workspace_bytes(M, S, I)
    if n == 0:
        raise Fp8bsError(FP8BS_ERR_SHAPE, "fp8bs_moe_w4a16_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def fp8bs_moe_w4a16(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, w13: torch.Tensor,
                    s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor, fmt: int = FP8BS_W4_MXFP4,
                    group: int = 32, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """One small-batch MoE layer on 4-bit weights: bf16 x [M, H]; int32 topk_ids
    and fp32 topk_w [M, S]; codes w13 [E, 2I, H/2], w2 [E, H, I/2] (uint8) with
    scales s13 [E, 2I, H/group], s2 [E, H, I/group].  Returns bf16 y [M, H]."""
    device = x.get_device()
    if device < 0 or not (device == topk_ids.get_device() == topk_w.get_device() == w13.get_device() ==
                          s13.get_device() == w2.get_device() == s2.get_device() == torch._C._cuda_getDevice()):
        _wrong_device(x, topk_ids, topk_w, w13, s13, w2, s2)
    scale_dtype = _w4_scale_dtype(fmt, group, "fp8bs_moe_w4a16")
    M, H = x.shape
    ldx, x1 = x.stride()
    routing = topk_ids.shape
    S = routing[1]
    E, H2, half = w2.shape
    I = 2 * half
    assert x.dtype is torch.bfloat16 and x1 == 1
    assert topk_ids.dtype is torch.int32 and topk_ids.is_contiguous() and routing[0] == M
    assert topk_w.dtype is torch.float32 and topk_w.is_contiguous() and topk_w.shape == routing
    assert w13.dtype is torch.uint8 and w13.is_contiguous() and w13.shape == (E, 2 * I, H // 2)
    assert w2.dtype is torch.uint8 and w2.is_contiguous() and H2 == H
    assert s13.dtype is scale_dtype and s13.is_contiguous() and s13.shape == (E, 2 * I, H // group)
    assert s2.dtype is scale_dtype and s2.is_contiguous() and s2.shape == (E, H, I // group)
    if y is None or workspace is None:
        with _on_stream(stream, device):
            if y is None:
                y = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
            if workspace is None:
                workspace = new_moe_w4_workspace(M, S, I, x.device)
    if not device == y.get_device() == workspace.get_device():
        _wrong_device(x, y, workspace)
    assert y.dtype is torch.bfloat16 and y.is_contiguous() and y.shape == (M, H)
    assert workspace.dtype is torch.uint8 and workspace.is_contiguous()
    rc = (_lib or lib()).fp8bs_moe_w4a16(x.data_ptr(), M, H, ldx, topk_ids.data_ptr(), topk_w.data_ptr(), S,
                                         w13.data_ptr(), s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), E, I, fmt,
                                         group, y.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                         torch._C._cuda_getCurrentRawStream(device) if stream is None else
                                         _raw_stream(stream, device))
    if rc:
        raise Fp8bsError(rc, "fp8bs_moe_w4a16")
    return y


def fp8bs_quant_weight(w: torch.Tensor, scale_kind: int = FP8BS_SCALE_F32, stream=None):
    """fp32 w [N, K] -> (wq uint8 [N, K], ws [N/128, K/128]) in 128x128 blocks."""
    _require_cuda(w)
    assert w.dtype == torch.float32 and w.dim() == 2 and w.stride(1) == 1
    N, K = w.shape
    with _on_stream(stream, w.get_device()):
        wq = torch.empty((N, K), dtype=torch.uint8, device=w.device)
        ws = torch.empty((N // 128, K // 128), dtype=_scale_dtype(scale_kind), device=w.device)
    rc = lib().fp8bs_quant_weight(_ptr(w), N, K, w.stride(0), int(scale_kind), _ptr(wq), _ptr(ws),
                                  _stream(stream))
    _check(rc, "fp8bs_quant_weight")
    return wq, ws


def fp8bs_packed_weight_bytes(N: int, K: int, scale_kind: int = FP8BS_SCALE_F32) -> int:
    return int(lib().fp8bs_packed_weight_bytes(int(N), int(K), int(scale_kind)))


def fp8bs_prepack_weight(wq: torch.Tensor, ws: torch.Tensor, scale_kind: int = FP8BS_SCALE_F32,
                         packed: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """wq uint8 [N, K] + ws [N/128, K/128] -> packed uint8 buffer (GB300 tile layout)."""
    _require_cuda(wq, ws)
    assert wq.dtype == torch.uint8 and wq.dim() == 2 and wq.stride(1) == 1
    assert ws.is_contiguous() and ws.dtype == _scale_dtype(scale_kind)
    N, K = wq.shape
    nbytes = fp8bs_packed_weight_bytes(N, K, scale_kind)
    if nbytes == 0:
        raise Fp8bsError(-2, "fp8bs_packed_weight_bytes")
    if packed is None:
        with _on_stream(stream, wq.get_device()):
            packed = torch.empty(nbytes, dtype=torch.uint8, device=wq.device)
    rc = lib().fp8bs_prepack_weight(_ptr(wq), wq.stride(0), _ptr(ws), N, K, int(scale_kind),
                                    _ptr(packed), packed.numel(), _stream(stream))
    _check(rc, "fp8bs_prepack_weight")
    return packed


def fp8bs_workspace_bytes(N: int, K: int, sm_count: int = 0) -> int:
    return int(lib().fp8bs_workspace_bytes(int(N), int(K), int(sm_count)))


def fp8bs_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _require_cuda(workspace)
    rc = lib().fp8bs_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check(rc, "fp8bs_workspace_init")


def new_workspace(N: int, K: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (with torch) and initialise a workspace for an N x K weight."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    n = fp8bs_workspace_bytes(N, K)
    if n == 0:
        raise Fp8bsError(-2, "fp8bs_workspace_bytes")
    with _on_stream(stream, torch.device(device).index):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    fp8bs_workspace_init(ws, stream)
    return ws


def fp8bs_gemm_fused(x: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                     scale_kind: int = FP8BS_SCALE_F32, y: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, xq_out: torch.Tensor | None = None,
                     xs_out: torch.Tensor | None = None, pdl: bool = False,
                     stream=None) -> torch.Tensor:
    """Y = bf16(quant(x) . W^T) for bf16 x [M <= 64, K] and a packed weight.

    pdl=True launches with programmatic dependent launch (FP8BS_FLAG_PDL); use
    it only when no unfinished work on the stream, however far back, writes
    `packed`.
    """
    _require_cuda(x, packed, y, workspace, xq_out, xs_out)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M = x.shape[0]
    assert x.shape[1] == K
    with _on_stream(stream, x.get_device()):
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            workspace = new_workspace(N, K, x.device, stream)
    rc = lib().fp8bs_gemm_fused(
        _ptr(x), M, x.stride(0), _ptr(packed), packed.numel(), N, K, int(scale_kind), _ptr(y),
        y.stride(0), _ptr(workspace), workspace.numel(), _ptr(xq_out), _ptr(xs_out),
        FP8BS_FLAG_PDL if pdl else 0, _stream(stream))
    _check(rc, "fp8bs_gemm_fused")
    return y


def fp8bs_gemm_prequant(xq: torch.Tensor, xs: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                        scale_kind: int = FP8BS_SCALE_F32, y: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, pdl: bool = False,
                        stream=None) -> torch.Tensor:
    """Y = bf16(xq . W^T) with the block scales, for pre-quantised activations
    (uint8 e4m3 codes [M, K], scales [M, K/128] fp32 or uint8 e8m0): the
    second launch of the two-launch path."""
    _require_cuda(xq, xs, packed, y, workspace)
    assert xq.dtype == torch.uint8 and xq.dim() == 2 and xq.stride(1) == 1 and xq.shape[1] == K
    assert xs.is_contiguous() and xs.shape == (xq.shape[0], K // 128)
    M = xq.shape[0]
    with _on_stream(stream, xq.get_device()):
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
        if workspace is None:
            workspace = new_workspace(N, K, xq.device, stream)
    rc = lib().fp8bs_gemm_prequant(
        _ptr(xq), M, xq.stride(0), _ptr(xs), _ptr(packed), packed.numel(), N, K, int(scale_kind),
        _ptr(y), y.stride(0), _ptr(workspace), workspace.numel(), FP8BS_FLAG_PDL if pdl else 0,
        _stream(stream))
    _check(rc, "fp8bs_gemm_prequant")
    return y


def fp8bs_gemm_fused_static(x: torch.Tensor, packed: torch.Tensor, N: int, K: int,
                            scale_kind: int = FP8BS_SCALE_F32, y: torch.Tensor | None = None,
                            xq_out: torch.Tensor | None = None, xs_out: torch.Tensor | None = None,
                            status_out: torch.Tensor | None = None, pdl: bool = False,
                            stream=None) -> torch.Tensor:
    """fp8bs_gemm_fused with the library's fixed per-device scratch instead of a
    workspace (K <= FP8BS_STATIC_MAX_K).  The C call allocates nothing; pass
    `y` to keep this wrapper from allocating it.  `status_out` (int32 [1] on
    the device, optional) receives the sticky device status after the kernel.
    """
    _require_cuda(x, packed, y, xq_out, xs_out, status_out)
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    M = x.shape[0]
    assert x.shape[1] == K
    if y is None:
        with _on_stream(stream, x.get_device()):
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    rc = lib().fp8bs_gemm_fused_static(
        _ptr(x), M, x.stride(0), _ptr(packed), packed.numel(), N, K, int(scale_kind), _ptr(y),
        y.stride(0), _ptr(xq_out), _ptr(xs_out), _ptr(status_out),
        FP8BS_FLAG_PDL if pdl else 0, _stream(stream))
    _check(rc, "fp8bs_gemm_fused_static")
    return y


FP8BS_TRACE_CALLS, FP8BS_TRACE_CTAS, FP8BS_TRACE_POINTS = 256, 160, 64


def fp8bs_trace_read():
    """The traced library's timeline as a numpy uint64 array
    [calls][CTAs][points][2] (globaltimer ns, clock64); raises in a plain build."""
    import numpy as np
    buf = np.zeros((FP8BS_TRACE_CALLS, FP8BS_TRACE_CTAS, FP8BS_TRACE_POINTS, 2), dtype=np.uint64)
    rc = lib().fp8bs_trace_read(ctypes.c_void_p(buf.ctypes.data), buf.nbytes)
    _check(rc, "fp8bs_trace_read")
    return buf


def fp8bs_debug_config(timeout_cycles: int = 0, sm_count_override: int = 0) -> None:
    """Diagnostic overrides of the fused GEMM's launches (tests only): the
    bounded waits' limit in SM cycles and the multiprocessor count grids and
    workspaces are sized for; 0 restores each default."""
    _check(lib().fp8bs_debug_config(int(timeout_cycles), int(sm_count_override)), "fp8bs_debug_config")


def fp8bs_check_error(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(lib().fp8bs_check_error(_ptr(workspace), _stream(stream)))
