// C ABI of the fp8bs library (declared in include/fp8bs.h).
//
// Every entry point checks its arguments on the host first, in this order:
// null pointers and the scale kind (FP8BS_ERR_ARG), shapes (FP8BS_ERR_SHAPE),
// strides and alignment (FP8BS_ERR_ALIGN), buffer sizes (FP8BS_ERR_WORKSPACE).
// Nothing is enqueued when a check fails, and no check touches the GPU, so the
// checks run on machines without one.  The support rules follow "[AMD] Small-M
// FP8 block-scale GEMM with fused activation quant for gfx950 (Qwen3.5)",
// "Modifications" (bf16 input with 16-byte aligned rows, a contiguous
// [N/128, K/128] weight scale, M <= 32); a mismatching scale kind is refused
// rather than reinterpreted, as "[Perf] [AMD] dsv4: optional e8m0 mxscale GEMM
// for dense 128x128 fp8 linears (6/8)", "Modifications" requires.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <mutex>

#include "attn.cuh"
#include "internal.cuh"
#include "moe.cuh"
#include "producer.cuh"
#include "trace.cuh"
#include "w4.cuh"

namespace {

using namespace fp8bs;

constexpr int64_t kMaxDim = int64_t(1) << 24;  // N, K bound (keeps every index in range)
constexpr long long kDefaultTimeoutCycles = 2000000000LL;  // ~1 s at 2 GHz

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool kind_ok(int kind) { return kind == FP8BS_SCALE_F32 || kind == FP8BS_SCALE_UE8M0; }

bool nk_ok(int64_t N, int64_t K) {
    return N >= kTile && K >= kTile && N % kTile == 0 && K % kTile == 0 && N <= kMaxDim && K <= kMaxDim;
}

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return FP8BS_OK;
    // the launchers' refusal of a grid that cannot be resident at once
    return e == cudaErrorCooperativeLaunchTooLarge ? FP8BS_ERR_RESIDENCY : FP8BS_ERR_CUDA;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// Diagnostic overrides (fp8bs_debug_config); 0: the defaults.
std::atomic<long long> g_timeout_override{0};
std::atomic<int> g_sm_override{0};

long long timeout_cycles() {
    const long long t = g_timeout_override.load(std::memory_order_relaxed);
    return t > 0 ? t : kDefaultTimeoutCycles;
}

// Multiprocessor count of the current device, cached per device (relaxed
// atomics: concurrent first calls from several host threads may both query).
int current_sm_count(int* out) {
    const int forced = g_sm_override.load(std::memory_order_relaxed);
    if (forced > 0) {
        *out = forced;
        return FP8BS_OK;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FP8BS_ERR_CUDA;
    static std::atomic<int> cache[64];
    if (dev >= 0 && dev < 64) {
        const int n = cache[dev].load(std::memory_order_relaxed);
        if (n > 0) {
            *out = n;
            return FP8BS_OK;
        }
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return FP8BS_ERR_CUDA;
    if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    *out = n;
    return FP8BS_OK;
}

// A 4-bit weight format with a group size that it has.
bool w4_ok(int format, int group) {
    return format == FP8BS_W4_MXFP4 ? group == 32
                                    : format == FP8BS_W4_INT4 && (group == 32 || group == 64 || group == 128);
}
int64_t w4_scale_size(int format) { return format == FP8BS_W4_MXFP4 ? 1 : 2; }

// A heads tensor [tokens, heads, D] of bf16: rows on 16 bytes.
bool heads_aligned(const uint16_t* p, int64_t ld, int64_t hs) { return aligned(p, 16) && ld % 8 == 0 && hs % 8 == 0; }

bool head_dim_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements: a tensor map's strides are below 2^40 bytes

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// The host description of a paged cache: FP8BS_OK or why not.
int cache_check(const fp8bs_kv_cache* c) {
    if (!c || (c->kind != FP8BS_KV_BF16 && c->kind != FP8BS_KV_E4M3) || !c->k || !c->v) return FP8BS_ERR_ARG;
    const bool codes = c->kind == FP8BS_KV_E4M3;
    if (codes && (!c->k_scale || !c->v_scale)) return FP8BS_ERR_ARG;
    if (!stride_ok(c->page_stride) || !stride_ok(c->slot_stride) || !stride_ok(c->head_stride)) return FP8BS_ERR_ARG;
    if (codes && (!stride_ok(c->scale_page_stride) || !stride_ok(c->scale_slot_stride) || !stride_ok(c->scale_head_stride)))
        return FP8BS_ERR_ARG;
    if (!head_dim_ok(c->head_dim) || c->kv_heads < 1 || c->kv_heads > kMaxHeads || c->page_size < 1 ||
        c->page_size > 65536 || (c->page_size & (c->page_size - 1)) != 0 || c->pages < 1 || c->pages > 0x7FFFFFFF)
        return FP8BS_ERR_SHAPE;
    // rows of one axis apart from each other
    if ((c->pages > 1 && c->page_stride < c->head_dim) || (c->page_size > 1 && c->slot_stride < c->head_dim) ||
        (c->kv_heads > 1 && c->head_stride < c->head_dim))
        return FP8BS_ERR_ARG;
    if (codes && ((c->pages > 1 && c->scale_page_stride < 1) || (c->page_size > 1 && c->scale_slot_stride < 1) ||
                  (c->kv_heads > 1 && c->scale_head_stride < 1)))
        return FP8BS_ERR_ARG;
    const int64_t unit = codes ? 16 : 8;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % unit || c->slot_stride % unit || c->head_stride % unit)
        return FP8BS_ERR_ALIGN;
    return FP8BS_OK;
}

// Checks common to the calls that norm and rotate heads.
int rope_check(const RopeArgs& a) {
    if (a.layout != FP8BS_ROPE_HALF && a.layout != FP8BS_ROPE_INTERLEAVED) return FP8BS_ERR_ARG;
    if (!std::isfinite(a.amplitude) || !std::isfinite(a.eps) || a.eps < 0.0f) return FP8BS_ERR_ARG;
    if (a.T < 0 || a.T > kMaxDim || a.Hq < 0 || a.Hq > kMaxHeads || a.Hk < 0 || a.Hk > kMaxHeads || a.Hq + a.Hk < 1 ||
        !head_dim_ok(a.D) || a.R < 0 || a.R > a.D || a.R % (a.layout == FP8BS_ROPE_HALF ? 16 : 2) != 0)
        return FP8BS_ERR_SHAPE;
    if (a.T == 0) return FP8BS_OK;
    if (a.Hq && (!a.q || !a.qo)) return FP8BS_ERR_ARG;
    if (a.Hk && (!a.k || (a.append ? !a.v : !a.ko))) return FP8BS_ERR_ARG;
    if (a.R && (!a.positions || !a.freqs)) return FP8BS_ERR_ARG;
    if (a.append && !a.slots) return FP8BS_ERR_ARG;
    // rows of one tensor apart from each other where they are written, not negative elsewhere
    auto apart = [&](int64_t ld, int64_t hs, int H) {
        return stride_ok(ld) && stride_ok(hs) && (H < 2 || hs >= a.D) && (a.T < 2 || ld >= a.D);
    };
    // (head strides count 32 bits of bytes in the kernel)
    for (int64_t hs : {a.Hq ? a.hsq : 0, a.Hq ? a.hsqo : 0, a.Hk ? a.hsk : 0, a.Hk && a.append ? a.hsv : 0, a.Hk && !a.append ? a.hsko : 0})
        if (hs >= int64_t(1) << 31) return FP8BS_ERR_ARG;
    if (a.Hq && (!stride_ok(a.ldq) || !stride_ok(a.hsq) || !apart(a.ldqo, a.hsqo, a.Hq))) return FP8BS_ERR_ARG;
    if (a.Hk && (!stride_ok(a.ldk) || !stride_ok(a.hsk))) return FP8BS_ERR_ARG;
    if (a.Hk && (a.append ? !stride_ok(a.ldv) || !stride_ok(a.hsv) : !apart(a.ldko, a.hsko, a.Hk))) return FP8BS_ERR_ARG;
    if (a.Hq && (!heads_aligned(a.q, a.ldq, a.hsq) || !heads_aligned(a.qo, a.ldqo, a.hsqo))) return FP8BS_ERR_ALIGN;
    if (a.Hk && (!heads_aligned(a.k, a.ldk, a.hsk) ||
                 !(a.append ? heads_aligned(a.v, a.ldv, a.hsv) : heads_aligned(a.ko, a.ldko, a.hsko))))
        return FP8BS_ERR_ALIGN;
    if (a.R && (!aligned(a.positions, 8) || !aligned(a.freqs, 8))) return FP8BS_ERR_ALIGN;
    if (a.append && (!aligned(a.slots, 8) || (a.err && !aligned(a.err, 256)))) return FP8BS_ERR_ALIGN;
    if ((a.gq && !aligned(a.gq, 16)) || (a.gk && !aligned(a.gk, 16))) return FP8BS_ERR_ALIGN;
    return FP8BS_OK;
}

int run_rope(RopeArgs& a, void* stream) {
    const int bad = rope_check(a);
    if (bad != FP8BS_OK || a.T == 0) return bad;
    const int rc = current_sm_count(&a.sm_count);
    if (rc != FP8BS_OK) return rc;
    return status_of(launch_qk_norm_rope(a, as_stream(stream)));
}

size_t workspace_bytes_for(int64_t K, int sm_count) { return ws_total_bytes(sm_count, K); }

// Above kFusedMaxM tokens the fused call runs the quant and the GEMM on its
// codes as two launches: the single launch has no 64-token tile that
// quantises, and [P1] "Motivation" likewise keeps larger inputs on the
// library path.
constexpr int kTwoLaunchMinM = kFusedMaxM + 1;

// The fused call, routed: below kTwoLaunchMinM one launch; from it on the
// 1x128 quant, then the GEMM on those codes.  The codes and scales go to
// xq_out / xs_out when the caller asked for them, else to the workspace's
// activation records, which the GEMM on given codes does not use (room for
// 64 rows of codes and fp32 scales per K block).
cudaError_t launch_fused_routed(FusedArgs a, cudaStream_t stream) {
    if (a.M < kTwoLaunchMinM) return launch_fused(a, stream);
    uint8_t* act = a.workspace + ws_act_offset(a.sm_count);
    uint8_t* xq = a.xq_out ? a.xq_out : act;
    void* xs = a.xs_out ? a.xs_out : static_cast<void*>(act + static_cast<size_t>(FP8BS_MAX_M) * a.K);
    const cudaError_t e = launch_quant(a.x, a.M, a.K, a.ldx, a.kind, xq, xs, stream, a.pdl != 0);
    if (e != cudaSuccess) return e;
    a.xq_in = xq;
    a.ldxq = a.K;
    a.xs_in = xs;
    a.xq_out = nullptr;
    a.xs_out = nullptr;
    return launch_fused(a, stream);
}

// Scratch of fp8bs_gemm_fused_static: one fixed array per device, laid out like
// a caller's workspace for FP8BS_STATIC_MAX_SMS CTAs and K up to
// FP8BS_STATIC_MAX_K.
constexpr size_t kStaticScratchBytes = ws_total_bytes(FP8BS_STATIC_MAX_SMS, FP8BS_STATIC_MAX_K);
static_assert(kStaticScratchBytes == 22057216, "fp8bs.h states the scratch size");

__device__ __align__(256) uint8_t g_static_scratch[kStaticScratchBytes];

constexpr int kStaticMaxDevices = 64;
std::mutex g_static_mu;
uint8_t* g_static_ptr[kStaticMaxDevices] = {};

// Address of the current device's scratch; the first call per device looks it
// up and zeroes it on `s` (the error word and the epoch words must start at
// zero), then waits for that, so a call from another thread or stream never
// sees a half-cleared scratch.  That set-up synchronises `s`, which would
// invalidate a stream capture: on a capturing stream it is refused
// (FP8BS_ERR_ARG) before the stream is touched.
int static_scratch(cudaStream_t s, uint8_t** out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FP8BS_ERR_CUDA;
    if (dev < 0 || dev >= kStaticMaxDevices) return FP8BS_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_static_mu);
    if (!g_static_ptr[dev]) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) return FP8BS_ERR_CUDA;
        if (cap != cudaStreamCaptureStatusNone) return FP8BS_ERR_ARG;
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_static_scratch) != cudaSuccess) return FP8BS_ERR_CUDA;
        if (cudaMemsetAsync(p, 0, kStaticScratchBytes, s) != cudaSuccess) return FP8BS_ERR_CUDA;
        if (cudaStreamSynchronize(s) != cudaSuccess) return FP8BS_ERR_CUDA;
        g_static_ptr[dev] = static_cast<uint8_t*>(p);
    }
    *out = g_static_ptr[dev];
    return FP8BS_OK;
}

}  // namespace

extern "C" {

const char* fp8bs_status_string(int status) {
    switch (status) {
        case FP8BS_OK: return "ok";
        case FP8BS_ERR_ARG: return "invalid argument (null pointer, scale kind or stride)";
        case FP8BS_ERR_SHAPE: return "unsupported shape (M, N or K)";
        case FP8BS_ERR_ALIGN: return "pointer or row stride not 16-byte aligned";
        case FP8BS_ERR_SCALE_KIND: return "packed weight has another scale kind or shape";
        case FP8BS_ERR_WORKSPACE: return "workspace or packed buffer too small or misaligned";
        case FP8BS_ERR_CUDA: return "CUDA runtime error";
        case FP8BS_ERR_TIMEOUT: return "device wait timed out";
        case FP8BS_ERR_DEVICE: return "device-side check failed";
        case FP8BS_ERR_RESIDENCY: return "the launch's CTAs cannot all be resident at once";
        default: return "unknown status";
    }
}

int fp8bs_version(void) { return (1 << 16) | 0; }

int fp8bs_encode_e4m3(const float* v, int64_t n, uint8_t* codes, void* stream) {
    if (n < 0 || n % 4 != 0) return FP8BS_ERR_SHAPE;
    if (n == 0) return FP8BS_OK;
    if (!v || !codes) return FP8BS_ERR_ARG;
    if (!aligned(v, 16) || !aligned(codes, 4)) return FP8BS_ERR_ALIGN;
    return status_of(launch_encode_e4m3(v, n, codes, as_stream(stream)));
}

int fp8bs_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int scale_kind, uint8_t* xq,
                void* xs, void* stream) {
    if (!kind_ok(scale_kind)) return FP8BS_ERR_ARG;
    if (M < 0 || K < kTile || K % kTile != 0 || K > kMaxDim || M > kMaxDim) return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !xq || !xs) return FP8BS_ERR_ARG;
    if (ldx < K) return FP8BS_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(xq, 8) ||
        (scale_kind == FP8BS_SCALE_F32 && !aligned(xs, 4)))
        return FP8BS_ERR_ALIGN;
    return status_of(launch_quant(x, M, K, ldx, scale_kind, xq, xs, as_stream(stream)));
}

int fp8bs_rmsnorm_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint16_t* gamma, float eps,
                        int scale_kind, uint8_t* xq, void* xs, uint16_t* y, int64_t ldy, void* stream) {
    if (!kind_ok(scale_kind) || !(eps >= 0.0f) || !(eps <= 3.4e38f)) return FP8BS_ERR_ARG;
    if (M < 0 || K < kTile || K % kTile != 0 || K > FP8BS_RMSNORM_MAX_K || M > kMaxDim) return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !gamma || !xq || !xs) return FP8BS_ERR_ARG;
    if (ldx < K || (y && ldy < K)) return FP8BS_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(gamma, 16) || !aligned(xq, 8) ||
        (scale_kind == FP8BS_SCALE_F32 && !aligned(xs, 4)) || (y && (!aligned(y, 16) || ldy % 8 != 0)))
        return FP8BS_ERR_ALIGN;
    return status_of(launch_rmsnorm_quant(x, M, K, ldx, gamma, eps, scale_kind, xq, xs, y, ldy, as_stream(stream)));
}
size_t fp8bs_moe_workspace_bytes(int64_t M, int64_t S, int64_t H, int64_t I) {
    if (M < 0 || S < 1 || M * S > FP8BS_MOE_MAX_PAIRS || H < 512 || H % 512 != 0 || H > kMaxDim ||
        (I != 128 && I != 256 && I != FP8BS_MOE_MAX_I))
        return 0;
    return moe_workspace_bytes(M, S, H, I);
}
int fp8bs_moe_w8a16(const uint16_t* x, int64_t M, int64_t H, const int32_t* topk_ids, const float* topk_w,
                    int64_t S, const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2, int64_t E,
                    int64_t I, uint16_t* y, void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || S < 1 || M * S > FP8BS_MOE_MAX_PAIRS || E < 1 || E > FP8BS_MOE_MAX_EXPERTS || H < 512 ||
        H % 512 != 0 || H > kMaxDim || (I != 128 && I != 256 && I != FP8BS_MOE_MAX_I))
        return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !topk_ids || !topk_w || !w13 || !s13 || !w2 || !s2 || !y || !workspace) return FP8BS_ERR_ARG;
    if (!aligned(x, 16) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(w13, 16) || !aligned(s13, 4) ||
        !aligned(w2, 16) || !aligned(s2, 4) || !aligned(y, 8) || !aligned(workspace, 256))
        return FP8BS_ERR_ALIGN;
    if (workspace_bytes < moe_workspace_bytes(M, S, H, I)) return FP8BS_ERR_WORKSPACE;
    int sm = 0;
    const int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    MoeArgs a;
    a.x = x;
    a.ids = topk_ids;
    a.tw = topk_w;
    a.w13 = w13;
    a.s13 = s13;
    a.w2 = w2;
    a.s2 = s2;
    a.y = y;
    a.workspace = static_cast<uint8_t*>(workspace);
    a.M = static_cast<int>(M);
    a.S = static_cast<int>(S);
    a.H = static_cast<int>(H);
    a.I = static_cast<int>(I);
    a.E = static_cast<int>(E);
    a.sm_count = sm;
    return status_of(launch_moe(a, as_stream(stream)));
}
int fp8bs_quant_weight(const float* w, int64_t N, int64_t K, int64_t ldw, int scale_kind, uint8_t* wq,
                       void* ws, void* stream) {
    if (!kind_ok(scale_kind)) return FP8BS_ERR_ARG;
    if (!nk_ok(N, K)) return FP8BS_ERR_SHAPE;
    if (!w || !wq || !ws) return FP8BS_ERR_ARG;
    if (ldw < K) return FP8BS_ERR_ARG;
    if (!aligned(w, 16) || ldw % 4 != 0 || !aligned(wq, 16) ||
        (scale_kind == FP8BS_SCALE_F32 && !aligned(ws, 4)))
        return FP8BS_ERR_ALIGN;
    return status_of(launch_quant_weight(w, N, K, ldw, scale_kind, wq, ws, as_stream(stream)));
}

int fp8bs_quant_weight_w4(const float* w, int64_t N, int64_t K, int64_t ldw, int format, int group, uint8_t* codes,
                          void* scales, void* stream) {
    if (!w4_ok(format, group)) return FP8BS_ERR_ARG;
    if (N < 1 || N > kMaxDim || K < kTile || K % kTile != 0 || K > kMaxDim) return FP8BS_ERR_SHAPE;
    if (!w || !codes || !scales) return FP8BS_ERR_ARG;
    if (ldw < K) return FP8BS_ERR_ARG;
    if (!aligned(w, 16) || ldw % 4 != 0 || !aligned(codes, 4) || !aligned(scales, w4_scale_size(format)))
        return FP8BS_ERR_ALIGN;
    int sm = 0;
    const int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    return status_of(launch_quant_weight_w4(w, N, K, ldw, format, group, codes, scales, sm, as_stream(stream)));
}

int fp8bs_gemv_w4a16(const uint16_t* x, int64_t M, int64_t ldx, const uint8_t* codes, int64_t ldc, const void* scales,
                     int64_t lds, int64_t N, int64_t K, int format, int group, uint16_t* y, int64_t ldy,
                     unsigned flags, void* stream) {
    if (!w4_ok(format, group) || (flags & ~static_cast<unsigned>(FP8BS_FLAG_PDL)) != 0) return FP8BS_ERR_ARG;
    if (M < 0 || M > FP8BS_W4_MAX_M || N < 1 || N > kMaxDim || K < kTile || K % kTile != 0 || K > kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !codes || !scales || !y) return FP8BS_ERR_ARG;
    if (ldx < K || ldc < K / 2 || ldc > FP8BS_W4_MAX_LDC || lds < K / group || ldy < N) return FP8BS_ERR_ARG;
    const int64_t size = w4_scale_size(format), chunk = size * (kTile / group);
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(codes, 16) || ldc % 16 != 0 || !aligned(scales, chunk) ||
        lds * size % chunk != 0 || !aligned(y, 2))
        return FP8BS_ERR_ALIGN;
    int sm = 0;
    const int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    GemvW4Args a;
    a.x = x;
    a.ldx = ldx;
    a.codes = codes;
    a.ldc = ldc;
    a.scales = static_cast<const uint8_t*>(scales);
    a.lds = lds * size;
    a.y = y;
    a.ldy = ldy;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.format = format;
    a.group = group;
    a.sm_count = sm;
    a.pdl = (flags & FP8BS_FLAG_PDL) ? 1 : 0;
    return status_of(launch_gemv_w4(a, as_stream(stream)));
}

size_t fp8bs_moe_route_workspace_bytes(int64_t M, int64_t E, int64_t H) {
    if (M < 0 || M > FP8BS_ROUTE_MAX_M || E < 1 || E > FP8BS_ROUTE_MAX_E || H < kTile || H % kTile != 0 || H > kMaxDim)
        return 0;
    return moe_route_workspace_bytes(M, E, H);
}

int fp8bs_moe_route(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* w, int64_t E, int64_t k,
                    int renorm, int shared, int32_t* topk_ids, float* topk_w, void* workspace,
                    size_t workspace_bytes, void* stream) {
    if (shared < FP8BS_ROUTE_SHARED_NONE || shared > FP8BS_ROUTE_SHARED_GATE) return FP8BS_ERR_ARG;
    if (M < 0 || M > FP8BS_ROUTE_MAX_M || E < 1 || E > FP8BS_ROUTE_MAX_E || k < 1 || k > E || k > FP8BS_ROUTE_MAX_K ||
        H < kTile || H % kTile != 0 || H > kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !w || !topk_ids || !topk_w || !workspace) return FP8BS_ERR_ARG;
    if (ldx < H) return FP8BS_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(w, 16) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
        !aligned(workspace, 256))
        return FP8BS_ERR_ALIGN;
    if (workspace_bytes < moe_route_workspace_bytes(M, E, H)) return FP8BS_ERR_WORKSPACE;
    MoeRouteArgs a;
    a.x = x;
    a.ldx = ldx;
    a.w = w;
    a.ids = topk_ids;
    a.weights = topk_w;
    a.workspace = static_cast<uint8_t*>(workspace);
    a.M = static_cast<int>(M);
    a.H = static_cast<int>(H);
    a.E = static_cast<int>(E);
    a.k = static_cast<int>(k);
    a.renorm = renorm != 0;
    a.shared = shared;
    return status_of(launch_moe_route(a, as_stream(stream)));
}

size_t fp8bs_moe_w4a16_workspace_bytes(int64_t M, int64_t S, int64_t I) {
    if (M < 0 || S < 1 || M > FP8BS_MOE_MAX_PAIRS || S > FP8BS_MOE_MAX_PAIRS || M * S > FP8BS_MOE_MAX_PAIRS ||
        I < kTile || I % kTile != 0 || I > FP8BS_MOE_W4_MAX_I)
        return 0;
    return moe_w4_workspace_bytes(M, S, I);
}

int fp8bs_moe_w4a16(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const int32_t* topk_ids, const float* topk_w,
                    int64_t S, const uint8_t* w13, const void* s13, const uint8_t* w2, const void* s2, int64_t E,
                    int64_t I, int format, int group, uint16_t* y, void* workspace, size_t workspace_bytes,
                    void* stream) {
    if (!w4_ok(format, group)) return FP8BS_ERR_ARG;
    if (fp8bs_moe_w4a16_workspace_bytes(M, S, I) == 0 || E < 1 || E > FP8BS_MOE_MAX_EXPERTS || H < kTile ||
        H % kTile != 0 || H > FP8BS_MOE_W4_MAX_H)
        return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !topk_ids || !topk_w || !w13 || !s13 || !w2 || !s2 || !y || !workspace) return FP8BS_ERR_ARG;
    if (ldx < H) return FP8BS_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(w13, 16) ||
        !aligned(s13, 8) || !aligned(w2, 16) || !aligned(s2, 8) || !aligned(y, 2) || !aligned(workspace, 256))
        return FP8BS_ERR_ALIGN;
    if (workspace_bytes < moe_w4_workspace_bytes(M, S, I)) return FP8BS_ERR_WORKSPACE;
    int sm = 0;
    const int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    MoeW4Args a;
    a.x = x;
    a.ldx = ldx;
    a.ids = topk_ids;
    a.tw = topk_w;
    a.w13 = w13;
    a.s13 = static_cast<const uint8_t*>(s13);
    a.w2 = w2;
    a.s2 = static_cast<const uint8_t*>(s2);
    a.y = y;
    a.workspace = static_cast<uint8_t*>(workspace);
    a.M = static_cast<int>(M);
    a.S = static_cast<int>(S);
    a.H = static_cast<int>(H);
    a.I = static_cast<int>(I);
    a.E = static_cast<int>(E);
    a.format = format;
    a.group = group;
    a.sm_count = sm;
    return status_of(launch_moe_w4(a, as_stream(stream)));
}

int fp8bs_rope_freqs(int rotary_dim, double theta, int scaling, double factor, double original_length,
                     double beta_fast, double beta_slow, uint64_t* freqs, float* amplitude) {
    const double pi = 3.14159265358979323846;
    if (!freqs || !std::isfinite(theta) || !(theta > 1.0) || scaling < FP8BS_ROPE_PLAIN || scaling > FP8BS_ROPE_BY_PARTS)
        return FP8BS_ERR_ARG;
    if (rotary_dim < 2 || rotary_dim > 256 || rotary_dim % 2 != 0) return FP8BS_ERR_SHAPE;
    if (scaling != FP8BS_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return FP8BS_ERR_ARG;
    double low = 0.0, span = 1.0;
    if (scaling == FP8BS_ROPE_BY_PARTS) {
        if (!(std::isfinite(original_length) && original_length > 0.0 && std::isfinite(beta_fast) && beta_slow > 0.0 &&
              beta_fast > beta_slow))
            return FP8BS_ERR_ARG;
        auto pair = [&](double turns) {
            return rotary_dim * std::log(original_length / (turns * 2.0 * pi)) / (2.0 * std::log(theta));
        };
        low = std::fmax(std::floor(pair(beta_fast)), 0.0);
        const double high = std::fmin(std::ceil(pair(beta_slow)), rotary_dim - 1.0);
        span = std::fmax(high - low, 1e-3);
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rotary_dim);
        if (scaling == FP8BS_ROPE_LINEAR) f /= factor;
        if (scaling == FP8BS_ROPE_BY_PARTS) {
            const double s = std::fmin(std::fmax((i - low) / span, 0.0), 1.0);
            f = f * (1.0 - s) + f / factor * s;
        }
        freqs[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f / (2.0 * pi), 64)));  // f <= 1: below 2^62
    }
    if (amplitude) *amplitude = scaling == FP8BS_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return FP8BS_OK;
}

int fp8bs_qk_norm_rope(const uint16_t* q, int64_t ldq, int64_t hsq, const uint16_t* k, int64_t ldk, int64_t hsk,
                       int64_t T, int64_t Hq, int64_t Hk, int64_t D, const int64_t* positions,
                       const uint64_t* freqs, int R, int layout, float amplitude, const uint16_t* gamma_q,
                       const uint16_t* gamma_k, float eps, uint16_t* q_out, int64_t ldqo, int64_t hsqo,
                       uint16_t* k_out, int64_t ldko, int64_t hsko, void* stream) {
    if (Hq < 0 || Hq > kMaxHeads || Hk < 0 || Hk > kMaxHeads || !head_dim_ok(D)) return FP8BS_ERR_SHAPE;
    RopeArgs a = {};
    a.q = q, a.ldq = ldq, a.hsq = hsq, a.k = k, a.ldk = ldk, a.hsk = hsk;
    a.T = T, a.Hq = static_cast<int>(Hq), a.Hk = static_cast<int>(Hk), a.D = static_cast<int>(D);
    a.positions = positions, a.freqs = freqs, a.R = R, a.layout = layout, a.amplitude = amplitude;
    a.gq = gamma_q, a.gk = gamma_k, a.eps = eps;
    a.qo = q_out, a.ldqo = ldqo, a.hsqo = hsqo, a.ko = k_out, a.ldko = ldko, a.hsko = hsko;
    return run_rope(a, stream);
}

int fp8bs_qk_norm_rope_append(const uint16_t* q, int64_t ldq, int64_t hsq, const uint16_t* k, int64_t ldk,
                              int64_t hsk, const uint16_t* v, int64_t ldv, int64_t hsv, int64_t T, int64_t Hq,
                              const int64_t* positions, const int64_t* slots, const uint64_t* freqs, int R,
                              int layout, float amplitude, const uint16_t* gamma_q, const uint16_t* gamma_k,
                              float eps, uint16_t* q_out, int64_t ldqo, int64_t hsqo, const fp8bs_kv_cache* cache,
                              void* error, void* stream) {
    const int bad = cache_check(cache);
    if (bad != FP8BS_OK) return bad;
    if (Hq < 0 || Hq > kMaxHeads) return FP8BS_ERR_SHAPE;
    RopeArgs a = {};
    a.q = q, a.ldq = ldq, a.hsq = hsq, a.k = k, a.ldk = ldk, a.hsk = hsk, a.v = v, a.ldv = ldv, a.hsv = hsv;
    a.T = T, a.Hq = static_cast<int>(Hq), a.Hk = cache->kv_heads, a.D = cache->head_dim;
    a.positions = positions, a.freqs = freqs, a.R = R, a.layout = layout, a.amplitude = amplitude;
    a.gq = gamma_q, a.gk = gamma_k, a.eps = eps;
    a.qo = q_out, a.ldqo = ldqo, a.hsqo = hsqo;
    a.slots = slots, a.cache = *cache, a.err = static_cast<uint32_t*>(error), a.append = 1;
    return run_rope(a, stream);
}

size_t fp8bs_attn_paged_workspace_bytes(int64_t D, int sm_count) {
    if (!head_dim_ok(D)) return 0;
    if (sm_count <= 0 && current_sm_count(&sm_count) != FP8BS_OK) return 0;
    return sm_count > kMaxCtas ? 0 : attn_workspace_bytes(static_cast<int>(D), sm_count);
}

int fp8bs_attn_paged(const uint16_t* q, int64_t ldq, int64_t hsq, int64_t T, int64_t Hq,
                     const fp8bs_kv_cache* cache, const int32_t* block_table, int64_t table_stride, int64_t cols,
                     int64_t B, const int32_t* cu_q, const int32_t* kv_len, float scale, int64_t window,
                     uint16_t* o, int64_t ldo, int64_t hso, void* workspace, size_t workspace_bytes, void* stream) {
    const int bad = cache_check(cache);
    if (bad != FP8BS_OK) return bad;
    if (!(scale > 0.0f && scale <= 65536.0f) || window < 0) return FP8BS_ERR_ARG;
    if (T < 0 || T > kMaxDim || Hq < 1 || Hq > kMaxHeads || Hq % cache->kv_heads != 0 || B < 0 ||
        B > FP8BS_ATTN_MAX_SEQS || cols < 0 || cols > 0x7FFFFFFF || T * (Hq / cache->kv_heads) > kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (T == 0 || B == 0) return FP8BS_OK;
    if (!q || !o || !block_table || !cu_q || !kv_len || !workspace) return FP8BS_ERR_ARG;
    const int64_t D = cache->head_dim;
    if (!stride_ok(ldq) || !stride_ok(hsq) || !stride_ok(ldo) || !stride_ok(hso) || (T > 1 && ldo < D) ||
        (Hq > 1 && hso < D) || table_stride < cols || table_stride > kMaxStride)
        return FP8BS_ERR_ARG;
    if (!heads_aligned(q, ldq, hsq) || !heads_aligned(o, ldo, hso) || !aligned(block_table, 4) || !aligned(cu_q, 4) ||
        !aligned(kv_len, 4) || !aligned(workspace, 256))
        return FP8BS_ERR_ALIGN;
    int sm = 0;
    const int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    if (sm > kMaxCtas || workspace_bytes < attn_workspace_bytes(static_cast<int>(D), sm)) return FP8BS_ERR_WORKSPACE;
    const bool codes = cache->kind == FP8BS_KV_E4M3;
    const int64_t size = codes ? 1 : 2;
    AttnArgs a = {};
    a.q = q, a.ldq = ldq, a.hsq = hsq;
    a.k = static_cast<const uint8_t*>(cache->k), a.v = static_cast<const uint8_t*>(cache->v);
    a.ks = cache->k_scale, a.vs = cache->v_scale;
    a.pstride = cache->page_stride * size, a.sstride = cache->slot_stride * size, a.hstride = cache->head_stride * size;
    a.zpstride = cache->scale_page_stride, a.zsstride = cache->scale_slot_stride, a.zhstride = cache->scale_head_stride;
    a.pages = cache->pages;
    while ((1 << a.page_log2) < cache->page_size) ++a.page_log2;
    a.table = block_table, a.table_stride = table_stride, a.table_cols = static_cast<int>(cols);
    a.cu = cu_q, a.len = kv_len;
    a.B = static_cast<int>(B), a.T = static_cast<int>(T);
    a.Hk = cache->kv_heads, a.G = static_cast<int>(Hq / cache->kv_heads);
    while ((1 << a.g_shift) < a.G) ++a.g_shift;
    a.g_shift += 31;
    a.g_mul = static_cast<uint32_t>(((uint64_t(1) << a.g_shift) + a.G - 1) / a.G);
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.window = static_cast<int>(window < kAttnMaxKeys ? window : 0);
    a.o = o, a.ldo = ldo, a.hso = hso;
    a.err = static_cast<uint32_t*>(workspace);
    a.ws = static_cast<uint8_t*>(workspace) + kWsErrorBytes;
    a.timeout_cycles = timeout_cycles();
    a.D = static_cast<int>(D), a.kind = cache->kind, a.sm_count = sm;
    return status_of(launch_attn_paged(a, as_stream(stream)));
}

size_t fp8bs_packed_weight_bytes(int64_t N, int64_t K, int scale_kind) {
    if (!kind_ok(scale_kind) || !nk_ok(N, K)) return 0;
    const size_t tiles = static_cast<size_t>(N / kTile) * static_cast<size_t>(K / kTile);
    const size_t scale_bytes = tiles * (scale_kind == FP8BS_SCALE_F32 ? 4 : 1);
    return round_up(packed_scales_offset(N, K) + scale_bytes, 256);
}

int fp8bs_prepack_weight(const uint8_t* wq, int64_t ldw, const void* ws, int64_t N, int64_t K,
                         int scale_kind, void* packed, size_t packed_bytes, void* stream) {
    if (!kind_ok(scale_kind)) return FP8BS_ERR_ARG;
    if (!nk_ok(N, K)) return FP8BS_ERR_SHAPE;
    if (!wq || !ws || !packed) return FP8BS_ERR_ARG;
    if (ldw < K) return FP8BS_ERR_ARG;
    if (!aligned(wq, 16) || ldw % 16 != 0 || !aligned(packed, 256) ||
        (scale_kind == FP8BS_SCALE_F32 && !aligned(ws, 4)))
        return FP8BS_ERR_ALIGN;
    if (packed_bytes < fp8bs_packed_weight_bytes(N, K, scale_kind)) return FP8BS_ERR_WORKSPACE;
    return status_of(launch_prepack(wq, ldw, ws, N, K, scale_kind, packed, as_stream(stream)));
}

size_t fp8bs_workspace_bytes(int64_t N, int64_t K, int sm_count) {
    if (!nk_ok(N, K)) return 0;
    if (sm_count <= 0 && current_sm_count(&sm_count) != FP8BS_OK) return 0;
    if (!fused_shape_supported(N, K, sm_count)) return 0;
    return workspace_bytes_for(K, sm_count);
}

int fp8bs_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
    if (!workspace) return FP8BS_ERR_ARG;
    if (!aligned(workspace, 256)) return FP8BS_ERR_ALIGN;
    if (workspace_bytes < kWsErrorBytes) return FP8BS_ERR_WORKSPACE;
    return status_of(cudaMemsetAsync(workspace, 0, workspace_bytes, as_stream(stream)));
}

int fp8bs_gemm_fused(const uint16_t* x, int64_t M, int64_t ldx, const void* packed, size_t packed_bytes,
                     int64_t N, int64_t K, int scale_kind, uint16_t* y, int64_t ldy, void* workspace,
                     size_t workspace_bytes, uint8_t* xq_out, void* xs_out, unsigned flags, void* stream) {
    if (!kind_ok(scale_kind) || (flags & ~static_cast<unsigned>(FP8BS_FLAG_PDL)) != 0) return FP8BS_ERR_ARG;
    if (M < 0 || M > FP8BS_MAX_M || !nk_ok(N, K)) return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !packed || !y || !workspace) return FP8BS_ERR_ARG;
    if (ldx < K || ldy < N) return FP8BS_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(y, 16) || ldy % 8 != 0 || !aligned(packed, 256) ||
        !aligned(workspace, 256) || (xq_out && !aligned(xq_out, 16)) ||
        (xs_out && scale_kind == FP8BS_SCALE_F32 && !aligned(xs_out, 4)))
        return FP8BS_ERR_ALIGN;
    if (packed_bytes < fp8bs_packed_weight_bytes(N, K, scale_kind)) return FP8BS_ERR_WORKSPACE;
    int sm = 0;
    const int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    if (!fused_shape_supported(N, K, sm)) return FP8BS_ERR_SHAPE;
    if (workspace_bytes < workspace_bytes_for(K, sm)) return FP8BS_ERR_WORKSPACE;
    FusedArgs a;
    a.x = x;
    a.ldx = ldx;
    a.packed = static_cast<const uint8_t*>(packed);
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.kind = scale_kind;
    a.y = y;
    a.ldy = ldy;
    a.workspace = static_cast<uint8_t*>(workspace);
    a.xq_out = xq_out;
    a.xs_out = xs_out;
    a.sm_count = sm;
    a.timeout_cycles = timeout_cycles();
    a.pdl = (flags & FP8BS_FLAG_PDL) ? 1 : 0;
    return status_of(launch_fused_routed(a, as_stream(stream)));
}

int fp8bs_gemm_prequant(const uint8_t* xq, int64_t M, int64_t ldxq, const void* xs, const void* packed,
                        size_t packed_bytes, int64_t N, int64_t K, int scale_kind, uint16_t* y, int64_t ldy,
                        void* workspace, size_t workspace_bytes, unsigned flags, void* stream) {
    if (!kind_ok(scale_kind) || (flags & ~static_cast<unsigned>(FP8BS_FLAG_PDL)) != 0) return FP8BS_ERR_ARG;
    if (M < 0 || M > FP8BS_MAX_M || !nk_ok(N, K)) return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!xq || !xs || !packed || !y || !workspace) return FP8BS_ERR_ARG;
    if (ldxq < K || ldy < N) return FP8BS_ERR_ARG;
    if (!aligned(xq, 16) || ldxq % 16 != 0 || !aligned(y, 16) || ldy % 8 != 0 || !aligned(packed, 256) ||
        !aligned(workspace, 256) || (scale_kind == FP8BS_SCALE_F32 && !aligned(xs, 4)))
        return FP8BS_ERR_ALIGN;
    if (packed_bytes < fp8bs_packed_weight_bytes(N, K, scale_kind)) return FP8BS_ERR_WORKSPACE;
    int sm = 0;
    const int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    if (!fused_shape_supported(N, K, sm)) return FP8BS_ERR_SHAPE;
    if (workspace_bytes < workspace_bytes_for(K, sm)) return FP8BS_ERR_WORKSPACE;
    FusedArgs a;
    a.x = nullptr;
    a.ldx = 0;
    a.packed = static_cast<const uint8_t*>(packed);
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.kind = scale_kind;
    a.y = y;
    a.ldy = ldy;
    a.workspace = static_cast<uint8_t*>(workspace);
    a.xq_out = nullptr;
    a.xs_out = nullptr;
    a.sm_count = sm;
    a.timeout_cycles = timeout_cycles();
    a.pdl = (flags & FP8BS_FLAG_PDL) ? 1 : 0;
    a.xq_in = xq;
    a.ldxq = ldxq;
    a.xs_in = xs;
    return status_of(launch_fused(a, as_stream(stream)));
}

int fp8bs_gemm_fused_static(const uint16_t* x, int64_t M, int64_t ldx, const void* packed,
                            size_t packed_bytes, int64_t N, int64_t K, int scale_kind, uint16_t* y,
                            int64_t ldy, uint8_t* xq_out, void* xs_out, uint32_t* status_out,
                            unsigned flags, void* stream) {
    if (!kind_ok(scale_kind) || (flags & ~static_cast<unsigned>(FP8BS_FLAG_PDL)) != 0) return FP8BS_ERR_ARG;
    if (M < 0 || M > FP8BS_MAX_M || !nk_ok(N, K)) return FP8BS_ERR_SHAPE;
    if (M == 0) return FP8BS_OK;
    if (!x || !packed || !y) return FP8BS_ERR_ARG;
    if (ldx < K || ldy < N) return FP8BS_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(y, 16) || ldy % 8 != 0 || !aligned(packed, 256) ||
        (xq_out && !aligned(xq_out, 16)) || (xs_out && scale_kind == FP8BS_SCALE_F32 && !aligned(xs_out, 4)) ||
        (status_out && !aligned(status_out, 4)))
        return FP8BS_ERR_ALIGN;
    if (packed_bytes < fp8bs_packed_weight_bytes(N, K, scale_kind)) return FP8BS_ERR_WORKSPACE;
    if (K > FP8BS_STATIC_MAX_K) return FP8BS_ERR_WORKSPACE;
    int sm = 0;
    int rc = current_sm_count(&sm);
    if (rc != FP8BS_OK) return rc;
    if (sm > FP8BS_STATIC_MAX_SMS) sm = FP8BS_STATIC_MAX_SMS;
    if (!fused_shape_supported(N, K, sm)) return FP8BS_ERR_SHAPE;
    if (workspace_bytes_for(K, sm) > kStaticScratchBytes) return FP8BS_ERR_WORKSPACE;
    uint8_t* scratch = nullptr;
    rc = static_scratch(as_stream(stream), &scratch);
    if (rc != FP8BS_OK) return rc;
    FusedArgs a;
    a.x = x;
    a.ldx = ldx;
    a.packed = static_cast<const uint8_t*>(packed);
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.kind = scale_kind;
    a.y = y;
    a.ldy = ldy;
    a.workspace = scratch;
    a.xq_out = xq_out;
    a.xs_out = xs_out;
    a.sm_count = sm;
    a.timeout_cycles = timeout_cycles();
    a.pdl = (flags & FP8BS_FLAG_PDL) ? 1 : 0;
    rc = status_of(launch_fused_routed(a, as_stream(stream)));
    if (rc != FP8BS_OK || !status_out) return rc;
    // this call's status, then a clean error word for the next call (both in
    // stream order; a memset allocates nothing)
    if (cudaMemcpyAsync(status_out, scratch, sizeof(uint32_t), cudaMemcpyDeviceToDevice, as_stream(stream)) !=
        cudaSuccess)
        return FP8BS_ERR_CUDA;
    return status_of(cudaMemsetAsync(scratch, 0, sizeof(uint32_t), as_stream(stream)));
}

int fp8bs_debug_config(long long timeout_cycles, int sm_count_override) {
    g_timeout_override.store(timeout_cycles > 0 ? timeout_cycles : 0, std::memory_order_relaxed);
    g_sm_override.store(sm_count_override > 0 ? sm_count_override : 0, std::memory_order_relaxed);
    return FP8BS_OK;
}

int fp8bs_trace_read(void* host_dst, size_t bytes) {
    static_assert(FP8BS_TRACE_CALLS == kTraceCalls && FP8BS_TRACE_CTAS == kTraceCtas &&
                      FP8BS_TRACE_POINTS == kTracePoints,
                  "fp8bs.h states the trace layout");
    if (!host_dst) return FP8BS_ERR_ARG;
    const cudaError_t e = trace_copy(host_dst, bytes);
    if (e == cudaErrorNotSupported) return FP8BS_ERR_ARG;
    return status_of(e);
}

int fp8bs_check_error(void* workspace, void* stream) {
    if (!workspace) return FP8BS_ERR_ARG;
    if (!aligned(workspace, 256)) return FP8BS_ERR_ALIGN;
    cudaStream_t s = as_stream(stream);
    uint32_t word = 0;
    if (cudaStreamSynchronize(s) != cudaSuccess) return FP8BS_ERR_CUDA;
    if (cudaMemcpy(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return FP8BS_ERR_CUDA;
    if (word != 0) {
        const uint32_t zero = 0;
        if (cudaMemcpy(workspace, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
            return FP8BS_ERR_CUDA;
        return -static_cast<int>(word);
    }
    return FP8BS_OK;
}

}  // extern "C"
