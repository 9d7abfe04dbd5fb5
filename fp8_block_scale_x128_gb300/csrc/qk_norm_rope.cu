// Norms and rotation of query and key heads, and appending keys and values to a
// paged cache, in one pass over a token's heads.
//
// A row (token, head) of D values lies in D/8 lanes of a warp, 16 bytes a lane:
// the sum of squares and the largest magnitude are butterflies over those lanes,
// and the partner of a rotated value is in the same lane (interleaved layout) or
// R/16 lanes away (half layout), one shuffle a value.  A lane keeps its columns
// from row to row, so gamma is loaded once, and a token's sines and cosines are
// computed once by the block and shared by all its heads.
//
// Angles: position * freqs[i] modulo 2^64 is the exact fraction of a turn (freqs
// in units of 2^-64 turns), so far positions cost no accuracy; its top 32 bits,
// rounded to fp32, go to sincospif.
//
// Everything is fp32 from the bf16 inputs to one rounding at the end.
#include "attn.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct RopeParams {
    const uint16_t *q, *k, *v;
    int64_t ldq, hsq, ldk, hsk, ldv, hsv;
    int Hq, Hk, rows;  // rows of a token: queries, keys, values
    const int64_t* positions;
    const uint64_t* freqs;
    int half;  // R / 2
    int interleaved;
    float amplitude, eps;
    const uint16_t *gq, *gk;
    uint16_t *qo, *ko;
    int64_t ldqo, hsqo, ldko, hsko;
    const int64_t* slots;
    uint8_t *ck, *cv, *zk, *zv;
    int64_t cps, css, chs, zps, zss, zhs;  // bytes
    int64_t cslots;
    int page_log2;
    uint32_t* err;
    int parts;  // blocks of a token
};

enum { kDense = 0, kBf16 = 1, kE4m3 = 2 };

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// A row's codes and scale byte from fp32 values in L lanes: the ue8m0 rule.  Its
// largest magnitude is compared by bits, so that infinities and NaNs are seen.
template <int L>
__device__ __forceinline__ uint2 quant_row(const float (&v)[8], uint32_t* byte) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, off));
    if (most >= 0x7F800000u) {
        *byte = 255;
        return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
    *byte = e8m0_ceil_byte(__fdiv_rn(__uint_as_float(most), 448.0f));
    const float inv = e8m0_to_float(254u - *byte);  // a power of two: products are exact
    uint2 c;
    c.x = e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16);
    c.y = e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16);
    return c;
}

template <int D, int DEST>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeParams p) {
    constexpr int L = D / 8;               // lanes of a row
    constexpr int kRows = kWarps * 32 / L;  // rows of a pass
    __shared__ float cosines[D / 2], sines[D / 2];
    const int lane = threadIdx.x & 31, l = lane & (L - 1);
    const int slot_row = threadIdx.x / L;
    const int64_t t = blockIdx.x / p.parts;
    const int part = blockIdx.x - static_cast<int>(t) * p.parts;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int first = part * kRows + slot_row;
    auto load = [&](int r) {
        const uint16_t* src = r < p.Hq                ? p.q + t * p.ldq + r * p.hsq
                              : r < p.Hq + p.Hk ? p.k + t * p.ldk + (r - p.Hq) * p.hsk
                                                : p.v + t * p.ldv + (r - p.Hq - p.Hk) * p.hsv;
        return r < p.rows ? *reinterpret_cast<const uint4*>(src + 8 * l) : make_uint4(0, 0, 0, 0);
    };
    uint4 raw = load(first);
    int64_t slot = -1;
    if (DEST != kDense) {
        slot = p.slots[t];
        if (slot >= p.cslots) {
            if (threadIdx.x == 0) record_error(p.err, FP8BS_ERR_DEVICE);
            slot = -1;
        }
    }
    for (int i = threadIdx.x; i < p.half; i += kThreads) {
        const uint64_t turn = static_cast<uint64_t>(p.positions[t]) * p.freqs[i];
        float s, c;
        sincospif(__int2float_rn(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
        sines[i] = s * p.amplitude;
        cosines[i] = c * p.amplitude;
    }
    __syncthreads();

    // the rotation of this lane's columns; untouched ones turn by nothing
    float co[8], si[8];
    const int R = 2 * p.half;
    const bool turns = 8 * l < R;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int col = 8 * l + i;
        co[i] = 1.0f;
        si[i] = 0.0f;
        if (col < R) {
            const int at = p.interleaved ? col >> 1 : (col < p.half ? col : col - p.half);
            co[i] = cosines[at];
            // y = x cos +- partner sin: minus for the first of a pair
            si[i] = (p.interleaved ? (col & 1) == 0 : col < p.half) ? -sines[at] : sines[at];
        }
    }
    const int away = p.half >> 3;  // lanes between the halves
    const int partner = 8 * l < p.half ? lane + away : lane - away;

    // a pass is kRows rows; whole warps leave together only past the last row
    for (int r0 = part * kRows; r0 < p.rows; r0 += p.parts * kRows) {
        const int r = r0 + slot_row;
        const uint4 now = raw;
        if (r0 + p.parts * kRows < p.rows) raw = load(r + p.parts * kRows);
        float v[8];
        unpack_bf16x8(now, v);
        const bool value = r >= p.Hq + p.Hk;
        const uint16_t* gamma = r < p.Hq ? p.gq : p.gk;
        const bool norm = !value && gamma != nullptr;
        if (__any_sync(0xFFFFFFFFu, norm)) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
            for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
            if (norm) {
                const float ms = ss * (1.0f / D) + p.eps;
                const float inv = ms > 0.0f ? __frsqrt_rn(ms) : (ms == 0.0f ? 0.0f : ms);
                float g[8];
                unpack_bf16x8(*reinterpret_cast<const uint4*>(gamma + 8 * l), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * g[i];
            }
        }
        if (p.half && __any_sync(0xFFFFFFFFu, !value)) {
            float w[8];
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = v[i ^ 1];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __shfl_sync(0xFFFFFFFFu, v[i], partner);
            }
            if (!value && turns) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (8 * l + i < R) v[i] = fmaf(v[i], co[i], w[i] * si[i]);
            }
        }
        if (DEST == kE4m3 && __any_sync(0xFFFFFFFFu, r >= p.Hq)) {
            uint32_t byte;
            const uint2 codes = quant_row<L>(v, &byte);
            if (r >= p.Hq && r < p.rows && slot >= 0) {
                const int64_t page = slot >> p.page_log2, at = slot & ((int64_t(1) << p.page_log2) - 1);
                const int h = r - p.Hq - (value ? p.Hk : 0);
                *reinterpret_cast<uint2*>((value ? p.cv : p.ck) + page * p.cps + at * p.css + h * p.chs + 8 * l) = codes;
                if (l == 0) (value ? p.zv : p.zk)[page * p.zps + at * p.zss + h * p.zhs] = static_cast<uint8_t>(byte);
            }
        }
        if (r < p.Hq) {
            *reinterpret_cast<uint4*>(p.qo + t * p.ldqo + r * p.hsqo + 8 * l) = pack8(v);
        } else if (r < p.rows && DEST == kDense) {
            *reinterpret_cast<uint4*>(p.ko + t * p.ldko + (r - p.Hq) * p.hsko + 8 * l) = pack8(v);
        } else if (r < p.rows && DEST == kBf16 && slot >= 0) {
            const int64_t page = slot >> p.page_log2, at = slot & ((int64_t(1) << p.page_log2) - 1);
            const int h = r - p.Hq - (value ? p.Hk : 0);
            // values are copied, whatever their bits
            *reinterpret_cast<uint4*>((value ? p.cv : p.ck) + page * p.cps + at * p.css + h * p.chs + 16 * l) =
                value ? now : pack8(v);
        }
    }
}

template <int D>
cudaError_t launch_d(const RopeParams& p0, int64_t T, int dest, int sm_count, cudaStream_t stream) {
    RopeParams p = p0;
    constexpr int kRows = kWarps * 32 / (D / 8);
    const int passes = (p.rows + kRows - 1) / kRows;
    p.parts = T * passes <= 8 * static_cast<int64_t>(sm_count) ? passes : 1;
    const int64_t grid = T * p.parts;
    auto kernel = dest == kDense ? qk_norm_rope_kernel<D, kDense>
                  : dest == kBf16 ? qk_norm_rope_kernel<D, kBf16>
                                  : qk_norm_rope_kernel<D, kE4m3>;
    return w4::launch_dependent(kernel, static_cast<int>(grid), kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream) {
    RopeParams p = {};
    p.q = a.q, p.k = a.k, p.v = a.v;
    p.ldq = a.ldq, p.hsq = a.hsq, p.ldk = a.ldk, p.hsk = a.hsk, p.ldv = a.ldv, p.hsv = a.hsv;
    p.Hq = a.Hq, p.Hk = a.Hk;
    p.rows = a.Hq + a.Hk + (a.append ? a.Hk : 0);
    p.positions = a.positions, p.freqs = a.freqs;
    p.half = a.R / 2;
    p.interleaved = a.layout == FP8BS_ROPE_INTERLEAVED;
    p.amplitude = a.amplitude, p.eps = a.eps;
    p.gq = a.gq, p.gk = a.gk;
    p.qo = a.qo, p.ko = a.ko;
    p.ldqo = a.ldqo, p.hsqo = a.hsqo, p.ldko = a.ldko, p.hsko = a.hsko;
    int dest = kDense;
    if (a.append) {
        const fp8bs_kv_cache& c = a.cache;
        const int64_t size = c.kind == FP8BS_KV_BF16 ? 2 : 1;
        dest = c.kind == FP8BS_KV_BF16 ? kBf16 : kE4m3;
        p.slots = a.slots;
        p.ck = static_cast<uint8_t*>(c.k), p.cv = static_cast<uint8_t*>(c.v);
        p.zk = c.k_scale, p.zv = c.v_scale;
        p.cps = c.page_stride * size, p.css = c.slot_stride * size, p.chs = c.head_stride * size;
        p.zps = c.scale_page_stride, p.zss = c.scale_slot_stride, p.zhs = c.scale_head_stride;
        while ((1 << p.page_log2) < c.page_size) ++p.page_log2;
        p.cslots = c.pages << p.page_log2;
        p.err = a.err;
    }
    if (a.D == 64) return launch_d<64>(p, a.T, dest, a.sm_count, stream);
    if (a.D == 128) return launch_d<128>(p, a.T, dest, a.sm_count, stream);
    return launch_d<256>(p, a.T, dest, a.sm_count, stream);
}

}  // namespace fp8bs
