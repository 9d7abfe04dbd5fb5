// Shared pieces of the 4-bit-weight kernels (w4_gemv.cu, w4_moe.cu): what one
// warp does with 16 weight rows and a slice of K.
//
// Arithmetic.  A weight is code * scale with an e2m1 value or an integer
// -8..7 as code: both are exact in fp16.  A bf16 activation has 8 significant
// bits, so after an exact power-of-two scaling that brings the largest
// magnitude of a token's slice into [2^14, 2^15) every element down to 2^-32
// of it is exact in fp16 as well (smaller ones are rounded at 2^-40 of the
// largest).  Codes times activations go through the warp-level matrix
// instruction (fp16 in, fp32 sums): products are exact, one scale group is
// summed at a time, and the group's sum times its scale is added in fp32.
// The matrix instruction is used for its decode rate: at a few tokens the
// products are bound by the bytes of the codes, and an MMA of 16 rows x 8
// token columns costs one issue slot for 256 weights where scalar products
// would cost 8 a token.
//
// Layout.  For the m16n8k16 fragments lane (g, t) = (lane / 4, lane % 4)
// holds rows g and g + 8 of the weight and token column g.  The k order
// within an MMA is free as long as both operands agree, so a lane takes one
// 32-bit word (8 codes) per 32-wide group: word t of the group is k = 8t ..
// 8t+7, two MMAs a group.  Codes reach shared memory in row-major order with
// a row pitch of 16 bytes more than the slice, which makes these word reads
// conflict-free; activations sit at [token][k] fp16, read as 16-byte words.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "fp8bs.h"
#include "ptx.cuh"

namespace fp8bs {
namespace w4 {

constexpr int kChunk = 128;    // k per chunk: the unit of slices
constexpr int kTileRows = 16;  // weight rows of a warp tile
constexpr int kMaxBlockShared = 227 * 1024;  // dynamic shared memory a block may have
constexpr int kMaxSmShared = 228 * 1024;     // shared memory of a multiprocessor (1 KB of it per block reserved)

// Format constants.  GP: scale groups per chunk; SB: scale bytes per row and chunk.
template <int FMT, int GP>
struct Format {
    static constexpr int kScaleBytes = FMT == FP8BS_W4_MXFP4 ? GP : 2 * GP;
};

// Shared memory of one warp's stage: PC chunks of 16 rows.
template <int GP, int PC>
struct Stage {
    static constexpr int kPitch = PC * 64 + 16;                // bytes of a code row
    static constexpr int kCodeBytes = kTileRows * kPitch;
    static constexpr int kScalePitch = PC * GP + 4;            // floats of a scale row
    static constexpr int kScaleTableBytes = kTileRows * kScalePitch * 4;
    static constexpr int kTokenPitch = PC * 256 + 64;          // bytes of a token's slice
};

// Scale words of a stage as loaded: lane l holds row l / 2, PC / 2 chunks from
// (l % 2) * PC / 2 on (PC = 1: row l % 16 by the first 16 lanes).
template <int PC>
struct RawScales {
    uint2 w[PC > 1 ? PC / 2 : 1];
};

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool pred) {
    const uint32_t n = pred ? 16u : 0u;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_addr(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Start the copy of nch (1..PC) chunks of 16 code rows to dst.  codes points
// at row 0's first byte of the slice; row r >= rows repeats the last row (its
// outputs are dropped), so every access stays inside the weight.
template <int GP, int PC>
__device__ __forceinline__ void load_codes(uint8_t* dst, const uint8_t* codes, int64_t ldc, int rows, int nch, int lane) {
    constexpr int kSegs = PC * 4;  // 16-byte pieces of a row
#pragma unroll
    for (int j = 0; j < kTileRows * kSegs / 32; ++j) {
        const int idx = lane + 32 * j, r = idx / kSegs, s = idx % kSegs;
        if (s < nch * 4)
            ptx::cp_async16(dst + r * Stage<GP, PC>::kPitch + s * 16, codes + static_cast<int64_t>(r < rows ? r : rows - 1) * ldc + s * 16);
    }
}

// The stage's scale words into registers (row pitch lds bytes); zeros past nch.
template <int FMT, int GP, int PC>
__device__ __forceinline__ RawScales<PC> load_scales(const uint8_t* scales, int64_t lds, int rows, int nch, int lane) {
    constexpr int SB = Format<FMT, GP>::kScaleBytes;
    constexpr int kPer = PC > 1 ? PC / 2 : 1;
    RawScales<PC> raw;
    const int r0 = PC > 1 ? lane >> 1 : lane & 15;
    const int r = r0 < rows ? r0 : rows - 1;
    const int c0 = PC > 1 ? (lane & 1) * kPer : 0;
    const uint8_t* p = scales + static_cast<int64_t>(r) * lds + c0 * SB;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        raw.w[j] = make_uint2(0, 0);
        if (c0 + j < nch) {
            if constexpr (SB == 8)
                raw.w[j] = __ldg(reinterpret_cast<const uint2*>(p + j * SB));
            else if constexpr (SB == 4)
                raw.w[j].x = __ldg(reinterpret_cast<const uint32_t*>(p + j * SB));
            else
                raw.w[j].x = __ldg(reinterpret_cast<const uint16_t*>(p + j * SB));
        }
    }
    return raw;
}

// Their fp32 values into the stage's table [row][chunk * GP + group].  An e8m0
// byte b is 2^(b - 127): its bits shifted into the exponent, 0 being the
// subnormal 2^-127.  A stage with a scale of 2^97 or more has its table divided
// by 2^64 (kBigScale), so that a group's sum, up to 2^27 at the activations'
// fixed scaling, times its scale stays finite; returns the factor to put back.
constexpr float kBigScale = 0x1p64f;
template <int FMT, int GP, int PC>
__device__ __forceinline__ float store_scales(float* table, const RawScales<PC>& raw, int lane) {
    constexpr int kPer = PC > 1 ? PC / 2 : 1;
    uint32_t high = 0;  // the three top exponent bits of some scale all set
#pragma unroll
    for (int j = 0; j < kPer; ++j) high |= (raw.w[j].x & raw.w[j].x << 1 & raw.w[j].x << 2) | (raw.w[j].y & raw.w[j].y << 1 & raw.w[j].y << 2);
    const bool big = __any_sync(0xFFFFFFFFu, (high & (FMT == FP8BS_W4_MXFP4 ? 0x80808080u : 0x40004000u)) != 0);
    const float fit = big ? 1.0f / kBigScale : 1.0f, back = big ? kBigScale : 1.0f;
    const int r = PC > 1 ? lane >> 1 : lane & 15;
    const int c0 = PC > 1 ? (lane & 1) * kPer : 0;
    float* dst = table + r * Stage<GP, PC>::kScalePitch + c0 * GP;
    if (PC == 1 && lane >= 16) return back;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint32_t w[2] = {raw.w[j].x, raw.w[j].y};
        float v[GP];
#pragma unroll
        for (int i = 0; i < GP; ++i) {
            if constexpr (FMT == FP8BS_W4_MXFP4)
                v[i] = __uint_as_float(max(((w[0] >> (8 * i)) & 0xFFu) << 23, 0x00400000u));
            else
                v[i] = __uint_as_float((w[i / 2] >> (16 * (i % 2))) << 16);
            v[i] *= fit;
        }
        if constexpr (GP == 4)
            *reinterpret_cast<float4*>(dst + j * GP) = make_float4(v[0], v[1], v[2], v[3]);
        else if constexpr (GP == 2)
            *reinterpret_cast<float2*>(dst + j * GP) = make_float2(v[0], v[1]);
        else
            dst[j] = v[0];
    }
    return back;
}

// tot += a stage's sums, their token's and their scales' factors put back.
__device__ __forceinline__ void add_stage(float (&tot)[4], const float (&acc)[4], float i0, float i1, float back) {
    tot[0] += acc[0] * i0 * back;
    tot[1] += acc[1] * i1 * back;
    tot[2] += acc[2] * i0 * back;
    tot[3] += acc[3] * i1 * back;
}

// 2^(14 - e) and its inverse for a slice whose largest magnitude has the
// biased exponent ef = e + 127 (clamped so that both are normal; ef = 255,
// infinities and NaN, takes the largest finite exponent and they stay what
// they are).
__device__ __forceinline__ float slice_scale(uint32_t ef, float& inverse) {
    ef = min(max(ef, 15u), 254u);
    inverse = __uint_as_float((ef - 14u) << 23);
    return __uint_as_float((268u - ef) << 23);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Eight activations, scaled, as fp16 in the pair order the code decode yields:
// e2m1 words give the pairs (0,1)(2,3)(4,5)(6,7), integer words (0,4)(1,5)(2,6)(3,7).
template <int FMT>
__device__ __forceinline__ uint4 pack_slice8(const float (&v)[8], float s) {
    if constexpr (FMT == FP8BS_W4_MXFP4)
        return make_uint4(pack_half2(v[0] * s, v[1] * s), pack_half2(v[2] * s, v[3] * s),
                          pack_half2(v[4] * s, v[5] * s), pack_half2(v[6] * s, v[7] * s));
    else
        return make_uint4(pack_half2(v[0] * s, v[4] * s), pack_half2(v[1] * s, v[5] * s),
                          pack_half2(v[2] * s, v[6] * s), pack_half2(v[3] * s, v[7] * s));
}

__device__ __forceinline__ void unpack8(const uint4& raw, float (&v)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// One token's slice of nch chunks, bf16 from global memory, into dst (fp16,
// zeros past nch); returns the inverse scale.  The whole warp takes part.
template <int FMT, int PC>
__device__ __forceinline__ float stage_token_bf16(uint8_t* dst, const uint16_t* src, int nch, int lane) {
    constexpr int kJ = (PC + 1) / 2;  // 256 k per warp-wide 16-byte load
    uint4 raw[kJ];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        const int k = 8 * lane + 256 * j;
        if (k < nch * kChunk) raw[j] = *reinterpret_cast<const uint4*>(src + k);
        const uint32_t m = __vmaxu2(__vmaxu2(raw[j].x & 0x7FFF7FFFu, raw[j].y & 0x7FFF7FFFu),
                                    __vmaxu2(raw[j].z & 0x7FFF7FFFu, raw[j].w & 0x7FFF7FFFu));
        top = max(top, max(m & 0xFFFFu, m >> 16));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    float inverse;
    const float s = slice_scale(top >> 7, inverse);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int k = 8 * lane + 256 * j;
        float v[8];
        unpack8(raw[j], v);
        if (k < PC * kChunk) *reinterpret_cast<uint4*>(dst + 2 * k) = pack_slice8<FMT>(v, s);
    }
    return inverse;
}

// The same from fp32 (rounded to fp16's 11 bits: 2^-12 of each value, 16 times
// finer than the bf16 of the outputs).
template <int FMT, int PC>
__device__ __forceinline__ float stage_token_f32(uint8_t* dst, const float* src, int nch, int lane) {
    constexpr int kJ = (PC + 1) / 2;
    float v[kJ][8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int k = 8 * lane + 256 * j;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (k < nch * kChunk) {
            a = __ldcg(reinterpret_cast<const float4*>(src + k));
            b = __ldcg(reinterpret_cast<const float4*>(src + k + 4));
        }
        v[j][0] = a.x, v[j][1] = a.y, v[j][2] = a.z, v[j][3] = a.w;
        v[j][4] = b.x, v[j][5] = b.y, v[j][6] = b.z, v[j][7] = b.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    float inverse;
    const float s = slice_scale(top >> 23, inverse);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int k = 8 * lane + 256 * j;
        if (k < PC * kChunk) *reinterpret_cast<uint4*>(dst + 2 * k) = pack_slice8<FMT>(v[j], s);
    }
    return inverse;
}

// One word (8 codes) -> four fp16 pairs, exact.  e2m1: the hardware conversion.
// Integers: a nibble q in the low mantissa bits under the exponent of 1024 is
// 1024 + q (16 q one nibble up), so one subtraction, or one multiply-add by
// 1/16, leaves q - 8.
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&r)[4]) {
    if constexpr (FMT == FP8BS_W4_MXFP4) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
            : "r"(w));
    } else {
        const uint32_t u = w >> 8;
        const uint32_t p[4] = {(w & 0x000F000Fu) | 0x64006400u, (w & 0x00F000F0u) | 0x64006400u,
                               (u & 0x000F000Fu) | 0x64006400u, (u & 0x00F000F0u) | 0x64006400u};
        const __half2 sub = __half2half2(__ushort_as_half(0xE408));   // -1032
        const __half2 mul = __half2half2(__ushort_as_half(0x2C00));   // 1/16
        const __half2 add = __half2half2(__ushort_as_half(0xD480));   // -72
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 h = *reinterpret_cast<const __half2*>(&p[i]);
            h = (i & 1) ? __hfma2(h, mul, add) : __hadd2(h, sub);
            r[i] = *reinterpret_cast<uint32_t*>(&h);
        }
    }
}

// d (+)= a(16x16) b(16x8), fp16 in, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc[j] += the stage's product for token columns 8j .. 8j+7: D fragment
// (rows g, g + 8; columns 2t, 2t + 1), still carrying the tokens' slice
// scales.  xs: [token][kTokenPitch]; columns past n repeat token n - 1.
template <int FMT, int GP, int PC, int NT>
__device__ __forceinline__ void stage_mma(float (&acc)[NT][4], const uint8_t* codes, const float* table, const uint8_t* xs,
                                          int n, int nch, int lane) {
    using S = Stage<GP, PC>;
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* c0 = codes + g * S::kPitch + t * 4;
    const float* s0 = table + g * S::kScalePitch;
    const uint8_t* x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = xs + min(8 * j + g, n - 1) * S::kTokenPitch + t * 16;
#pragma unroll
    for (int c = 0; c < PC; ++c) {
        if (c >= nch) break;
        constexpr int kPerScale = 4 / GP;  // 32-wide groups under one scale
#pragma unroll
        for (int q = 0; q < GP; ++q) {
            float part[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) part[j][0] = part[j][1] = part[j][2] = part[j][3] = 0.0f;
#pragma unroll
            for (int i = q * kPerScale; i < (q + 1) * kPerScale; ++i) {
                uint32_t lo[4], hi[4];
                decode8<FMT>(*reinterpret_cast<const uint32_t*>(c0 + c * 64 + i * 16), lo);
                decode8<FMT>(*reinterpret_cast<const uint32_t*>(c0 + 8 * S::kPitch + c * 64 + i * 16), hi);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 b = *reinterpret_cast<const uint4*>(x[j] + c * 256 + i * 64);
                    mma16816(part[j], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                    mma16816(part[j], lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                }
            }
            const float sa = s0[c * GP + q], sb = s0[8 * S::kScalePitch + c * GP + q];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[j][0] = fmaf(part[j][0], sa, acc[j][0]);
                acc[j][1] = fmaf(part[j][1], sa, acc[j][1]);
                acc[j][2] = fmaf(part[j][2], sb, acc[j][2]);
                acc[j][3] = fmaf(part[j][3], sb, acc[j][3]);
            }
        }
    }
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
    return r;
}

// Calls launch(FMT, GP) with both as compile-time constants, for a format and
// group size the C ABI accepted.
template <int V>
using Const = std::integral_constant<int, V>;
template <typename F>
cudaError_t dispatch_format(int format, int group, F&& launch) {
    if (format == FP8BS_W4_MXFP4) return launch(Const<FP8BS_W4_MXFP4>{}, Const<4>{});
    if (group == 32) return launch(Const<FP8BS_W4_INT4>{}, Const<4>{});
    if (group == 64) return launch(Const<FP8BS_W4_INT4>{}, Const<2>{});
    return launch(Const<FP8BS_W4_INT4>{}, Const<1>{});
}

// Raises a kernel's dynamic shared memory limit to the most a block may have,
// once per kernel and device.
template <typename K>
cudaError_t allow_shared(K* kernel, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done.load(std::memory_order_relaxed) >> dev & 1) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBlockShared);
    if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

}  // namespace w4

// Launchers (argument checks are done by the C ABI before these run).

cudaError_t launch_quant_weight_w4(const float* w, int64_t N, int64_t K, int64_t ldw, int format, int group,
                                   uint8_t* codes, void* scales, cudaStream_t stream);

struct GemvW4Args {
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* codes;
    int64_t ldc;  // bytes
    const uint8_t* scales;
    int64_t lds;  // bytes
    uint16_t* y;
    int64_t ldy;
    int M, N, K;
    int format, group;
    int sm_count;
    int pdl;
};
cudaError_t launch_gemv_w4(const GemvW4Args& a, cudaStream_t stream);

struct MoeRouteArgs {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* w;
    int32_t* ids;
    float* weights;
    uint8_t* workspace;
    int M, H, E, k;
    int renorm, shared;
};
size_t moe_route_workspace_bytes(int64_t M, int64_t E, int64_t H);
cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t stream);

struct MoeW4Args {
    const uint16_t* x;
    int64_t ldx;
    const int32_t* ids;
    const float* tw;
    const uint8_t* w13;
    const uint8_t* s13;
    const uint8_t* w2;
    const uint8_t* s2;
    uint16_t* y;
    uint8_t* workspace;
    int M, S, H, I, E;
    int format, group;
    int sm_count;
};
size_t moe_w4_workspace_bytes(int64_t M, int64_t S, int64_t I);
cudaError_t launch_moe_w4(const MoeW4Args& a, cudaStream_t stream);

}  // namespace fp8bs
