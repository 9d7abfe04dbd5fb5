// Shared pieces of the 4-bit-weight kernels (w4_gemv.cu, w4_moe.cu): what one
// warp does with 16 weight rows and a slice of K.
//
// Arithmetic.  A weight is code * scale with an e2m1 value or an integer
// -8..7 as code: both are exact in fp16.  A bf16 activation has 8 significant
// bits, so after an exact power-of-two scaling that brings the largest
// magnitude of a token's slice into [2^14, 2^15) every element down to 2^-31
// of it is exact in fp16 as well (smaller ones are off by at most 2^-39 of the
// largest: half of fp16's smallest step over 2^14).  Codes times activations go through the warp-level matrix
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
// 8t+7, two MMAs a group.  A row's 16 bytes of a group are a row of an 8x8
// matrix of 16-bit values to ldmatrix, which hands lane (g, t) word t of row
// g: one ldmatrix.x4 fetches two groups of 16 rows.  Codes reach shared memory
// in row-major order with a row pitch of 144 bytes (the 128 of a stage and 16
// more), conflict-free for that; activations sit at [token][k] fp16, the
// 64-byte halves of each 128 swapped for odd tokens, read as 16-byte words.
//
// What bounds it.  Measured on GB300, per multiprocessor quarter: this MMA takes
// 8 cycles, the e2m1 conversion of a pair, an integer operation and an fp16 pair
// operation 2, an fp32 FMA 1; together the MMAs and the integer pipe take about
// the sum of their cycles.  Codes at the measured copy bandwidth arrive as 1088
// bytes (16 rows x 128 k with e8m0 scales) per 186 cycles; decoding, multiplying
// and scaling them (stage_mma alone, 4 warps a quarter) takes 116 to 135 cycles
// with one tile of token columns, 220 with two, 150 for integer codes.  What a
// stage needs besides -- addresses, copies, scale tables, sums -- comes on top.
// The kernels are bound by latency in that chain, not by memory and by no pipe:
// with 4 warps a scheduler (128 registers) 0.4 to 0.5 instructions issue a cycle,
// and a warp waits 1.3 to 1.9 issues on the instruction before, 0.6 to 2.2 on
// global and 0.7 to 1.1 on shared memory.  Stages are made as large as shared
// memory lets them be, for fewer instructions in the chain: two tiles a stage
// where they fit.
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
constexpr int kMaxBlockShared = 226 * 1024;  // dynamic shared memory of a block (1 KB of the 227 for static)
constexpr int kMaxSmShared = 228 * 1024;     // shared memory of a multiprocessor (1 KB of it per block reserved)

// Format constants.  GP: scale groups per chunk; SB: scale bytes per row and chunk.
template <int FMT, int GP>
struct Format {
    static constexpr int kScaleBytes = FMT == FP8BS_W4_MXFP4 ? GP : 2 * GP;
};

// A stage: kPC chunks of 16 rows, copied and multiplied together by one warp.
constexpr int kPC = 2;
constexpr int kStageK = kPC * kChunk;
constexpr int kCodePitch = kPC * 64 + 16;  // bytes of a code row
constexpr int kCodeBytes = kTileRows * kCodePitch;
constexpr int kTokenBytes = kStageK * 2;   // fp16 of a token
template <int GP>
constexpr int kScalePitch = kPC * GP;  // floats of a scale row
template <int GP>
constexpr int kTableBytes = kTileRows * kScalePitch<GP> * 4;

// Shared memory by its 32-bit address: the loops below keep every address as a
// lane constant plus a slot's offset.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float2 lds_float2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds_float(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts_float2(uint32_t a, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void sts_float(uint32_t a, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// p + a * b bytes as one wide multiply-add.
__device__ __forceinline__ const uint8_t* at(const uint8_t* p, uint32_t a, uint32_t b) {
    return p + static_cast<uint64_t>(a) * b;
}

// Start the copy of a stage: nch (1..kPC) chunks of 16 code rows.  src points
// at this lane's first 16 bytes: row lane / 8 of the tile, byte 16 (lane % 8)
// of the stage, dst at their place (code_dst); it takes the rows 4, 8 and 12
// further on as well.  last: the tile's last row; rows past it repeat it (their
// outputs are dropped), so every access stays inside the weight.
__device__ __forceinline__ uint32_t code_dst(int lane) { return (lane >> 3) * kCodePitch + (lane & 7) * 16; }
__device__ __forceinline__ void load_codes(uint32_t dst, const uint8_t* src, uint32_t ldc, int last, int nch, int lane) {
    if ((lane & 7) >= nch * 4) return;
    if (last == kTileRows - 1) {
        cp_async16(dst, src);
        cp_async16(dst + 4 * kCodePitch, at(src, ldc, 4));
        cp_async16(dst + 8 * kCodePitch, at(src, ldc, 8));
        cp_async16(dst + 12 * kCodePitch, at(src, ldc, 12));
    } else {
#pragma unroll
        for (int j = 0; j < kTileRows / 4; ++j) {
            const int r = (lane >> 3) + 4 * j;
            cp_async16(dst + 4 * j * kCodePitch, src + static_cast<int64_t>(min(r, last) - (lane >> 3)) * ldc);
        }
    }
}

// The stage's scale words as loaded: lane l holds row l / 2, chunk l % 2; zeros
// past nch.  src points at the lane's own scales (row min(l / 2, last)).
template <int FMT, int GP>
__device__ __forceinline__ uint2 load_scales(const uint8_t* src, int nch, int lane) {
    constexpr int SB = Format<FMT, GP>::kScaleBytes;
    uint2 w = make_uint2(0, 0);
    if ((lane & 1) < nch) {
        if constexpr (SB == 8)
            w = __ldg(reinterpret_cast<const uint2*>(src));
        else if constexpr (SB == 4)
            w.x = __ldg(reinterpret_cast<const uint32_t*>(src));
        else
            w.x = __ldg(reinterpret_cast<const uint16_t*>(src));
    }
    return w;
}

// Their fp32 values into the stage's table [row][chunk * GP + group].  Returns
// whether one of the stage's scales is 2^97 or more: a group's sum, up to 2^27
// at the activations' fixed scaling, times such a scale may leave fp32's range
// where the result does not, and the stage is multiplied by stage_far.
template <int FMT>
__device__ __forceinline__ bool far_scale(uint2 raw) {  // some scale's three top exponent bits all set
    const uint32_t high = (raw.x & raw.x << 1 & raw.x << 2) | (raw.y & raw.y << 1 & raw.y << 2);
    return (high & (FMT == FP8BS_W4_MXFP4 ? 0x80808080u : 0x40004000u)) != 0;
}
template <int FMT, int GP>
__device__ __forceinline__ void store_scales_of(uint32_t dst, uint2 raw) {
    uint32_t w[2] = {raw.x, raw.y};
    if constexpr (FMT == FP8BS_W4_MXFP4)  // four e8m0 bytes to four bf16
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\tcvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
            : "=r"(w[0]), "=r"(w[1])
            : "r"(raw.x));
    float v[GP];
#pragma unroll
    for (int i = 0; i < GP; ++i) v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    if constexpr (GP == 4)
        sts128(dst, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    else if constexpr (GP == 2)
        sts_float2(dst, v[0], v[1]);
    else
        sts_float(dst, v[0]);
}
// dst: this lane's place in the table (scale_dst).
template <int GP>
__device__ __forceinline__ uint32_t scale_dst(int lane) {
    return ((lane >> 1) * kScalePitch<GP> + (lane & 1) * GP) * 4;
}
template <int FMT, int GP, int T>
__device__ __forceinline__ bool store_scales(uint32_t dst, const uint2 (&raw)[T]) {
    bool far = far_scale<FMT>(raw[0]);
    if constexpr (T == 2) far |= far_scale<FMT>(raw[1]);
#pragma unroll
    for (int i = 0; i < T; ++i) store_scales_of<FMT, GP>(dst + i * kTableBytes<GP>, raw[i]);
    return __any_sync(0xFFFFFFFFu, far);
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

// What that rounding leaves of them, as fp16 in the same order.
__device__ __forceinline__ uint32_t pack_rest2(float lo, float hi, uint32_t rounded) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&rounded));
    return pack_half2(lo - f.x, hi - f.y);
}
template <int FMT>
__device__ __forceinline__ uint4 pack_rest8(const float (&v)[8], float s, const uint4& r) {
    if constexpr (FMT == FP8BS_W4_MXFP4)
        return make_uint4(pack_rest2(v[0] * s, v[1] * s, r.x), pack_rest2(v[2] * s, v[3] * s, r.y),
                          pack_rest2(v[4] * s, v[5] * s, r.z), pack_rest2(v[6] * s, v[7] * s, r.w));
    else
        return make_uint4(pack_rest2(v[0] * s, v[4] * s, r.x), pack_rest2(v[1] * s, v[5] * s, r.y),
                          pack_rest2(v[2] * s, v[6] * s, r.z), pack_rest2(v[3] * s, v[7] * s, r.w));
}

__device__ __forceinline__ void unpack8(const uint4& raw, float (&v)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Where the 16-byte word w (8 k) of a token's stage sits.
__device__ __forceinline__ uint32_t token_word(int token, int w) { return token * kTokenBytes + (w ^ (token & 1) << 2) * 16; }

// A stage of up to four bf16 tokens, as loaded: lane l holds k = 8l .. 8l+7
// (zeros past nch chunks).  src(i): token i's first element of the stage.
struct RawBf16 {
    static constexpr int kTokens = 4;
    uint4 r[kTokens];
    template <typename Src>
    __device__ __forceinline__ void load(int n, int nch, int lane, Src src) {
        const bool in = lane < nch * (kChunk / 8);
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            if (i >= n) break;
            r[i] = make_uint4(0, 0, 0, 0);
            if (in) r[i] = *reinterpret_cast<const uint4*>(src(i) + 8 * lane);
        }
    }
    __device__ __forceinline__ uint32_t exponent(int i) const {
        const uint32_t m = __vmaxu2(__vmaxu2(r[i].x & 0x7FFF7FFFu, r[i].y & 0x7FFF7FFFu),
                                    __vmaxu2(r[i].z & 0x7FFF7FFFu, r[i].w & 0x7FFF7FFFu));
        return __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16)) >> 7;
    }
    __device__ __forceinline__ void values(int i, float (&v)[8]) const { unpack8(r[i], v); }
};

// Where value k of a kept fp32 token sits: a chunk's 8l + 4h + i at 64h + 4l + i,
// so that each of a lane's two 16-byte loads is next to its neighbours'.
__device__ __forceinline__ int kept_place(int k) { return (k & ~127) | (k & 4) << 4 | (k & 0x78) >> 1 | (k & 3); }
__device__ __forceinline__ uint32_t kept_src(int lane) { return (lane >> 4) * (kChunk * 4) + (lane & 15) * 16; }

// A stage of up to two fp32 tokens.  A token takes two columns of the matrix
// product, 2i and 2i + 1: fp16(v s) and fp16 of what that leaves, with one
// power of two s as for bf16 tokens.  Their sum is off by at most 2^-22 of the
// value, or 2^-39 of the slice's largest (half of fp16's smallest step over
// 2^14) where that is more.
struct RawFp32 {
    static constexpr int kTokens = 2;
    uint4 r[kTokens][2];
    // a: this lane's values (kept_src) of pair 0's stage, la bytes a pair; pair(i): the i-th pair
    template <typename Pair>
    __device__ __forceinline__ void load(const uint8_t* a, uint32_t la, int n, int nch, int lane, Pair pair) {
        const bool in = lane < nch * (kChunk / 8);
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            if (i >= n) break;
            r[i][0] = r[i][1] = make_uint4(0, 0, 0, 0);
            if (in) {
                const uint4* p = reinterpret_cast<const uint4*>(at(a, pair(i), la));
                r[i][0] = __ldcg(p);
                r[i][1] = __ldcg(p + kChunk / 8);
            }
        }
    }
    template <int FMT>
    __device__ __forceinline__ void store(uint32_t dst, uint32_t inv, int i0, int n, int lane) const {
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            if (i0 + i >= n) break;
            const uint32_t w[8] = {r[i][0].x, r[i][0].y, r[i][0].z, r[i][0].w, r[i][1].x, r[i][1].y, r[i][1].z, r[i][1].w};
            float v[8], top = 0.0f;  // (a NaN does not reach top, but stays what it is)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __uint_as_float(w[j]);
                top = fmaxf(top, fabsf(v[j]));
            }
            const uint32_t ef = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)) >> 23;
            float inverse;
            const uint4 hi = pack_slice8<FMT>(v, slice_scale(ef, inverse));
            // infinities and NaN are whole in the first column
            uint4 lo = make_uint4(0, 0, 0, 0);
            if (ef < 255) lo = pack_rest8<FMT>(v, slice_scale(ef, inverse), hi);
            sts128(dst + token_word(2 * (i0 + i), lane), hi);
            sts128(dst + token_word(2 * (i0 + i) + 1, lane), lo);
            if (lane == 0) sts_float2(inv + 8 * (i0 + i), inverse, inverse);
        }
    }
};

// The stage of n tokens as fp16 at dst, with the inverse scales in inv.  raw
// holds the first tokens, loaded beforehand; the others are loaded here.  The
// whole warp takes part and must synchronise before it reads.
template <int FMT, typename Src>
__device__ __forceinline__ void stage_tokens(uint32_t dst, uint32_t inv, RawBf16& raw, int n, int nch, int lane, Src src) {
    for (int i0 = 0; i0 < n; i0 += RawBf16::kTokens) {
        if (i0 > 0) raw.load(n - i0, nch, lane, [&](int i) { return src(i0 + i); });
#pragma unroll
        for (int i = 0; i < RawBf16::kTokens; ++i) {
            if (i0 + i >= n) break;
            float inverse, v[8];
            const float s = slice_scale(raw.exponent(i), inverse);
            raw.values(i, v);
            sts128(dst + token_word(i0 + i, lane), pack_slice8<FMT>(v, s));
            if (lane == 0) sts_float(inv + 4 * (i0 + i), inverse);
        }
    }
}

// (a & b) | c as one instruction (written out: a compiler that sees both
// constants makes two of it).
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// One word (8 codes) -> four fp16 pairs, exact.  e2m1: the hardware conversion.
// Integers by an offset in the exponent, a published method (Y. J. Kim, R. Henry,
// R. Fahim, H. H. Awadalla, "Who Says Elephants Can't Run", 2022): a nibble q in
// the low mantissa bits under the exponent of 1024 is 1024 + q (16 q one nibble
// up), so one subtraction, or one multiply-add by 1/16, leaves q - 8.
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
        const uint32_t p[4] = {and_or(w, 0x000F000Fu, 0x64006400u), and_or(w, 0x00F000F0u, 0x64006400u),
                               and_or(u, 0x000F000Fu, 0x64006400u), and_or(u, 0x00F000F0u, 0x64006400u)};
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

// d = a b
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// tot[i][j] += the stage's products of tile i and token columns 8j .. 8j+7, as D
// fragments (rows g, g + 8; columns 2t, 2t + 1).  Tile i's codes and scale
// table follow tile i - 1's.  inv holds 8 NT factors; columns past n repeat
// token n - 1 and take whatever factor is there, they are never read.
//
// All addresses are a lane's: codes at code_src, table at scale_src, inv at
// inv_src, x[j] at token_src of column 8j + g.
__device__ __forceinline__ uint32_t code_src(int lane) {  // ldmatrix: lanes 0-15 rows 0-15 of an even group, 16-31 of the odd one
    return (lane & 15) * kCodePitch + (lane >> 4) * 16;
}
template <int GP>
__device__ __forceinline__ uint32_t scale_src(int lane) {
    return (lane >> 2) * kScalePitch<GP> * 4;
}
__device__ __forceinline__ uint32_t inv_src(int lane) { return (lane & 3) * 8; }
// Relative to a 128-byte aligned stage of n tokens; bit 6 says which half of
// each 128 bytes the even groups are in.
__device__ __forceinline__ uint32_t token_src(int column, int n, int lane) {
    const int tok = min(column, n - 1);
    return tok * kTokenBytes + (tok & 1) * 64 + (lane & 3) * 16;
}
template <int FMT, int GP, int NT, int T>
__device__ __forceinline__ void stage_mma(float (&tot)[T][NT][4], uint32_t codes, uint32_t table, const uint32_t (&x)[NT],
                                          uint32_t inv, int nch) {
    float acc[T][NT][4];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        float sa[T][GP], sb[T][GP];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const uint32_t p = table + i * kTableBytes<GP> + c * GP * 4;
            if constexpr (GP == 4) {
                const uint4 u = lds128(p), v = lds128(p + 8 * kScalePitch<GP> * 4);
                sa[i][0] = __uint_as_float(u.x), sa[i][1] = __uint_as_float(u.y), sa[i][2] = __uint_as_float(u.z), sa[i][3] = __uint_as_float(u.w);
                sb[i][0] = __uint_as_float(v.x), sb[i][1] = __uint_as_float(v.y), sb[i][2] = __uint_as_float(v.z), sb[i][3] = __uint_as_float(v.w);
            } else {
#pragma unroll
                for (int q = 0; q < GP; ++q) sa[i][q] = lds_float(p + 4 * q), sb[i][q] = lds_float(p + 8 * kScalePitch<GP> * 4 + 4 * q);
            }
        }
        constexpr int kPerScale = 4 / GP;  // 32-wide groups under one scale
        float part[T][NT][4];
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
            uint32_t w[T][4];  // group 2 i2: rows g, g + 8; group 2 i2 + 1: the same
#pragma unroll
            for (int i = 0; i < T; ++i) ldmatrix4(w[i], codes + i * kCodeBytes + c * 64 + i2 * 32);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int grp = 2 * i2 + h;
                uint4 b[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) b[j] = lds128((h ? x[j] ^ 64 : x[j]) + c * 256 + i2 * 128);
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    uint32_t lo[4], hi[4];
                    decode8<FMT>(w[i][2 * h], lo);
                    decode8<FMT>(w[i][2 * h + 1], hi);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (grp % kPerScale == 0)
                            mma16816_zero(part[i][j], lo[0], hi[0], lo[1], hi[1], b[j].x, b[j].y);
                        else
                            mma16816(part[i][j], lo[0], hi[0], lo[1], hi[1], b[j].x, b[j].y);
                        mma16816(part[i][j], lo[2], hi[2], lo[3], hi[3], b[j].z, b[j].w);
                    }
                    if (grp % kPerScale == kPerScale - 1) {
                        const int q = grp / kPerScale;
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            acc[i][j][0] = fmaf(part[i][j][0], sa[i][q], acc[i][j][0]);
                            acc[i][j][1] = fmaf(part[i][j][1], sa[i][q], acc[i][j][1]);
                            acc[i][j][2] = fmaf(part[i][j][2], sb[i][q], acc[i][j][2]);
                            acc[i][j][3] = fmaf(part[i][j][3], sb[i][q], acc[i][j][3]);
                        }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const float2 f = lds_float2(inv + 32 * j);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            tot[i][j][0] = fmaf(acc[i][j][0], f.x, tot[i][j][0]);
            tot[i][j][1] = fmaf(acc[i][j][1], f.y, tot[i][j][1]);
            tot[i][j][2] = fmaf(acc[i][j][2], f.x, tot[i][j][2]);
            tot[i][j][3] = fmaf(acc[i][j][3], f.y, tot[i][j][3]);
        }
    }
}

// The same for one tile of a stage that has scales of 2^97 and more, whose
// groups are summed apart at 2^-64 of their size: no other group of the stage,
// in its row or another, loses range to them.  Never seen in quantised weights,
// so it is kept out of the kernels' own code.
template <int NT>
struct FarTile {
    uint32_t x[NT];
    float sum[NT][4];
};
constexpr float kFarScale = 0x1p64f;
template <int FMT, int GP, int NT>
__device__ __noinline__ void stage_far(FarTile<NT>* tile, uint32_t codes, uint32_t table, uint32_t inv, int nch) {
    float near[NT][4] = {}, far[NT][4] = {}, part[NT][4] = {};
#pragma unroll 1
    for (int i2 = 0; i2 < 2 * nch; ++i2) {
        uint32_t w[4];
        ldmatrix4(w, codes + i2 * 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            constexpr int kPerScale = 4 / GP;
            const int grp = 2 * i2 + h;
            uint32_t lo[4], hi[4];
            decode8<FMT>(w[2 * h], lo);
            decode8<FMT>(w[2 * h + 1], hi);
            const bool ends = grp % kPerScale == kPerScale - 1;
            const uint32_t p = table + grp / kPerScale * 4;
            const float scale[2] = {lds_float(p), lds_float(p + 8 * kScalePitch<GP> * 4)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint4 b = lds128((h ? tile->x[j] ^ 64 : tile->x[j]) + i2 * 128);
                mma16816(part[j], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                mma16816(part[j], lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                if (!ends) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float s = scale[q / 2];
                    if ((__float_as_uint(s) & 0x7F800000u) >= 224u << 23)
                        far[j][q] = fmaf(part[j][q], s * (1.0f / kFarScale), far[j][q]);
                    else
                        near[j][q] = fmaf(part[j][q], s, near[j][q]);
                    part[j][q] = 0.0f;
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const float2 f = lds_float2(inv + 32 * j);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float e = q % 2 ? f.y : f.x;
            tile->sum[j][q] = fmaf(far[j][q] * e, kFarScale, near[j][q] * e);
        }
    }
}

// A stage by one or the other.
template <int FMT, int GP, int NT, int T>
__device__ __forceinline__ void multiply_stage(float (&tot)[T][NT][4], uint32_t codes, uint32_t table, const uint32_t (&x)[NT],
                                               uint32_t inv, bool far, int nch) {
    if (!far) {
        stage_mma<FMT, GP, NT, T>(tot, codes, table, x, inv, nch);
        return;
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
        FarTile<NT> tile;
#pragma unroll
        for (int j = 0; j < NT; ++j) tile.x[j] = x[j];
        stage_far<FMT, GP, NT>(&tile, codes + i * kCodeBytes, table + i * kTableBytes<GP>, inv, nch);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) tot[i][j][q] += tile.sum[j][q];
    }
}

// D fragments of a warp as [column][kSumPitch], conflict-free to write and read.
constexpr int kSumPitch = kTileRows + 4;  // floats
template <int NT>
constexpr int kSumBytes = 8 * NT * kSumPitch * 4;  // of a tile
template <int NT>
__device__ __forceinline__ void store_sums(uint32_t dst, const float (&tot)[NT][4], int lane) {
    const uint32_t r = dst + (2 * (lane & 3) * kSumPitch + (lane >> 2)) * 4;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        sts_float(r + 8 * j * kSumPitch * 4, tot[j][0]);
        sts_float(r + (8 * j + 1) * kSumPitch * 4, tot[j][1]);
        sts_float(r + (8 * j * kSumPitch + 8) * 4, tot[j][2]);
        sts_float(r + ((8 * j + 1) * kSumPitch + 8) * 4, tot[j][3]);
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

// Every kernel of these files is launched with programmatic dependent launch:
// it waits for its predecessor (griddep_wait) before it touches memory -- but
// for weights that the caller says no unfinished work writes -- and lets
// its successor start (launch_dependents) only after that wait, so that what a
// successor reads before its own wait is complete up to the kernel before it.
// Back-to-back calls overlap one call's start-up with the other's tail.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), int grid, int block, int smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace w4

// Launchers (argument checks are done by the C ABI before these run).

cudaError_t launch_quant_weight_w4(const float* w, int64_t N, int64_t K, int64_t ldw, int format, int group,
                                   uint8_t* codes, void* scales, int sm_count, cudaStream_t stream);

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
