// fp32 weights -> 4-bit codes and one scale per 1xG group along K.
//
// MXFP4 (e2m1 codes, e8m0 scales, G = 32): s = the smallest power of two >=
// RN32(amax / 6), so no finite weight saturates; code = the e2m1 value nearest
// to w / s, ties to even.  INT4 (codes q for q - 8, bf16 scales): s =
// bf16(RN32(amax / 7)), q = clamp(rint(RN32(w / s)), -8, 7) + 8; a group whose
// scale is 0 gets q = 8.  A group with an infinity or a NaN gets a NaN as its
// scale (the codes have none): e8m0's 255 or bf16's.
//
// Memory-bound: each lane takes 8 consecutive weights (two 16-byte loads) and
// writes one word of codes, G / 8 lanes share a group's maximum by shuffles.
// Measured at 16384x8192: 134 us to MXFP4 (4.5 TB/s, 0.67 of the measured copy
// bandwidth), 167 us to INT4; what keeps it from the rest was not looked for.
#include <algorithm>

#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

template <int FMT, int G>
__global__ void __launch_bounds__(kThreads)
    quant_weight_w4_kernel(const float* __restrict__ w, int64_t words, int K, int64_t ldw, uint32_t* __restrict__ codes,
                           void* __restrict__ scales) {
    const int per_row = K / 8;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    // words is a multiple of 16 and every lane runs the same trip count, so a
    // group's lanes are active together and the shuffles stay converged
    const int64_t trips = (words + stride - 1) / stride;
    for (int64_t i = 0; i < trips; ++i) {
        const int64_t at = first + i * stride;
        const bool valid = at < words;
        const int64_t row = valid ? at / per_row : 0;
        const int col = valid ? static_cast<int>(at - row * per_row) : 0;
        float v[8] = {};
        if (valid) {
            const float4* src = reinterpret_cast<const float4*>(w + row * ldw + static_cast<int64_t>(col) * 8);
            const float4 a = src[0], b = src[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max_or_nan(amax, fabsf(v[j]));
#pragma unroll
        for (int off = 1; off < G / 8; off <<= 1) amax = max_or_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
        const bool finite = amax <= 3.402823466e38f;
        uint32_t word = 0;
        if constexpr (FMT == FP8BS_W4_MXFP4) {
            const uint32_t byte = e8m0_ceil_byte(__fdiv_rn(amax, 6.0f));
            const float s = e8m0_to_float(byte);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t two;
                asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
                    : "=r"(two)
                    : "f"(__fdiv_rn(v[2 * j + 1], s)), "f"(__fdiv_rn(v[2 * j], s)));
                word |= two << (8 * j);
            }
            if (valid && (col & (G / 8 - 1)) == 0)
                static_cast<uint8_t*>(scales)[row * (K / G) + col / (G / 8)] = finite ? static_cast<uint8_t>(byte) : uint8_t(255);
        } else {
            const uint16_t bits = w4::to_bf16(__fdiv_rn(amax, 7.0f));
            const float s = bf16_bits_to_float(bits);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = s > 0.0f ? rintf(__fdiv_rn(v[j], s)) : 0.0f;
                word |= static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(q, -8.0f), 7.0f)) + 8) << (4 * j);
            }
            if (valid && (col & (G / 8 - 1)) == 0) static_cast<uint16_t*>(scales)[row * (K / G) + col / (G / 8)] = finite ? bits : uint16_t(0x7FC0);
        }
        if (!finite) word = FMT == FP8BS_W4_MXFP4 ? 0u : 0x88888888u;  // zeros, times a NaN
        if (valid) codes[at] = word;
    }
}

}  // namespace

cudaError_t launch_quant_weight_w4(const float* w, int64_t N, int64_t K, int64_t ldw, int format, int group,
                                   uint8_t* codes, void* scales, int sm_count, cudaStream_t stream) {
    // 16 blocks a multiprocessor, two or more waves of them (us to MXFP4 with 8, 16,
    // 32 and 64: 5120x4096 35.5, 35.5, 41.7, 60.1; 16384x8192 156, 134, 139, 140)
    const int64_t words = N * (K / 8), most = int64_t(sm_count) * 16;
    const int64_t blocks = std::min((words + kThreads - 1) / kThreads, most);
    return w4::dispatch_format(format, group, [&](auto fmt, auto gp) {
        quant_weight_w4_kernel<fmt(), 128 / gp()><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
            w, words, static_cast<int>(K), ldw, reinterpret_cast<uint32_t*>(codes), scales);
        return cudaGetLastError();
    });
}

}  // namespace fp8bs
