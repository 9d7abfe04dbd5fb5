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
//
// It reads and writes each head once.  8192 tokens of 32 + 8 heads of 128 take 38.5 us
// (4.4 TB/s, 0.64 of a copy's rate; a block a token, without a ring of its own, 56),
// 40 + 8 + 8 into a bf16 cache 47.5 (5.0 TB/s; 67).  One token takes 2.2 us in a graph.
#include "attn.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 8;  // passes under way in a block: 16 KB

struct RopeParams {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv, ldqo, ldko;     // bytes, as all strides here
    uint32_t hsq, hsk, hsv, hsqo, hsko;
    int Hq, Hk, rows;  // rows of a token: queries, keys, values
    const int64_t* positions;
    const uint64_t* freqs;
    int half;  // R / 2
    float amplitude, eps;
    const uint16_t *gq, *gk;
    uint16_t *qo, *ko;
    const int64_t* slots;
    uint8_t *ck, *cv, *zk, *zv;
    int64_t cps, css, chs, zps, zss, zhs;  // bytes
    int64_t cslots;
    int page_log2;
    uint32_t* err;
    int parts;  // tasks of a token
    int64_t tasks;
};

enum { kDense = 0, kBf16 = 1, kE4m3 = 2 };

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

// Pairs of fp32 operations in one instruction each.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ void widen8(const uint4& w, uint64_t (&v)[4]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
}

template <int D, int DEST, bool HALF>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int L = D / 8;               // lanes of a row
    constexpr int kRows = kWarps * 32 / L;  // rows of a pass
    // what a column is multiplied by, and its partner: 1 and 0 where nothing turns
    __shared__ __align__(16) float cosines[2][D], sines[2][D];
    __shared__ __align__(16) float gammas[2][D];  // of queries and keys
    const int lane = threadIdx.x & 31, l = lane & (L - 1), slot_row = threadIdx.x / L;
    const int R = 2 * p.half;
    for (int i = threadIdx.x; i < 2 * D; i += kThreads)
        if (i % D >= R) cosines[i / D][i % D] = 1.0f, sines[i / D][i % D] = 0.0f;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    for (int i = threadIdx.x; i < D; i += kThreads) {
        if (p.gq) gammas[0][i] = bf16_bits_to_float(p.gq[i]);
        if (p.gk) gammas[1][i] = bf16_bits_to_float(p.gk[i]);
    }
    const bool turns = 8 * l < R;  // half layout: all of this lane's columns do
    const int away = p.half >> 3;  // lanes between the halves
    const int partner = 8 * l < p.half ? lane + away : lane - away;
    const int keys = p.Hq, values = p.Hq + p.Hk;  // first rows

    // A thread's own pieces, kStages - 1 passes ahead, in its own places of shared memory.
    extern __shared__ __align__(16) uint8_t ring[];
    const uint32_t mine = ptx::smem_addr(ring) + 16 * threadIdx.x;
    int64_t task = blockIdx.x;
    int64_t next_task = task;
    int next_row = 0, stage_in = 0, stage = 0;  // the pass to fetch
    const uint8_t *nq, *nk, *nv;                // its token
    auto next_token = [&] {
        const int64_t t = p.parts == 1 ? next_task : next_task / p.parts;
        nq = reinterpret_cast<const uint8_t*>(p.q) + t * p.ldq + 16 * l;
        nk = reinterpret_cast<const uint8_t*>(p.k) + t * p.ldk + 16 * l;
        nv = reinterpret_cast<const uint8_t*>(p.v) + t * p.ldv + 16 * l;
        next_row = static_cast<int>(next_task - t * p.parts) * kRows;
    };
    next_token();
    auto fetch = [&] {
        if (next_task < p.tasks) {
            const int r = next_row + slot_row;
            const uint8_t* base = r < keys ? nq : r < values ? nk : nv;
            const uint32_t hs = r < keys ? p.hsq : r < values ? p.hsk : p.hsv;
            const uint32_t h = r - (r < keys ? 0 : r < values ? keys : values);
            if (r < p.rows) cp_async16(mine + stage_in * (kThreads * 16), base + static_cast<uint64_t>(h) * hs);
            next_row += p.parts * kRows;
            if (next_row >= p.rows) {
                next_task += gridDim.x;
                if (next_task < p.tasks) next_token();
            }
            if (++stage_in == kStages) stage_in = 0;
        }
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fetch();
    int64_t position = 0, slot = -1;
    auto look = [&](int64_t t) {
        if (p.half) position = p.positions[t];
        if (DEST != kDense) slot = p.slots[t];
    };
    look(p.parts == 1 ? task : task / p.parts);
    int buffer = 0;
#pragma unroll 1
    for (; task < p.tasks; task += gridDim.x, buffer ^= 1) {
        const int64_t t = p.parts == 1 ? task : task / p.parts;
        const int part = static_cast<int>(task - t * p.parts);
        for (int i = threadIdx.x; i < p.half; i += kThreads) {
            const uint64_t turn = static_cast<uint64_t>(position) * p.freqs[i];
            float s, c;
            sincospif(__int2float_rn(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
            s *= p.amplitude, c *= p.amplitude;
            // y = x cos -+ partner sin: minus for the first of a pair
            const int first = HALF ? i : 2 * i, second = HALF ? i + p.half : 2 * i + 1;
            cosines[buffer][first] = cosines[buffer][second] = c;
            sines[buffer][first] = -s, sines[buffer][second] = s;
        }
        __syncthreads();  // (a block that is a token ahead fills the other table)
        int64_t to = -1, scale_to = -1;  // offsets of the slot in the cache
        if (DEST != kDense) {
            if (slot >= p.cslots) {
                if (threadIdx.x == 0) record_error(p.err, FP8BS_ERR_DEVICE);
            } else if (slot >= 0) {
                const int64_t page = slot >> p.page_log2, at = slot & ((int64_t(1) << p.page_log2) - 1);
                to = page * p.cps + at * p.css;
                scale_to = page * p.zps + at * p.zss;
            }
        }
        if (task + gridDim.x < p.tasks) look(p.parts == 1 ? task + gridDim.x : (task + gridDim.x) / p.parts);
        uint64_t co[4], si[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const ulonglong2 c = reinterpret_cast<const ulonglong2*>(&cosines[buffer][8 * l])[i];
            const ulonglong2 n = reinterpret_cast<const ulonglong2*>(&sines[buffer][8 * l])[i];
            co[2 * i] = c.x, co[2 * i + 1] = c.y, si[2 * i] = n.x, si[2 * i + 1] = n.y;
        }
        uint8_t* oq = reinterpret_cast<uint8_t*>(p.qo) + t * p.ldqo + 16 * l;
        uint8_t* ok = reinterpret_cast<uint8_t*>(p.ko) + t * p.ldko + 16 * l;
        uint8_t* ck = p.ck + to + (DEST == kE4m3 ? 8 : 16) * l;
        uint8_t* cv = p.cv + to + (DEST == kE4m3 ? 8 : 16) * l;
#pragma unroll 1
        for (int r0 = part * kRows; r0 < p.rows; r0 += p.parts * kRows) {
            const int r = r0 + slot_row;
            fetch();
            cp_wait<kStages - 1>();
            // (a row past the last has what was there before: nothing is made of it)
            const uint4 now = *reinterpret_cast<const uint4*>(ring + stage * (kThreads * 16) + 16 * threadIdx.x);
            if (++stage == kStages) stage = 0;
            const bool key = r >= keys && r < values, value = r >= values;
            uint64_t v[4];
            widen8(now, v);
            const bool norm = key ? p.gk != nullptr : !value && p.gq != nullptr;
            if (__any_sync(0xFFFFFFFFu, norm)) {
                uint64_t squares = mul2(v[0], v[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) squares = fma2(v[i], v[i], squares);
                const float2 s2 = halves(squares);
                float ss = s2.x + s2.y;
#pragma unroll
                for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
                if (norm) {
                    const float ms = ss * (1.0f / D) + p.eps;
                    const float inv = ms == 0.0f ? 0.0f : rsqrtf(ms);
                    const uint64_t inv2 = pair(inv, inv);
                    const ulonglong2* g = reinterpret_cast<const ulonglong2*>(&gammas[key][8 * l]);
                    const ulonglong2 g0 = g[0], g1 = g[1];
                    v[0] = mul2(mul2(v[0], inv2), g0.x), v[1] = mul2(mul2(v[1], inv2), g0.y);
                    v[2] = mul2(mul2(v[2], inv2), g1.x), v[3] = mul2(mul2(v[3], inv2), g1.y);
                }
            }
            if (p.half && __any_sync(0xFFFFFFFFu, !value)) {
                if (HALF) {
                    uint64_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = halves(v[i]);
                        w[i] = pair(__shfl_sync(0xFFFFFFFFu, x.x, partner), __shfl_sync(0xFFFFFFFFu, x.y, partner));
                    }
                    // (a column that does not turn keeps its value, whatever other columns hold)
                    if (turns && !value)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = fma2(w[i], si[i], mul2(v[i], co[i]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (8 * l + 2 * i < R && !value) {
                            const float2 x = halves(v[i]);
                            v[i] = fma2(pair(x.y, x.x), si[i], mul2(v[i], co[i]));
                        }
                }
            }
            if (DEST == kE4m3 && __any_sync(0xFFFFFFFFu, r >= keys)) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[2 * i] = halves(v[i]).x, x[2 * i + 1] = halves(v[i]).y;
                uint32_t byte;
                const uint2 codes = quant_row<L>(x, &byte);
                if (r >= keys && r < p.rows && to >= 0) {
                    const int h = r - (value ? values : keys);
                    *reinterpret_cast<uint2*>((value ? cv : ck) + h * p.chs) = codes;
                    if (l == 0) (value ? p.zv : p.zk)[scale_to + h * p.zhs] = static_cast<uint8_t>(byte);
                }
            }
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16(halves(v[i]).x, halves(v[i]).y);
            const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
            if (r < keys) {
                *reinterpret_cast<uint4*>(oq + static_cast<uint64_t>(r) * p.hsqo) = out;
            } else if (r < p.rows && DEST == kDense) {
                *reinterpret_cast<uint4*>(ok + static_cast<uint64_t>(r - keys) * p.hsko) = out;
            } else if (r < p.rows && DEST == kBf16 && to >= 0) {
                // values are copied, whatever their bits
                const int h = r - (value ? values : keys);
                *reinterpret_cast<uint4*>((value ? cv : ck) + h * p.chs) = value ? now : out;
            }
        }
    }
}

template <int D, int DEST, bool HALF>
cudaError_t launch_to(const RopeParams& p, int sm_count, cudaStream_t stream) {
    // as many blocks as the device holds at once, each through its share of the tokens:
    // gammas are read once, and a token's table is computed while others are stored
    static std::atomic<int> held{0};
    int blocks = held.load(std::memory_order_relaxed);
    if (!blocks) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, qk_norm_rope_kernel<D, DEST, HALF>, kThreads, kStages * kThreads * 16);
        if (e != cudaSuccess) return e;
        held.store(blocks < 1 ? 1 : blocks, std::memory_order_relaxed);
    }
    const int64_t most = static_cast<int64_t>(sm_count) * (blocks < 1 ? 1 : blocks);
    return w4::launch_dependent(qk_norm_rope_kernel<D, DEST, HALF>, static_cast<int>(p.tasks < most ? p.tasks : most), kThreads,
                                kStages * kThreads * 16, stream, p);
}

template <int D>
cudaError_t launch_d(const RopeParams& p0, int64_t T, int dest, bool half, int sm_count, cudaStream_t stream) {
    RopeParams p = p0;
    constexpr int kRows = kWarps * 32 / (D / 8);
    const int passes = (p.rows + kRows - 1) / kRows;
    // a block a pass where that leaves the machine unfilled
    p.parts = T * passes <= 4 * static_cast<int64_t>(sm_count) ? passes : 1;
    p.tasks = T * p.parts;
    if (dest == kDense) return half ? launch_to<D, kDense, true>(p, sm_count, stream) : launch_to<D, kDense, false>(p, sm_count, stream);
    if (dest == kBf16) return half ? launch_to<D, kBf16, true>(p, sm_count, stream) : launch_to<D, kBf16, false>(p, sm_count, stream);
    return half ? launch_to<D, kE4m3, true>(p, sm_count, stream) : launch_to<D, kE4m3, false>(p, sm_count, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream) {
    RopeParams p = {};
    p.q = a.q, p.k = a.k, p.v = a.v;
    p.ldq = 2 * a.ldq, p.ldk = 2 * a.ldk, p.ldv = 2 * a.ldv;
    p.hsq = static_cast<uint32_t>(2 * a.hsq), p.hsk = static_cast<uint32_t>(2 * a.hsk), p.hsv = static_cast<uint32_t>(2 * a.hsv);
    p.Hq = a.Hq, p.Hk = a.Hk;
    p.rows = a.Hq + a.Hk + (a.append ? a.Hk : 0);
    p.positions = a.positions, p.freqs = a.freqs;
    p.half = a.R / 2;
    const bool half = a.layout == FP8BS_ROPE_HALF;
    p.amplitude = a.amplitude, p.eps = a.eps;
    p.gq = a.gq, p.gk = a.gk;
    p.qo = a.qo, p.ko = a.ko;
    p.ldqo = 2 * a.ldqo, p.ldko = 2 * a.ldko;
    p.hsqo = static_cast<uint32_t>(2 * a.hsqo), p.hsko = static_cast<uint32_t>(2 * a.hsko);
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
    if (a.D == 64) return launch_d<64>(p, a.T, dest, half, a.sm_count, stream);
    if (a.D == 128) return launch_d<128>(p, a.T, dest, half, a.sm_count, stream);
    return launch_d<256>(p, a.T, dest, half, a.sm_count, stream);
}

}  // namespace fp8bs
