// Attention of a few new tokens a sequence over a paged cache, and the join of
// items that several blocks share (attn.cuh says how the work is dealt out).
//
// A tile is 8 or 16 rows, (token, query head) pairs of one key head, so every key is
// read once for all the query heads that share it.  The four warps of a block take
// alternate slices of 16 or 32 consecutive keys, each through a ring of its own
// (cp.async, no block-wide step), and keep their own maximum, sum and weighted
// values; they meet once an item.  Keys and values are the 16-row operand of mma.sync
// m16n8k16, the few query rows its 8 columns: scores are [key][row], a transposition
// of 8x8 blocks makes the weights the next product's operand, outputs are
// [dimension][row].
//
// Precision.  Scores, maxima, sums and outputs are fp32.  Over bf16 keys a weight enters
// the product with the values as the sum of two bf16 numbers (off by at most 2^-16 of
// it), since the memory leaves the tensor cores idle.  The maximum that weights
// are taken against may lag by 8 in units of log2: the sums then hold values up
// to 2^8 larger, and most slices need no rescaling.
//
// Codes.  e4m3 codes are exact in fp16, and the products run in it.  A row of q is
// multiplied by the power of two that brings its largest magnitude into [2^14, 2^15):
// exact down to 2^-31 of that, below off by at most 2^-39 of it.  A key's scale
// multiplies its score.  A value's scale 2^e is part of its weight, 2^(x + e), the
// maximum is taken of these, and 2^7 more uses fp16's range: a weight is off by at most
// 2^-11 of itself, or 2^-32 of the largest.  The sum takes 2^((x + e) - e), so that what
// the large numbers lose is the same in both.  (e below -80 counts as that, so that no sum
// of the weights 2^x alone overflows.)
//
// Masks.  A slice that some row masks a part of has a branch of its own.  Values that are
// not finite would reach a row that masks them as zero times them: over bf16 such a slice is
// weighed key by key; over codes zeros stand in their place, and the rows that see them get
// their NaNs at once.
// A 16-bit load of two bytes of a row, transposed, gives two dimensions of a key side
// by side: output tiles hold even dimensions in their upper and odd ones in their lower
// half.
//
// Over bf16 the memory bounds it: one token over 131072 keys of 8 heads of 128 takes 86 us
// (6.2 TB/s, 0.92 of a copy's rate).  Over codes their conversion and the weights do: 48
// tokens over up to 8192 keys 96 us (4.7 TB/s, 0.70).  Few keys wait for two launches, one
// behind the other: 777 take 9.7 us, in a graph 9.2.
#include "attn.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLag = 8.0f;

template <int D, int KIND, int NT>
struct Cfg {
    static constexpr bool kCodes = KIND == FP8BS_KV_E4M3;
    static constexpr int kRows = 8 * NT;
    static constexpr int kRowBytes = kCodes ? D : 2 * D;
    static constexpr int kSlice = kRowBytes <= 64 ? 32 : 16;  // keys
    static constexpr int kUnit = kSlice * kWarps;
    static constexpr int kStageBytes = 2 * kSlice * kRowBytes;
    static constexpr int kStages = kStageBytes <= 4096 ? 3 : 2;
    static constexpr int kPitch = D + 4;  // floats of a joined row: no bank conflicts
    static constexpr int kRedBytes = kRows * kPitch * 4;
    static constexpr int kScaleBytes = kCodes ? kWarps * kStages * 2 * kSlice * 4 : 0;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kSmem = kRing + kRedBytes + kScaleBytes;
    // of an SM: as many as its shared memory holds (Shared and 1 KB beside).  Of codes four
    // at most: three take 98 us at 48 sequences of up to 8192, two 115; of bf16 two, whose
    // longer shares fill the memory's pages: one token over 131072 keys 87 us, by three 92
    static constexpr int kFit = 228 * 1024 / (kSmem + 7 * 1024), kMost = kCodes ? 4 : 2;
    static constexpr int kBlocks = kFit > kMost ? kMost : kFit;
};

struct Shared {
    PlanShared plan;
    Cursor items[kWarps][4];  // of each warp: the ones that it has begun to fetch
    float2 parts[kWarps][16];  // (maximum, sum)
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {  // an 8x8 block of 16-bit numbers
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Byte offset of 16-byte chunk c of row r: no two rows of an ldmatrix phase share
// a bank.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return r * RB + ((RB >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// Codes 0 and 1 (WHICH 0) or 2 and 3 of a word as fp16 numbers.
template <int WHICH>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    uint32_t r;
    if (WHICH == 0)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// 2^(b - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7FFFFFFFu) : e8m0_to_float(b);
}

// The item after `c`, into *to.  Whole warp.
template <int ROWS, int UNIT>
__device__ __noinline__ void next_item(const AttnParams& p, const PlanShared& plan, const Cursor* from, Cursor* to) {
    Cursor c = *from;
    if (c.head + 1 < p.Hk) {
        ++c.head;
        c.unit = 0;
    } else if (c.tile + 1 < plan.first[p.B]) {
        c = attn_enter<ROWS, UNIT>(p, plan, c.tile + 1, c.b, 0);
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) *to = c;
    __syncwarp();
}
template <int ROWS, int UNIT>
__device__ __noinline__ void first_item(const AttnParams& p, const PlanShared& plan, Cursor* to) {
    const AttnShare& a = plan.share;
    Cursor c = attn_enter<ROWS, UNIT>(p, plan, a.tile, a.b, a.head);
    c.unit = a.unit;
    if ((threadIdx.x & 31) == 0) *to = c;
    __syncwarp();
}

template <int D, int KIND, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, KIND, NT>::kBlocks)
    attn_decode_kernel(const __grid_constant__ AttnParams p) {
    using C = Cfg<D, KIND, NT>;
    constexpr int RB = C::kRowBytes, SL = C::kSlice, ST = C::kStages;
    constexpr int KT = SL / 16;                // 16-key tiles of a slice
    constexpr int kChunks = RB / 16;           // of a row
    constexpr int kRowsACopy = 32 / kChunks;   // rows that one cp.async of the warp covers
    constexpr int kCopies = SL / kRowsACopy;
    constexpr int kSteps = D / 16;             // k16 steps of a score, and output tiles
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int mrow = lane & 7, mid = lane >> 3;
    float* red = reinterpret_cast<float*>(smem + C::kRing);
    const uint32_t ring = ptx::smem_addr(smem) + warp * ST * C::kStageBytes;
    float* zring = reinterpret_cast<float*>(smem + C::kRing + C::kRedBytes) + warp * ST * 2 * SL;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    if (tid == 0) reinterpret_cast<AttnSplit*>(p.ws)[blockIdx.x].rows = 0;
    attn_share<C::kRows, C::kUnit, kThreads>(p, sh.plan);
    const int units = static_cast<int>(sh.plan.share.end - sh.plan.share.begin);
    if (units == 0) return;

    Cursor* items = sh.items[warp];
    first_item<C::kRows, C::kUnit>(p, sh.plan, &items[0]);
    Cursor in = items[0], at = in;
    int in_item = 0, at_item = 0;
    int left = units;  // units still to fetch

    // Rows of the next slice to fetch: lane r < SL looks after row r, or all after the
    // page where one holds the slice.  The table is read a slice before it is used,
    // scales are stored a slice after they are read.
    const bool one_page = (1 << p.page_log2) >= SL;
    int page = -1, fetch_stage = 0, zstage = -1;
    uint32_t zk = 0, zv = 0;
    auto look_up = [&] {
        page = -1;
        if (left == 0) return;
        const int j = (in.lo + in.unit) * C::kUnit + warp * SL + (lane < SL ? lane : 0);
        int id;
        if (j >= in.first && j < in.past && attn_page(p, p.table + in.b * p.table_stride, j, &id)) page = id;
    };
    auto store_scales = [&] {
        if (C::kCodes && zstage >= 0 && lane < SL) {
            zring[zstage * 2 * SL + lane] = scale_of(zk);
            zring[zstage * 2 * SL + SL + lane] = zv == 255u ? __uint_as_float(0x7FFFFFFFu) : static_cast<float>(max(static_cast<int>(zv), 47) - 127);
        }
        zstage = -1;
    };
    auto fetch = [&] {
        store_scales();
        if (left > 0) {
            const int j = (in.lo + in.unit) * C::kUnit + warp * SL + (lane < SL ? lane : 0);
            const int slot = j & ((1 << p.page_log2) - 1);
            long long off = -1;
            if (page >= 0) off = page * p.pstride + slot * p.sstride + in.head * p.hstride;
            if (C::kCodes) {
                zk = zv = 0;
                zstage = fetch_stage;
                if (page >= 0) {
                    const long long z = page * p.zpstride + slot * p.zsstride + in.head * p.zhstride;
                    zk = p.ks[z], zv = p.vs[z];
                }
            }
            const uint32_t base = ring + fetch_stage * C::kStageBytes;
            const int r0 = lane / kChunks, c = lane % kChunks;
            if (one_page && __all_sync(0xFFFFFFFFu, page >= 0)) {  // every row is there
                long long o = __shfl_sync(0xFFFFFFFFu, off, 0) + r0 * p.sstride + 16 * c;
                const long long step = kRowsACopy * p.sstride;
#pragma unroll
                for (int i = 0; i < kCopies; ++i, o += step) {
                    const uint32_t to = base + chunk_at<RB>(i * kRowsACopy + r0, c);
                    cp_async16(to, p.k + o);
                    cp_async16(to + SL * RB, p.v + o);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kCopies; ++i) {
                    const int r = i * kRowsACopy + r0;
                    const long long o = __shfl_sync(0xFFFFFFFFu, off, r);
                    const long long src = o >= 0 ? o + 16 * c : 0;
                    const uint32_t to = base + chunk_at<RB>(r, c);
                    cp_async16_zfill(to, p.k + src, o >= 0);
                    cp_async16_zfill(to + SL * RB, p.v + src, o >= 0);
                }
            }
            --left;
            if (++fetch_stage == ST) fetch_stage = 0;
            if (++in.unit >= in.n && left > 0) {
                next_item<C::kRows, C::kUnit>(p, sh.plan, &items[in_item & 3], &items[(in_item + 1) & 3]);
                in = items[++in_item & 3];
            }
        }
        cp_commit();
        look_up();
    };
    look_up();
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) fetch();

    uint32_t qf[kSteps][NT][2];
    float out[kSteps][NT][4];
    float m[NT][2], l[NT][2];  // of rows 8 n + 2 t + i; sums over this lane's keys
    int place[NT][2];
    float unit[NT][2];  // codes: what a row's scores are multiplied by

    auto load_q = [&] {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * t + i;
                place[n][i] = r < at.rows ? at.base + div_g(p, at.row0 + r) : -1;
                m[n][i] = -INFINITY, l[n][i] = 0.0f;
            }
#pragma unroll
            for (int o = 0; o < kSteps; ++o)
#pragma unroll
                for (int i = 0; i < 4; ++i) out[o][n][i] = 0.0f;
            const int r = at.row0 + 8 * n + g, token = div_g(p, r);
            const bool there = 8 * n + g < at.rows;
            const uint16_t* q = p.q;
            if (there) q += static_cast<int64_t>(at.q0 + token) * p.ldq + (at.head * p.G + r - token * p.G) * p.hsq;
            uint32_t most = 0;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                uint2 w = make_uint2(0, 0);
                if (there && C::kCodes) w = *reinterpret_cast<const uint2*>(q + 16 * ks + 4 * t);
                if (there && !C::kCodes) {
                    w.x = *reinterpret_cast<const uint32_t*>(q + 16 * ks + 2 * t);
                    w.y = *reinterpret_cast<const uint32_t*>(q + 16 * ks + 8 + 2 * t);
                }
                qf[ks][n][0] = w.x, qf[ks][n][1] = w.y;
                if (C::kCodes)
                    most = max(max(most, max(w.x & 0x7FFFu, w.y & 0x7FFFu)), max(w.x >> 16 & 0x7FFFu, w.y >> 16 & 0x7FFFu));
            }
            if (C::kCodes) {
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                // the exponent of the factor 2^(14 - exponent of the largest), within fp32's;
                // rows of zeros, and with an infinity or a NaN, stay
                const int e = static_cast<int>(most >> 7);
                const int up = most == 0 || e == 255 ? 0 : min(14 - (e - 127), 126);
                const float factor = __int_as_float((up + 127) << 23);
                auto narrow = [&](uint32_t w) {
                    uint32_t r;
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(w & 0xFFFF0000u) * factor),
                        "f"(__uint_as_float(w << 16) * factor));
                    return r;
                };
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) qf[ks][n][i] = narrow(qf[ks][n][i]);
                // (up is in -114 .. 126, so 2^-up is a normal number)
                const float back = __int_as_float((127 - up) << 23) * p.scale_log2;
#pragma unroll
                for (int i = 0; i < 2; ++i) unit[n][i] = __shfl_sync(0xFFFFFFFFu, back, 4 * (2 * t + i));
            }
        }
    };

    int begun = at.unit == 0;  // whether the item began in this block
    // The four warps' parts of the item become one, which goes to o or to a slot.
    auto finish = [&](bool whole, int u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], off);
                if (l[n][i] == 0.0f && place[n][i] >= 0) l[n][i] = kNoWeight;
                if (g == 0) sh.parts[warp][8 * n + 2 * t + i] = make_float2(m[n][i], l[n][i]);
            }
        __syncthreads();
        float part[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * t + i;
                float most = sh.parts[0][r].x;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) most = fmaxf(most, sh.parts[w][r].x);
                part[n][i] = m[n][i] == -INFINITY ? 0.0f : ex2(m[n][i] - most);
            }
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int o = 0; o < kSteps; ++o)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // rows 2t, 2t + 1 of dimensions g and g + 8, or 2g and 2g + 1, of 16
                            float* to = red + (8 * n + 2 * t + (i & 1)) * C::kPitch + 16 * o +
                                        (C::kCodes ? 2 * g + (i >> 1) : g + 8 * (i >> 1));
                            *to = (w == 0 ? 0.0f : *to) + out[o][n][i] * part[n][i & 1];
                        }
            }
            __syncthreads();
        }
        float* slot = attn_slot(p, gridDim.x, C::kRows, D, blockIdx.x, begun);
        constexpr int kPer = D / 8;  // threads of a row
#pragma unroll 1
        for (int row = tid / kPer; row < at.rows; row += kThreads / kPer) {
            const int col = tid % kPer * 8;
            float most = sh.parts[0][row].x, sum = 0.0f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) most = fmaxf(most, sh.parts[w][row].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += sh.parts[w][row].x == -INFINITY ? sh.parts[w][row].y : fallen(sh.parts[w][row].y, sh.parts[w][row].x - most);
            const float4 x = *reinterpret_cast<const float4*>(red + row * C::kPitch + col);
            const float4 y = *reinterpret_cast<const float4*>(red + row * C::kPitch + col + 4);
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const int r = at.row0 + row, token = div_g(p, r);
                uint16_t* dst = p.o + static_cast<int64_t>(at.q0 + token) * p.ldo + (at.head * p.G + r - token * p.G) * p.hso + col;
                *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv),
                                                            pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
            } else {
                *reinterpret_cast<float4*>(slot + row * D + col) = x;
                *reinterpret_cast<float4*>(slot + row * D + col + 4) = y;
                if (col == 0) slot[C::kRows * D + row] = most, slot[C::kRows * D + C::kRows + row] = sum;
            }
        }
        if (!whole && begun && tid == 0) {
            const long long start = sh.plan.share.begin + u - at.unit;  // where the item begins
            AttnSplit rec = {at.rows, at.q0, at.row0, at.head, attn_last_block(sh.plan.share, start, at.n), {0, 0, 0}};
            reinterpret_cast<AttnSplit*>(p.ws)[blockIdx.x] = rec;
        }
        __syncthreads();
    };

    load_q();
    int stage = 0;
#pragma unroll 1
    for (int u = 0; u < units; ++u) {
        fetch();
        cp_wait<ST - 1>();
        __syncwarp();
        const uint32_t ks = ring + stage * C::kStageBytes, vs = ks + SL * RB;
        const float* z = zring + stage * 2 * SL;
        const int j0 = (at.lo + at.unit) * C::kUnit + warp * SL;
        if (j0 < at.past && j0 + SL > at.first) {
            float s[KT][NT][4];
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[k][n][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < kSteps; i += C::kCodes ? 2 : 1)
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    uint32_t b[4];
                    const int row = k * 16 + (mid & 1) * 8 + mrow;
                    if (C::kCodes) {
                        ldsm(b, ks + chunk_at<RB>(row, i + (mid >> 1)));
                        const uint32_t a0[4] = {code_pair<0>(b[0]), code_pair<0>(b[1]), code_pair<1>(b[0]), code_pair<1>(b[1])};
                        const uint32_t a1[4] = {code_pair<0>(b[2]), code_pair<0>(b[3]), code_pair<1>(b[2]), code_pair<1>(b[3])};
                        const int next = i + 1 < kSteps ? i + 1 : i;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16(s[k][n], a0, qf[i][n][0], qf[i][n][1]);
                            mma_f16(s[k][n], a1, qf[next][n][0], qf[next][n][1]);
                        }
                    } else {
                        ldsm(b, ks + chunk_at<RB>(row, 2 * i + (mid >> 1)));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_bf16(s[k][n], b, qf[i][n][0], qf[i][n][1]);
                    }
                }
            // scores in units of log2, masked ones at minus infinity
            float most[NT][2], in[KT][2];  // of a key: what its score has of its value's scale
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = k * 16 + 8 * h + g;
                    const float scale = C::kCodes ? z[key] : 0.0f, more = C::kCodes ? z[SL + key] : 0.0f;
                    if (C::kCodes) in[k][h] = more == more ? more : 0.0f;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // codes: twice a factor, as their product may leave fp32's range
                            float& x = s[k][n][2 * h + i];
                            x = C::kCodes ? x * unit[n][i] * scale + more : x * p.scale_log2;  // with the value's scale
                        }
                }
            bool odd = false;  // a value that is not finite where some row masks its key
            if (!(j0 + SL <= at.lowest + 1 && (p.window == 0 || j0 >= at.past - p.window))) {
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int j = j0 + k * 16 + 8 * h + g, w = place[n][i];
                                if (j > w || (p.window && j <= w - p.window)) s[k][n][2 * h + i] = -INFINITY;
                            }
                // (rows of one token see the same keys; the others are zeros here)
                if (at.lowest + 1 < at.past) {
                    uint32_t acc = 0;
#pragma unroll 1
                    for (int i = lane; i < SL * kChunks; i += 32) {
                        const uint4 x = *reinterpret_cast<const uint4*>(smem + (vs - ptx::smem_addr(smem)) + 16 * i);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            acc |= C::kCodes ? odd_codes(w[c]) : ((w[c] & 0x7F80u) == 0x7F80u) | ((w[c] & 0x7F800000u) == 0x7F800000u);
                    }
                    odd = __any_sync(0xFFFFFFFFu, acc != 0);
                }
                if (C::kCodes && odd) {
                    // NaNs for the rows that see such a code, and a zero in its place.  (A scale of
                    // 255 is in the weights of the rows that see its key.)
                    uint8_t* rows = smem + (vs - ptx::smem_addr(smem));
#pragma unroll 1
                    for (int key = 0; key < SL; ++key) {
                        const int j = j0 + key;
                        bool sees[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) sees[n][i] = j <= place[n][i] && (!p.window || j > place[n][i] - p.window);
#pragma unroll
                        for (int o = 0; o < kSteps; ++o) {
                            const uint32_t w = odd_codes(*reinterpret_cast<const uint16_t*>(rows + chunk_at<RB>(key, o) + 2 * g));
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if ((w >> (8 * (i >> 1)) & 0x80u) && sees[n][i & 1]) out[o][n][i] = __uint_as_float(0x7FFFFFFFu);
                        }
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int i = lane; i < SL * kChunks * 4; i += 32) {
                        uint32_t* w = reinterpret_cast<uint32_t*>(rows) + i;
                        *w = without_odd_codes(*w);
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    most[n][i] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int h = 0; h < 2; ++h) most[n][i] = fmaxf(most[n][i], s[k][n][2 * h + i]);
                }
            bool grown = false;
            float fall[NT][2], from[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) most[n][i] = fmaxf(most[n][i], __shfl_xor_sync(0xFFFFFFFFu, most[n][i], off));
                    fall[n][i] = 0.0f;
                    // (roundings that keep weights of codes within fp16's range, however large scores are)
                    if (most[n][i] > __fadd_rd(m[n][i], kLag)) {
                        fall[n][i] = m[n][i] - most[n][i];
                        m[n][i] = most[n][i];
                        grown = true;
                    }
                    from[n][i] = __fsub_ru(m[n][i] == -INFINITY ? 0.0f : m[n][i], C::kCodes ? 7.0f : 0.0f);
                }
            if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float shrink[2] = {ex2(fall[n][0]), ex2(fall[n][1])};  // 0 from minus infinity
                    l[n][0] = fallen(l[n][0], fall[n][0]), l[n][1] = fallen(l[n][1], fall[n][1]);
#pragma unroll
                    for (int o = 0; o < kSteps; ++o)
#pragma unroll
                        for (int i = 0; i < 4; ++i) out[o][n][i] *= shrink[i & 1];
                }
            }
            uint32_t hi[KT][NT][2], low[KT][NT][2];  // [8 keys]: the product's operand
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float x = s[k][n][2 * h + i] - from[n][i];
                            w[i] = ex2(x);
                            l[n][i] += C::kCodes ? ex2(x - in[k][h]) : w[i];
                            s[k][n][2 * h + i] = w[i];
                        }
                        if (C::kCodes) {
                            uint32_t both;
                            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(both) : "f"(w[1]), "f"(w[0]));
                            hi[k][n][h] = transposed(both);
                        } else {
                            const uint32_t both = pack_bf16(w[0], w[1]);
                            hi[k][n][h] = transposed(both);
                            low[k][n][h] = transposed(pack_bf16(w[0] - __uint_as_float(both << 16),
                                                                w[1] - __uint_as_float(both & 0xFFFF0000u)));
                        }
                    }
                }
            if (C::kCodes || !odd) {
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int o = 0; o < kSteps; o += C::kCodes ? 2 : 1) {
                        uint32_t b[4];
                        if (C::kCodes) {
                            ldsm_t(b, vs + chunk_at<RB>(k * 16 + (mid & 1) * 8 + mrow, o + (mid >> 1)));
                            // a word: (d, d + 1) of a key, then of the next; wanted: pairs of keys
#pragma unroll
                            for (int e = 0; e < 4; ++e) b[e] = __byte_perm(b[e], 0, 0x3120);
                            const uint32_t a0[4] = {code_pair<0>(b[0]), code_pair<1>(b[0]), code_pair<0>(b[1]), code_pair<1>(b[1])};
                            const uint32_t a1[4] = {code_pair<0>(b[2]), code_pair<1>(b[2]), code_pair<0>(b[3]), code_pair<1>(b[3])};
                            const int next = o + 1 < kSteps ? o + 1 : o;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma_f16(out[o][n], a0, hi[k][n][0], hi[k][n][1]);
                                mma_f16(out[next][n], a1, hi[k][n][0], hi[k][n][1]);
                            }
                        } else {
                            ldsm_t(b, vs + chunk_at<RB>(k * 16 + (mid >> 1) * 8 + mrow, 2 * o + (mid & 1)));
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma_bf16(out[o][n], b, hi[k][n][0], hi[k][n][1]);
                                mma_bf16(out[o][n], b, low[k][n][0], low[k][n][1]);
                            }
                        }
                    }
            } else if constexpr (!C::kCodes) {
                // key by key, so that no masked value is multiplied
                const uint8_t* rows = smem + (vs - ptx::smem_addr(smem));
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll 1
                        for (int e = 0; e < 8; ++e) {
                            const int key = k * 16 + 8 * h + e, j = j0 + key;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float w[2];
                                bool sees[2];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    w[i] = __shfl_sync(0xFFFFFFFFu, s[k][n][2 * h + i], 4 * e + t);
                                    sees[i] = j <= place[n][i] && (!p.window || j > place[n][i] - p.window);
                                }
#pragma unroll
                                for (int o = 0; o < kSteps; ++o)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const int d = 16 * o + g + 8 * (i >> 1);
                                        const uint16_t v = *reinterpret_cast<const uint16_t*>(rows + chunk_at<RB>(key, d >> 3) + 2 * (d & 7));
                                        if (sees[i & 1]) out[o][n][i] = fmaf(w[i & 1], bf16_bits_to_float(v), out[o][n][i]);
                                    }
                            }
                        }
            }
        }
        __syncwarp();  // the stage is read; the warp's next fetch may overwrite it
        if (++stage == ST) stage = 0;
        const bool last = at.unit + 1 == at.n;
        if (last || u + 1 == units) {
            finish(last && begun, u);
            if (u + 1 < units) {
                at = items[++at_item & 3];
                begun = 1;
                load_q();
            }
        } else {
            ++at.unit;
        }
    }
}

// Rows of items that several blocks share: blockIdx.x names the block that began one,
// 8 values a thread.  An item's parts are dealt to up to 8 threads of the same values,
// each of which keeps a maximum of its own; they meet in shared memory, in the order
// of the parts.
constexpr int kJoin = 256;
template <int D>
__global__ void __launch_bounds__(kJoin) attn_join_kernel(const __grid_constant__ AttnParams p, int MT, int grid) {
    constexpr int kPer = D / 8, kLanes = kJoin / kPer;  // threads of a row; rows that the block has threads for
    __shared__ float met[kJoin][11];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const AttnSplit rec = reinterpret_cast<const AttnSplit*>(p.ws)[blockIdx.x];
    if (rec.rows == 0) return;
    const int first = blockIdx.x, n = rec.last - first + 1;
    int ways = 1;
    while (ways < 8 && 2 * ways < n && 2 * ways * rec.rows <= kLanes * static_cast<int>(gridDim.y)) ways *= 2;
    const int col = threadIdx.x % kPer * 8, lane = threadIdx.x / kPer;
    const int way = lane % ways, per = (n + ways - 1) / ways, rows = kLanes / ways;
    for (int row0 = blockIdx.y * rows; row0 < rec.rows; row0 += gridDim.y * rows) {
        const int row = row0 + lane / ways;
        float most = -INFINITY, sum = 0.0f, v[8] = {};
        if (row < rec.rows) {
#pragma unroll 4
            for (int i = way * per; i < min(n, (way + 1) * per); ++i) {
                const float* s = attn_slot(p, grid, MT, D, first + i, i == 0);
                const float m = s[MT * D + row], l = s[MT * D + MT + row];
                const float4 x = *reinterpret_cast<const float4*>(s + row * D + col);
                const float4 y = *reinterpret_cast<const float4*>(s + row * D + col + 4);
                const float top = fmaxf(most, m), at = top == -INFINITY ? 0.0f : top;
                const float keep1 = ex2(0.5f * (most - at)), w1 = ex2(0.5f * (m - at)), keep = keep1 * keep1, w = w1 * w1;
                sum = m == -INFINITY ? sum + l : fmaf(l * w1, w1, sum * keep1 * keep1);  // (as fallen)
                most = top;
                v[0] = fmaf(x.x, w, v[0] * keep), v[1] = fmaf(x.y, w, v[1] * keep);
                v[2] = fmaf(x.z, w, v[2] * keep), v[3] = fmaf(x.w, w, v[3] * keep);
                v[4] = fmaf(y.x, w, v[4] * keep), v[5] = fmaf(y.y, w, v[5] * keep);
                v[6] = fmaf(y.z, w, v[6] * keep), v[7] = fmaf(y.w, w, v[7] * keep);
            }
        }
        if (ways > 1) {
            float* mine = met[threadIdx.x];
            __syncthreads();
            mine[0] = most, mine[1] = sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) mine[2 + i] = v[i];
            __syncthreads();
            if (way == 0) {
                for (int j = 1; j < ways; ++j) {
                    const float* o = met[threadIdx.x + j * kPer];
                    const float top = fmaxf(most, o[0]), at = top == -INFINITY ? 0.0f : top;
                    const float keep1 = ex2(0.5f * (most - at)), w1 = ex2(0.5f * (o[0] - at)), keep = keep1 * keep1, w = w1 * w1;
                    sum = o[0] == -INFINITY ? sum + o[1] : fmaf(o[1] * w1, w1, sum * keep1 * keep1);
                    most = top;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = fmaf(o[2 + i], w, v[i] * keep);
                }
            }
        }
        if (way == 0 && row < rec.rows) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int r = rec.row0 + row, token = div_g(p, r);
            uint16_t* dst = p.o + static_cast<int64_t>(rec.q0 + token) * p.ldo + (rec.head * p.G + r - token * p.G) * p.hso + col;
            *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                                                        pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
        }
    }
}

template <int D, int KIND, int NT>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    using C = Cfg<D, KIND, NT>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = attn_allow_shared(attn_decode_kernel<D, KIND, NT>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    const int grid = a.sm_count * C::kBlocks;
    const cudaError_t r = w4::launch_dependent(attn_decode_kernel<D, KIND, NT>, grid, kThreads, C::kSmem, stream,
                                               static_cast<const AttnParams&>(a));
    return r == cudaSuccess ? launch_attn_join(a, C::kRows, grid, stream) : r;
}

// 16 rows a tile where a sequence has more than 8 on average: its keys are then read
// half as often, and every step costs twice as much.
template <int D, int KIND>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
    if constexpr (D < 256)
        if (static_cast<int64_t>(a.T) * a.G > 8 * static_cast<int64_t>(a.B)) return launch<D, KIND, 2>(a, stream);
    return launch<D, KIND, 1>(a, stream);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, int MT, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    const int rows = kJoin / (a.D / 8);  // of a pass, where nothing is dealt out
    const int most = MT * 8 / rows;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), static_cast<unsigned>(most < 1 ? 1 : most > 16 ? 16 : most));
    cfg.blockDim = dim3(kJoin);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kernel = a.D == 64 ? attn_join_kernel<64> : a.D == 128 ? attn_join_kernel<128> : attn_join_kernel<256>;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const AttnParams&>(a), MT, grid);
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t stream) {
    if (a.kind == FP8BS_KV_BF16) {
        if (a.D == 64) return launch_rows<64, FP8BS_KV_BF16>(a, stream);
        if (a.D == 128) return launch_rows<128, FP8BS_KV_BF16>(a, stream);
        return launch_rows<256, FP8BS_KV_BF16>(a, stream);
    }
    if (a.D == 64) return launch_rows<64, FP8BS_KV_E4M3>(a, stream);
    if (a.D == 128) return launch_rows<128, FP8BS_KV_E4M3>(a, stream);
    return launch_rows<256, FP8BS_KV_E4M3>(a, stream);
}

size_t attn_workspace_bytes(int D, int sm_count) {
    const size_t few = static_cast<size_t>(4 * sm_count) * 2 * attn_slot_floats(16, D);
    const size_t many = static_cast<size_t>(sm_count) * 2 * attn_chunk_slot_floats(D);
    return kWsErrorBytes + attn_records_bytes(4 * sm_count) + (few > many ? few : many) * sizeof(float);
}

// Rows of a sequence, on average, from which the tensor core's kernel takes the call.  This
// file's kernel reads a sequence's keys once for 16 rows (8 with heads of 256), the other
// once for 256 (128), at a higher cost of each step.  At 64 sequences of up to 8192 keys
// (4560 on average), us by this one against the other, with so many rows on average:
//   heads of 128: 12 rows bf16 198 / 237, codes 260 / 374; 23 rows 353 / 239, 462 / 377
//   heads of 256: 14 rows bf16 184 / 109, codes 100 / 145; codes 19 rows 137 / 147, 24 171 / 147
//   heads of 64 (which take the value of 128): 12 rows 135 / 200, 115 / 352; 23 rows 235 / 200, 186 / 352
static int64_t chunk_rows(const AttnArgs& a) {
    return a.D < 256 ? 17 : a.kind == FP8BS_KV_BF16 ? 9 : 20;
}

cudaError_t launch_attn_paged(const AttnArgs& a, cudaStream_t stream) {
    // (boxes of one row of 64 codes would not begin on 128 bytes of shared memory)
    const bool boxes = a.kind == FP8BS_KV_BF16 || a.D > 64 || a.page_log2 > 0;
    if (static_cast<int64_t>(a.T) * a.G >= chunk_rows(a) * a.B && boxes) return launch_attn_chunk(a, stream);
    return launch_attn_decode(a, stream);
}

}  // namespace fp8bs
