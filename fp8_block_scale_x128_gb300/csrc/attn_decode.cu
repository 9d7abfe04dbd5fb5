// Attention of a few new tokens a sequence over a paged cache, and the join of
// items that several blocks share (attn.cuh says how the work is dealt out).
//
// A tile is 16 rows, (token, query head) pairs of one key head, so every key is
// read once for all the query heads that share it.  The four warps of a block
// take alternate slices of 16 or 32 consecutive keys, each through a ring of its
// own (cp.async, no block-wide step), and keep their own maximum, sum and
// weighted values; they meet once an item.  A slice: scores by mma.sync m16n8k16
// (16 rows x 8 keys a step), softmax weights in registers, whose accumulator
// layout is the next product's operand layout, values by ldmatrix.trans.
//
// Precision.  Scores, maxima, sums and outputs are fp32.  A weight enters the
// product with the values as the sum of two bf16 numbers (off by at most 2^-18 of
// it), since the memory leaves the tensor cores idle.  The maximum that weights
// are taken against may lag by 8 in units of log2: the sums then hold values up
// to 2^8 larger, and most slices need no rescaling.
//
// Codes.  An e4m3 code's bits shifted into a bf16's exponent and fraction are its
// value times 2^-120, exactly, subnormals included; q carries 2^64 and the weights
// 2^64 against it.  Scales are powers of two: a key's multiplies its scores, a
// value's its weights.  The pairing of bytes that the decode gives (even bytes,
// odd bytes) is met by a permutation of q's dimensions, and by two tiles of even
// and odd dimensions of the output.
#include "attn.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;
constexpr float kLag = 8.0f;

template <int D, int KIND>
struct Cfg {
    static constexpr bool kCodes = KIND == FP8BS_KV_E4M3;
    static constexpr int kRowBytes = kCodes ? D : 2 * D;
    static constexpr int kSlice = kRowBytes * 32 <= 4096 ? 32 : 16;  // keys
    static constexpr int kUnit = kSlice * kWarps;
    static constexpr int kStageBytes = 2 * kSlice * kRowBytes;
    static constexpr int kStages = kStageBytes <= 4096 ? 4 : 3;
    static constexpr bool kQShared = D == 256;  // else q stays in registers
    static constexpr int kRedPitch = 136;       // floats; 128 columns at a time
    static constexpr int kRedBytes = kRows * kRedPitch * 4;
    static constexpr int kScaleBytes = kCodes ? kWarps * kStages * 2 * kSlice : 0;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kSmem = kRing + kRedBytes + kScaleBytes;
    static constexpr int kBlocks = kSmem <= 108 * 1024 ? 2 : 1;  // of an SM
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

// Byte offset of 16-byte chunk c of row r: no two rows of an ldmatrix phase share
// a bank.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return r * RB + ((RB >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// 2^(b - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7FFFFFFFu) : e8m0_to_float(b);
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, Cfg<D, KIND>::kBlocks) attn_decode_kernel(const AttnParams p) {
    using C = Cfg<D, KIND>;
    constexpr int RB = C::kRowBytes, SL = C::kSlice, ST = C::kStages;
    constexpr int kChunks = RB / 16;           // of a row
    constexpr int kRowsACopy = 32 / kChunks;   // rows that one cp.async of the warp covers (kChunks <= 32)
    constexpr int kSteps = D / 16;             // k16 steps of a score
    constexpr int kOut = D / 8;                // output tiles
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PlanShared plan;
    __shared__ float2 parts[kWarps][kRows];    // (maximum, sum)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    float* red = reinterpret_cast<float*>(smem + C::kRing);
    const uint32_t ring = ptx::smem_addr(smem) + warp * ST * C::kStageBytes;
    const uint32_t qshared = ptx::smem_addr(red);  // q and the joined rows take turns
    uint8_t* zring = smem + C::kRing + C::kRedBytes + warp * ST * 2 * SL;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const AttnShare share = attn_share<kRows, C::kUnit, kThreads>(p, plan, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0) {
        AttnSplit* rec = reinterpret_cast<AttnSplit*>(p.ws) + blockIdx.x;
        rec->rows = 0;
    }
    if (share.begin >= share.end) return;

    Cursor<kRows, C::kUnit> in, at;
    in.start(p, plan, share);
    at = in;
    long long left = share.end - share.begin;  // units still to fetch

    // A slice's rows: lane r < SL looks after row r.  The table's entries are read a
    // slice before they are used, the scales stored a slice after they are read.
    int page = -1;
    uint32_t zk = 0, zv = 0;
    int zstage = -1, fetch_stage = 0;
    auto look_up = [&] {  // the page of this lane's row of `in`'s slice, -1: no key
        page = -1;
        const int j = (in.lo + in.unit) * C::kUnit + warp * SL + lane;
        if (left > 0 && lane < SL && j >= in.first && j < in.past) {
            int id;
            if (attn_page(p, p.table + in.b * p.table_stride, j, &id)) page = id;
        }
    };
    auto store_scales = [&] {
        if (C::kCodes && zstage >= 0 && lane < SL) {
            zring[zstage * 2 * SL + lane] = static_cast<uint8_t>(zk);
            zring[zstage * 2 * SL + SL + lane] = static_cast<uint8_t>(zv);
        }
        zstage = -1;
    };
    auto fetch = [&] {
        store_scales();
        if (left > 0) {
            const int j = (in.lo + in.unit) * C::kUnit + warp * SL + lane;
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
#pragma unroll
            for (int i = 0; i < SL / kRowsACopy; ++i) {
                const int r = i * kRowsACopy + lane / kChunks, c = lane % kChunks;
                const long long o = __shfl_sync(0xFFFFFFFFu, off, r);
                const bool there = o >= 0;
                const long long src = there ? o + 16 * c : 0;
                cp_async16_zfill(base + chunk_at<RB>(r, c), p.k + src, there);
                cp_async16_zfill(base + SL * RB + chunk_at<RB>(r, c), p.v + src, there);
            }
            --left;
            in.next(p, plan);
            if (++fetch_stage == ST) fetch_stage = 0;
        }
        cp_commit();
        look_up();
    };
    look_up();
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) fetch();

    uint32_t qf[C::kQShared ? 1 : kSteps][4];
    float out[kOut][4];
    float m[2], l[2];
    int place[2];
    int stage = 0;
    int begun = 1;  // whether the item began in this block

    auto load_q = [&] {
        const int base = at.s.kv - at.s.nq;
        const uint16_t* rows[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = at.row0 + g + 8 * i;
            const bool there = g + 8 * i < at.rows;
            place[i] = there ? base + r / p.G : -1;
            const int token = at.s.q0 + r / p.G, head = at.head * p.G + r % p.G;
            rows[i] = there ? p.q + static_cast<int64_t>(token) * p.ldq + head * p.hsq : nullptr;
            m[i] = -INFINITY, l[i] = 0.0f;
        }
#pragma unroll
        for (int o = 0; o < kOut; ++o)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[o][i] = 0.0f;
        auto big = [](uint32_t w) {  // * 2^64
            return pack_bf16(__uint_as_float(w << 16) * 0x1p64f, __uint_as_float(w & 0xFFFF0000u) * 0x1p64f);
        };
        auto piece = [&](int i, int ks, uint32_t& lo, uint32_t& hi) {
            lo = hi = 0;
            if (!rows[i]) return;
            if (C::kCodes) {
                const uint2 w = *reinterpret_cast<const uint2*>(rows[i] + 16 * ks + 4 * t);
                const uint32_t x = big(w.x), y = big(w.y);
                lo = __byte_perm(x, y, 0x5410), hi = __byte_perm(x, y, 0x7632);
            } else {
                lo = *reinterpret_cast<const uint32_t*>(rows[i] + 16 * ks + 2 * t);
                hi = *reinterpret_cast<const uint32_t*>(rows[i] + 16 * ks + 8 + 2 * t);
            }
        };
        if constexpr (C::kQShared) {
            if (warp == 0) {
                for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t lo, hi;
                        piece(i, ks, lo, hi);
                        uint8_t* q8 = reinterpret_cast<uint8_t*>(red);
                        *reinterpret_cast<uint32_t*>(q8 + chunk_at<2 * D>(g + 8 * i, 2 * ks) + 4 * t) = lo;
                        *reinterpret_cast<uint32_t*>(q8 + chunk_at<2 * D>(g + 8 * i, 2 * ks + 1) + 4 * t) = hi;
                    }
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                piece(0, ks, qf[ks][0], qf[ks][2]);
                piece(1, ks, qf[ks][1], qf[ks][3]);
            }
        }
    };

    // The four warps' parts of the item become one, which goes to o or to a slot.
    auto finish = [&](bool whole) {
        float part[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
            if (t == 0) parts[warp][g + 8 * i] = make_float2(m[i], l[i]);
        }
        __syncthreads();  // q in shared memory is read no more, too
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float most = parts[0][g + 8 * i].x;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) most = fmaxf(most, parts[w][g + 8 * i].x);
            part[i] = m[i] == -INFINITY ? 0.0f : ex2(m[i] - most);
            if (C::kCodes) part[i] *= 0x1p56f;
        }
        const int row = tid / 8, sub = tid % 8;
        float most = parts[0][row].x, sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) most = fmaxf(most, parts[w][row].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            sum += parts[w][row].x == -INFINITY ? 0.0f : parts[w][row].y * ex2(parts[w][row].x - most);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        float* slot = attn_slot(p, gridDim.x, kRows, D, blockIdx.x, begun);
        const int r = at.row0 + row;
        const int token = at.s.q0 + r / p.G, head = at.head * p.G + r % p.G;
        uint16_t* dst = p.o + static_cast<int64_t>(token) * p.ldo + head * p.hso;
        constexpr int kCols = D < 128 ? D : 128;
#pragma unroll
        for (int cb = 0; cb < D / kCols; ++cb) {
#pragma unroll 1
            for (int w = kWarps - 1; w >= 0; --w) {
                if (warp == w) {
#pragma unroll
                    for (int o = 0; o < kCols / 8; ++o)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float* v = &out[cb * kCols / 8 + o][2 * i];
                            float* to = red + (g + 8 * i) * C::kRedPitch;
                            float2* both;
                            if (C::kCodes) {  // even or odd dimensions of 16: one of the lane's four
                                float* q4 = to + 16 * (o / 2) + 4 * t + (o & 1);
                                q4[0] = (w == kWarps - 1 ? 0.0f : q4[0]) + v[0] * part[i];
                                q4[2] = (w == kWarps - 1 ? 0.0f : q4[2]) + v[1] * part[i];
                            } else {
                                both = reinterpret_cast<float2*>(to + 8 * o + 2 * t);
                                float2 x = w == kWarps - 1 ? make_float2(0.0f, 0.0f) : *both;
                                x.x += v[0] * part[i], x.y += v[1] * part[i];
                                *both = x;
                            }
                        }
                }
                __syncthreads();
            }
            constexpr int kMine = kCols / 8;  // columns of a thread
            const float* from = red + row * C::kRedPitch;
            if (row < at.rows) {
                if (whole) {
#pragma unroll
                    for (int c = 0; c < kMine; c += 8) {
                        const int col = (c / 8 * 8 + sub) * 8;
                        const float4 x = *reinterpret_cast<const float4*>(from + col);
                        const float4 y = *reinterpret_cast<const float4*>(from + col + 4);
                        *reinterpret_cast<uint4*>(dst + cb * kCols + col) =
                            make_uint4(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv),
                                       pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kMine; c += 4) {
                        const int col = (c / 4 * 8 + sub) * 4;
                        *reinterpret_cast<float4*>(slot + row * D + cb * kCols + col) =
                            *reinterpret_cast<const float4*>(from + col);
                    }
                    if (cb == 0 && sub == 0) {
                        slot[kRows * D + row] = most;
                        slot[kRows * D + kRows + row] = sum;
                    }
                }
            }
            __syncthreads();
        }
        // the item's unit past this block's share, counted from its start
        if (!whole && begun && tid == 0) {
            const long long start = share.end - (at.unit + 1);  // where the item begins
            AttnSplit* rec = reinterpret_cast<AttnSplit*>(p.ws) + blockIdx.x;
            rec->q0 = at.s.q0;
            rec->row0 = at.row0;
            rec->head = at.head;
            rec->last = static_cast<int32_t>(((start + at.n) * share.blocks - 1) / share.total);
            rec->rows = at.rows;
        }
    };

    begun = at.unit == 0;
    load_q();
    const long long units = share.end - share.begin;
#pragma unroll 1
    for (long long u = 0; u < units; ++u) {
        fetch();
        cp_wait<ST - 1>();
        __syncwarp();
        const uint32_t ks = ring + stage * C::kStageBytes, vs = ks + SL * RB;
        const uint8_t* z = zring + stage * 2 * SL;
        const int j0 = (at.lo + at.unit) * C::kUnit + warp * SL;
        const int base = at.s.kv - at.s.nq;
        const int lowest = base + at.row0 / p.G;
        if (j0 < at.past && j0 + SL > at.first) {
            float s[SL / 8][4];
#pragma unroll
            for (int n = 0; n < SL / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
            const int mrow = lane & 7, mid = lane >> 3;
#pragma unroll
            for (int k = 0; k < kSteps; k += C::kCodes ? 2 : 1) {
                uint32_t a[2][4];
                if constexpr (C::kQShared) {
                    ldsm(a[0], qshared + chunk_at<2 * D>(mrow + (mid & 1) * 8, 2 * k + (mid >> 1)));
                    if (C::kCodes) ldsm(a[1], qshared + chunk_at<2 * D>(mrow + (mid & 1) * 8, 2 * k + 2 + (mid >> 1)));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[0][i] = qf[k][i];
                        if (C::kCodes) a[1][i] = qf[k + 1 < kSteps ? k + 1 : k][i];
                    }
                }
#pragma unroll
                for (int n = 0; n < SL / 8; n += 2) {
                    uint32_t b[4];
                    const int row = n * 8 + (mid >> 1) * 8 + mrow;
                    if (C::kCodes) {
                        ldsm(b, ks + chunk_at<RB>(row, k + (mid & 1)));
                        mma_bf16(s[n], a[0], codes_even(b[0]), codes_odd(b[0]));
                        mma_bf16(s[n + 1], a[0], codes_even(b[2]), codes_odd(b[2]));
                        mma_bf16(s[n], a[1], codes_even(b[1]), codes_odd(b[1]));
                        mma_bf16(s[n + 1], a[1], codes_even(b[3]), codes_odd(b[3]));
                    } else {
                        ldsm(b, ks + chunk_at<RB>(row, 2 * k + (mid & 1)));
                        mma_bf16(s[n], a[0], b[0], b[1]);
                        mma_bf16(s[n + 1], a[0], b[2], b[3]);
                    }
                }
            }
            // scores in units of log2, masked ones at minus infinity
            const bool all = j0 + SL <= lowest + 1 && (p.window == 0 || j0 >= at.past - p.window);
            float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < SL / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = s[n][i] * (C::kCodes ? p.scale_log2 * 0x1p56f : p.scale_log2);
                    if (C::kCodes) x *= scale_of(z[n * 8 + 2 * t + (i & 1)]);
                    if (!all) {
                        const int j = j0 + n * 8 + 2 * t + (i & 1);
                        const int w = place[i >> 1];
                        if (j > w || (p.window && j <= w - p.window)) x = -INFINITY;
                    }
                    s[n][i] = x;
                    most[i >> 1] = fmaxf(most[i >> 1], x);
                }
            bool grown = false;
            float shrink[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                most[i] = fmaxf(most[i], __shfl_xor_sync(0xFFFFFFFFu, most[i], 1));
                most[i] = fmaxf(most[i], __shfl_xor_sync(0xFFFFFFFFu, most[i], 2));
                const bool up = most[i] > m[i] + kLag;
                shrink[i] = 1.0f;
                if (up) {
                    shrink[i] = ex2(m[i] - most[i]);  // 0 from minus infinity
                    m[i] = most[i];
                    grown = true;
                }
            }
            if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
                for (int o = 0; o < kOut; ++o)
#pragma unroll
                    for (int i = 0; i < 4; ++i) out[o][i] *= shrink[i >> 1];
                l[0] *= shrink[0], l[1] *= shrink[1];
            }
            const float from[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
            uint32_t hi[SL / 8][2], low[SL / 8][2];
#pragma unroll
            for (int n = 0; n < SL / 8; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float w0 = ex2(s[n][2 * i] - from[i]), w1 = ex2(s[n][2 * i + 1] - from[i]);
                    l[i] += w0 + w1;
                    if (C::kCodes) {
                        const float v0 = scale_of(z[SL + n * 8 + 2 * t]), v1 = scale_of(z[SL + n * 8 + 2 * t + 1]);
                        // a masked key's scale may be a NaN
                        w0 = s[n][2 * i] == -INFINITY ? 0.0f : w0 * 0x1p64f * v0;
                        w1 = s[n][2 * i + 1] == -INFINITY ? 0.0f : w1 * 0x1p64f * v1;
                    }
                    s[n][2 * i] = w0, s[n][2 * i + 1] = w1;
                    hi[n][i] = pack_bf16(w0, w1);
                    low[n][i] = pack_bf16(w0 - __uint_as_float(hi[n][i] << 16),
                                          w1 - __uint_as_float(hi[n][i] & 0xFFFF0000u));
                }
            bool odd = false;  // a value that is not finite where some row masks its key
            if (!C::kCodes && !all) {
                uint32_t acc = 0;
                for (int i = lane; i < SL * kChunks; i += 32) {
                    const uint4 x = *reinterpret_cast<const uint4*>(smem + (vs - ptx::smem_addr(smem)) + 16 * i);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc |= ((w[c] & 0x7F80u) == 0x7F80u) | ((w[c] & 0x7F800000u) == 0x7F800000u);
                }
                odd = __any_sync(0xFFFFFFFFu, acc != 0);
            }
            if (!odd) {
#pragma unroll
                for (int n = 0; n < SL / 16; ++n) {
                    const uint32_t ph[4] = {hi[2 * n][0], hi[2 * n][1], hi[2 * n + 1][0], hi[2 * n + 1][1]};
                    const uint32_t pl[4] = {low[2 * n][0], low[2 * n][1], low[2 * n + 1][0], low[2 * n + 1][1]};
#pragma unroll
                    for (int c = 0; c < kChunks; c += 2) {
                        uint32_t b[4];
                        ldsm_t(b, vs + chunk_at<RB>(n * 16 + (mid & 1) * 8 + mrow, c + (mid >> 1)));
                        if (C::kCodes) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t e0 = codes_even(b[2 * i]), e1 = codes_even(b[2 * i + 1]);
                                const uint32_t o0 = codes_odd(b[2 * i]), o1 = codes_odd(b[2 * i + 1]);
                                mma_bf16(out[2 * (c + i)], ph, e0, e1);
                                mma_bf16(out[2 * (c + i) + 1], ph, o0, o1);
                                mma_bf16(out[2 * (c + i)], pl, e0, e1);
                                mma_bf16(out[2 * (c + i) + 1], pl, o0, o1);
                            }
                        } else {
                            mma_bf16(out[c], ph, b[0], b[1]);
                            mma_bf16(out[c + 1], ph, b[2], b[3]);
                            mma_bf16(out[c], pl, b[0], b[1]);
                            mma_bf16(out[c + 1], pl, b[2], b[3]);
                        }
                    }
                }
            } else {
                // key by key, so that no masked value is multiplied
#pragma unroll
                for (int n = 0; n < SL / 8; ++n)
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        const int src = (lane & 28) | (k >> 1);
                        const float a0 = __shfl_sync(0xFFFFFFFFu, s[n][0], src), a1 = __shfl_sync(0xFFFFFFFFu, s[n][1], src);
                        const float b0 = __shfl_sync(0xFFFFFFFFu, s[n][2], src), b1 = __shfl_sync(0xFFFFFFFFu, s[n][3], src);
                        const float wa = k & 1 ? a1 : a0, wb = k & 1 ? b1 : b0;
                        const int j = j0 + n * 8 + k;
                        const bool sa = j <= place[0] && (!p.window || j > place[0] - p.window);
                        const bool sb = j <= place[1] && (!p.window || j > place[1] - p.window);
                        const uint32_t row = vs - ptx::smem_addr(smem);
#pragma unroll
                        for (int o = 0; o < kOut; ++o) {
                            if constexpr (!C::kCodes) {
                                const uint32_t w = *reinterpret_cast<const uint32_t*>(smem + row + chunk_at<RB>(n * 8 + k, o) + 4 * t);
                                const float v0 = __uint_as_float(w << 16), v1 = __uint_as_float(w & 0xFFFF0000u);
                                if (sa) out[o][0] = fmaf(wa, v0, out[o][0]), out[o][1] = fmaf(wa, v1, out[o][1]);
                                if (sb) out[o][2] = fmaf(wb, v0, out[o][2]), out[o][3] = fmaf(wb, v1, out[o][3]);
                            }
                        }
                    }
            }
        }
        __syncwarp();  // the stage is read; the warp's next fetch may overwrite it
        if (++stage == ST) stage = 0;
        const bool last = at.unit + 1 == at.n;
        if (last || u + 1 == units) {
            finish(last && begun);
            if (u + 1 < units) {
                at.next(p, plan);
                begun = 1;
                load_q();
            }
        } else {
            ++at.unit;
        }
    }
}

// Rows of items that several blocks share: blockIdx.x names the block that began
// one, blockIdx.y some of its rows, 8 values a thread.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p, int MT, int grid) {
    constexpr int kTh = D / 8;  // threads of a row
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const AttnSplit rec = reinterpret_cast<const AttnSplit*>(p.ws)[blockIdx.x];
    const int row = blockIdx.y * (256 / kTh) + threadIdx.x / kTh, col = threadIdx.x % kTh * 8;
    if (row >= rec.rows) return;
    const int first = blockIdx.x, n = rec.last - first + 1;
    auto slot = [&](int i) { return attn_slot(p, grid, MT, D, first + i, i == 0); };
    float most = -INFINITY;
    for (int i = 0; i < n; ++i) most = fmaxf(most, slot(i)[MT * D + row]);
    float sum = 0.0f, v[8] = {};
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float* s = slot(i);
        const float mi = s[MT * D + row], w = mi == -INFINITY ? 0.0f : ex2(mi - most);
        const float4 x = *reinterpret_cast<const float4*>(s + row * D + col);
        const float4 y = *reinterpret_cast<const float4*>(s + row * D + col + 4);
        sum = fmaf(w, s[MT * D + MT + row], sum);
        v[0] = fmaf(w, x.x, v[0]), v[1] = fmaf(w, x.y, v[1]), v[2] = fmaf(w, x.z, v[2]), v[3] = fmaf(w, x.w, v[3]);
        v[4] = fmaf(w, y.x, v[4]), v[5] = fmaf(w, y.y, v[5]), v[6] = fmaf(w, y.z, v[6]), v[7] = fmaf(w, y.w, v[7]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int r = rec.row0 + row;
    uint16_t* dst = p.o + static_cast<int64_t>(rec.q0 + r / p.G) * p.ldo + (rec.head * p.G + r % p.G) * p.hso + col;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                                                pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
}

template <int D, int KIND>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    using C = Cfg<D, KIND>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = attn_allow_shared(attn_decode_kernel<D, KIND>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    const int grid = a.sm_count * C::kBlocks;
    const cudaError_t r = w4::launch_dependent(attn_decode_kernel<D, KIND>, grid, kThreads, C::kSmem, stream,
                                               static_cast<const AttnParams&>(a));
    return r == cudaSuccess ? launch_attn_join(a, kRows, grid, stream) : r;
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, int MT, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    const int rows = 256 / (a.D / 8);
    cfg.gridDim = dim3(static_cast<unsigned>(grid), static_cast<unsigned>((MT + rows - 1) / rows));
    cfg.blockDim = dim3(256);
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
        if (a.D == 64) return launch<64, FP8BS_KV_BF16>(a, stream);
        if (a.D == 128) return launch<128, FP8BS_KV_BF16>(a, stream);
        return launch<256, FP8BS_KV_BF16>(a, stream);
    }
    if (a.D == 64) return launch<64, FP8BS_KV_E4M3>(a, stream);
    if (a.D == 128) return launch<128, FP8BS_KV_E4M3>(a, stream);
    return launch<256, FP8BS_KV_E4M3>(a, stream);
}

size_t attn_workspace_bytes(int D, int sm_count) {
    const size_t few = static_cast<size_t>(2 * sm_count) * 2 * attn_slot_floats(kRows, D);
    const size_t many = static_cast<size_t>(sm_count) * 2 * attn_chunk_slot_floats(D);
    return kWsErrorBytes + attn_records_bytes(2 * sm_count) + (few > many ? few : many) * sizeof(float);
}

// Rows of a sequence, on average, from which the tensor core's kernel takes the call.
constexpr int64_t kChunkRows = 33;

cudaError_t launch_attn_paged(const AttnArgs& a, cudaStream_t stream) {
    if (static_cast<int64_t>(a.T) * a.G >= kChunkRows * a.B) return launch_attn_chunk(a, stream);
    return launch_attn_decode(a, stream);
}

}  // namespace fp8bs
