// Mixture-of-experts router: l = x . w^T (bf16 in, fp32 sums), softmax over the
// experts, the k largest per token (ties to the lowest index), their weights.
//
// The logits are a skinny matrix product bound by the bytes of w and, at one
// token, by latency: 16 expert rows x one slice of H per warp (bf16 matrix
// instructions straight from global memory, each operand read as 16-byte words
// in a k order both share), the slices of a block summed in warp order, those
// of several blocks through the workspace, in slice order.  One warp selects
// for a token.  Up to kOneLaunchM tokens that is done by the last block to
// arrive (a counter that it also resets; no block waits for another), which
// saves a launch; with more tokens one block's warps would take them in turn,
// so a second kernel, a block per token, selects (programmatic dependent
// launch).  Measured (in a graph, w in the second-level cache): 7.1 us for one
// token of 512 experts, hidden 4096, 7.3 for 16 in two launches, 10.3 for 64; all
// of it is latency: two trips to memory, the arrival, the selection.
//
// The order of the chosen experts is decided by fp32 logits unless two of them
// (or the last chosen and the first left out) are closer than twice the bound
// of an fp32 logit's error: those are summed again with a compensated sum.  The
// error goes with the sum of magnitudes S = sum |x w|, not with the logit, so S
// is taken beside it, by the same matrix instruction on operands without their
// signs.  In units of 2^-24 S: 10 for an MMA (exact products, cut below 2^-25 of
// the largest of the 16, the sum below 2^-23 of itself: measured on GB300; each
// starts from zero, so that the cuts are of its own 16 products), 3 for the 8
// MMAs of a chunk, added in pairs, as are the 8 warps' sums, and one for each
// further chunk of a warp and slice.
//
// On N(0, 1) tokens with 1% outliers about one token in a hundred has such a pair
// (hidden 4096, 10 of 512): 3.2 us more for the call, most of it the latency of
// instructions that are not in the cache.  64 tokens take 12.5 us on average (24
// inputs), 10.3 without a pair.
#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

using namespace w4;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kOneLaunchM = kWarps;  // a warp per token in the last block
constexpr size_t kHeader = 256;  // workspace: the arrival counter, then the partial logits
// Blocks wanted: one a multiprocessor of a GB300.  A constant, not the device's
// count: the workspace's size goes by it and is asked for without a device.
constexpr int kTargetBlocks = 152;
constexpr int kMaxCand = 64;

struct RouteParams {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* w;  // [rows, H]
    int32_t* ids;
    float* weights;
    uint32_t* counter;
    float* part;  // [KS][M][pitch]: the logits of rows, then each tile's largest S
    int M, H, E, k, S;
    int rows, tiles, pitch, KS;
    float tie;  // logits closer than tie S may be in the wrong order
    int renorm, shared;
};

// K slices over blocks: enough blocks for the machine, at least one chunk per warp.
__host__ int k_splits(int64_t rows, int64_t H) {
    const int64_t tiles = (rows + kTileRows - 1) / kTileRows, chunks = H / kChunk;
    const int64_t want = (kTargetBlocks + tiles - 1) / tiles, most = (chunks + kWarps - 1) / kWarps;
    return static_cast<int>(want < most ? want : most);
}

__host__ int tiles_of(int64_t rows) { return static_cast<int>((rows + kTileRows - 1) / kTileRows); }
__host__ int pitch_of(int64_t rows) { return static_cast<int>((rows + tiles_of(rows) + 15) / 16 * 16); }

__device__ __forceinline__ void mma16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a b
__device__ __forceinline__ void mma16816_bf16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint4 magnitudes(const uint4& v) {
    constexpr uint32_t m = 0x7FFF7FFFu;
    return make_uint4(v.x & m, v.y & m, v.z & m, v.w & m);
}

// Order-preserving key of a logit; NaN ranks below everything, 0 is "taken".
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    if (v != v) return 1u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t key) {
    if (key == 1u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// The sum of two fp32 numbers, about 2^-48 of it exact.
struct Exact {
    float hi, lo;
    // this + v, the rounding error kept (D. E. Knuth's two-sum)
    __device__ __forceinline__ void add(float v) {
        const float t = __fadd_rn(hi, v), z = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(v, z)));
        hi = t;
    }
    // hi the nearest fp32 number, so that two compare by hi, then lo
    __device__ __forceinline__ void normalise() {
        const float t = __fadd_rn(hi, lo);
        lo = __fsub_rn(lo, __fsub_rn(t, hi));
        hi = t;
    }
    __device__ __forceinline__ bool operator>(const Exact& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
    __device__ __forceinline__ bool operator==(const Exact& o) const { return hi == o.hi && lo == o.lo; }
    __device__ __forceinline__ bool nan() const { return hi != hi; }
    __device__ __forceinline__ Exact shfl(int from) const {
        return {__shfl_sync(0xFFFFFFFFu, hi, from), __shfl_sync(0xFFFFFFFFu, lo, from)};
    }
};

// x[m] . w[e0] and x[m] . w[e1], compensated (products of two bf16 are exact in
// fp32).  Every lane returns them.  A warp has the latency of memory to itself:
// both rows together, the next words loaded before these are summed.
__device__ void exact_logits(const RouteParams& p, int m, int e0, int e1, int lane, Exact (&s)[2]) {
    constexpr int kWords = 4;
    const uint16_t *x = p.x + m * p.ldx, *w0 = p.w + static_cast<int64_t>(e0) * p.H, *w1 = p.w + static_cast<int64_t>(e1) * p.H;
    uint4 xr[kWords], wr[2][kWords];
    auto load = [&](int k0) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const int k = k0 + 256 * j + 8 * lane;
            xr[j] = wr[0][j] = wr[1][j] = make_uint4(0, 0, 0, 0);
            if (k < p.H) {
                xr[j] = *reinterpret_cast<const uint4*>(x + k);
                wr[0][j] = ptx::ld_global_v4(w0 + k);
                wr[1][j] = ptx::ld_global_v4(w1 + k);
            }
        }
    };
    s[0] = s[1] = {0.0f, 0.0f};
    load(0);
    for (int k0 = 0; k0 < p.H; k0 += 256 * kWords) {
        uint4 xn[kWords], wn[2][kWords];
#pragma unroll
        for (int j = 0; j < kWords; ++j) xn[j] = xr[j], wn[0][j] = wr[0][j], wn[1][j] = wr[1][j];
        load(k0 + 256 * kWords);
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            float a[8];
            unpack8(xn[j], a);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float b[8];
                unpack8(wn[q][j], b);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[q].add(__fmul_rn(a[i], b[i]));
            }
        }
    }
#pragma unroll 1
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const Exact o = {__shfl_xor_sync(0xFFFFFFFFu, s[q].hi, off), __shfl_xor_sync(0xFFFFFFFFu, s[q].lo, off)};
            // both lanes add the lower one's to the upper one's, so that they agree
            const bool upper = (lane & off) != 0;
            Exact sum = upper ? o : s[q];
            const Exact more = upper ? s[q] : o;
            sum.add(more.hi);
            sum.lo = __fadd_rn(sum.lo, more.lo);
            s[q] = sum;
        }
    s[0].normalise();
    s[1].normalise();
}

// A warp's scratch.
struct Select {
    uint32_t key[kMaxCand];
    float value[FP8BS_ROUTE_MAX_K + 1];
    int16_t expert[FP8BS_ROUTE_MAX_K + 1];
    int16_t cand[kMaxCand];
};

// The k + 1 largest of a token's logits in order, by one warp.  v[j]: expert
// lane + 32 j.
template <int PER>
__device__ void select_token(const RouteParams& p, Select& sel, int m, int lane) {
    constexpr int kTiles = PER / 16 + 1;  // of E + 1 rows, a lane's
    float v[PER], s[kTiles];
    uint32_t key[PER];
    const float* part = p.part + static_cast<int64_t>(m) * p.pitch + lane;
    const int64_t pitch = static_cast<int64_t>(p.M) * p.pitch;
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = 0.0f;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) s[j] = 0.0f;
    // four slices' loads in flight together, added in slice order
    for (int ks = 0; ks < p.KS; ks += 4) {
        float u[4][PER], us[4][kTiles];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                u[i][j] = ks + i < p.KS && lane + 32 * j < p.E ? __ldcg(part + (ks + i) * pitch + 32 * j) : 0.0f;
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
                us[i][j] = ks + i < p.KS && lane + 32 * j < p.tiles ? __ldcg(part + (ks + i) * pitch + p.rows + 32 * j) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < PER; ++j) v[j] += u[i][j];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) s[j] += us[i][j];
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = lane + 32 * j < p.E ? order_key(v[j]) : 0;
    uint32_t largest_s = 0;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) largest_s = max(largest_s, __float_as_uint(s[j]) & 0x7FFFFFFFu);
    largest_s = __reduce_max_sync(0xFFFFFFFFu, largest_s);
    const int kk = min(p.k + 1, p.E);
    // The kk-th largest of the lanes' maxima is a bound that at least kk experts
    // reach; the few that do are ranked against each other.
    int n_top = kMaxCand + 1;
    if (kk <= 32) {
        uint32_t most = key[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) most = max(most, key[j]);
        int rank = 0;
#pragma unroll
        for (int o = 0; o < 32; ++o) {
            const uint32_t other = __shfl_sync(0xFFFFFFFFu, most, o);
            rank += other > most || (other == most && o < lane);
        }
        const uint32_t bound = max(__shfl_sync(0xFFFFFFFFu, most, __ffs(__ballot_sync(0xFFFFFFFFu, rank == kk - 1)) - 1), 1u);
        n_top = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t bal = __ballot_sync(0xFFFFFFFFu, key[j] >= bound);
            const int at = n_top + __popc(bal & ((1u << lane) - 1u));
            if (key[j] >= bound && at < kMaxCand) {
                sel.key[at] = key[j];
                sel.cand[at] = static_cast<int16_t>(lane + 32 * j);
            }
            n_top += __popc(bal);
        }
        __syncwarp();
    }
    if (n_top <= kMaxCand) {
        for (int i = lane; i < n_top; i += 32) {
            const uint32_t mine = sel.key[i];
            const int e = sel.cand[i];
            int rank = 0;
            for (int o = 0; o < n_top; ++o) rank += sel.key[o] > mine || (sel.key[o] == mine && sel.cand[o] < e);
            if (rank < kk) {
                sel.value[rank] = key_value(mine);
                sel.expert[rank] = static_cast<int16_t>(e);
            }
        }
    } else {
        // many equal logits (or 32 experts to choose): every lane holds its best,
        // the warp's best of them is taken round by round
        uint32_t best;
        int best_j;
        auto rescan = [&]() {
            uint32_t m[PER];
            int at[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) m[j] = key[j];
#pragma unroll
            for (int w = PER / 2; w > 0; w /= 2)
#pragma unroll
                for (int j = 0; j < w; ++j) m[j] = max(m[j], m[j + w]);
            best = m[0];
#pragma unroll
            for (int j = 0; j < PER; ++j) at[j] = key[j] == best ? j : PER;
#pragma unroll
            for (int w = PER / 2; w > 0; w /= 2)
#pragma unroll
                for (int j = 0; j < w; ++j) at[j] = min(at[j], at[j + w]);
            best_j = at[0];
        };
        rescan();
        for (int r = 0; r < kk; ++r) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, best == top);
            int e = best_j * 32 + lane;
            if (who & (who - 1))  // several lanes: the lowest expert of them
                e = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, best == top ? static_cast<uint32_t>(e) : 0xFFFFFFFFu));
            if (best == top && e == best_j * 32 + lane) {
                sel.value[r] = key_value(top);
                sel.expert[r] = static_cast<int16_t>(e);
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (j == best_j) key[j] = 0;
                rescan();
            }
        }
    }
    __syncwarp();
    const float largest = sel.value[0];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (lane + 32 * j < p.E) sum += expf(v[j] - largest);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);

    // near ties: order them by their exact values (no order among infinite sums)
    const float tol = largest_s < 0x7F800000u ? __uint_as_float(largest_s) * p.tie : 0.0f;
    const uint32_t gaps = __ballot_sync(0xFFFFFFFFu, lane + 1 < kk && sel.value[lane] - sel.value[lane + 1] < tol);
    if (gaps != 0 && (gaps >> (p.k - 1) & 1) == 0) {  // among the chosen: lane r holds the r-th
        const int e = lane < p.k ? sel.expert[lane] : 0;
        Exact d = {lane < p.k ? sel.value[lane] : 0.0f, 0.0f};
        for (uint32_t near = gaps | gaps << 1; near != 0;) {
            const int r0 = __ffs(near) - 1;
            near &= near - 1;
            const int r1 = near != 0 ? __ffs(near) - 1 : r0;
            near &= near - 1;
            Exact both[2];
            exact_logits(p, m, __shfl_sync(0xFFFFFFFFu, e, r0), __shfl_sync(0xFFFFFFFFu, e, r1), lane, both);
            if (lane == r0) d = both[0];
            if (lane == r1) d = both[1];
        }
        int rank = 0;
#pragma unroll 1
        for (int o = 0; o < p.k; ++o) {
            const Exact b = d.shfl(o);
            const int eb = __shfl_sync(0xFFFFFFFFu, e, o);
            rank += b > d || (b == d && eb < e) || (d.nan() && (!b.nan() || o < lane));
        }
        if (lane < p.k) {
            sel.expert[rank] = static_cast<int16_t>(e);
            sel.value[rank] = d.hi;
        }
        __syncwarp();
    } else if (gaps != 0) {  // at their end too: any other expert may belong to them
        // the candidates in ascending order, each put in its place among the
        // best so far: lane i holds the i-th
        float floor_v = sel.value[p.k - 1];
        floor_v = floor_v == floor_v ? floor_v - tol : __uint_as_float(0xFF800000u);
        Exact held = {0.0f, 0.0f};
        int held_e = -1, n = 0;
        for (int j = 0; 32 * j < p.E; ++j) {
            float mine = v[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) mine = i == j ? v[i] : mine;
            uint32_t left = __ballot_sync(0xFFFFFFFFu, lane + 32 * j < p.E && mine >= floor_v);
            while (left) {
                const int src = __ffs(left) - 1, e = 32 * j + src;
                left &= left - 1;
                const float c = __shfl_sync(0xFFFFFFFFu, mine, src);
                bool near = false;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    near |= lane + 32 * i < p.E && fabsf(v[i] - c) < tol && lane + 32 * i != e;
                Exact d = {c, 0.0f};
                if (__any_sync(0xFFFFFFFFu, near)) {
                    Exact both[2];
                    exact_logits(p, m, e, e, lane, both);
                    d = both[0];
                }
                // behind those at least as large: they have lower indices
                const int at = __popc(__ballot_sync(0xFFFFFFFFu, lane < n && !(d > held)));
                const Exact prev = {__shfl_up_sync(0xFFFFFFFFu, held.hi, 1), __shfl_up_sync(0xFFFFFFFFu, held.lo, 1)};
                const int prev_e = __shfl_up_sync(0xFFFFFFFFu, held_e, 1);
                if (lane >= at) held = lane == at ? d : prev, held_e = lane == at ? e : prev_e;
                n = min(n + 1, 32);
            }
        }
        if (lane < min(n, p.k)) {  // (fewer where the rest are NaN: those keep their places)
            sel.expert[lane] = static_cast<int16_t>(held_e);
            sel.value[lane] = held.hi;
        }
        __syncwarp();
    }

    float chosen = 0.0f;
    for (int r = lane; r < p.k; r += 32) chosen += expf(sel.value[r] - largest);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) chosen += __shfl_xor_sync(0xFFFFFFFFu, chosen, off);
    const float denom = sum != sum ? sum : (p.renorm ? chosen : sum);
    for (int r = lane; r < p.k; r += 32) {
        p.ids[m * p.S + r] = sel.expert[r];
        p.weights[m * p.S + r] = expf(sel.value[r] - largest) / denom;
    }
    if (p.shared && lane == 0) {
        float g = 1.0f;
        if (p.shared == FP8BS_ROUTE_SHARED_GATE) {
            float l = 0.0f;
            for (int ks = 0; ks < p.KS; ++ks) l += __ldcg(p.part + (static_cast<int64_t>(ks) * p.M + m) * p.pitch + p.E);
            g = 1.0f / (1.0f + expf(-l));
        }
        p.ids[m * p.S + p.k] = p.E;
        p.weights[m * p.S + p.k] = g;
    }
    __syncwarp();
}

__device__ void select_any(const RouteParams& p, Select& sel, int m, int lane) {
    if (p.E <= 256)
        select_token<8>(p, sel, m, lane);
    else if (p.E <= 512)
        select_token<16>(p, sel, m, lane);
    else
        select_token<FP8BS_ROUTE_MAX_E / 32>(p, sel, m, lane);
}

// Eight numbers in pairs: three roundings on any path.
template <typename F>
__device__ __forceinline__ float sum8(F at) {
    static_assert(kWarps == 8, "a number a warp");
    return ((at(0) + at(1)) + (at(2) + at(3))) + ((at(4) + at(5)) + (at(6) + at(7)));
}

// NT: tiles of 8 tokens taken together (their operands are in flight together).
template <int NT, bool LAST>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const __grid_constant__ RouteParams p) {
    constexpr int kTok = 8 * NT, kPitch = kTok + 1;
    __shared__ float red[kWarps][kTileRows][kPitch];
    __shared__ float red_s[kWarps][kTok];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.x / p.KS, ks = blockIdx.x - tile * p.KS;
    const int chunks = p.H / kChunk;
    const int r0 = min(tile * kTileRows + g, p.rows - 1), r1 = min(tile * kTileRows + g + 8, p.rows - 1);
    const uint16_t* w0 = p.w + static_cast<int64_t>(r0) * p.H + 8 * t;
    const uint16_t* w1 = p.w + static_cast<int64_t>(r1) * p.H + 8 * t;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (int m0 = 0; m0 < p.M; m0 += kTok) {
        float acc[NT][4] = {}, mag[NT][4] = {};
        for (int c = ks * kWarps + warp; c < chunks; c += p.KS * kWarps) {
            uint4 a0[4], a1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a0[i] = ptx::ld_global_v4(w0 + c * kChunk + 32 * i);
                a1[i] = ptx::ld_global_v4(w1 + c * kChunk + 32 * i);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                // columns past M repeat the last token and are not stored
                const uint16_t* x = p.x + min(m0 + 8 * j + g, p.M - 1) * p.ldx + c * kChunk + 8 * t;
                uint4 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const uint4*>(x + 32 * i);
                float part[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float other[4];
                    mma16816_bf16_zero(part[i], a0[i].x, a1[i].x, a0[i].y, a1[i].y, b[i].x, b[i].y);
                    mma16816_bf16_zero(other, a0[i].z, a1[i].z, a0[i].w, a1[i].w, b[i].z, b[i].w);
#pragma unroll
                    for (int q = 0; q < 4; ++q) part[i][q] += other[q];
                    const uint4 ma = magnitudes(a0[i]), mb = magnitudes(a1[i]), mx = magnitudes(b[i]);
                    mma16816_bf16(mag[j], ma.x, mb.x, ma.y, mb.y, mx.x, mx.y);
                    mma16816_bf16(mag[j], ma.z, mb.z, ma.w, mb.w, mx.z, mx.w);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[j][q] += (part[0][q] + part[1][q]) + (part[2][q] + part[3][q]);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            red[warp][g][8 * j + 2 * t] = acc[j][0];
            red[warp][g][8 * j + 2 * t + 1] = acc[j][1];
            red[warp][g + 8][8 * j + 2 * t] = acc[j][2];
            red[warp][g + 8][8 * j + 2 * t + 1] = acc[j][3];
            // S: the largest of the 16 rows (as bits: NaN above infinity)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t s = max(__float_as_uint(mag[j][q]) & 0x7FFFFFFFu, __float_as_uint(mag[j][q + 2]) & 0x7FFFFFFFu);
#pragma unroll
                for (int off = 4; off < 32; off *= 2) s = max(s, __shfl_xor_sync(0xFFFFFFFFu, s, off));
                if (g == 0) red_s[warp][8 * j + 2 * t + q] = __uint_as_float(s);
            }
        }
        __syncthreads();
        const int n = min(kTok, p.M - m0);
        for (int o = threadIdx.x; o < n * kTileRows; o += kThreads) {
            const int m = o / kTileRows, r = o % kTileRows;
            const float v = sum8([&](int w) { return red[w][r][m]; });
            if (tile * kTileRows + r < p.rows)
                p.part[(static_cast<int64_t>(ks) * p.M + m0 + m) * p.pitch + tile * kTileRows + r] = v;
        }
        if (const int m = kThreads - 1 - static_cast<int>(threadIdx.x); m < n) {
            const float v = sum8([&](int w) { return red_s[w][m]; });
            p.part[(static_cast<int64_t>(ks) * p.M + m0 + m) * p.pitch + p.rows + tile] = v;
        }
        __syncthreads();
    }
    if constexpr (LAST) {
        __shared__ Select sel[kWarps];
        __shared__ int is_last;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) is_last = atomicAdd(p.counter, 1u) == gridDim.x - 1;
        __syncthreads();
        if (!is_last) return;
        __threadfence();
        if (threadIdx.x == 0) *p.counter = 0;
        if (warp < p.M) select_any(p, sel[warp], warp, lane);
    }
}

__global__ void __launch_bounds__(32) moe_select_kernel(const __grid_constant__ RouteParams p) {
    __shared__ Select sel;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    select_any(p, sel, blockIdx.x, threadIdx.x);
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t M, int64_t E, int64_t H) {
    const int64_t rows = E + 1;
    // with and without a gate row: the larger of the two
    const int64_t ks = k_splits(E, H) > k_splits(rows, H) ? k_splits(E, H) : k_splits(rows, H);
    return kHeader + static_cast<size_t>(ks) * M * pitch_of(rows) * sizeof(float);
}

cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t stream) {
    RouteParams p;
    p.x = a.x;
    p.ldx = a.ldx;
    p.w = a.w;
    p.ids = a.ids;
    p.weights = a.weights;
    p.counter = reinterpret_cast<uint32_t*>(a.workspace);
    p.part = reinterpret_cast<float*>(a.workspace + kHeader);
    p.M = a.M;
    p.H = a.H;
    p.E = a.E;
    p.k = a.k;
    p.S = a.k + (a.shared != FP8BS_ROUTE_SHARED_NONE ? 1 : 0);
    p.rows = a.E + (a.shared == FP8BS_ROUTE_SHARED_GATE ? 1 : 0);
    p.tiles = tiles_of(p.rows);
    p.pitch = pitch_of(p.rows);
    p.KS = k_splits(p.rows, a.H);
    // twice the bound of the head comment, and 1 for the comparison's own rounding;
    // S itself is short by at most 8 MMAs' cuts a chunk
    const int chunks = a.H / kChunk, per_warp = (chunks + p.KS * kWarps - 1) / (p.KS * kWarps);
    p.tie = 2.0f * (10 + 3 + (per_warp - 1) + 3 + (p.KS - 1) + 1) * 0x1p-24f * (1.0f + per_warp * 0x1p-16f);
    p.renorm = a.renorm;
    p.shared = a.shared;
    const int grid = p.tiles * p.KS;
    if (a.M <= kOneLaunchM) return launch_dependent(moe_route_kernel<1, true>, grid, kThreads, 0, stream, p);
    const cudaError_t e = a.M <= 16   ? launch_dependent(moe_route_kernel<2, false>, grid, kThreads, 0, stream, p)
                          : a.M <= 32 ? launch_dependent(moe_route_kernel<4, false>, grid, kThreads, 0, stream, p)
                                      : launch_dependent(moe_route_kernel<8, false>, grid, kThreads, 0, stream, p);
    return e != cudaSuccess ? e : launch_dependent(moe_select_kernel, a.M, 32, 0, stream, p);
}

}  // namespace fp8bs
