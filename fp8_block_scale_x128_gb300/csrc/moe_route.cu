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
// launch).  Measured (in a graph, w in the second-level cache): 7.0 us for one
// token of 512 experts, hidden 4096, 7.4 for 9 in two launches, 10.5 for 64; all
// of it is latency: two trips to memory, the arrival, the selection.
//
// The order of the chosen experts is decided by fp32 logits unless two of them
// (or the last chosen and the first left out) are within 2^-20 of the largest
// logit: those are summed again with a compensated sum, which orders them as a
// 64-bit sum would.
#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

using namespace w4;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kOneLaunchM = kWarps;  // a warp per token in the last block
constexpr size_t kHeader = 256;  // workspace: the arrival counter, then the partial logits
constexpr int kTargetBlocks = 152;
constexpr int kMaxCand = 64;

struct RouteParams {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* w;  // [rows, H]
    int32_t* ids;
    float* weights;
    uint32_t* counter;
    float* part;  // [KS][M][rows16]
    int M, H, E, k, S;
    int rows, rows16, KS;
    int renorm, shared;
};

// K slices over blocks: enough blocks for the machine, at least one chunk per warp.
__host__ int k_splits(int64_t rows, int64_t H) {
    const int64_t tiles = (rows + kTileRows - 1) / kTileRows, chunks = H / kChunk;
    const int64_t want = (kTargetBlocks + tiles - 1) / tiles, most = (chunks + kWarps - 1) / kWarps;
    return static_cast<int>(want < most ? want : most);
}

__device__ __forceinline__ void mma16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// x[m] . w[e] with a compensated fp32 sum (products of two bf16 are exact in
// fp32; each addition's rounding error is kept: D. E. Knuth's two-sum), the
// lanes' sums joined in 64 bits.  Every lane returns it.
__device__ double exact_logit(const RouteParams& p, int m, int e, int lane) {
    float s = 0.0f, c = 0.0f;
    const uint16_t *x = p.x + m * p.ldx, *w = p.w + static_cast<int64_t>(e) * p.H;
    for (int k0 = 8 * lane; k0 < p.H; k0 += 4 * 256) {
        uint4 xr[4], wr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + 256 * j;
            xr[j] = wr[j] = make_uint4(0, 0, 0, 0);
            if (k < p.H) xr[j] = *reinterpret_cast<const uint4*>(x + k), wr[j] = ptx::ld_global_v4(w + k);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a[8], b[8];
            unpack8(xr[j], a);
            unpack8(wr[j], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = __fmul_rn(a[i], b[i]), t = __fadd_rn(s, v), z = __fsub_rn(t, s);
                c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(v, z)));
                s = t;
            }
        }
    }
    double d = static_cast<double>(s) + static_cast<double>(c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, off);
    return d;
}

// A warp's scratch.
struct Select {
    double cand_value[kMaxCand];
    uint32_t key[kMaxCand];
    float value[FP8BS_ROUTE_MAX_K + 1];
    int16_t expert[FP8BS_ROUTE_MAX_K + 1];
    int16_t cand[kMaxCand];
};

// The k + 1 largest of a token's logits in order, by one warp.  v[j]: expert
// lane + 32 j.
template <int PER>
__device__ void select_token(const RouteParams& p, Select& sel, int m, int lane) {
    float v[PER];
    uint32_t key[PER];
    uint32_t top_abs = 0;
    const float* part = p.part + static_cast<int64_t>(m) * p.rows16 + lane;
    const int64_t pitch = static_cast<int64_t>(p.M) * p.rows16;
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = 0.0f;
    // four slices' loads in flight together, added in slice order
    for (int ks = 0; ks < p.KS; ks += 4) {
        float u[4][PER];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < PER; ++j)
                u[i][j] = ks + i < p.KS && lane + 32 * j < p.E ? __ldcg(part + (ks + i) * pitch + 32 * j) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < PER; ++j) v[j] += u[i][j];
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const bool in = lane + 32 * j < p.E;
        key[j] = in ? order_key(v[j]) : 0;
        if (in) top_abs = max(top_abs, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
    top_abs = __reduce_max_sync(0xFFFFFFFFu, top_abs);
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

    // near ties: order them by their exact values
    const float tol = top_abs < 0x7F800000u ? __uint_as_float(top_abs) * 0x1p-20f : 0.0f;
    bool close = false;
    for (int r = lane; r + 1 < kk; r += 32) close |= sel.value[r] - sel.value[r + 1] < tol;
    if (__any_sync(0xFFFFFFFFu, close)) {
        const float floor_v = sel.value[p.k - 1] - tol;
        int n = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const bool in = lane + 32 * j < p.E && v[j] >= floor_v;
            const uint32_t bal = __ballot_sync(0xFFFFFFFFu, in);
            const int at = n + __popc(bal & ((1u << lane) - 1u));
            if (in && at < kMaxCand) {
                sel.cand[at] = static_cast<int16_t>(lane + 32 * j);
                sel.cand_value[at] = v[j];
            }
            n += __popc(bal);
        }
        __syncwarp();
        if (n <= kMaxCand) {
            uint64_t unclear = 0;
            for (int i = 0; i < n; ++i) {
                bool near = false;
                for (int o = lane; o < n; o += 32)
                    near |= o != i && fabs(sel.cand_value[i] - sel.cand_value[o]) < tol;
                if (__any_sync(0xFFFFFFFFu, near)) unclear |= uint64_t(1) << i;
            }
            __syncwarp();
            for (int i = 0; i < n; ++i)
                if (unclear >> i & 1) {
                    const double d = exact_logit(p, m, sel.cand[i], lane);
                    if (lane == 0) sel.cand_value[i] = d;
                }
            __syncwarp();
            // the candidates are in ascending blocks of 32 experts, not sorted: rank each one
            for (int i = lane; i < n; i += 32) {
                const double a = sel.cand_value[i];
                const int e = sel.cand[i];
                int rank = 0;
                for (int o = 0; o < n; ++o) {
                    const double b = sel.cand_value[o];
                    rank += b > a || (b == a && sel.cand[o] < e);
                }
                if (rank < p.k) {
                    sel.expert[rank] = static_cast<int16_t>(e);
                    sel.value[rank] = static_cast<float>(a);
                }
            }
            __syncwarp();
        }
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
            for (int ks = 0; ks < p.KS; ++ks) l += __ldcg(p.part + (static_cast<int64_t>(ks) * p.M + m) * p.rows16 + p.E);
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

// NT: tiles of 8 tokens taken together (their operands are in flight together).
template <int NT, bool LAST>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const __grid_constant__ RouteParams p) {
    constexpr int kTok = 8 * NT, kPitch = kTok + 1;
    __shared__ float red[kWarps][kTileRows][kPitch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.x / p.KS, ks = blockIdx.x - tile * p.KS;
    const int chunks = p.H / kChunk;
    const int r0 = min(tile * kTileRows + g, p.rows - 1), r1 = min(tile * kTileRows + g + 8, p.rows - 1);
    const uint16_t* w0 = p.w + static_cast<int64_t>(r0) * p.H + 8 * t;
    const uint16_t* w1 = p.w + static_cast<int64_t>(r1) * p.H + 8 * t;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (int m0 = 0; m0 < p.M; m0 += kTok) {
        float acc[NT][4] = {};
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
                float part[4] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma16816_bf16(part, a0[i].x, a1[i].x, a0[i].y, a1[i].y, b[i].x, b[i].y);
                    mma16816_bf16(part, a0[i].z, a1[i].z, a0[i].w, a1[i].w, b[i].z, b[i].w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] += part[i];
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            red[warp][g][8 * j + 2 * t] = acc[j][0];
            red[warp][g][8 * j + 2 * t + 1] = acc[j][1];
            red[warp][g + 8][8 * j + 2 * t] = acc[j][2];
            red[warp][g + 8][8 * j + 2 * t + 1] = acc[j][3];
        }
        __syncthreads();
        const int n = min(kTok, p.M - m0);
        for (int o = threadIdx.x; o < n * kTileRows; o += kThreads) {
            const int m = o / kTileRows, r = o % kTileRows;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[w][r][m];
            p.part[(static_cast<int64_t>(ks) * p.M + m0 + m) * p.rows16 + tile * kTileRows + r] = v;
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
    const int64_t rows = E + 1, rows16 = (rows + kTileRows - 1) / kTileRows * kTileRows;
    // with and without a gate row: the larger of the two
    const int64_t ks = k_splits(E, H) > k_splits(rows, H) ? k_splits(E, H) : k_splits(rows, H);
    return kHeader + static_cast<size_t>(ks) * M * rows16 * sizeof(float);
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
    p.rows16 = (p.rows + kTileRows - 1) / kTileRows * kTileRows;
    p.KS = k_splits(p.rows, a.H);
    p.renorm = a.renorm;
    p.shared = a.shared;
    const int grid = p.rows16 / kTileRows * p.KS;
    if (a.M <= kOneLaunchM) return launch_dependent(moe_route_kernel<1, true>, grid, kThreads, 0, stream, p);
    const cudaError_t e = a.M <= 16   ? launch_dependent(moe_route_kernel<2, false>, grid, kThreads, 0, stream, p)
                          : a.M <= 32 ? launch_dependent(moe_route_kernel<4, false>, grid, kThreads, 0, stream, p)
                                      : launch_dependent(moe_route_kernel<8, false>, grid, kThreads, 0, stream, p);
    return e != cudaSuccess ? e : launch_dependent(moe_select_kernel, a.M, 32, 0, stream, p);
}

}  // namespace fp8bs
