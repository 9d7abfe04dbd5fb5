// Small-batch mixture-of-experts layer on 4-bit weights, two launches.
//
//   h = x[m] . w13[e]^T              (gate rows 0..I-1 over up rows I..2I-1)
//   a = silu(h_gate) * h_up          (fp32, kept in the workspace)
//   y[m] = bf16(sum over s, in slot order, of tw[m, s] * (a . w2[e]^T))
//
// 1. gate/up: items of (expert, up to 8 of its pairs, 16 gate rows and the 16
//    up rows that go with them); the 8 warps of a block split H, their sums are
//    added in warp order and the activation applied to the whole sum.
// 2. down: a block owns 16 rows of the output for every token, its warps deal
//    out the experts; the pairs' products meet in shared memory and are summed
//    in slot order.  No partial sums in global memory, no atomics on values.
//
// An expert's codes are read once for up to 8 pairs.  Every block builds the
// expert lists itself: a histogram of the routed pairs and its running sums.
// The second launch is a programmatic dependent one: its lists and its first
// codes do not wait for the first.
#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

using namespace w4;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBatch = 8;  // pairs of an entry: the token columns of one MMA
constexpr size_t kHeader = 256;  // workspace: the device error word, then a

struct MoeParams {
    const uint16_t* x;  // [M, H] bf16, row pitch ldx
    int64_t ldx;
    const int32_t* ids;  // [M, S]
    const float* tw;     // [M, S]
    const uint8_t* w13;  // [E, 2I, H/2]
    const uint8_t* s13;
    const uint8_t* w2;  // [E, H, I/2]
    const uint8_t* s2;
    uint16_t* y;    // [M, H]
    uint32_t* err;  // workspace error word
    float* a;       // [M*S][I]
    int M, S, H, I, E;
};

// Shared-memory tables of the routed pairs, built by every block.
struct Lists {
    int n_entries;
    int sums[kWarps];
    int16_t pairs[FP8BS_MOE_MAX_PAIRS];        // pairs grouped by expert, ascending experts
    int16_t unsorted[FP8BS_MOE_MAX_PAIRS];     // of experts with more than one entry
    int16_t entry_expert[FP8BS_MOE_MAX_PAIRS];
    int16_t entry_first[FP8BS_MOE_MAX_PAIRS];  // into pairs
    int8_t entry_n[FP8BS_MOE_MAX_PAIRS];       // 1..kBatch
};

// counts: E ints of shared memory, free afterwards.  The order of the pairs of
// an expert with one entry may differ between blocks and runs: it only decides
// which MMA column serves a pair, and columns do not mix.  An expert with more
// pairs has them sorted, so that every block splits them into the same entries.
__device__ void build_lists(const MoeParams& p, Lists& L, int* counts) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.M * p.S;
    constexpr int kMine = FP8BS_MOE_MAX_PAIRS / kThreads;
    int id[kMine], rank[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int q = tid + j * kThreads;
        id[j] = q < P ? p.ids[q] : -1;
        if (q < P && (id[j] < 0 || id[j] >= p.E)) {
            record_error(p.err, FP8BS_ERR_DEVICE);
            id[j] = -1;
        }
    }
    for (int e = tid; e < p.E; e += kThreads) counts[e] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j) rank[j] = id[j] >= 0 ? atomicAdd(&counts[id[j]], 1) : 0;
    __syncthreads();
    // running sums over the experts: pairs in the low half, entries in the high one
    const int per = (p.E + kThreads - 1) / kThreads;
    const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += counts[e] | ((counts[e] + kBatch - 1) / kBatch << 16);
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) L.sums[warp] = incl;
    __syncthreads();
    int at = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) at += L.sums[w];
    if (tid == kThreads - 1) L.n_entries = (at + mine) >> 16;
    for (int e = e0; e < e1; ++e) {
        const int n = counts[e], first = at & 0xFFFF;
        counts[e] = first | n << 16;
        for (int b = 0; b * kBatch < n; ++b) {
            const int i = (at >> 16) + b;
            L.entry_expert[i] = static_cast<int16_t>(e);
            L.entry_first[i] = static_cast<int16_t>(first + b * kBatch);
            L.entry_n[i] = static_cast<int8_t>(min(n - b * kBatch, kBatch));
        }
        at += n | ((n + kBatch - 1) / kBatch << 16);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j)
        if (id[j] >= 0) {
            const int c = counts[id[j]];
            (c >> 16 > kBatch ? L.unsorted : L.pairs)[(c & 0xFFFF) + rank[j]] = static_cast<int16_t>(tid + j * kThreads);
        }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j)
        if (id[j] >= 0 && counts[id[j]] >> 16 > kBatch) {
            const int n = counts[id[j]] >> 16, first = counts[id[j]] & 0xFFFF, q = tid + j * kThreads;
            int r = 0;
            for (int i = 0; i < n; ++i) r += L.unsorted[first + i] < q;
            L.pairs[first + r] = static_cast<int16_t>(q);
        }
    __syncthreads();
}

__host__ __device__ constexpr int lists_bytes() { return (sizeof(Lists) + 15) / 16 * 16; }
__host__ __device__ constexpr int counts_bytes(int E) { return (E * 4 + 15) / 16 * 16; }

template <int GP, int PC>
__host__ __device__ constexpr int warp_bytes(int n) {
    using S = Stage<GP, PC>;
    return 2 * S::kCodeBytes + S::kScaleTableBytes + n * (S::kTokenPitch + 16);
}

// ---- 1. gate / up ------------------------------------------------------------
constexpr int kUpPC = 4;
constexpr int kRedBytes = kWarps * 2 * kTileRows * kBatch * 4;

template <int FMT, int GP>
__global__ void __launch_bounds__(kThreads, 2) moe_w4_up_kernel(const __grid_constant__ MoeParams p) {
    constexpr int PC = kUpPC, SB = Format<FMT, GP>::kScaleBytes;
    using S = Stage<GP, PC>;
    extern __shared__ __align__(16) uint8_t smem[];
    Lists& L = *reinterpret_cast<Lists*>(smem);
    float* red = reinterpret_cast<float*>(smem + lists_bytes());  // [kWarps][2][16][kBatch]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nmax = min(p.M * p.S, kBatch);
    uint8_t* base = smem + lists_bytes() + kRedBytes;
    uint8_t* codes = base + warp * warp_bytes<GP, PC>(nmax);
    float* table = reinterpret_cast<float*>(codes + 2 * S::kCodeBytes);
    uint8_t* xs = codes + 2 * S::kCodeBytes + S::kScaleTableBytes;
    float* xinv = reinterpret_cast<float*>(xs + nmax * S::kTokenPitch);
    build_lists(p, L, reinterpret_cast<int*>(base));
    ptx::griddep_launch_dependents();

    const int chunks = p.H / kChunk, slice = (chunks + kWarps - 1) / kWarps, pieces = (slice + PC - 1) / PC;
    const int first = warp * slice, last = min(first + slice, chunks);
    const int per = p.I / kTileRows, items = L.n_entries * per;
    const int64_t ldc = p.H / 2, lds = static_cast<int64_t>(chunks) * SB;

    RawScales<PC> raw = {};
    // stage u of an item: piece u / 2, gate (0) or up (1) rows u % 2
    auto issue = [&](int item, int u, int b) {
        const int c = first + u / 2 * PC, nch = min(last - c, PC);
        if (item < items && nch > 0) {
            const int entry = item / per, j = item - entry * per;
            const int64_t row = static_cast<int64_t>(L.entry_expert[entry]) * 2 * p.I + (u & 1) * p.I + j * kTileRows;
            load_codes<GP, PC>(codes + b * S::kCodeBytes, p.w13 + row * ldc + c * 64, ldc, kTileRows, nch, lane);
            raw = load_scales<FMT, GP, PC>(p.s13 + row * lds + c * SB, lds, kTileRows, nch, lane);
        }
        cp_async_commit();
    };
    issue(blockIdx.x, 0, 0);
    int b = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int entry = item / per, j = item - entry * per;
        const int n = L.entry_n[entry], pf = L.entry_first[entry];
        float tot[2][4] = {};
        for (int piece = 0; piece < pieces; ++piece) {
            const int c = first + piece * PC, nch = min(last - c, PC);
#pragma unroll
            for (int half = 0; half < 2; ++half, b ^= 1) {
                const RawScales<PC> cur = raw;
                const int u = 2 * piece + half + 1;
                const bool more = u < 2 * pieces;
                issue(more ? item : item + static_cast<int>(gridDim.x), more ? u : 0, b ^ 1);
                if (nch > 0) {
                    if (half == 0)
                        for (int i = 0; i < n; ++i) {
                            const int m = L.pairs[pf + i] / p.S;
                            const float inv = stage_token_bf16<FMT, PC>(xs + i * S::kTokenPitch, p.x + m * p.ldx + c * kChunk, nch, lane);
                            if (lane == 0) xinv[i] = inv;
                        }
                    const float back = store_scales<FMT, GP, PC>(table, cur, lane);
                    cp_async_wait<1>();
                    __syncwarp();
                    float acc[1][4] = {};
                    stage_mma<FMT, GP, PC, 1>(acc, codes + b * S::kCodeBytes, table, xs, n, nch, lane);
                    const int col = 2 * (lane & 3);
                    const float i0 = xinv[min(col, n - 1)], i1 = xinv[min(col + 1, n - 1)];
                    add_stage(tot[half], acc[0], i0, i1, back);
                }
                __syncwarp();
            }
        }
        float* r = red + (warp * 2 * kTileRows + (lane >> 2)) * kBatch + 2 * (lane & 3);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            *reinterpret_cast<float2*>(r + half * kTileRows * kBatch) = make_float2(tot[half][0], tot[half][1]);
            *reinterpret_cast<float2*>(r + (half * kTileRows + 8) * kBatch) = make_float2(tot[half][2], tot[half][3]);
        }
        __syncthreads();
        if (threadIdx.x < kTileRows * kBatch) {
            const int i = threadIdx.x / kTileRows, row = threadIdx.x % kTileRows;
            if (i < n) {
                float g = 0.0f, v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    g += red[(w * 2 * kTileRows + row) * kBatch + i];
                    v += red[((w * 2 + 1) * kTileRows + row) * kBatch + i];
                }
                p.a[static_cast<int64_t>(L.pairs[pf + i]) * p.I + j * kTileRows + row] = g / (1.0f + expf(-g)) * v;
            }
        }
        __syncthreads();  // red is rewritten by the next item
    }
}

// ---- 2. down -----------------------------------------------------------------
template <int FMT, int GP, int PC>
__global__ void __launch_bounds__(kThreads, 2) moe_w4_down_kernel(const __grid_constant__ MoeParams p) {
    constexpr int SB = Format<FMT, GP>::kScaleBytes;
    using S = Stage<GP, PC>;
    extern __shared__ __align__(16) uint8_t smem[];
    Lists& L = *reinterpret_cast<Lists*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.M * p.S, nmax = min(P, kBatch);
    float* out = reinterpret_cast<float*>(smem + lists_bytes());  // [P][16]
    uint8_t* base = smem + lists_bytes() + P * kTileRows * 4;
    uint8_t* codes = base + warp * warp_bytes<GP, PC>(nmax);
    float* table = reinterpret_cast<float*>(codes + 2 * S::kCodeBytes);
    uint8_t* xs = codes + 2 * S::kCodeBytes + S::kScaleTableBytes;
    float* xinv = reinterpret_cast<float*>(xs + nmax * S::kTokenPitch);
    build_lists(p, L, reinterpret_cast<int*>(base));

    const int chunks = p.I / kChunk, pieces = (chunks + PC - 1) / PC;
    const int64_t ldc = p.I / 2, lds = static_cast<int64_t>(chunks) * SB;
    const int tiles = p.H / kTileRows;
    RawScales<PC> raw = {};
    auto issue = [&](int tile, int entry, int piece, int b) {
        if (tile < tiles && entry < L.n_entries) {
            const int c = piece * PC, nch = min(chunks - c, PC);
            const int64_t row = static_cast<int64_t>(L.entry_expert[entry]) * p.H + tile * kTileRows;
            load_codes<GP, PC>(codes + b * S::kCodeBytes, p.w2 + row * ldc + c * 64, ldc, kTileRows, nch, lane);
            raw = load_scales<FMT, GP, PC>(p.s2 + row * lds + c * SB, lds, kTileRows, nch, lane);
        }
        cp_async_commit();
    };
    issue(blockIdx.x, warp, 0, 0);
    ptx::griddep_wait();
    int b = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        for (int q = tid; q < P * kTileRows; q += kThreads) out[q] = 0.0f;  // pairs with an invalid id stay 0
        __syncthreads();
        for (int entry = warp; entry < L.n_entries; entry += kWarps) {
            const int n = L.entry_n[entry], pf = L.entry_first[entry];
            float tot[4] = {};
            for (int piece = 0; piece < pieces; ++piece, b ^= 1) {
                const int c = piece * PC, nch = min(chunks - c, PC);
                const RawScales<PC> cur = raw;
                if (piece + 1 < pieces)
                    issue(tile, entry, piece + 1, b ^ 1);
                else if (entry + kWarps < L.n_entries)
                    issue(tile, entry + kWarps, 0, b ^ 1);
                else
                    issue(tile + gridDim.x, warp, 0, b ^ 1);
                for (int i = 0; i < n; ++i) {
                    const float inv = stage_token_f32<FMT, PC>(xs + i * S::kTokenPitch, p.a + static_cast<int64_t>(L.pairs[pf + i]) * p.I + c * kChunk, nch, lane);
                    if (lane == 0) xinv[i] = inv;
                }
                const float back = store_scales<FMT, GP, PC>(table, cur, lane);
                cp_async_wait<1>();
                __syncwarp();
                float acc[1][4] = {};
                stage_mma<FMT, GP, PC, 1>(acc, codes + b * S::kCodeBytes, table, xs, n, nch, lane);
                const int col = 2 * (lane & 3);
                const float i0 = xinv[min(col, n - 1)], i1 = xinv[min(col + 1, n - 1)];
                add_stage(tot, acc[0], i0, i1, back);
                __syncwarp();
            }
            const int col = 2 * (lane & 3), row = lane >> 2;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (col + h < n) {
                    float* o = out + L.pairs[pf + col + h] * kTileRows + row;
                    o[0] = tot[h];
                    o[8] = tot[2 + h];
                }
        }
        __syncthreads();
        for (int o = tid; o < p.M * kTileRows; o += kThreads) {
            const int m = o / kTileRows, row = o % kTileRows;
            float v = 0.0f;
            for (int s = 0; s < p.S; ++s) {
                const int q = m * p.S + s, e = p.ids[q];
                if (e >= 0 && e < p.E) v = fmaf(p.tw[q], out[q * kTileRows + row], v);
            }
            p.y[static_cast<int64_t>(m) * p.H + tile * kTileRows + row] = to_bf16(v);
        }
        __syncthreads();  // out is cleared for the next tile
    }
}

cudaError_t launch_pdl(void (*kernel)(MoeParams), const MoeParams& p, int grid, int smem, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int FMT, int GP>
cudaError_t launch_up(const MoeParams& p, int sm_count, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(moe_w4_up_kernel<FMT, GP>, allowed);
    if (e != cudaSuccess) return e;
    const int P = p.M * p.S;
    const int smem = lists_bytes() + kRedBytes + max(counts_bytes(p.E), kWarps * warp_bytes<GP, kUpPC>(min(P, kBatch)));
    const int per_sm = min(2, kMaxSmShared / (smem + 1024));
    const int grid = static_cast<int>(min(static_cast<int64_t>(P) * (p.I / kTileRows), static_cast<int64_t>(sm_count) * per_sm));
    return launch_pdl(moe_w4_up_kernel<FMT, GP>, p, grid, smem, false, stream);
}

template <int FMT, int GP, int PC>
cudaError_t launch_down(const MoeParams& p, int sm_count, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(moe_w4_down_kernel<FMT, GP, PC>, allowed);
    if (e != cudaSuccess) return e;
    const int P = p.M * p.S;
    const int smem = lists_bytes() + P * kTileRows * 4 + max(counts_bytes(p.E), kWarps * warp_bytes<GP, PC>(min(P, kBatch)));
    const int per_sm = min(2, kMaxSmShared / (smem + 1024));
    return launch_pdl(moe_w4_down_kernel<FMT, GP, PC>, p, min(p.H / kTileRows, sm_count * per_sm), smem, true, stream);
}

}  // namespace

size_t moe_w4_workspace_bytes(int64_t M, int64_t S, int64_t I) {
    return kHeader + static_cast<size_t>(M) * S * I * sizeof(float);
}

cudaError_t launch_moe_w4(const MoeW4Args& a, cudaStream_t stream) {
    MoeParams p;
    p.x = a.x;
    p.ldx = a.ldx;
    p.ids = a.ids;
    p.tw = a.tw;
    p.w13 = a.w13;
    p.s13 = a.s13;
    p.w2 = a.w2;
    p.s2 = a.s2;
    p.y = a.y;
    p.err = reinterpret_cast<uint32_t*>(a.workspace);
    p.a = reinterpret_cast<float*>(a.workspace + kHeader);
    p.M = a.M;
    p.S = a.S;
    p.H = a.H;
    p.I = a.I;
    p.E = a.E;
    return dispatch_format(a.format, a.group, [&](auto fmt, auto gp) {
        const cudaError_t e = launch_up<fmt(), gp()>(p, a.sm_count, stream);
        if (e != cudaSuccess) return e;
        if (p.I == 128) return launch_down<fmt(), gp(), 1>(p, a.sm_count, stream);
        if (p.I == 256) return launch_down<fmt(), gp(), 2>(p, a.sm_count, stream);
        return launch_down<fmt(), gp(), 4>(p, a.sm_count, stream);
    });
}

}  // namespace fp8bs
