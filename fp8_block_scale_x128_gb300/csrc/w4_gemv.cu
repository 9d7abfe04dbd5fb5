// y[M, N] = bf16(x . W^T) for up to 16 bf16 tokens and a 4-bit weight.
//
// One warp works on 16 weight rows and a slice of K (w4.cuh).  The warps of a
// block are WK slices of K times WR row tiles; each warp keeps its slice of x
// (fp16, staged once where it fits) and streams codes through a two-stage ring
// of its own, so the only block-wide steps are the sums over the slices, in
// slice order: repeated calls give the same bits.  A persistent grid deals out
// the row tiles.
#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

using namespace w4;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

struct GemvParams {
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* codes;
    int64_t ldc;
    const uint8_t* scales;
    int64_t lds;
    uint16_t* y;
    int64_t ldy;
    int M, N, chunks;  // chunks of 128 k
    int WK;            // K slices (a power of two, at most kWarps)
    int slice;         // chunks of a slice
    int pieces;        // stages of a slice
    int resident;      // whether the whole slice of x stays staged
    int pdl;
};

template <int GP, int PC>
__host__ __device__ constexpr int warp_bytes(int M, int staged_pieces) {
    using S = Stage<GP, PC>;
    return 2 * S::kCodeBytes + S::kScaleTableBytes + staged_pieces * M * (S::kTokenPitch + 16);
}
template <int NT>
constexpr int reduce_bytes() {
    return kWarps * kTileRows * 8 * NT * 4;
}

// PC chunks a stage, NT tiles of 8 token columns.
template <int FMT, int GP, int PC, int NT>
__global__ void __launch_bounds__(kThreads, 2) gemv_w4_kernel(const __grid_constant__ GemvParams p) {
    using S = Stage<GP, PC>;
    constexpr int SB = Format<FMT, GP>::kScaleBytes;
    extern __shared__ __align__(16) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem);  // [kWarps][16][8 NT]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wk = warp & (p.WK - 1), wr = warp / p.WK, WR = kWarps / p.WK;
    const int staged = p.resident ? p.pieces : 1;
    uint8_t* mine = smem + reduce_bytes<NT>() + warp * warp_bytes<GP, PC>(p.M, staged);
    uint8_t* codes = mine;                                                  // [2][kCodeBytes]
    float* table = reinterpret_cast<float*>(mine + 2 * S::kCodeBytes);      // scales
    uint8_t* xs = mine + 2 * S::kCodeBytes + S::kScaleTableBytes;           // [staged][M][kTokenPitch]
    float* xinv = reinterpret_cast<float*>(xs + staged * p.M * S::kTokenPitch);  // [staged][M] (16-byte slots)

    const int first = wk * p.slice, last = min(first + p.slice, p.chunks);
    const int tiles = (p.N + kTileRows - 1) / kTileRows;
    const int rounds = (tiles + WR - 1) / WR;

    RawScales<PC> raw = {};
    // start stage (round, piece) into ring slot b
    auto issue = [&](int round, int piece, int b) {
        const int tile = round * WR + wr, c = first + piece * PC, nch = min(last - c, PC);
        if (round < rounds && tile < tiles && nch > 0) {
            const int64_t row = static_cast<int64_t>(tile) * kTileRows;
            const int rows = min(p.N - tile * kTileRows, kTileRows);
            load_codes<GP, PC>(codes + b * S::kCodeBytes, p.codes + row * p.ldc + c * 64, p.ldc, rows, nch, lane);
            raw = load_scales<FMT, GP, PC>(p.scales + row * p.lds + c * SB, p.lds, rows, nch, lane);
        }
        cp_async_commit();
    };
    auto stage_x = [&](int piece, int slot) {
        const int c = first + piece * PC, nch = min(last - c, PC);
        if (nch <= 0) return;
        for (int m = 0; m < p.M; ++m) {
            const float inv = stage_token_bf16<FMT, PC>(xs + (slot * p.M + m) * S::kTokenPitch, p.x + m * p.ldx + c * kChunk, nch, lane);
            if (lane == 0) xinv[slot * p.M + m] = inv;
        }
    };

    issue(blockIdx.x, 0, 0);
    if (p.pdl) {
        ptx::griddep_launch_dependents();
        ptx::griddep_wait();
    }
    if (p.resident)
        for (int q = 0; q < p.pieces; ++q) stage_x(q, q);

    int b = 0;
    for (int round = blockIdx.x; round < rounds; round += gridDim.x) {
        const int tile = round * WR + wr;
        float tot[NT][4] = {};
        for (int piece = 0; piece < p.pieces; ++piece, b ^= 1) {
            const int nch = min(last - first - piece * PC, PC);
            const RawScales<PC> cur = raw;
            const bool more = piece + 1 < p.pieces;
            issue(more ? round : round + static_cast<int>(gridDim.x), more ? piece + 1 : 0, b ^ 1);
            if (tile < tiles && nch > 0) {
                const float back = store_scales<FMT, GP, PC>(table, cur, lane);
                if (!p.resident) stage_x(piece, 0);
                cp_async_wait<1>();
                __syncwarp();
                const int slot = p.resident ? piece : 0;
                float acc[NT][4] = {};
                stage_mma<FMT, GP, PC, NT>(acc, codes + b * S::kCodeBytes, table, xs + slot * p.M * S::kTokenPitch, p.M, nch, lane);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int col = 8 * j + 2 * (lane & 3);
                    const float i0 = xinv[slot * p.M + min(col, p.M - 1)], i1 = xinv[slot * p.M + min(col + 1, p.M - 1)];
                    add_stage(tot[j], acc[j], i0, i1, back);
                }
            }
            __syncwarp();  // the slot and the tables are rewritten by the next stage
        }
        // [warp][row][token]
        float* r = red + warp * kTileRows * 8 * NT + (lane >> 2) * 8 * NT + 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            *reinterpret_cast<float2*>(r + 8 * j) = make_float2(tot[j][0], tot[j][1]);
            *reinterpret_cast<float2*>(r + 8 * 8 * NT + 8 * j) = make_float2(tot[j][2], tot[j][3]);
        }
        __syncthreads();
        for (int o = threadIdx.x; o < p.M * WR * kTileRows; o += kThreads) {
            const int m = o / (WR * kTileRows), rr = o - m * WR * kTileRows;
            const int64_t row = static_cast<int64_t>(round) * WR * kTileRows + rr;
            if (row < p.N) {
                const float* s = red + (rr / kTileRows * p.WK * kTileRows + rr % kTileRows) * 8 * NT + m;
                float v = s[0];
                for (int k = 1; k < p.WK; ++k) v += s[k * kTileRows * 8 * NT];
                p.y[m * p.ldy + row] = to_bf16(v);
            }
        }
        __syncthreads();  // red is rewritten by the next round
    }
}

template <int FMT, int GP, int PC, int NT>
cudaError_t launch(const GemvW4Args& a, cudaStream_t stream) {
    GemvParams p;
    p.x = a.x;
    p.ldx = a.ldx;
    p.codes = a.codes;
    p.ldc = a.ldc;
    p.scales = a.scales;
    p.lds = a.lds;
    p.y = a.y;
    p.ldy = a.ldy;
    p.M = a.M;
    p.N = a.N;
    p.chunks = a.K / kChunk;
    p.WK = kWarps;
    while (p.WK > p.chunks) p.WK /= 2;
    p.slice = (p.chunks + p.WK - 1) / p.WK;
    p.pieces = (p.slice + PC - 1) / PC;
    p.pdl = a.pdl;
    auto bytes = [&](int staged) { return reduce_bytes<NT>() + kWarps * warp_bytes<GP, PC>(p.M, staged); };
    p.resident = bytes(p.pieces) <= kMaxBlockShared;
    const int smem = bytes(p.resident ? p.pieces : 1);
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(gemv_w4_kernel<FMT, GP, PC, NT>, allowed);
    if (e != cudaSuccess) return e;
    const int per_sm = min(2, kMaxSmShared / (smem + 1024));
    const int WR = kWarps / p.WK;
    const int rounds = ((a.N + kTileRows - 1) / kTileRows + WR - 1) / WR;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(min(rounds, a.sm_count * per_sm)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = a.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gemv_w4_kernel<FMT, GP, PC, NT>, p);
}

}  // namespace

cudaError_t launch_gemv_w4(const GemvW4Args& a, cudaStream_t stream) {
    return dispatch_format(a.format, a.group, [&](auto fmt, auto gp) {
        return a.M <= 8 ? launch<fmt(), gp(), 4, 1>(a, stream) : launch<fmt(), gp(), 2, 2>(a, stream);
    });
}

}  // namespace fp8bs
