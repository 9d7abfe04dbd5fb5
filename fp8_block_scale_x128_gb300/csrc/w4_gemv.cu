// y[M, N] = bf16(x . W^T) for up to 16 bf16 tokens and a 4-bit weight.
//
// A block owns a contiguous range of 16-row tiles; its warps split K (WK
// slices), or K and the tiles where K has fewer than 16 chunks.  A warp keeps
// its slice of x as fp16 (all of it where it fits, and then a tile's stages
// follow each other; else one stage at a time for kGroup tiles, staged again
// for the next ones) and streams its part of the codes through a ring of its
// own, so no step but the sums over the slices is block-wide.  Those go in
// slice order: repeated calls give the same bits.
//
// Bound by latency in a long chain of instructions (w4.cuh), at the smallest sizes
// by the launch.  Measured in a graph on weights that are not in the second-level
// cache: 4.0 us for 1x4096x2048 (MXFP4; 0.66 at the measured copy bandwidth), 7.0
// for 1x5120x4096 (INT4, groups of 128; 1.6), 18.3 for 1x16384x8192 (MXFP4; 10.5,
// 58% of the bandwidth; the other way round, groups of tiles in pieces, took
// 21.0), 24.5 for 8 tokens of it and 39 for 16, where x does not fit beside the
// codes and is staged twice.  16 warps in one block, not 8 in two: the slices are
// half as long, and x is held once.  Of 128 registers a thread 16 columns spill 32
// bytes (MXFP4; 4 with integer groups of 32 or 128), two tiles a stage with kept
// x 24 (MXFP4) and 16 (integer groups of 32).
#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

using namespace w4;

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 4;  // tiles summed in registers before the slices meet

struct GemvParams {
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* codes;
    int64_t ldc;
    const uint8_t* scales;
    int64_t lds;
    uint16_t* y;
    int64_t ldy;
    int M, N, tiles;
    int chunks;    // chunks of 128 k
    int WK, WR;    // K slices, row tiles at a time: WK * WR <= kWarps
    int pieces;    // stages of the longest slice
    int pdl;
};

template <int NT>
constexpr int kRedBytes = kGroup * kSumBytes<NT>;  // of a warp

// Bytes of a warp: the ring, the scale table, staged x and its inverse scales,
// and the partial sums, which take the place of x where that is staged anew.
template <int GP, int NT, int T, int D>
__host__ __device__ constexpr int warp_bytes(int M, int pieces, bool resident) {
    const int kept = resident ? pieces : 1, x = kept * M * kTokenBytes, inv = (kept * 8 * NT * 4 + 127) / 128 * 128;
    return D * T * kCodeBytes + T * kTableBytes<GP> + inv + (resident ? x + kRedBytes<NT> : (x > kRedBytes<NT> ? x : kRedBytes<NT>));
}

// NT: tiles of 8 token columns; T: tiles of a stage; D: ring depth; RES: whether
// all pieces of x stay staged.
template <int FMT, int GP, int NT, int T, int D, bool RES>
__global__ void __launch_bounds__(kThreads, 1) gemv_w4_kernel(const __grid_constant__ GemvParams p) {
    constexpr int SB = Format<FMT, GP>::kScaleBytes;
    constexpr int kSlot = T * kCodeBytes, kTableAt = D * kSlot, kInvAt = kTableAt + T * kTableBytes<GP>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wr = warp / p.WK, wk = warp - wr * p.WK;
    const int kept = RES ? p.pieces : 1;
    const int mine_bytes = warp_bytes<GP, NT, T, D>(p.M, p.pieces, RES);
    // a warp's memory: codes [D][T], scale tables [T], inv [kept][8 NT],
    // x [kept][M][kTokenBytes], and the sums behind x or in its place
    const int x_at = kInvAt + (kept * 8 * NT * 4 + 127) / 128 * 128;
    const int red_at = x_at + (RES ? kept * p.M * kTokenBytes : 0);
    const uint32_t mine = ptx::smem_addr(smem) + warp * mine_bytes, xs = mine + x_at;
    const uint32_t to_codes = mine + code_dst(lane), to_table = mine + kTableAt + scale_dst<GP>(lane);
    const uint32_t from_codes = mine + code_src(lane), from_table = mine + kTableAt + scale_src<GP>(lane);
    const uint32_t from_inv = mine + kInvAt + inv_src(lane);
    uint32_t from_x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) from_x[j] = xs + token_src(8 * j + (lane >> 2), p.M, lane);

    // a warp past WK * WR has no slice; it only takes part in the sums
    const bool works = wr < p.WR;
    const int first = works ? wk * p.chunks / p.WK : 0, last = works ? (wk + 1) * p.chunks / p.WK : 0;
    const int t0 = static_cast<int>(static_cast<int64_t>(blockIdx.x) * p.tiles / gridDim.x);
    const int t1 = static_cast<int>((static_cast<int64_t>(blockIdx.x) + 1) * p.tiles / gridDim.x);
    const int steps = (t1 - t0 + p.WR - 1) / p.WR;  // tiles of a warp

    // the order of a warp's stages.  RES: its tiles, T at a time, in them the
    // pieces of the slice; else groups of kGroup tiles, in a group the pieces, in
    // a piece the tiles.  (Of two tiles the second may be missing at the end of
    // a range.)  codes and scales are this lane's pointers into the stage.
    struct Cursor {
        int group, piece, t;
        const uint8_t *codes, *scales;
    };
    const int64_t tile_codes = kTileRows * p.WR * p.ldc, tile_scales = kTileRows * p.WR * p.lds;
    Cursor ahead = {0, 0, 0, nullptr, nullptr};
    ahead.codes = p.codes + (static_cast<int64_t>(t0 + wr) * kTileRows + (lane >> 3)) * p.ldc + first * 64 + (lane & 7) * 16;
    ahead.scales = p.scales + (static_cast<int64_t>(t0 + wr) * kTileRows + (lane >> 1)) * p.lds + (first + (lane & 1)) * SB;
    const uint32_t ldc = static_cast<uint32_t>(p.ldc);
    const int whole = min(t1, p.N / kTileRows);  // tiles before this one have 16 rows
    auto issue = [&](int slot, uint2 (&raw)[T]) {
        const int nch = min(last - first - ahead.piece * kPC, kPC), step = ahead.group + ahead.t;
        if (step < steps && nch > 0) {
            const int tile = t0 + wr + step * p.WR;
            if (tile + (T - 1) * p.WR < whole && (RES || ahead.t + T <= kGroup)) {
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    load_codes(to_codes + slot * kSlot + i * kCodeBytes, ahead.codes + i * tile_codes, ldc, kTileRows - 1, nch, lane);
                    raw[i] = load_scales<FMT, GP>(ahead.scales + i * tile_scales, nch, lane);
                }
            } else {
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    raw[i] = make_uint2(0, 0);
                    if (tile + i * p.WR < t1) {
                        const int last_row = min(p.N - (tile + i * p.WR) * kTileRows, kTileRows) - 1;
                        load_codes(to_codes + slot * kSlot + i * kCodeBytes, ahead.codes + i * tile_codes, ldc, last_row, nch, lane);
                        raw[i] = load_scales<FMT, GP>(ahead.scales + i * tile_scales - max((lane >> 1) - last_row, 0) * p.lds, nch, lane);
                    }
                }
            }
        }
        cp_async_commit();
        // on to the next stage
        if constexpr (RES) {
            if (++ahead.piece < p.pieces) {
                ahead.codes += kPC * 64;
                ahead.scales += kPC * SB;
            } else {
                ahead.piece = 0;
                ahead.group += T;
                ahead.codes += T * tile_codes - (p.pieces - 1) * kPC * 64;
                ahead.scales += T * tile_scales - (p.pieces - 1) * kPC * SB;
            }
        } else {
            const int count = min(kGroup, steps - ahead.group);
            if ((ahead.t += T) < count) {
                ahead.codes += T * tile_codes;
                ahead.scales += T * tile_scales;
            } else {
                const int back = ahead.t - T;
                ahead.t = 0;
                if (++ahead.piece < p.pieces) {
                    ahead.codes += kPC * 64 - back * tile_codes;
                    ahead.scales += kPC * SB - back * tile_scales;
                } else {
                    ahead.piece = 0;
                    ahead.group += kGroup;
                    ahead.codes += T * tile_codes - (p.pieces - 1) * kPC * 64;
                    ahead.scales += T * tile_scales - (p.pieces - 1) * kPC * SB;
                }
            }
        }
    };
    auto stage_x = [&](int piece, int slot) {
        const int at = first + piece * kPC, nch = min(last - at, kPC);
        if (nch > 0) {
            auto src = [&](int m) { return p.x + m * p.ldx + at * kChunk; };
            RawBf16 first_tokens;
            first_tokens.load(p.M, nch, lane, src);
            stage_tokens<FMT>(xs + slot * p.M * kTokenBytes, mine + kInvAt + slot * 8 * NT * 4, first_tokens, p.M, nch, lane, src);
        }
    };

    if (!p.pdl) ptx::griddep_wait();
    uint2 raw[D - 1][T] = {};
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i, raw[i]);
    if (p.pdl) ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (RES)
        for (int q = 0; q < p.pieces; ++q) stage_x(q, q);

    int slot = 0;
    // multiply the stage at the front of the ring and start the one that takes
    // its predecessor's slot
    auto multiply = [&](float (&tot)[T][NT][4], int nch, int kept_at) {
        uint2 cur[T];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            cur[i] = raw[0][i];
#pragma unroll
            for (int k = 0; k + 2 < D; ++k) raw[k][i] = raw[k + 1][i];
        }
        issue(slot == 0 ? D - 1 : slot - 1, raw[D - 2]);
        if (nch > 0) {
            const bool far = store_scales<FMT, GP, T>(to_table, cur);
            uint32_t x[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) x[j] = from_x[j] + kept_at * p.M * kTokenBytes;
            cp_async_wait<D - 1>();
            __syncwarp();
            multiply_stage<FMT, GP, NT, T>(tot, from_codes + slot * kSlot, from_table, x, from_inv + kept_at * 8 * NT * 4, far, nch);
        }
        __syncwarp();  // the slot, the table and x are rewritten by later stages
        slot = slot + 1 == D ? 0 : slot + 1;
    };
    for (int group = 0; group < steps; group += kGroup) {
        const int count = min(kGroup, steps - group);
        // sums as [warp][tile of the group][token][row]
        if constexpr (RES) {
            for (int t = 0; t < count; t += T) {
                float tot[T][NT][4] = {};
                for (int piece = 0; piece < p.pieces; ++piece) multiply(tot, min(last - first - piece * kPC, kPC), piece);
#pragma unroll
                for (int i = 0; i < T; ++i) store_sums<NT>(mine + red_at + (t + i) * kSumBytes<NT>, tot[i], lane);
            }
        } else {
            float tot[kGroup / T][T][NT][4] = {};
            for (int piece = 0; piece < p.pieces; ++piece) {
                stage_x(piece, 0);
#pragma unroll
                for (int t = 0; t < kGroup / T; ++t)
                    if (t * T < count) multiply(tot[t], min(last - first - piece * kPC, kPC), 0);
            }
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                if (u < count) store_sums<NT>(mine + red_at + u * kSumBytes<NT>, tot[u / T][u % T], lane);
        }
        __syncthreads();
        const int rows = count * p.WR * kTileRows;
        const int64_t row0 = static_cast<int64_t>(t0 + group * p.WR) * kTileRows;
        const int64_t row_end = min(static_cast<int64_t>(p.N), static_cast<int64_t>(t1) * kTileRows);
        for (int o = threadIdx.x; o < p.M * rows; o += kThreads) {
            const int m = o / rows, rr = o - m * rows;
            if (row0 + rr < row_end) {
                const int tile = rr / kTileRows, u = tile / p.WR, w0 = (tile - u * p.WR) * p.WK;
                const uint8_t* s = smem + w0 * mine_bytes + red_at + u * kSumBytes<NT> + (m * kSumPitch + rr % kTileRows) * 4;
                float v = *reinterpret_cast<const float*>(s);
                for (int k = 1; k < p.WK; ++k) v += *reinterpret_cast<const float*>(s + k * mine_bytes);
                p.y[m * p.ldy + row0 + rr] = to_bf16(v);
            }
        }
        __syncthreads();  // the sums' place is rewritten by the next group
    }
}

template <int FMT, int GP, int NT, int T, int D, bool RES>
cudaError_t launch(const GemvParams& p, int sm_count, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(gemv_w4_kernel<FMT, GP, NT, T, D, RES>, allowed);
    if (e != cudaSuccess) return e;
    const int smem = kWarps * warp_bytes<GP, NT, T, D>(p.M, p.pieces, RES);
    return launch_dependent(gemv_w4_kernel<FMT, GP, NT, T, D, RES>, min((p.tiles + p.WR - 1) / p.WR, sm_count), kThreads, smem, stream, p);
}

// Whether a block with this ring fits, all of x staged (RES) or a stage of it.
template <int GP, int NT, int T, int D, bool RES>
bool fits(const GemvParams& p) {
    return kWarps * warp_bytes<GP, NT, T, D>(p.M, p.pieces, RES) <= kMaxBlockShared;
}

}  // namespace

cudaError_t launch_gemv_w4(const GemvW4Args& a, cudaStream_t stream) {
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
    p.tiles = (a.N + kTileRows - 1) / kTileRows;
    p.chunks = a.K / kChunk;
    p.WK = min(p.chunks, kWarps);
    p.WR = kWarps / p.WK;
    p.pieces = ((p.chunks + p.WK - 1) / p.WK + kPC - 1) / kPC;
    p.pdl = a.pdl;
    return dispatch_format(a.format, a.group, [&](auto fmt, auto gp) {
        constexpr int F = fmt(), G = gp();
        const int sm = a.sm_count, blocks = min((p.tiles + p.WR - 1) / p.WR, sm);
        const int steps = ((p.tiles + blocks - 1) / blocks + p.WR - 1) / p.WR;  // tiles of a warp
        // (from 9 tokens on the sums leave no room for x beside them at any size)
        if (a.M > 8) return launch<F, G, 2, 1, 2, false>(p, sm, stream);
        // two tiles a stage share its activations; where a warp has one tile,
        // half of such a stage would be idle.  (A slice of one stage is staged
        // once for kGroup tiles without being kept.)
        if (steps > 1 && fits<G, 1, 2, 2, true>(p)) return launch<F, G, 1, 2, 2, true>(p, sm, stream);
        if (steps > 1 && p.pieces == 1 && fits<G, 1, 2, 2, false>(p)) return launch<F, G, 1, 2, 2, false>(p, sm, stream);
        if (fits<G, 1, 1, 3, true>(p)) return launch<F, G, 1, 1, 3, true>(p, sm, stream);
        if (fits<G, 1, 1, 2, true>(p)) return launch<F, G, 1, 1, 2, true>(p, sm, stream);
        return launch<F, G, 1, 1, 3, false>(p, sm, stream);
    });
}

}  // namespace fp8bs
