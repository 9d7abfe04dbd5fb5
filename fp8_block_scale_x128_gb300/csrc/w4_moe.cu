// Small-batch mixture-of-experts layer on 4-bit weights, two launches.
//
//   h = x[m] . w13[e]^T              (gate rows 0..I-1 over up rows I..2I-1)
//   a = silu(h_gate) * h_up          (kept in the workspace as fp32)
//   y[m] = bf16(sum over s, in slot order, of tw[m, s] * (a . w2[e]^T))
//
// 1. gate/up: items of (expert, up to 8 of its pairs, 16 gate rows and the 16
//    up rows that go with them), dealt out in contiguous runs, so that a block
//    stages an expert's tokens once for its run; the 8 warps of a block split
//    H, their sums are added in warp order and the activation applied to the
//    whole sum.
// 2. down: a block owns 16 or 32 rows of the output for every token, its warps
//    deal out the experts; the pairs' products meet in shared memory and are summed
//    in slot order.  No partial sums in global memory, no atomics on values.
//    a takes two of an MMA's columns, as the sum of two fp16 numbers.  (As one
//    of 11 bits it left y off from its form in fp32 by 8.6e-4 of the 2-norm, now
//    2e-5; 32 tokens of 513x256 took 100.6 us, now 103.7.)
//
// An expert's codes are read once for a batch of its pairs.  Every block builds
// the expert lists itself: a histogram of the routed pairs and its running
// sums (up to 32 pairs by one warp with a match across its lanes: 12.1 us
// instead of 14.4 for one token of 513x256).  The second launch's lists and
// first codes do not wait for the first.
//
// Bound by latency in a long chain of instructions (w4.cuh).  Measured on MXFP4
// experts of 513x256, hidden 4096, 32 tokens with 10 routed and a shared one:
// gate/up 64.1 us for 271 MB read (0.62 of the measured copy bandwidth), down
// 48.9 us for 135 MB (0.41), each launched alone; 102.6 us for both in a graph;
// 11.7 us for one token.  Gate/up spills 20 bytes a thread with 32-wide groups
// (128 registers, two blocks a multiprocessor; with 48 bytes it took 14 us more),
// the down projection with two tiles 4.
#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

using namespace w4;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// pairs of an entry at most: the token columns of one MMA, two a pair in the
// down projection
constexpr int kMaxBatch = 8;
constexpr int kMaxDownBatch = kMaxBatch / 2;
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
    float* a;       // [M*S][I], in kept_place's order
    int M, S, H, I, E;
};

// Shared-memory tables of the routed pairs, built by every block, of P = M * S
// elements each.
struct Lists {
    ushort4* entry;      // expert, first (place of its first pair), n (its pairs: 1 .. batch)
    uint32_t* pair;      // by place, grouped by entry: pair | token << 16
    uint16_t* place;     // of a pair
    uint16_t* unsorted;  // pairs of experts with more than one entry
    int entries;
};
__host__ __device__ constexpr int lists_bytes(int P) { return (16 * P + 127) / 128 * 128; }
__host__ __device__ constexpr int counts_bytes(int E) { return (E * 4 + 15) / 16 * 16; }

// counts: E ints of shared memory, free afterwards.  The order of the pairs of
// an expert with one entry may differ between blocks and runs: it only decides
// which MMA column serves a pair, and columns do not mix.  An expert with more
// pairs has them sorted, so that every block splits them into the same entries.
template <int THREADS>
__device__ Lists build_lists(const MoeParams& p, int batch, uint8_t* mem, int* counts) {
    __shared__ int sums[THREADS / 32];
    __shared__ int n_entries;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.M * p.S;
    Lists L;
    L.entry = reinterpret_cast<ushort4*>(mem);
    L.pair = reinterpret_cast<uint32_t*>(L.entry + P);
    L.place = reinterpret_cast<uint16_t*>(L.pair + P);
    L.unsorted = L.place + P;
    if (P <= 32) {  // one warp, lane q pair q, without the histogram: entries by their first pair
        if (warp == 0) {
            int e = lane < P ? p.ids[lane] : -1;
            if (lane < P && (e < 0 || e >= p.E)) record_error(p.err, FP8BS_ERR_DEVICE);
            if (e >= p.E) e = -1;
            const bool valid = e >= 0;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, valid ? e : -1 - lane), below = (1u << lane) - 1u;
            const int rank = __popc(same & below), n = __popc(same);
            const bool leads = valid && rank % batch == 0;  // the first pair of an entry
            const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
            const int size = leads ? min(batch, n - rank) : 0;
            int incl = size;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
                if (lane >= off) incl += v;
            }
            // the last leader of the same expert at or below this lane
            const uint32_t mine = leaders & same & (below | 1u << lane);
            const int from = mine ? 31 - __clz(mine) : lane;
            const int first = __shfl_sync(0xFFFFFFFFu, incl - size, from);
            if (leads)
                L.entry[__popc(leaders & below)] = make_ushort4(static_cast<unsigned short>(e), static_cast<unsigned short>(first),
                                                                static_cast<unsigned short>(size), 0);
            if (valid) L.pair[first + rank % batch] = static_cast<uint32_t>(lane) | static_cast<uint32_t>(lane / p.S) << 16;
            if (lane < P) L.place[lane] = valid ? static_cast<uint16_t>(first + rank % batch) : 0xFFFF;
            if (lane == 0) n_entries = __popc(leaders);
        }
        __syncthreads();
        L.entries = n_entries;
        return L;
    }
    constexpr int kMine = (FP8BS_MOE_MAX_PAIRS + THREADS - 1) / THREADS;
    int id[kMine], rank[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int q = tid + j * THREADS;
        id[j] = q < P ? p.ids[q] : -1;
        if (q < P && (id[j] < 0 || id[j] >= p.E)) {
            record_error(p.err, FP8BS_ERR_DEVICE);
            id[j] = -1;
        }
    }
    for (int e = tid; e < p.E; e += THREADS) counts[e] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j) rank[j] = id[j] >= 0 ? atomicAdd(&counts[id[j]], 1) : 0;
    __syncthreads();
    // running sums over the experts: pairs in the low half, entries in the high one
    const int per = (p.E + THREADS - 1) / THREADS;
    const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += counts[e] | ((counts[e] + batch - 1) / batch << 16);
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int at = incl - mine;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w)
        if (w < warp) at += sums[w];
    if (tid == THREADS - 1) n_entries = (at + mine) >> 16;
    for (int e = e0; e < e1; ++e) {
        const int n = counts[e], first = at & 0xFFFF;
        counts[e] = first | n << 16;
        for (int b = 0; b * batch < n; ++b)
            L.entry[(at >> 16) + b] = make_ushort4(static_cast<unsigned short>(e), static_cast<unsigned short>(first + b * batch),
                                                   static_cast<unsigned short>(min(n - b * batch, batch)), 0);
        at += n | ((n + batch - 1) / batch << 16);
    }
    __syncthreads();
    auto set = [&](int place, int q) {
        L.pair[place] = static_cast<uint32_t>(q) | static_cast<uint32_t>(q / p.S) << 16;
        L.place[q] = static_cast<uint16_t>(place);
    };
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int q = tid + j * THREADS;
        if (id[j] >= 0) {
            const int c = counts[id[j]], place = (c & 0xFFFF) + rank[j];
            if (c >> 16 > batch)
                L.unsorted[place] = static_cast<uint16_t>(q);
            else
                set(place, q);
        } else if (q < P) {
            L.place[q] = 0xFFFF;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j)
        if (id[j] >= 0 && counts[id[j]] >> 16 > batch) {
            const int n = counts[id[j]] >> 16, first = counts[id[j]] & 0xFFFF, q = tid + j * THREADS;
            int r = 0;
            for (int i = 0; i < n; ++i) r += L.unsorted[first + i] < q;
            set(first + r, q);
        }
    L.entries = n_entries;
    __syncthreads();
    return L;
}

// ---- 1. gate / up ------------------------------------------------------------
constexpr int kUpDepth = 2;

// Bytes of a warp: the ring of gate and up tiles, their scale tables (whose
// place the sums take between items), the inverse scales and the tokens of the
// whole slice (pieces stages) for n pairs.
template <int GP>
constexpr int kUpTableBytes = 2 * (kTableBytes<GP> > kSumBytes<1> ? kTableBytes<GP> : kSumBytes<1>);
__host__ __device__ constexpr int up_inv_bytes(int pieces) { return (pieces * kMaxBatch * 4 + 127) / 128 * 128; }
template <int GP>
__host__ __device__ constexpr int up_bytes(int n, int pieces) {
    return kUpDepth * 2 * kCodeBytes + kUpTableBytes<GP> + up_inv_bytes(pieces) + pieces * n * kTokenBytes;
}
__host__ __device__ constexpr int up_pieces(int H) { return ((H / kChunk + kWarps - 1) / kWarps + kPC - 1) / kPC; }

template <int FMT, int GP>
__global__ void __launch_bounds__(kThreads, 2) moe_w4_up_kernel(const __grid_constant__ MoeParams p, int batch) {
    constexpr int SB = Format<FMT, GP>::kScaleBytes, D = kUpDepth, kSlot = 2 * kCodeBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int P = p.M * p.S, kept = min(P, batch), pieces = up_pieces(p.H);
    uint8_t* base = smem + lists_bytes(P);
    const int mine_bytes = up_bytes<GP>(kept, pieces);
    // a warp's memory: codes [D][gate, up], their scale tables, inv [pieces][8],
    // x [pieces][kept]
    constexpr int kTableAt = D * kSlot, kInvAt = kTableAt + kUpTableBytes<GP>;
    const uint32_t mine = ptx::smem_addr(base) + warp * mine_bytes, xs = mine + kInvAt + up_inv_bytes(pieces);
    const uint32_t to_codes = mine + code_dst(lane), to_table = mine + kTableAt + scale_dst<GP>(lane);
    const uint32_t from_codes = mine + code_src(lane), from_table = mine + kTableAt + scale_src<GP>(lane);
    const uint32_t from_inv = mine + kInvAt + inv_src(lane);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const Lists L = build_lists<kThreads>(p, batch, smem, reinterpret_cast<int*>(base));

    const int chunks = p.H / kChunk;
    const int first = warp * chunks / kWarps, last = (warp + 1) * chunks / kWarps;
    const int per = p.I / kTileRows;
    const uint32_t ldc = p.H / 2, lds = chunks * SB;
    const uint32_t up_codes = p.I * ldc, up_scales = p.I * lds;  // from a gate tile to its up tile
    const uint32_t lane_codes = (lane >> 3) * ldc + first * 64 + (lane & 7) * 16;
    const uint32_t lane_scales = (lane >> 1) * lds + (first + (lane & 1)) * SB;

    // the block's run of items (entry, tile j)
    const int64_t items = static_cast<int64_t>(L.entries) * per;
    const int item0 = static_cast<int>(blockIdx.x * items / gridDim.x);
    const int count = static_cast<int>((blockIdx.x + 1) * items / gridDim.x) - item0;
    int entry = item0 / per, j = item0 - entry * per;

    // a warp's stages: the items of the run, in an item the pieces of the slice
    struct Cursor {
        int entry, j, piece, left;
        const uint8_t *gate, *scales;  // this lane's, of the gate tile
    };
    Cursor ahead = {entry, j, 0, count, nullptr, nullptr};
    auto locate = [&]() {
        if (ahead.left <= 0) return;
        const uint32_t e = L.entry[ahead.entry].x;
        ahead.gate = at(at(p.w13, e, 2 * up_codes), ahead.j * kTileRows, ldc) + lane_codes;
        ahead.scales = at(at(p.s13, e, 2 * up_scales), ahead.j * kTileRows, lds) + lane_scales;
    };
    const int next_codes = static_cast<int>(kTileRows * ldc) - (pieces - 1) * kPC * 64, next_scales = static_cast<int>(kTileRows * lds) - (pieces - 1) * kPC * SB;
    auto issue = [&](int slot, uint2 (&raw)[2]) {
        const int nch = min(last - first - ahead.piece * kPC, kPC);
        if (ahead.left > 0 && nch > 0) {
            load_codes(to_codes + slot * kSlot, ahead.gate, ldc, kTileRows - 1, nch, lane);
            load_codes(to_codes + slot * kSlot + kCodeBytes, ahead.gate + up_codes, ldc, kTileRows - 1, nch, lane);
            raw[0] = load_scales<FMT, GP>(ahead.scales, nch, lane);
            raw[1] = load_scales<FMT, GP>(ahead.scales + up_scales, nch, lane);
        }
        cp_async_commit();
        if (++ahead.piece < pieces) {
            ahead.gate += kPC * 64;
            ahead.scales += kPC * SB;
            return;
        }
        ahead.piece = 0;
        --ahead.left;
        if (++ahead.j < per) {
            ahead.gate += next_codes;
            ahead.scales += next_scales;
        } else {
            ahead.j = 0;
            ++ahead.entry;
            locate();
        }
    };

    locate();
    uint2 raw[D - 1][2] = {};
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i, raw[i]);
    int slot = 0, staged = -1, n = 0, pf = 0;
    uint32_t x0 = 0;
    for (int item = 0; item < count; ++item) {
        if (entry != staged) {  // the expert's tokens, two pieces' loads in flight together
            staged = entry;
            n = L.entry[entry].z;
            pf = L.entry[entry].y;
            x0 = xs + token_src(lane >> 2, n, lane);
            auto source = [&](int piece) {
                const uint32_t* pair = L.pair + pf;
                const uint16_t* x = p.x + (first + piece * kPC) * kChunk;
                return [=](int i) { return x + (pair[i] >> 16) * p.ldx; };
            };
            for (int q = 0; q < pieces; q += 2) {
                const int nch0 = min(last - first - q * kPC, kPC), nch1 = min(last - first - (q + 1) * kPC, kPC);
                RawBf16 t0, t1;
                if (nch0 > 0) t0.load(n, nch0, lane, source(q));
                if (nch1 > 0) t1.load(n, nch1, lane, source(q + 1));
                if (nch0 > 0) stage_tokens<FMT>(xs + q * kept * kTokenBytes, mine + kInvAt + q * kMaxBatch * 4, t0, n, nch0, lane, source(q));
                if (nch1 > 0) stage_tokens<FMT>(xs + (q + 1) * kept * kTokenBytes, mine + kInvAt + (q + 1) * kMaxBatch * 4, t1, n, nch1, lane, source(q + 1));
            }
        }
        float tot[2][1][4] = {};
        for (int piece = 0; piece < pieces; ++piece) {
            const int nch = min(last - first - piece * kPC, kPC);
            const uint2 cur[2] = {raw[0][0], raw[0][1]};
#pragma unroll
            for (int i = 0; i + 2 < D; ++i) raw[i][0] = raw[i + 1][0], raw[i][1] = raw[i + 1][1];
            issue(slot == 0 ? D - 1 : slot - 1, raw[D - 2]);
            if (nch > 0) {
                const bool far = store_scales<FMT, GP, 2>(to_table, cur);
                const uint32_t x[1] = {x0 + piece * kept * kTokenBytes};
                cp_async_wait<D - 1>();
                __syncwarp();
                multiply_stage<FMT, GP, 1, 2>(tot, from_codes + slot * kSlot, from_table, x, from_inv + piece * kMaxBatch * 4, far, nch);
            }
            __syncwarp();  // the slot and the table are rewritten by later stages
            slot = slot + 1 == D ? 0 : slot + 1;
        }
        // [warp][gate, up][pair][row]
        store_sums<1>(mine + kTableAt, tot[0], lane);
        store_sums<1>(mine + kTableAt + kSumBytes<1>, tot[1], lane);
        __syncthreads();
        if (threadIdx.x < kMaxBatch * kTileRows) {  // 16 lanes a pair
            const int i = min(static_cast<int>(threadIdx.x) / kTileRows, n - 1), row = threadIdx.x % kTileRows;
            const uint32_t s = mine - warp * mine_bytes + kTableAt + (i * kSumPitch + row) * 4;
            float g = 0.0f, v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                g += lds_float(s + w * mine_bytes);
                v += lds_float(s + w * mine_bytes + kSumBytes<1>);
            }
            const float a = g / (1.0f + expf(-g)) * v;
            if (static_cast<int>(threadIdx.x) < n * kTileRows)
                p.a[(L.pair[pf + i] & 0xFFFF) * p.I + kept_place(j * kTileRows + row)] = a;
        }
        __syncthreads();  // the sums' place is rewritten by the next item
        if (++j == per) j = 0, ++entry;
    }
}

// ---- 2. down -----------------------------------------------------------------
// Bytes of a warp: a ring of stages of T tiles, their scale tables, the inverse
// scales and a stage of a for n pairs, two columns each.
constexpr int kInvBytes = 128;  // 8 factors, the next part aligned
__host__ __device__ constexpr int down_depth(int T) { return T == 2 ? 2 : 3; }
template <int GP>
__host__ __device__ constexpr int down_bytes(int n, int T) {
    return down_depth(T) * T * kCodeBytes + T * kTableBytes<GP> + kInvBytes + 2 * n * kTokenBytes;
}
// the pairs' products for the rows by place, and the pairs' routing weights
__host__ __device__ constexpr int out_bytes(int P, int T) { return (P * (T * kTileRows + 1) * 4 + 127) / 128 * 128; }

// ONE: the whole of I in one stage; T: tiles of a block; WARPS: 8, two blocks a
// multiprocessor, or 16.
template <int FMT, int GP, bool ONE, int T, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) moe_w4_down_kernel(const __grid_constant__ MoeParams p, int batch) {
    constexpr int SB = Format<FMT, GP>::kScaleBytes, D = down_depth(T), kSlot = T * kCodeBytes, kRows = T * kTileRows;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.M * p.S;
    float* out = reinterpret_cast<float*>(smem + lists_bytes(P));  // [P][kRows]
    float* weight = out + P * kRows;
    uint8_t* base = smem + lists_bytes(P) + out_bytes(P, T);
    // a warp's memory: codes [D][T], the scale tables, inv, the entry's a
    constexpr int kTableAt = D * kSlot, kInvAt = kTableAt + T * kTableBytes<GP>, kXsAt = kInvAt + kInvBytes;
    const uint32_t mine = ptx::smem_addr(base) + warp * down_bytes<GP>(min(P, batch), T), xs = mine + kXsAt;
    const uint32_t to_codes = mine + code_dst(lane), to_table = mine + kTableAt + scale_dst<GP>(lane);
    const uint32_t from_codes = mine + code_src(lane), from_table = mine + kTableAt + scale_src<GP>(lane);
    const uint32_t from_inv = mine + kInvAt + inv_src(lane);
    // the routing is complete: the first launch has waited for what wrote it
    for (int q = tid; q < P; q += (WARPS * 32)) weight[q] = p.tw[q];
    const Lists L = build_lists<WARPS * 32>(p, batch, smem, reinterpret_cast<int*>(base));

    const int chunks = p.I / kChunk, pieces = ONE ? 1 : (chunks + kPC - 1) / kPC;
    const uint32_t ldc = p.I / 2, lds = chunks * SB;
    const uint32_t expert_codes = p.H * ldc, expert_scales = p.H * lds;
    const uint8_t* lane_a = reinterpret_cast<const uint8_t*>(p.a) + kept_src(lane);
    const uint32_t la = p.I * 4;
    const int tiles = p.H / kRows;
    RawFp32 tokens;
    auto load_tokens = [&](const ushort4& entry, int piece, int i0) {
        const uint32_t* pair = L.pair + entry.y + i0;
        tokens.load(lane_a + piece * (kStageK * 4), la, entry.z - i0, min(chunks - piece * kPC, kPC), lane,
                    [=](int i) { return pair[i] & 0xFFFFu; });
    };

    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const uint8_t* lane_codes = at(p.w2 + static_cast<int64_t>(lane >> 3) * ldc + (lane & 7) * 16, tile * kRows, ldc);
        const uint8_t* lane_scales = at(p.s2 + static_cast<int64_t>(lane >> 1) * lds + (lane & 1) * SB, tile * kRows, lds);
        // a warp's stages: its entries, in an entry the pieces of I
        int ahead = warp, ahead_piece = 0;
        auto issue = [&](uint32_t slot_at, uint2 (&raw)[T]) {
            if (ahead < L.entries) {
                const uint32_t e = L.entry[ahead].x;
                const int nch = min(chunks - ahead_piece * kPC, kPC);
                const uint8_t* c = at(lane_codes, e, expert_codes) + ahead_piece * kPC * 64;
                const uint8_t* s = at(lane_scales, e, expert_scales) + ahead_piece * kPC * SB;
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    load_codes(to_codes + slot_at + i * kCodeBytes, at(c, ldc, i * kTileRows), ldc, kTileRows - 1, nch, lane);
                    raw[i] = load_scales<FMT, GP>(at(s, lds, i * kTileRows), nch, lane);
                }
            }
            cp_async_commit();
            if (ONE || ++ahead_piece == pieces) ahead_piece = 0, ahead += WARPS;
        };
        uint2 raw[D - 1][T] = {};
#pragma unroll
        for (int i = 0; i < D - 1; ++i) issue(i * kSlot, raw[i]);
        if (tile == static_cast<int>(blockIdx.x)) {
            ptx::griddep_wait();
            ptx::griddep_launch_dependents();
        }
        ushort4 now = L.entry[min(warp, max(L.entries - 1, 0))];
        if (warp < L.entries) load_tokens(now, 0, 0);
        uint32_t slot_at = 0;
        for (int entry = warp; entry < L.entries; entry += WARPS) {
            const int n = now.z, pf = now.y;
            const ushort4 next = L.entry[min(entry + WARPS, L.entries - 1)];
            const uint32_t x[1] = {xs + token_src(lane >> 2, 2 * n, lane)};
            float tot[T][1][4] = {};
            for (int piece = 0; piece < pieces; ++piece) {
                const int nch = min(chunks - piece * kPC, kPC);
                uint2 cur[T];
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    cur[i] = raw[0][i];
#pragma unroll
                    for (int k = 0; k + 2 < D; ++k) raw[k][i] = raw[k + 1][i];
                }
                issue(slot_at == 0 ? (D - 1) * kSlot : slot_at - kSlot, raw[D - 2]);
                tokens.store<FMT>(xs, mine + kInvAt, 0, n, lane);
                for (int i0 = RawFp32::kTokens; i0 < n; i0 += RawFp32::kTokens) {
                    load_tokens(now, piece, i0);
                    tokens.store<FMT>(xs, mine + kInvAt, i0, n, lane);
                }
                if (!ONE && piece + 1 < pieces)
                    load_tokens(now, piece + 1, 0);
                else
                    load_tokens(next, 0, 0);
                const bool far = store_scales<FMT, GP, T>(to_table, cur);
                cp_async_wait<D - 1>();
                __syncwarp();
                multiply_stage<FMT, GP, 1, T>(tot, from_codes + slot_at, from_table, x, from_inv, far, nch);
                __syncwarp();  // the slot, the table and the tokens are rewritten by later stages
                slot_at = slot_at == (D - 1) * kSlot ? 0 : slot_at + kSlot;
            }
            if ((lane & 3) < n) {  // a lane's two columns are one pair's
                float* o = out + (pf + (lane & 3)) * kRows + (lane >> 2);
#pragma unroll
                for (int i = 0; i < T; ++i, o += kTileRows) {
                    o[0] = tot[i][0][0] + tot[i][0][1];
                    o[8] = tot[i][0][2] + tot[i][0][3];
                }
            }
            now = next;
        }
        __syncthreads();
        for (int o = tid; o < p.M * kRows; o += WARPS * 32) {
            const int m = o / kRows, row = o % kRows;
            float v = 0.0f;
#pragma unroll 4
            for (int q = m * p.S; q < (m + 1) * p.S; ++q) {
                const int place = L.place[q];  // 0xFFFF: an invalid id contributes nothing
                if (place != 0xFFFF) v = fmaf(weight[q], out[place * kRows + row], v);
            }
            p.y[static_cast<int64_t>(m) * p.H + tile * kRows + row] = to_bf16(v);
        }
        __syncthreads();  // out is rewritten for the next tile
    }
}

// The pairs of an entry (at most `largest`) and the blocks of a multiprocessor (at most `most`): two
// blocks, with as many pairs as then fit, unless the experts have more than twice as many on
// average (their codes would be fetched and decoded over and over): then one.
template <typename F>
int batch_of(const MoeParams& p, F&& bytes, int largest, int most, int& per_sm) {
    constexpr int kHalf = kMaxSmShared / 2 - 1024 - 128;  // less a block's reserved and static shared memory
    int batch = largest;
    while (batch > 0 && bytes(batch) > kHalf) --batch;
    per_sm = 2;
    if (most > 1 && batch > 0 && (batch == largest || p.M * p.S <= 2 * batch * p.E)) return batch;
    per_sm = 1;
    for (batch = largest; batch > 1 && bytes(batch) > kMaxBlockShared; --batch) {}
    return batch;
}

template <int FMT, int GP>
cudaError_t launch_up(const MoeParams& p, int sm_count, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(moe_w4_up_kernel<FMT, GP>, allowed);
    if (e != cudaSuccess) return e;
    const int P = p.M * p.S, pieces = up_pieces(p.H);
    auto bytes = [&](int batch) {
        return lists_bytes(P) + max(counts_bytes(p.E), kWarps * up_bytes<GP>(min(P, batch), pieces));
    };
    int per_sm;
    const int batch = batch_of(p, bytes, kMaxBatch, 2, per_sm), smem = bytes(batch);
    if (smem > kMaxBlockShared) return cudaErrorInvalidValue;
    const int64_t most = static_cast<int64_t>(P) * (p.I / kTileRows);
    const int grid = static_cast<int>(min(most, static_cast<int64_t>(sm_count) * per_sm));
    return launch_dependent(moe_w4_up_kernel<FMT, GP>, grid, kThreads, smem, stream, p, batch);
}

template <int GP, int T, int WARPS>
int down_block_bytes(const MoeParams& p, int batch) {
    const int P = p.M * p.S;
    return lists_bytes(P) + out_bytes(P, T) + max(counts_bytes(p.E), WARPS * down_bytes<GP>(min(P, batch), T));
}

template <int FMT, int GP, bool ONE, int T, int WARPS>
cudaError_t launch_down_as(const MoeParams& p, int sm_count, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(moe_w4_down_kernel<FMT, GP, ONE, T, WARPS>, allowed);
    if (e != cudaSuccess) return e;
    int per_sm;
    const int batch = batch_of(p, [&](int n) { return down_block_bytes<GP, T, WARPS>(p, n); }, kMaxDownBatch,
                               16 / WARPS, per_sm);
    return launch_dependent(moe_w4_down_kernel<FMT, GP, ONE, T, WARPS>, min(p.H / (T * kTileRows), sm_count * per_sm), WARPS * 32,
                            down_block_bytes<GP, T, WARPS>(p, batch), stream, p, batch);
}

template <int FMT, int GP, bool ONE>
cudaError_t launch_down(const MoeParams& p, int sm_count, cudaStream_t stream) {
    const int tiles = p.H / kTileRows;
    // Three forms, the first two where 16 warps fit beside the pairs' products
    // with kWant pairs an entry (with one an expert's codes are fetched for each of
    // its pairs).  Whole layers, us, two tiles and 16 warps / one and 8 / one and
    // 16, INT4: 8 tokens of 64x256, 6 slots, hidden 2560 18.9 / 19.8 / 20.9, 3584
    // 21.7 / 22.4 / 24.4, 7168 40.2 / 42.5 / 43.5; 24 tokens of 128x256, 8 slots,
    // hidden 4096 48.3 / 52.3 / 54.0.  Two tiles share a stage's other costs, though
    // at hidden 2560 they leave half of the multiprocessors without a block; one
    // token of up to 8 slots takes up to 1 us less with one tile and 8 warps.
    // With no more tiles than multiprocessors (hidden 2048) a second block of 8
    // warps would have none: 19 tokens of 24x512, 4 slots 23.8 / 27.3 / 22.4, 64 of
    // 128x512, 8 slots 112 / 112 / 88.  Past kWant: 128 tokens of 64x256, 8 slots
    // (one pair an entry with 16 warps) 88 / 88 / 114.
    constexpr int kWant = 2;
    if (tiles > sm_count && down_block_bytes<GP, 2, 16>(p, kWant) <= kMaxBlockShared)
        return launch_down_as<FMT, GP, ONE, 2, 16>(p, sm_count, stream);
    if (tiles <= sm_count && down_block_bytes<GP, 1, 16>(p, kWant) <= kMaxBlockShared)
        return launch_down_as<FMT, GP, ONE, 1, 16>(p, sm_count, stream);
    return launch_down_as<FMT, GP, ONE, 1, 8>(p, sm_count, stream);
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
        return p.I <= kStageK ? launch_down<fmt(), gp(), true>(p, a.sm_count, stream)
                              : launch_down<fmt(), gp(), false>(p, a.sm_count, stream);
    });
}

}  // namespace fp8bs
