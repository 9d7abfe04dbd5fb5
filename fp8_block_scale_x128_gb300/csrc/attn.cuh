// Attention block over a paged cache: what its kernels share.  The operators are
// the norm and rotation of query and key heads (qk_norm_rope.cu), with or
// without appending to the cache, and attention of new tokens over it
// (attn_decode.cu, attn_chunk.cu).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "internal.cuh"
#include "ptx.cuh"

namespace fp8bs {

// ---------------------------------------------------------------------------
// Norm, rotation, append
// ---------------------------------------------------------------------------

struct RopeArgs {
    const uint16_t *q, *k, *v;       // v only when appending
    int64_t ldq, hsq, ldk, hsk, ldv, hsv;  // token and head strides, elements
    int64_t T;
    int Hq, Hk, D;
    const int64_t* positions;
    const uint64_t* freqs;           // turns a position, in 2^-64
    int R, layout;
    float amplitude;
    const uint16_t *gq, *gk;
    float eps;
    uint16_t *qo, *ko;               // ko only without a cache
    int64_t ldqo, hsqo, ldko, hsko;
    const int64_t* slots;
    fp8bs_kv_cache cache;            // used when append
    uint32_t* err;
    int append;
    int sm_count;
};
cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Attention: the deal of the work
// ---------------------------------------------------------------------------

constexpr int kAttnMaxSeqs = FP8BS_ATTN_MAX_SEQS;
constexpr int kAttnMaxKeys = 1 << 30;  // of a sequence

struct AttnParams {
    const uint16_t* q;
    int64_t ldq, hsq;
    const uint8_t *k, *v, *ks, *vs;
    int64_t pstride, sstride, hstride;     // bytes
    int64_t zpstride, zsstride, zhstride;  // of the scales
    int64_t pages;
    int page_log2;
    const int32_t* table;
    int64_t table_stride;
    int table_cols;
    const int32_t *cu, *len;
    int B, T, Hk, G;
    uint32_t g_mul;    // n / G = n * g_mul >> g_shift for n < 2^31
    int g_shift;
    float scale_log2;  // softmax scale * log2(e)
    int window;        // 0: none
    uint16_t* o;
    int64_t ldo, hso;
    uint32_t* err;
    uint8_t* ws;  // past the error word
    long long timeout_cycles;  // of a wait inside the kernel
};

__device__ __forceinline__ int div_g(const AttnParams& p, int n) {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * p.g_mul >> p.g_shift);
}

struct AttnArgs : AttnParams {
    int D, kind;
    int sm_count;
};
size_t attn_workspace_bytes(int D, int sm_count);
cudaError_t launch_attn_paged(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_chunk(const AttnArgs& a, cudaStream_t stream);
size_t attn_chunk_slot_floats(int D);

// The work is dealt out on the device, from the lengths that stand there, so a
// captured call follows them.  The rows of a sequence are its new tokens times
// the G query heads of a key head, packed token by token; MT of them make a
// tile, a tile and a key head an item, BN consecutive keys of an item a unit.
// All units in the order (sequence, tile, head, key) go to the blocks in equal
// contiguous shares.  An item that lies in one block's share is finished there;
// of the others each block leaves (sum, maximum, weighted values) in a slot of
// its own and a second launch joins them in block order: no atomics, and the
// same bits each time.
struct SeqInfo {
    int q0, nq, kv;
};

__device__ __forceinline__ SeqInfo attn_seq(const AttnParams& p, int b) {
    const int c0 = p.cu[b], c1 = p.cu[b + 1], kv = p.len[b];
    // lengths that do not fit the tensors are cut to them
    const int most = static_cast<int>(min(static_cast<int64_t>(p.table_cols) << p.page_log2, int64_t(kAttnMaxKeys)));
    SeqInfo s;
    s.q0 = min(max(c0, 0), p.T);
    s.nq = max(min(max(c1, 0), p.T) - s.q0, 0);
    s.kv = min(max(kv, 0), most);
    if (s.q0 != c0 || s.q0 + s.nq != c1 || s.kv != kv) record_error(p.err, FP8BS_ERR_DEVICE);
    return s;
}

// The units [lo, lo + n) of keys that rows [r0, r1) of a sequence need.
struct TileUnits {
    int lo, n;
};
template <int BN>
__device__ __forceinline__ TileUnits attn_units(const AttnParams& p, const SeqInfo& s, int r0, int r1) {
    const int base = s.kv - s.nq;
    const int hi = base + div_g(p, r1 - 1) + 1;  // past the last key seen
    const int lo = p.window ? max(base + div_g(p, r0) - p.window + 1, 0) : 0;
    TileUnits u;
    u.lo = hi > lo ? lo / BN : 0;
    u.n = hi > lo ? (hi + BN - 1) / BN - u.lo : 1;  // a tile that sees nothing still writes its rows
    return u;
}

// What a block knows of its share.
struct AttnShare {
    long long total;       // units of all items
    int blocks;            // that take part: each has a unit at least
    long long begin, end;  // units of this block
    int tile, b, head, unit;  // the place of the first one
};

// The place in the deal of the work: an item and a unit of it.
struct Cursor {
    int tile, b, head, unit, n, lo;  // unit: within the item
    int q0, rows, row0;              // the sequence's first token, packed rows of the tile
    int base;                        // place of the sequence's first new token
    int first, past;                 // keys that some row sees
    int lowest;                      // place of the first row
};

struct PlanShared {
    int first[kAttnMaxSeqs + 1];  // tiles before each sequence
    long long sums[2][32];        // of the warps
    AttnShare share;
};

// Inclusive sum over the block; *all: the block's.  Whole block; calls in turn take
// turns with the places of `sums`.
template <int THREADS, typename N>
__device__ __forceinline__ N block_scan(N v, long long* sums, N* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const N t = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += t;
    }
    N* of = reinterpret_cast<N*>(sums);
    if (lane == 31) of[warp] = v;
    __syncthreads();
    N before = 0, sum = 0;
#pragma unroll 4
    for (int w = 0; w < THREADS / 32; ++w) {
        const N t = of[w];
        if (w < warp) before += t;
        sum += t;
    }
    *all = sum;
    return before + v;
}

// a / b, b > 0: a division of 64 bits takes some hundred instructions.
__device__ __forceinline__ long long divide(long long a, long long b) {
    if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

__device__ __forceinline__ int attn_tile_seq(const PlanShared& sh, int B, int tile) {
    int lo = 0, hi = B;  // first[lo] <= tile < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.first[mid] <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Whole block; leaves sh.first and sh.share.
template <int MT, int BN, int THREADS>
__device__ __noinline__ void attn_share(const AttnParams& p, PlanShared& sh) {
    const int tid = threadIdx.x, block = blockIdx.x;
    if (tid == 0) sh.first[0] = 0;
    int tiles = 0, turn = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + tid;
        int all;
        const int n = b < p.B ? (attn_seq(p, b).nq * p.G + MT - 1) / MT : 0;
        const int upto = block_scan<THREADS, int>(n, sh.sums[turn ^= 1], &all);
        if (b < p.B) sh.first[b + 1] = tiles + upto;
        tiles += all;
    }
    __syncthreads();
    // twice over the tiles: the sum of all units, then the tile that this block's first
    // unit lies in (of up to THREADS tiles once)
    long long total = 0, begin = 0, before = 0, all = 0, upto = 0;
    int n = 0, b = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int t0 = 0; t0 < tiles; t0 += THREADS) {
            const int t = t0 + tid;
            if (pass == 0 || tiles > THREADS) {
                n = 0;
                if (t < tiles) {
                    b = attn_tile_seq(sh, p.B, t);
                    const SeqInfo s = attn_seq(p, b);
                    const int r0 = (t - sh.first[b]) * MT;
                    n = attn_units<BN>(p, s, r0, min(r0 + MT, s.nq * p.G)).n;
                }
                upto = block_scan<THREADS, long long>(n, sh.sums[turn ^= 1], &all);
            }
            if (pass == 0) {
                total += all;
                continue;
            }
            const long long mine = (before + upto - n) * p.Hk;
            if (n > 0 && mine <= begin && begin < mine + static_cast<long long>(n) * p.Hk) {
                sh.share.tile = t, sh.share.b = b;
                sh.share.head = static_cast<int>(divide(begin - mine, n));
                sh.share.unit = static_cast<int>(begin - mine - static_cast<long long>(sh.share.head) * n);
            }
            before += all;
        }
        if (pass == 0) {
            total *= p.Hk;
            const int blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
            // odd lanes: where the next block begins
            const long long bound = block < blocks ? divide((block + (tid & 1)) * total, blocks) : 0;
            begin = __shfl_sync(0xFFFFFFFFu, bound, 0);
            if (tid == 0) sh.share.total = total, sh.share.blocks = blocks, sh.share.begin = begin;
            if (tid == 1) sh.share.end = bound;
        }
    }
    __syncthreads();
}

// What a tile is, for a cursor that has come to it.
template <int ROWS, int UNIT>
__device__ __forceinline__ Cursor attn_enter(const AttnParams& p, const PlanShared& sh, int tile, int b, int head) {
    while (tile >= sh.first[b + 1]) ++b;
    const SeqInfo s = attn_seq(p, b);
    Cursor c;
    c.tile = tile, c.b = b, c.head = head, c.unit = 0;
    c.q0 = s.q0;
    c.row0 = (tile - sh.first[b]) * ROWS;
    c.rows = min(ROWS, s.nq * p.G - c.row0);
    const TileUnits u = attn_units<UNIT>(p, s, c.row0, c.row0 + c.rows);
    c.n = u.n, c.lo = u.lo;
    c.base = s.kv - s.nq;
    c.lowest = c.base + div_g(p, c.row0);
    c.past = c.base + div_g(p, c.row0 + c.rows - 1) + 1;
    c.first = p.window ? max(c.lowest - p.window + 1, 0) : 0;
    return c;
}

// Whether every row of the item sees every key of a unit.
template <int UNIT>
__device__ __forceinline__ bool attn_sees_all(const AttnParams& p, const Cursor& c) {
    const int j0 = (c.lo + c.unit) * UNIT;
    return j0 + UNIT <= c.lowest + 1 && (p.window == 0 || j0 >= c.past - p.window);
}

// The block that finishes an item begun in unit `start` of all.
static __device__ __noinline__ int attn_last_block(const AttnShare& a, long long start, int n) {
    return static_cast<int>(divide((start + n) * a.blocks - 1, a.total));
}

// What a block leaves for the second launch about an item that it begins and
// does not finish.
struct AttnSplit {
    int32_t rows;   // 0: none
    int32_t q0;     // the sequence's first token
    int32_t row0;   // the item's first packed row
    int32_t head;   // key head
    int32_t last;   // the block that finishes it
    int32_t pad[3];
};

// The sum of a row's weights where it sees keys, all at scores of minus infinity: values
// divided by it are NaN.  (Other sums of rows that see keys are above 2^-126.)
constexpr float kNoWeight = 0x1p-149f;

// Workspace past the error word: a record a block, then two slots a block:
// slot 0 for an item begun elsewhere, slot 1 for one begun here.  A slot holds
// values [rows][D], maxima [rows] (in units of log2) and sums [rows], all fp32.
__host__ __device__ constexpr size_t attn_slot_floats(int MT, int D) { return static_cast<size_t>(MT) * (D + 2); }
__host__ __device__ constexpr size_t attn_records_bytes(int grid) {
    return (static_cast<size_t>(grid) * sizeof(AttnSplit) + 255) / 256 * 256;
}
__device__ __forceinline__ float* attn_slot(const AttnParams& p, int grid, int MT, int D, int block, int slot) {
    return reinterpret_cast<float*>(p.ws + attn_records_bytes(grid)) +
           (static_cast<size_t>(block) * 2 + slot) * attn_slot_floats(MT, D);
}

// Key position -> byte offset of its row for one head; false where the table
// names no page of the cache (recorded).
__device__ __forceinline__ bool attn_page(const AttnParams& p, const int32_t* table, int j, int* page) {
    *page = table[j >> p.page_log2];
    if (*page < 0 || *page >= p.pages) {
        record_error(p.err, FP8BS_ERR_DEVICE);
        return false;
    }
    return true;
}

// ---------------------------------------------------------------------------
// Small device pieces
// ---------------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A sum of weights against a maximum that is 2^-x as large.  (Over codes the maximum is of
// weights times values' scales, so the sum may be far above it: 2^x alone would be nothing
// where the sum times it is not.)
__device__ __forceinline__ float fallen(float sum, float x) {
    const float half = ex2(0.5f * x);
    return sum * half * half;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The upper bit of each byte of a word that is a code without a value.
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u & 0x80808080u; }

// Zeros in their place.
__device__ __forceinline__ uint32_t without_odd_codes(uint32_t w) { return w & ~((odd_codes(w) >> 7) * 0xFFu); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros where !there (nothing is read then).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Raises a kernel's dynamic shared memory limit to `bytes`, once per kernel and device.
template <typename K>
cudaError_t attn_allow_shared(K* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done.load(std::memory_order_relaxed) >> dev & 1) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

cudaError_t launch_attn_join(const AttnArgs& a, int MT, int grid, cudaStream_t stream);

}  // namespace fp8bs
