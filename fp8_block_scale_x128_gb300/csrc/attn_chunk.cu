// Attention of many new tokens a sequence over a paged cache, on the 5th
// generation tensor core (attn.cuh says how the work is dealt out).
//
// A tile is 256 rows (128 with heads of 256), in streams of 128 with their own
// accumulators in tensor memory.  Warps have one task each:
//   loaders  copy a unit's keys and its values into a ring of shared memory
//            tiles in the operand layout (128-byte swizzle; a row's 64 dimensions are
//            a line, so keys are a K-major operand and values an MN-major one of the
//            same layout); codes become fp16 on the way;
//   one warp issues the products: scores S = Q K^T into tensor memory, then, once
//            the weights are there, O += P V with P as the operand in tensor memory;
//   a warpgroup a stream takes its rows' softmax, a thread a row: no shuffles.
// Two streams (heads up to 128) take turns on the tensor core: while one's weights
// are computed, the other's products run.  One stream (heads of 256) has two score
// buffers, and the next unit's scores are under way during a unit's softmax.
//
// Weights are rounded to bf16 once (2^-8 of each, at most; they average out) and
// summed before that in fp32.  The maximum that they are taken against may lag by 8
// in units of log2, so that outputs are rescaled in tensor memory only rarely.
//
// Codes.  e4m3 codes are exact in fp16, and the products run in it.  A row of q is
// multiplied by the power of two that brings its largest magnitude into [2^14, 2^15)
// (exact down to 2^-31 of that).  A code is multiplied by its scale over the largest of
// its unit, exactly where they differ by 2^14 at most; the unit's own scale multiplies the
// scores, and the values' is part of the weights, 2^(x + e), of which the maximum is taken.
// Where the scales of a unit's keys or of its values are further apart, codes stay as they
// are, and each score has its key's own scale and each weight its value's: a masked key, or
// one of no weight, may be as large as it likes.  2^7 more uses fp16's range: a weight is off
// by at most 2^-11 of itself, or 2^-32 of the largest.
//
// A value that is not finite and that some row of its unit masks would reach that row
// as zero times it.  In units with masks the loaders put zeros in the place of such
// values (codes without a value among them) and mark the item; its rows then add those
// that they see at their end.
//
// Scores from 2^16 on are rounded each for itself before the maximum is taken from them:
// below that a multiply-add takes a rounded maximum from an unrounded score, which is off by
// no power of two worth the name.
//
// 4096 tokens over 16384 keys, 32 + 8 heads of 128, take 664 to 729 us with pages of 64 (the
// same inputs again and again, or others each time; 1.44 to 1.32 PFLOP/s, 0.78 to 0.72 of a
// large matrix product's rate) and 670 to 695 with pages of 16 (the same inputs): some 3300
// cycles a unit, of which a stream's softmax 1800 and its two products 1024 follow one another,
// beside the other stream's.  Over codes 888 us with pages of 64, 1015 with pages of 16: the
// widening shares the issue slots and the shared memory with the softmax, and one warp looks
// pages up, reads scales and issues boxes.  (Below, what a variant that was not kept took
// stands beside what this took then.)
#include <cuda.h>
#include <cuda_fp16.h>

#include "attn.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

constexpr int kRows = 128;  // of a stream
constexpr float kLag = 8.0f;
constexpr float kFar = 65536.0f;  // scores whose rounding is 2^-8 and more
constexpr int kMarks = 8;
// That may be under way.  The loaders are at most three ahead of the outputs; warps that look
// values through wait for nothing in units without masks, so an item's place is given to
// another only once they have read it (`taken`).
constexpr int kItems = 8;

template <int D, int KIND>
struct Cfg {
    static constexpr bool kCodes = KIND == FP8BS_KV_E4M3;
    static constexpr int kStreams = D == 256 ? 1 : 2;
    static constexpr int kTile = kStreams * kRows;
    static constexpr int kKeys = D == 256 ? 64 : 128;  // of a unit
    static constexpr int kSoft = kStreams * 4;         // softmax warps, a thread a row (two
    // threads a row, each of half the keys, took 830 us where this takes 720: the softmax
    // of the two streams together is bound by its instructions, not by one's latency)
    static constexpr int kThreads = kStreams == 2 || kCodes ? 512 : 384;
    // Registers of a softmax thread and of the others, where the launch's are dealt out
    // anew: 256 (184 + 72) of 512 * 128.
    static constexpr bool kDeal = kStreams == 2;
    static constexpr int kMoreRegs = 184, kFewRegs = 72;
    static_assert(!kDeal || kSoft * 32 * kMoreRegs + (kThreads - kSoft * 32) * kFewRegs <= kThreads * (65536 / kThreads / 8 * 8),
                  "more registers than the launch has would be waited for without end");
    static constexpr int kLoadWarps = kThreads / 32 - kSoft - 2;
    // warps that issue copies: small pages make for many boxes, and a warp issues them one
    // by one (1024 tokens over 6000 keys, heads of 256, pages of 16: 171 us by one warp, 119
    // by two, 99 by four; 4096 over 16384 of 128: 1002, 713 and 736); of codes there are
    // half as many, and widening needs the warps
    static constexpr int kCopyWarps = kCodes ? 1 : D == 256 ? 4 : 2;
    static constexpr int kShare = kCopyWarps == 4 ? 2 : 1;  // of them, a tile
    static constexpr int kOthers = (kLoadWarps - kCopyWarps) * 32;  // threads that check or widen
    static constexpr int kTileBytes = kKeys * D * 2;
    static constexpr int kStages = kCodes ? 3 : 4;
    // codes as they are in the cache, on their way
    static constexpr int kRaw = 3, kRawBytes = kCodes ? kKeys * D : 0;
    static constexpr int kQBytes = kTile * D * 2;
    static constexpr int kOutBytes = 1024;  // of a softmax warp: outputs on their way
    static constexpr int kSmem = kQBytes + kStages * kTileBytes + kRaw * kRawBytes + kSoft * kOutBytes + 1024;
    // Columns of tensor memory: scores from 0 (a buffer's 128), outputs from 256.  The
    // weights stand beside the scores; with heads of 128, which leave no room, in their
    // place: the next scores are then issued behind the product that reads the weights, and
    // the tensor core takes one thread's products, which are all of one shape there, in
    // the order of their issue.  (To wait for that product first takes 810 us where this
    // takes 725, at 4096 tokens over 16384 keys.)
    static constexpr uint32_t kOut = 256;
    __device__ static constexpr uint32_t weights_of(uint32_t buffer) {
        return D == 128 ? buffer * 128 : D == 64 ? 384 + buffer * 64 : buffer * 128 + 64;
    }
};

struct Shared {
    PlanShared plan;
    Cursor items[kItems];
    uint64_t known[kItems];  // that an item stands there
    uint64_t taken[kItems];  // that the warps which look values through have read it
    long long next_start;    // units before the next item
    // scores, weights and joined (outputs): of a score buffer.  A phase's parity is that of
    // the one before last, too, so a barrier is waited for only where the phase before is
    // known to be over: a buffer's scores are issued after the product of its last weights.
    uint64_t full[4], raw[2], empty[4], scores[2], weights[2], joined[2], query[2], drained;
    uint64_t coded[3], widened[3];  // of the tiles of codes: they are there, they are free
    uint8_t row_scale[4][2][128];   // of a unit's keys and values
    uint32_t largest[4][2];         // 0: scales too far apart
    float2 scales[8];               // of a unit: 2^e of the keys, e of the values; 0, 0 if too far apart
    float unscale[2][2 * kRows];    // codes: what a row's scores are multiplied by, of an item and the next
    uint32_t tmem;
    int dead;
    int looked[2];  // warps that have looked a tile through, of either stage
    int mark[kMarks];
};

// Cycles in which copies and products that are under way are over, by far: a block in which
// a wait has run out stays so long, however short that wait's limit is.
constexpr long long kLanding = 1000000;

// One lane of the warp, the same every time.
__device__ __forceinline__ bool ptx_elect() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Steps of 16 along the products' inner dimension, issued by one elected lane: A and B
// from shared memory (descriptors that advance by `step` every time and by `part` more
// every fourth time), or A from tensor memory (8 columns a step).
template <int STEPS>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t a_part, uint32_t b_part, uint32_t idesc) {
    if (ptx_elect()) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                "l"(a + (k >> 2) * a_part + (k & 3) * 2), "l"(b + (k >> 2) * b_part + (k & 3) * 2), "r"(idesc), "r"(k > 0 ? 1 : 0)
                : "memory");
    }
    __syncwarp();
}
template <int STEPS>
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (ptx_elect()) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                "r"(a + 8 * k), "l"(b + 128 * k), "r"(idesc), "r"(k > 0 ? 1u : acc)
                : "memory");
    }
    __syncwarp();
}

__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
        : "memory");
}

// Two fp32 operations in one instruction.
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Instruction descriptor, kind::f16: D fp32 (bits 4-5 = 1), A and B bf16 or fp16 (bits
// 7-9, 10-12 = 1 or 0), A K-major (bit 15 = 0), B's major (bit 16: 1 MN-major), N >> 3 in bits
// 17-22, M >> 4 in bits 24-28.
constexpr uint32_t idesc_f16(uint32_t n, uint32_t b_mn, bool bf16) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// smem_desc_sw128 with the leading byte offset that an MN-major operand has: from
// one 64-element wide part to the next.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lead) {
    uint64_t d = ptx::smem_desc_sw128(saddr) & ~(uint64_t(0x3FFF) << 16);
    return d | static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
}

__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a)
        : "memory");
}

// Waits for a phase, with a limit; false when it ran out here or anywhere in the
// block.  (Inline: a call would have to keep a row's scores over it.)
// EASY: probes now and then, as what it waits for is far ahead of its use, and probes
// take issue slots from the softmax.
template <bool EASY = false>
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, const AttnParams& p) {
    if (ptx::mbar_test(bar, parity)) return true;
    const long long began = clock64();
#pragma unroll 1
    while (!ptx::mbar_test(bar, parity)) {
        if (EASY) __nanosleep(100);
        if (*reinterpret_cast<volatile int*>(&sh.dead)) return false;
        if (clock64() - began > p.timeout_cycles) {
            record_error(p.err, FP8BS_ERR_TIMEOUT);
            *reinterpret_cast<volatile int*>(&sh.dead) = 1;
            return false;
        }
    }
    return true;
}

// A box of 64 dimensions x some slots of one head and page, in the 128-byte swizzle.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int d, int slot, int head, int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            ptx::smem_addr(dst)),
        "l"(map), "r"(d), "r"(slot), "r"(head), "r"(page), "r"(ptx::smem_addr(bar))
        : "memory");
}

// The items of the block's share, one after the other: a copy warp, which comes to them
// first, finds out what they are, and the other tasks read it.  (The code that does it is
// long, and there is one copy of it: what the instruction cache does not hold costs
// more than the look-up.)
// PACED: see kItems.  False when that wait ran out.
template <int ROWS, int UNIT, bool PACED>
__device__ __noinline__ bool publish(const AttnParams& p, Shared& sh, int item) {
    if (PACED && item >= kItems &&
        !__all_sync(0xFFFFFFFFu, wait<true>(sh, &sh.taken[item & (kItems - 1)], (item / kItems - 1) & 1, p)))
        return false;
    Cursor c;
    if (item == 0) {
        const AttnShare& s0 = sh.plan.share;
        c = attn_enter<ROWS, UNIT>(p, sh.plan, s0.tile, s0.b, s0.head);
    } else {
        c = sh.items[(item - 1) & (kItems - 1)];
        if (c.head + 1 < p.Hk) ++c.head;
        else if (c.tile + 1 < sh.plan.first[p.B]) c = attn_enter<ROWS, UNIT>(p, sh.plan, c.tile + 1, c.b, 0);
    }
    const AttnShare& a = sh.plan.share;
    const long long start = item == 0 ? a.begin - a.unit : sh.next_start;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        sh.next_start = start + c.n;
        if (start >= a.begin && start < a.end && start + c.n > a.end) {  // begun here, finished elsewhere
            AttnSplit rec = {c.rows, c.q0, c.row0, c.head, attn_last_block(a, start, c.n), {0, 0, 0}};
            reinterpret_cast<AttnSplit*>(p.ws)[blockIdx.x] = rec;
        }
        sh.items[item & (kItems - 1)] = c;
        ptx::mbar_arrive(&sh.known[item & (kItems - 1)]);
    }
    __syncwarp();
    return true;
}

// A task's place: the unit of an item.
struct Place : Cursor {
    int item;

    __device__ __forceinline__ bool enter(const AttnParams& p, Shared& sh, int k) {
        item = k;
        if (!__all_sync(0xFFFFFFFFu, wait<true>(sh, &sh.known[k & (kItems - 1)], (k / kItems) & 1, p))) return false;
        *static_cast<Cursor*>(this) = sh.items[k & (kItems - 1)];
        return true;
    }
    __device__ __forceinline__ bool start(const AttnParams& p, Shared& sh) {
        const bool ok = enter(p, sh, 0);
        unit = sh.plan.share.unit;
        return ok;
    }
    __device__ __forceinline__ bool next(const AttnParams& p, Shared& sh) {
        return ++unit < n || enter(p, sh, item + 1);
    }
};

constexpr uint32_t kApart = 14;  // 2^-14 times a code is exact in fp16

// 16 codes -> 16 fp16 numbers times the scale over the largest, or 1 where that is the
// smaller (NaN for a scale of 255).
__device__ __forceinline__ void widen(const uint4& c, uint32_t scale, uint32_t largest, uint4& lo, uint4& hi) {
    const uint32_t down = largest - min(scale, largest);  // (past kApart: no key, or a row of zeros)
    const uint32_t bits = scale == 255u ? 0x7E00u : down > kApart ? 0u : (15u - down) << 10;
    const __half2 f = __half2half2(__ushort_as_half(static_cast<unsigned short>(bits)));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    __half2 r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, b;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(w[i]));
        r[2 * i] = __hmul2_rn(*reinterpret_cast<__half2*>(&a), f), r[2 * i + 1] = __hmul2_rn(*reinterpret_cast<__half2*>(&b), f);
    }
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    lo = make_uint4(u[0], u[1], u[2], u[3]);
    hi = make_uint4(u[4], u[5], u[6], u[7]);
}

// Bits 15 and 31: whether the lower and the upper bf16 of a word have no finite value.
__device__ __forceinline__ uint32_t odd_pair(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// One warp issues boxes (a lane each) of up to a page's slots.
// bf16: they go where the products read them.  A unit's values that some row masks
// land on a barrier of their own, and the other loader warps look them through before
// they hand them on: rows that are no keys, which the boxes may cover or leave, become
// zeros, as do values that are not finite.
// Codes: boxes go to a ring of their own, with a unit's scales beside them (a lane reads
// those of four keys), and the other loader warps widen them.
// The next unit's pages are looked up behind a unit's boxes, in few instructions: two
// units ahead 4096 tokens over 16384 keys take 857 us, before the boxes 771, so 681.
template <int D, int KIND>
__device__ __forceinline__ void copy_units(const AttnParams& p, Shared& sh, uint8_t* ring, const CUtensorMap* mk,
                                           const CUtensorMap* mv, int kv0, int kv1, int which) {  // keys: 0, values: 1
    using C = Cfg<D, KIND>;
    constexpr int kParts = C::kCodes ? 1 : D / 64, kWide = C::kCodes ? D : 64;  // boxes over a row, and their width
    constexpr int kMost = C::kKeys * kParts / (32 * C::kShare);  // boxes of a lane
    constexpr int kRing = C::kCodes ? C::kRaw : C::kStages, kBoxRow = C::kCodes ? D : 128;
    const int lane = threadIdx.x & 31;
    const int rows = min(1 << p.page_log2, C::kKeys), boxes = C::kKeys / rows * kParts;
    const int units = static_cast<int>(sh.plan.share.end - sh.plan.share.begin);
    Place at;
    const bool publishes = kv0 == 0 && which == 0;
    auto box = [&](int i) { return (lane + 32 * i) * C::kShare + which; };  // a lane's boxes
    if (publishes) publish<C::kTile, C::kKeys, !C::kCodes>(p, sh, 0);
    bool alive = at.start(p, sh);
    uint32_t fill = 0;  // tiles of both kinds
    int page[kMost];
    auto page_of = [&](int j) {
        int id;
        return j >= at.first && j < at.past && attn_page(p, p.table + at.b * p.table_stride, j, &id) ? id : -1;
    };
    auto find = [&] {
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            if (32 * i * C::kShare >= boxes) break;
            const int j = (at.lo + at.unit) * C::kKeys + box(i) / kParts * rows;
            // (a box may begin before the first key and end past the last)
            page[i] = box(i) < boxes && j + rows > at.first ? page_of(max(j, at.first)) : -1;
        }
    };
    uint32_t zk[C::kKeys / 32], zv[C::kKeys / 32];
    auto read_scales = [&] {
#pragma unroll
        for (int i = 0; i < C::kKeys / 32; ++i) {
            const int j = (at.lo + at.unit) * C::kKeys + lane + 32 * i, id = page_of(j);
            zk[i] = zv[i] = 256;  // no key
            if (id >= 0) {
                const long long z = id * p.zpstride + (j & ((1 << p.page_log2) - 1)) * p.zsstride + at.head * p.zhstride;
                zk[i] = p.ks[z], zv[i] = p.vs[z];
            }
        }
    };
    auto keep_scales = [&](int u) {
        uint32_t mostk = 0, mostv = 47, leastk = 255, leastv = 255;
#pragma unroll
        for (int i = 0; i < C::kKeys / 32; ++i) {
            // A value's scale below 2^-80 counts as that (the sum of the weights, which are
            // taken against those times values, would leave fp32's range).  Rows of byte 0, as
            // rows of zeros have it, are zeros beside others: they set no scales apart.
            if (zv[i] != 0) zv[i] = max(zv[i], 47u);
            sh.row_scale[u & 3][0][lane + 32 * i] = static_cast<uint8_t>(zk[i]);
            sh.row_scale[u & 3][1][lane + 32 * i] = static_cast<uint8_t>(zv[i]);
            mostk = max(mostk, zk[i] < 255u ? zk[i] : 0u), leastk = min(leastk, zk[i] - 1u);
            mostv = max(mostv, zv[i] < 255u ? zv[i] : 0u), leastv = min(leastv, zv[i] - 1u);
        }
        mostk = __reduce_max_sync(0xFFFFFFFFu, mostk), mostv = __reduce_max_sync(0xFFFFFFFFu, mostv);
        const bool apart = __any_sync(0xFFFFFFFFu, mostk > leastk + 1 + kApart || mostv > leastv + 1 + kApart);
        if (lane == 0) {
            sh.largest[u & 3][0] = apart ? 0u : mostk, sh.largest[u & 3][1] = apart ? 0u : mostv;
            sh.scales[u & 7] = apart ? make_float2(0.0f, 0.0f) : make_float2(e8m0_to_float(mostk), static_cast<float>(static_cast<int>(mostv) - 127));
        }
        __syncwarp();
    };
    if (alive) find();
    if (alive && C::kCodes) read_scales();
#pragma unroll 1
    for (int u = 0; u < units && alive; ++u) {
        const int j0 = (at.lo + at.unit) * C::kKeys, head = at.head;
        const bool check = !C::kCodes && !attn_sees_all<C::kKeys>(p, at);
        int count = 0;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            if (32 * i * C::kShare >= boxes) break;
            count += __popc(__ballot_sync(0xFFFFFFFFu, page[i] >= 0));
        }
        if (C::kCodes) keep_scales(u);
#pragma unroll 1
        for (int kv = kv0; kv <= kv1; ++kv) {
            fill = 2 * static_cast<uint32_t>(u) + kv;
            const uint32_t stage = fill % kRing;
            if (alive && fill >= kRing)
                alive = __all_sync(0xFFFFFFFFu, wait<true>(sh, C::kCodes ? &sh.widened[stage] : &sh.empty[stage], ((fill / kRing) - 1) & 1, p));
            if (!alive) break;
            uint64_t* bar = C::kCodes ? &sh.coded[stage] : kv && check ? &sh.raw[stage >> 1] : &sh.full[stage];
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, count * rows * kBoxRow);
            __syncwarp();
            uint8_t* tile = ring + stage * (C::kCodes ? C::kRawBytes : C::kTileBytes);
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                if (32 * i * C::kShare >= boxes) break;
                if (page[i] >= 0) {
                    const int q = box(i), part = q % kParts, r = q / kParts * rows;
                    tma_box(tile + part * (C::kKeys * 128) + r * kBoxRow, kv ? mv : mk, kWide * part,
                            (j0 + r) & ((1 << p.page_log2) - 1), head, page[i], bar);
                }
            }
        }
        if (u + 1 < units && alive) {  // the next unit's pages, while this one's tiles come
            if (publishes && at.unit + 1 == at.n) alive = publish<C::kTile, C::kKeys, !C::kCodes>(p, sh, at.item + 1);
            alive = alive && at.next(p, sh);
            if (alive) find();
            if (alive && C::kCodes) read_scales();
        }
    }
}

template <int D>
__device__ __forceinline__ void check_units(const AttnParams& p, Shared& sh, uint8_t* ring) {
    using C = Cfg<D, FP8BS_KV_BF16>;
    constexpr int kThreads = C::kOthers, kPer = D / 8;
    const int tid = threadIdx.x - (C::kThreads - kThreads);
    const int units = static_cast<int>(sh.plan.share.end - sh.plan.share.begin);
    Place at;
    bool alive = at.start(p, sh);
    auto take = [&] {  // the item is read, by all lanes
        __syncwarp();
        if ((tid & 31) == 0) ptx::mbar_arrive(&sh.taken[at.item & (kItems - 1)]);
    };
    if (alive) take();
    uint32_t checked[2] = {0, 0};
#pragma unroll 1
    for (int u = 0; u < units && alive; ++u) {
        const int j0 = (at.lo + at.unit) * C::kKeys;
        if (!attn_sees_all<C::kKeys>(p, at)) {
            const uint32_t stage = (2 * static_cast<uint32_t>(u) + 1) % C::kStages;
            alive = __all_sync(0xFFFFFFFFu, wait<true>(sh, &sh.raw[stage >> 1], checked[stage >> 1] & 1, p));
            ++checked[stage >> 1];
            if (alive) {
                uint8_t* tile = ring + stage * C::kTileBytes;
                for (int i = tid; i < C::kKeys * kPer; i += kThreads) {
                    const int r = i / kPer, c = i % kPer, j = j0 + r;
                    uint4* q = reinterpret_cast<uint4*>(tile + (c >> 3) * (C::kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                    if (j < at.first || j >= at.past) {
                        *q = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint32_t w[4] = {q->x, q->y, q->z, q->w};
                    if (!((odd_pair(w[0]) | odd_pair(w[1])) | (odd_pair(w[2]) | odd_pair(w[3])))) continue;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t x = odd_pair(w[k]);
                        w[k] &= ((x >> 15 & 1) - 1 & 0xFFFFu) | ((x >> 31) - 1 & 0xFFFF0000u);
                        reinterpret_cast<uint32_t*>(q)[k] = w[k];
                    }
                    sh.mark[at.item & (kMarks - 1)] = at.item + 1;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if ((tid & 31) == 0) {  // the last of the warps hands the tile on
                    __threadfence_block();
                    if ((atomicAdd(&sh.looked[stage >> 1], 1) + 1) % (kThreads / 32) == 0) {
                        __threadfence_block();
                        for (int i = 0; i < C::kShare; ++i) ptx::mbar_arrive(&sh.full[stage]);
                    }
                }
            }
        }
        if (alive && u + 1 < units) {
            const int item = at.item;
            alive = at.next(p, sh);
            if (alive && at.item != item) take();
        }
    }
}

// Tiles of codes become the products' tiles.
template <int D>
__device__ __forceinline__ void widen_units(const AttnParams& p, Shared& sh, const uint8_t* raw, uint8_t* ring) {
    using C = Cfg<D, FP8BS_KV_E4M3>;
    constexpr int kThreads = C::kOthers, kPer = D / 16;  // 16-byte pieces of a row
    constexpr int kStep = kThreads / kPer;               // rows between a thread's pieces
    const int tid = threadIdx.x - (C::kThreads - kThreads), piece = tid % kPer;
    const int first = tid < kStep * kPer ? tid / kPer : C::kKeys;
    const int units = static_cast<int>(sh.plan.share.end - sh.plan.share.begin);
    Place at;
    bool alive = at.start(p, sh);
    uint32_t fill = 0;
#pragma unroll 1
    for (int u = 0; u < units && alive; ++u) {
        const int j0 = (at.lo + at.unit) * C::kKeys;
        const bool masks = !attn_sees_all<C::kKeys>(p, at);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++fill) {
            const uint32_t from = fill % C::kRaw, to = fill % C::kStages;
            alive = wait(sh, &sh.coded[from], (fill / C::kRaw) & 1, p);
            if (alive && fill >= C::kStages) alive = wait(sh, &sh.empty[to], ((fill / C::kStages) - 1) & 1, p);
            alive = __all_sync(0xFFFFFFFFu, alive);
            if (!alive) break;
            const uint32_t largest = sh.largest[u & 3][kv];
            uint8_t* tile = ring + to * C::kTileBytes;
            const uint8_t* source = raw + from * C::kRawBytes + 16 * piece;
            // a piece at a time: two at once 1106 us, four 1130 (one 1010 then), as the softmax
            // waits for the same issue slots (nor do eight or ten warps help: 1050, five 997)
#pragma unroll 1
            for (int r = first; r < C::kKeys; r += kStep) {
                uint4 codes = *reinterpret_cast<const uint4*>(source + r * D);
                uint32_t scale = sh.row_scale[u & 3][kv][r];
                if (kv && masks) {
                    const bool key = j0 + r >= at.first && j0 + r < at.past;
                    const bool none = !key || scale == 255u;
                    if (none || ((odd_codes(codes.x) | odd_codes(codes.y)) | (odd_codes(codes.z) | odd_codes(codes.w)))) {
                        // see the head of this file
                        if (key) sh.mark[at.item & (kMarks - 1)] = at.item + 1;
                        if (none) scale = largest;
                        codes = none ? make_uint4(0, 0, 0, 0)
                                     : make_uint4(without_odd_codes(codes.x), without_odd_codes(codes.y), without_odd_codes(codes.z), without_odd_codes(codes.w));
                    }
                }
                uint4 lo, hi;
                widen(codes, scale, largest, lo, hi);
                uint8_t* line = tile + (piece >> 2) * (C::kKeys * 128) + r * 128;
                const int c = 2 * (piece & 3);
                *reinterpret_cast<uint4*>(line + ((c ^ (r & 7)) << 4)) = lo;
                *reinterpret_cast<uint4*>(line + ((c + 1 ^ (r & 7)) << 4)) = hi;
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if ((tid & 31) == 0) {
                ptx::mbar_arrive(&sh.widened[from]);
                ptx::mbar_arrive(&sh.full[to]);
            }
        }
        if (alive && u + 1 < units) alive = at.next(p, sh);
    }
}

// The order of the products, in steps: the watcher waits for what a step needs and
// lets the issuer go through a hardware barrier, as a probe of a barrier in shared
// memory from the warp that issues would wait behind the products' own reads.  A step's
// barrier comes round after eight steps; the watcher is never that far ahead, as it
// waits for what follows from the issuer's steps.
//   two streams: (first scores of both), then for each unit and stream
//     [weights, values there; the next unit's keys]  O += P V, next S = Q K^T
//   one stream: (first scores), then for each unit
//     [the next unit's keys]   next S = Q K^T in the other buffer
//     [weights, values there]  O += P V
// After an item's last unit the next S has a step of its own, the last, in which the
// next item's queries are waited for.  Once a wait has run out, here or in another task
// (sh.dead), the watcher lets one more step go and leaves; the issuer looks before each
// step, so it finds that step or the mark, and leaves too.  (Weights handed over in halves
// of a unit's keys, to begin the product earlier, took 757 us where this takes 697.)
constexpr uint32_t kStepBarrier = 2, kStepBarriers = 8;

template <int D, int KIND>
__device__ __forceinline__ void watch(const AttnParams& p, Shared& sh) {
    using C = Cfg<D, KIND>;
    const int units = static_cast<int>(sh.plan.share.end - sh.plan.share.begin);
    Place at;
    uint32_t step = 0;
    bool alive = at.start(p, sh);
    auto need = [&](uint64_t* bar, uint32_t parity) {
        if (alive) alive = __all_sync(0xFFFFFFFFu, wait(sh, bar, parity, p));
    };
    auto full = [&](uint32_t fill) { need(&sh.full[fill % C::kStages], (fill / C::kStages) & 1); };
    auto go = [&] {
        if (!alive) __threadfence_block();  // the mark is seen with the step
        ptx::named_arrive(kStepBarrier + step++ % kStepBarriers, 64);
        return alive;
    };
    uint32_t items = 0;
    need(&sh.query[0], 0);
    if (C::kStreams == 2) need(&sh.query[1], 0);
    full(0);
    if (!go()) return;
#pragma unroll 1
    for (int u = 0; u < units; ++u) {
        const uint32_t fv = 2 * static_cast<uint32_t>(u) + 1, fk = fv + 1;
        const bool more = u + 1 < units, last = at.unit + 1 == at.n;
        if (more) alive = at.next(p, sh);
        items += last;
        if (C::kStreams == 2) {
            full(fv);
            if (more) full(fk);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                need(&sh.weights[s], u & 1);
                if (!go()) return;
                if (more && last) {
                    need(&sh.query[s], items & 1);
                    if (!go()) return;
                }
            }
        } else {
            if (more && !last) {
                full(fk);
                if (!go()) return;
            }
            full(fv);
            need(&sh.weights[u & 1], (u >> 1) & 1);
            if (!go()) return;
            if (more && last) {
                full(fk);
                need(&sh.query[0], items & 1);
                if (!go()) return;
            }
        }
    }
}

template <int D, int KIND>
__device__ __forceinline__ void issue_products(const AttnParams& p, Shared& sh, uint32_t query, uint32_t ring) {
    using C = Cfg<D, KIND>;
    constexpr uint32_t kScoreDesc = idesc_f16(C::kKeys, 0, !C::kCodes), kValueDesc = idesc_f16(D, 1, !C::kCodes);
    const int units = static_cast<int>(sh.plan.share.end - sh.plan.share.begin);
    const uint32_t tmem = sh.tmem;
    uint32_t step = 0;
    auto over = [&] { return __any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(&sh.dead) != 0); };
    auto come = [&] {
        if (over()) return false;
        ptx::named_sync(kStepBarrier + step++ % kStepBarriers, 64);
        ptx::tc_fence_after();
        return true;
    };
    auto tile = [&](uint32_t fill) { return ring + fill % C::kStages * C::kTileBytes; };
    auto scores = [&](int stream, int buffer, uint32_t keys, int rows) {
        if (rows > stream * kRows)
            mma_scores<D / 16>(tmem + buffer * 128, ptx::smem_desc_sw128(query + stream * kRows * D * 2), ptx::smem_desc_sw128(keys),
                               kRows * 128 / 16, C::kKeys * 128 / 16, kScoreDesc);
        ptx::mma_commit_warp(&sh.scores[buffer]);
    };
    auto values = [&](int stream, int buffer, uint32_t vals, int rows, bool first) {
        if (rows > stream * kRows)
            mma_values<C::kKeys / 16>(tmem + C::kOut + stream * D, tmem + C::weights_of(buffer), desc_mn(vals, C::kKeys * 128), kValueDesc,
                                      !first);
        ptx::mma_commit_warp(&sh.joined[buffer]);
    };

    if (!come() || over()) return;
    // (the watcher has seen that the items which are read here are known; of one that is
    // not, in the step after a wait has run out, no more is used than how many rows it has)
    int item = 0, unit = sh.plan.share.unit, n = sh.items[0].n, rows = sh.items[0].rows;
    bool first = true;  // the unit is its item's first here
#pragma unroll 1
    for (int s = 0; s < C::kStreams; ++s) scores(s, s, tile(0), rows);
    ptx::mma_commit_warp(&sh.empty[0]);
#pragma unroll 1
    for (int u = 0; u < units; ++u) {
        const uint32_t fv = 2 * static_cast<uint32_t>(u) + 1, fk = fv + 1;
        const bool more = u + 1 < units, last = unit + 1 == n;
        const int rows_now = rows;
        auto go_on = [&] {  // to the next item, once the watcher has seen that it is known
            ++item;
            n = sh.items[item & (kItems - 1)].n, rows = sh.items[item & (kItems - 1)].rows;
        };
        unit = last ? 0 : unit + 1;
        if constexpr (C::kStreams == 2) {
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
                if (!come()) return;
                values(s, s, tile(fv), rows_now, first);
                if (s == 1) ptx::mma_commit_warp(&sh.empty[fv % C::kStages]);
                if (more) {
                    if (last) {
                        if (!come()) return;
                        if (s == 0) go_on();
                    }
                    scores(s, s, tile(fk), rows);
                    if (s == 1) ptx::mma_commit_warp(&sh.empty[fk % C::kStages]);
                }
            }
        } else {
            const int b = u & 1;
            auto next = [&] {
                if (!come()) return false;
                if (last) go_on();
                scores(0, b ^ 1, tile(fk), rows);
                ptx::mma_commit_warp(&sh.empty[fk % C::kStages]);
                return true;
            };
            if (more && !last && !next()) return;
            if (!come()) return;
            values(0, b, tile(fv), rows_now, first);
            ptx::mma_commit_warp(&sh.empty[fv % C::kStages]);
            if (more && last && !next()) return;
        }
        first = last;
    }
}

// Minus infinity in the place of the scores of keys past `hi` and before `lo`, in tensor
// memory: a short loop.  (This and all else that does not run for every unit is kept
// short: its code comes from far, as the loops over units fill the instruction cache.
// Masks, unrolled over a row in registers, took 12 us a unit.)
template <int KEYS>
__device__ __forceinline__ void mask_scores(uint32_t scores, int hi, int lo) {
#pragma unroll 1
    for (int c = 0; c < KEYS; c += 16) {
        uint32_t s[16];
        ptx::tmem_ld_32x32b_x16(scores + c, s);
        ptx::tmem_wait_ld();
        const int h = min(hi - c, 15), l = lo - c;
        uint32_t seen = h < 0 ? 0u : 0xFFFFu >> (15 - h);  // bit i: this row sees key c + i
        if (l > 0) seen = l > 15 ? 0u : seen >> l << l;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (!(seen >> i & 1)) s[i] = 0xFF800000u;
        tmem_st16(scores + c, s);
    }
    ptx::tmem_wait_st();
}

// Scores in units of log2 with the exponents of the values' scales, each rounded for itself,
// in the place of a row's products with the keys: x factor + e, or, where the scales of a
// unit are far apart (row_scale), with each key's own.
template <int KEYS>
__device__ __noinline__ void far_scores(uint32_t scores, const uint8_t (*row_scale)[128], float factor, float e) {
#pragma unroll 1
    for (int c = 0; c < KEYS; c += 16) {
        uint32_t s[16];
        ptx::tmem_ld_32x32b_x16(scores + c, s);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (s[i] != 0xFF800000u) {  // (masked: whatever scale that key has)
                const float x = __fmul_rn(__uint_as_float(s[i]), factor);
                s[i] = __float_as_uint(row_scale ? __fadd_rn(__fmul_rn(x, e8m0_to_float(row_scale[0][c + i])),
                                                             static_cast<float>(max(static_cast<int>(row_scale[1][c + i]), 47) - 127))
                                                 : __fadd_rn(x, e));
            }
        }
        tmem_st16(scores + c, s);
    }
    ptx::tmem_wait_st();
}

// The sum of a row's weights without the values' scales, which far_scores has put into them.
template <int KEYS>
__device__ __noinline__ float far_sum(uint32_t scores, const uint8_t (*row_scale)[128], float base) {
    float sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < KEYS; c += 16) {
        uint32_t s[16];
        ptx::tmem_ld_32x32b_x16(scores + c, s);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sum += ex2(__uint_as_float(s[i]) - base + static_cast<float>(127 - max(static_cast<int>(row_scale[1][c + i]), 47)));
    }
    return sum;
}

// The values that are not finite, among the keys that a row sees in the item's units
// with masks from `from` on, where zeros stood for them: added to what the row has in
// o or, without that, in a slot.
template <int D, int KIND>
__device__ __forceinline__ void add_odd(const AttnParams& p, Cursor c, int from, int place, uint16_t* o, float* slot) {
    constexpr int kKeys = Cfg<D, KIND>::kKeys;
    const int upto = c.unit;
#pragma unroll 1
    for (c.unit = from; c.unit <= upto; ++c.unit) {
        if (attn_sees_all<kKeys>(p, c)) continue;
        const int j0 = (c.lo + c.unit) * kKeys;
#pragma unroll 1
        for (int j = max(j0, c.first); j < min(j0 + kKeys, c.past); ++j) {
            int page;
            if (j > place || (p.window && j <= place - p.window)) continue;
            if (!attn_page(p, p.table + c.b * p.table_stride, j, &page)) continue;
            const int s = j & ((1 << p.page_log2) - 1);
            const bool codes = KIND == FP8BS_KV_E4M3;
            const bool none = codes && p.vs[page * p.zpstride + s * p.zsstride + c.head * p.zhstride] == 255;
            const uint8_t* v = p.v + page * p.pstride + s * p.sstride + c.head * p.hstride;
#pragma unroll 1
            for (int i = 0; i < D; ++i) {
                const float x = codes ? __uint_as_float(none || odd_codes(v[i]) ? 0x7FFFFFFFu : 0u)
                                      : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(v)[i]);
                if (isfinite(x)) continue;
                if (o) o[i] = static_cast<uint16_t>(pack_bf16(bf16_bits_to_float(o[i]) + x, 0.0f));
                else slot[i] += x;
            }
        }
    }
}

template <int D, int KIND>
__device__ __forceinline__ void weigh(const AttnParams& p, Shared& sh, uint8_t* query, uint8_t* way) {
    using C = Cfg<D, KIND>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3, stream = warp >> 2;
    const int row = quarter * 32 + lane;  // of the stream
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int units = static_cast<int>(sh.plan.share.end - sh.plan.share.begin);
    const uint32_t out = sh.tmem + C::kOut + stream * D + lanes;
    const uint32_t own = stream * kRows * D * 2;  // the stream's queries
    uint8_t* staged = way + warp * C::kOutBytes;
    Place at;
    if (!at.start(p, sh)) return;

    auto query_row = [&](int r, int* token, int* head) {  // of the stream; past the last: the last
        const int packed = at.row0 + min(stream * kRows + r, at.rows - 1);
        *token = div_g(p, packed);
        *head = at.head * p.G + packed - *token * p.G;
    };
    // The queries: eight lanes a row, four rows of a warp at a time, in turns with the
    // stream's other warps (few rows are then soon there: a thread a row took 8400 cycles
    // to bring 32 rows of 256 into fp16).  Rows that are not there keep what lies there:
    // no row's results depend on another's.
    const int part = lane & 7;
    auto piece = [&](int r, int i) { return own + r * 128 + i * (kRows * 128) + ((part ^ (r & 7)) << 4); };
    auto fetch_query = [&] {
#pragma unroll 1
        for (int r0 = 4 * quarter; r0 < min(kRows, at.rows - stream * kRows); r0 += 16) {
            const int r = r0 + (lane >> 3);
            int token, head;
            query_row(r, &token, &head);
            const uint16_t* src = p.q + static_cast<int64_t>(at.q0 + token) * p.ldq + head * p.hsq + 8 * part;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) cp_async16(ptx::smem_addr(query) + piece(r, i), src + 64 * i);
        }
        cp_commit();
    };
    auto query_ready = [&] {
        cp_wait<0>();
        if (C::kCodes) {  // the rows in fp16, in place
#pragma unroll 1
            for (int r0 = 4 * quarter; r0 < min(kRows, at.rows - stream * kRows); r0 += 16) {
                const int r = r0 + (lane >> 3);
                uint4 v[D / 64];
                uint32_t largest = 0;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    v[i] = *reinterpret_cast<const uint4*>(query + piece(r, i));
                    const uint32_t lo = max(max(v[i].x & 0x7FFFu, v[i].y & 0x7FFFu), max(v[i].z & 0x7FFFu, v[i].w & 0x7FFFu));
                    const uint32_t hi = max(max(v[i].x >> 16 & 0x7FFFu, v[i].y >> 16 & 0x7FFFu), max(v[i].z >> 16 & 0x7FFFu, v[i].w >> 16 & 0x7FFFu));
                    largest = max(largest, max(lo, hi));
                }
#pragma unroll
                for (int off = 1; off < 8; off <<= 1) largest = max(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, off));
                // zeros, and rows with an infinity or a NaN, stay
                const int e = static_cast<int>(largest >> 7), up = largest == 0 || e == 255 ? 0 : min(14 - (e - 127), 126);
                const float factor = __int_as_float((up + 127) << 23);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    float x[8];
                    unpack_bf16x8(v[i], x);
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[k]) : "f"(x[2 * k + 1] * factor), "f"(x[2 * k] * factor));
                    *reinterpret_cast<uint4*>(query + piece(r, i)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                if (part == 0) sh.unscale[at.item & 1][stream * kRows + r] = __int_as_float((127 - up) << 23) * p.scale_log2;
            }
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&sh.query[stream]);
    };
    fetch_query();
    query_ready();
    float now = 0.0f;  // codes: what the row's scores are multiplied by, beside their unit's scale
    float most = -INFINITY, sum = 0.0f;
    bool first = true;
    bool begun = at.unit == 0;
    int from = at.unit;
#pragma unroll 1
    for (int u = 0; u < units; ++u) {
        const int buffer = C::kStreams == 2 ? stream : static_cast<int>(u & 1);
        const uint32_t parity = C::kStreams == 2 ? u & 1 : (u >> 1) & 1;
        const uint32_t scores = sh.tmem + buffer * 128 + lanes, weights = sh.tmem + C::weights_of(buffer) + lanes;
        const bool active = at.rows > stream * kRows;
        const int j0 = (at.lo + at.unit) * C::kKeys;
        const bool last = at.unit + 1 == at.n, done = last || u + 1 == units;
        if (!__all_sync(0xFFFFFFFFu, wait(sh, &sh.scores[buffer], parity, p))) return;
        ptx::tc_fence_after();
        if (active) {
            // (the row's warps had it there before they let its scores begin)
            if (C::kCodes && first) now = sh.unscale[at.item & 1][stream * kRows + row];
            if (!attn_sees_all<C::kKeys>(p, at)) {
                int token, head;
                query_row(row, &token, &head);
                const int hi = at.base + token - j0;
                mask_scores<C::kKeys>(scores, hi, p.window ? hi - p.window + 1 : 0);
            }
            const float2 scale = C::kCodes ? sh.scales[u & 7] : make_float2(1.0f, 0.0f);
            const bool apart = C::kCodes && scale.x == 0.0f;
            if (apart) far_scores<C::kKeys>(scores, sh.row_scale[u & 3], now, 0.0f);
            // Codes: a loop over 32 scores, which are read again for their weights: the loaders'
            // code is long, and all of it has to stay in the instruction cache (4096 tokens over
            // 16384 keys 1065 us without, 997 so).  bf16: a row's scores in registers (681 us,
            // read twice in a loop 746).
            constexpr int kTimes = C::kCodes ? 1 : C::kKeys / 32;
            float s[32 * kTimes];
            if (!C::kCodes) {
#pragma unroll
                for (int i = 0; i < kTimes; ++i) tmem_ld32(scores + 32 * i, reinterpret_cast<uint32_t*>(s) + 32 * i);
                ptx::tmem_wait_ld();
            }
            auto some = [&](int c) {  // scores 32 c and on
                if (!C::kCodes) return s + 32 * c % (32 * kTimes);
                tmem_ld32(scores + 32 * c, reinterpret_cast<uint32_t*>(s));
                ptx::tmem_wait_ld();
                return s;
            };
            // eight chains, so that none is long
            float tops[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) tops[i] = -INFINITY;
#pragma unroll kTimes
            for (int c = 0; c < C::kKeys / 32; ++c) {
                const float* x = some(c);
#pragma unroll
                for (int i = 0; i < 32; i += 2) tops[(i >> 1) & 7] = fmaxf(tops[(i >> 1) & 7], fmaxf(x[i], x[i + 1]));
            }
            // (above zero, so that masked scores stay minus infinity; scores are below 2^34, and
            // 2^-126 of that is nothing)
            float factor = apart ? 1.0f : C::kCodes ? fminf(fmaxf(now * scale.x, 0x1p-126f), 0x1.fffffep127f) : p.scale_log2;
            const float top = __fadd_rn(scale.y, __fmul_rn(factor, fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                                                                         fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])))));
            // A score is not rounded before the maximum, which is, is taken from it.  Where that
            // rounding is no small part of a power of two, weights would leave their range.
            float with = scale.y;  // of the maximum, and not of the scores
            if (__any_sync(0xFFFFFFFFu, fabsf(top) > kFar && top > -INFINITY && stream * kRows + row < at.rows)) {
                if (!apart) far_scores<C::kKeys>(scores, nullptr, factor, scale.y);
                if (!C::kCodes) {
#pragma unroll
                    for (int i = 0; i < kTimes; ++i) tmem_ld32(scores + 32 * i, reinterpret_cast<uint32_t*>(s) + 32 * i);
                    ptx::tmem_wait_ld();
                }
                factor = 1.0f, with = 0.0f;
            }
            float fall = 0.0f;
            if (top > __fadd_rd(most, kLag)) {
                fall = most - top;
                most = top;
            }
            if (__any_sync(0xFFFFFFFFu, fall != 0.0f)) {
                const float shrink = ex2(fall);  // 0 from minus infinity
                sum = fallen(sum, fall);
                if (!first) {
                    // the products before this one are in the outputs
                    if (!__all_sync(0xFFFFFFFFu, wait(sh, &sh.joined[C::kStreams == 2 ? stream : buffer ^ 1], (C::kStreams == 2 ? u - 1 : (u - 1) >> 1) & 1, p))) return;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        ptx::tmem_ld_32x32b_x16(out + c, o);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
                        tmem_st16(out + c, o);
                    }
                    ptx::tmem_wait_st();
                }
            }
            const float base = __fsub_ru(most == -INFINITY ? 0.0f : most, with + (C::kCodes ? 7.0f : 0.0f));
            float own = 0.0f;
            if (apart) own = far_sum<C::kKeys>(scores, sh.row_scale[u & 3], base);
            const uint64_t factors = pair(factor, factor), minus = pair(-base, -base);
            uint64_t sums[4] = {0, 0, 0, 0};
#pragma unroll kTimes
            for (int c = 0; c < C::kKeys / 32; ++c) {
                const float* y = some(c);
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 x = halves(fma2(pair(y[2 * i], y[2 * i + 1]), factors, minus));
                    const float a = ex2(x.x), b = ex2(x.y);
                    sums[i & 3] = add2(sums[i & 3], pair(a, b));
                    if (C::kCodes) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
                    else w[i] = pack_bf16(a, b);
                }
                tmem_st16(weights + 16 * c, w);
            }
            const float2 both = halves(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
            sum += apart ? own : C::kCodes ? (both.x + both.y) * ex2(-scale.y) : both.x + both.y;
            ptx::tmem_wait_st();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&sh.weights[buffer]);
        first = false;
        if (!done) {
            ++at.unit;
            continue;
        }
        // the item's last unit here: the next one's queries, then this one's rows
        const Place was = at;
        int token, head;
        query_row(row, &token, &head);
        if (u + 1 < units) {
            if (!at.enter(p, sh, at.item + 1)) return;
            fetch_query();
        }
        if (u + 1 < units) query_ready();
        if (!__all_sync(0xFFFFFFFFu, wait(sh, &sh.joined[buffer], parity, p))) return;
        ptx::tc_fence_after();
        if (active) {
            const bool whole = last && begun, there = stream * kRows + row < was.rows;
            const bool odd = *reinterpret_cast<volatile int*>(&sh.mark[was.item & (kMarks - 1)]) == was.item + 1;
            if (sum == 0.0f && was.base + token >= 0) sum = kNoWeight;
            const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : __frcp_rn(sum);
            uint16_t* dst = p.o + static_cast<int64_t>(was.q0 + token) * p.ldo + head * p.hso;
            const int at_row = stream * kRows + row;
            float* slot = attn_slot(p, gridDim.x, C::kTile, D, blockIdx.x, begun) + at_row * D;
            // Whole rows go by way of shared memory, so that two lanes write 32 bytes of one:
            // a store's time goes with the lines that it touches.
            const unsigned long long own = there ? reinterpret_cast<unsigned long long>(dst) : 0;
            const unsigned long long to0 = __shfl_sync(0xFFFFFFFFu, own, lane >> 1);
            const unsigned long long to1 = __shfl_sync(0xFFFFFFFFu, own, 16 + (lane >> 1));
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                ptx::tmem_ld_32x32b_x16(out + c, o);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                    uint4* to = reinterpret_cast<uint4*>(staged + lane * 32);
                    const int swizzle = lane >> 2 & 1;
                    to[swizzle] = make_uint4(o[0], o[1], o[2], o[3]);
                    to[swizzle ^ 1] = make_uint4(o[4], o[5], o[6], o[7]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = 16 * i + (lane >> 1);
                        const uint4 v = reinterpret_cast<const uint4*>(staged + r * 32)[(lane & 1) ^ (r >> 2 & 1)];
                        const unsigned long long d = i ? to1 : to0;
                        if (d) *reinterpret_cast<uint4*>(d + 2 * c + 16 * (lane & 1)) = v;
                    }
                    __syncwarp();
                } else if (there) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<uint4*>(slot + c)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            if (there && !whole) {
                float* end = attn_slot(p, gridDim.x, C::kTile, D, blockIdx.x, begun) + C::kTile * D;
                end[at_row] = most;
                end[C::kTile + at_row] = sum;
            }
            if (odd) {  // (rows were written by other lanes of the warp)
                __syncwarp();
                if (there) add_odd<D, KIND>(p, was, from, was.base + token, whole ? dst : nullptr, slot);
            }
        }
        ptx::tc_fence_before();
        most = -INFINITY, sum = 0.0f;
        first = begun = true;
        from = 0;
    }
}

template <int D, int KIND>
__global__ void __launch_bounds__(Cfg<D, KIND>::kThreads, 1) attn_chunk_kernel(const __grid_constant__ AttnParams p,
                                                                          const __grid_constant__ CUtensorMap mk,
                                                                          const __grid_constant__ CUtensorMap mv) {
    using C = Cfg<D, KIND>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    static_assert(C::kSmem + sizeof(Shared) <= 227 * 1024, "more shared memory than a block has");
    uint8_t* query = raw + ((1024 - (ptx::smem_addr(raw) & 1023)) & 1023);
    uint8_t* ring = query + C::kQBytes;
    uint8_t* raws = ring + C::kStages * C::kTileBytes;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) ptx::mbar_init(&sh.full[i], C::kCodes ? C::kOthers / 32 : C::kShare), ptx::mbar_init(&sh.empty[i], 1);
        for (int i = 0; i < C::kRaw; ++i) ptx::mbar_init(&sh.coded[i], 1), ptx::mbar_init(&sh.widened[i], C::kOthers / 32);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.raw[i], C::kShare);
            ptx::mbar_init(&sh.scores[i], 1);
            ptx::mbar_init(&sh.weights[i], 128);
            ptx::mbar_init(&sh.joined[i], 1);
            ptx::mbar_init(&sh.query[i], 128);
        }
        ptx::mbar_init(&sh.drained, 1);
        for (int i = 0; i < kItems; ++i) ptx::mbar_init(&sh.known[i], 1), ptx::mbar_init(&sh.taken[i], C::kOthers / 32);
        ptx::fence_mbar_init();
        sh.dead = 0;
        sh.looked[0] = sh.looked[1] = 0;
        for (int i = 0; i < kMarks; ++i) sh.mark[i] = 0;
    }
    if (warp == C::kSoft) {
        ptx::tmem_alloc(&sh.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (threadIdx.x == 0) reinterpret_cast<AttnSplit*>(p.ws)[blockIdx.x].rows = 0;
    ptx::tc_fence_before();
    attn_share<C::kTile, C::kKeys, C::kThreads>(p, sh.plan);
    ptx::tc_fence_after();
    if (sh.plan.share.begin < sh.plan.share.end) {
        if (C::kDeal) {
            if (warp < C::kSoft) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kMoreRegs));
            else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kFewRegs));
        }
        if (warp < C::kSoft) weigh<D, KIND>(p, sh, query, raws + C::kRaw * C::kRawBytes);
        else if (warp == C::kSoft) issue_products<D, KIND>(p, sh, ptx::smem_addr(query), ptx::smem_addr(ring));
        else if (warp == C::kSoft + 1) watch<D, KIND>(p, sh);
        else if (warp < C::kSoft + 2 + C::kCopyWarps)
            copy_units<D, KIND>(p, sh, C::kCodes ? raws : ring, &mk, &mv, (warp - C::kSoft - 2) / C::kShare,
                                C::kCopyWarps == 1 ? 1 : (warp - C::kSoft - 2) / C::kShare, (warp - C::kSoft - 2) % C::kShare);
        else if constexpr (C::kCodes) widen_units<D>(p, sh, raws, ring);
        else check_units<D>(p, sh, ring);
        ptx::cp_async_wait_all();
        if (warp == C::kSoft) {
            // nothing of the tensor core's is under way when the memory is given back
            ptx::mma_commit_warp(&sh.drained);
            const long long began = clock64();
            while (!ptx::mbar_test(&sh.drained, 0) && clock64() - began < kLanding) {
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (sh.dead) {
        const long long began = clock64();
        while (clock64() - began < kLanding) __nanosleep(1000);
    }
    if (warp == C::kSoft) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(sh.tmem, 512);
    }
}

// The driver's tensor map encoder (looked up once; the library does not link to the driver).
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
    static std::atomic<Encode> found{nullptr};
    Encode e = found.load(std::memory_order_acquire);
    if (!e) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult got;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &got) != cudaSuccess ||
            got != cudaDriverEntryPointSuccess)
            return nullptr;
        e = reinterpret_cast<Encode>(f);
        found.store(e, std::memory_order_release);
    }
    return e;
}

// Keys or values as [page][head][slot][D], boxes of `rows` slots x 64 dimensions in the
// products' swizzle, or of codes x D.  An axis of one place takes any stride.
bool describe(CUtensorMap* map, const AttnArgs& a, const uint8_t* base, int rows) {
    const Encode e = encoder();
    if (!e) return false;
    const bool codes = a.kind == FP8BS_KV_E4M3;
    const int page = 1 << a.page_log2;
    const cuuint64_t own = static_cast<cuuint64_t>(a.D) * (codes ? 1 : 2);
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(a.Hk),
                                static_cast<cuuint64_t>(a.pages)};
    const cuuint64_t strides[3] = {page > 1 ? static_cast<cuuint64_t>(a.sstride) : own,
                                   a.Hk > 1 ? static_cast<cuuint64_t>(a.hstride) : own,
                                   a.pages > 1 ? static_cast<cuuint64_t>(a.pstride) : own};
    const cuuint32_t box[4] = {codes ? static_cast<cuuint32_t>(a.D) : 64u, static_cast<cuuint32_t>(rows), 1, 1}, step[4] = {1, 1, 1, 1};
    return e(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint8_t*>(base), dims,
             strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KIND>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    using C = Cfg<D, KIND>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = attn_allow_shared(attn_chunk_kernel<D, KIND>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    CUtensorMap mk = {}, mv = {};
    const int rows = min(1 << a.page_log2, C::kKeys);
    if (!describe(&mk, a, a.k, rows)) {
        // the first call of a host thread: the device's context is not current in it yet
        int dev = 0;
        cudaError_t s = cudaGetDevice(&dev);
        if (s == cudaSuccess) s = cudaSetDevice(dev);
        if (s != cudaSuccess) return s;
        if (!describe(&mk, a, a.k, rows)) return cudaErrorInvalidValue;
    }
    if (!describe(&mv, a, a.v, rows)) return cudaErrorInvalidValue;
    const cudaError_t r = w4::launch_dependent(attn_chunk_kernel<D, KIND>, a.sm_count, C::kThreads, C::kSmem, stream,
                                               static_cast<const AttnParams&>(a), mk, mv);
    return r == cudaSuccess ? launch_attn_join(a, C::kTile, a.sm_count, stream) : r;
}

}  // namespace

size_t attn_chunk_slot_floats(int D) {
    return D == 256 ? attn_slot_floats(Cfg<256, 0>::kTile, 256) : attn_slot_floats(Cfg<128, 0>::kTile, D);
}

cudaError_t launch_attn_chunk(const AttnArgs& a, cudaStream_t stream) {
    if (a.kind == FP8BS_KV_BF16) {
        if (a.D == 64) return launch<64, FP8BS_KV_BF16>(a, stream);
        if (a.D == 128) return launch<128, FP8BS_KV_BF16>(a, stream);
        return launch<256, FP8BS_KV_BF16>(a, stream);
    }
    if (a.D == 64) return launch<64, FP8BS_KV_E4M3>(a, stream);
    if (a.D == 128) return launch<128, FP8BS_KV_E4M3>(a, stream);
    return launch<256, FP8BS_KV_E4M3>(a, stream);
}

}  // namespace fp8bs
