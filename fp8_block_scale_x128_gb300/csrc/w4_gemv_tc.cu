// y[M, N] = bf16(x . W^T) for up to 16 bf16 tokens and an MXFP4 weight on the
// block-scaled tensor core (tcgen05.mma kind::mxf8f6f4): the e2m1 codes are the
// MMA's A operand as they are and the e8m0 group scales its scale factors, so
// no instruction decodes or scales a weight.
//
// The other operand is e4m3, 4 significant bits, and a bf16 value has 8.  A
// token becomes four columns: with x' = x 2^-e of its 32-wide group (the largest
// magnitude brought into [128, 256)),
//   t1 = e4m3(x'), t2 = e4m3((x' - t1) 2^5), t3 = e4m3((x' - t1 - t2 2^-5) 2^22),
//   t4 = e4m3((x' - t1 - t2 2^-5 - t3 2^-22) 2^27),
// each column with its own e8m0 scale.  t1 + t2 is x itself down to 2^-14 of the
// group's largest magnitude (a rounding to 4 bits leaves at most 4 bits), t3
// and t4 hold the smaller ones to 2^-40 of it.  Every product is exact, the sums
// are the tensor core's fp32.
//
// Swap-AB: D[128 weight rows][N columns], N = 4 M rounded up to 16, accumulated
// over the block's whole range of K in TMEM.  Warps 0-3 copy codes (8-byte
// cp.async: 16 codes fill the low half of a 16-byte unit, the operand's layout
// for 4-bit elements, 128-byte swizzle), store the rows' scale words into TMEM
// and issue the MMAs; warps 4-7 turn x into columns ahead of them.  A cluster
// splits K; its blocks' sums meet through distributed shared memory in rank
// order, so repeated calls give the same bits.
//
// A token with an infinity or NaN in a block's range of K is summed there by
// plain fp32 multiply-adds instead.
#include "internal.cuh"
#include "w4.cuh"

namespace fp8bs {
namespace {

using namespace w4;

constexpr int kThreads = 256;
constexpr int kRowsBlock = 128;
constexpr int kStages = 5;  // of the code ring: 2 chunks of 128 rows each
constexpr int kChunkBytes = 128 * 128;
constexpr int kStageBytes = 2 * kChunkBytes;
constexpr int kMaxSlots = 8;  // of the column ring
constexpr uint32_t kSfaCol = 64, kSfbCol = kSfaCol + 8 * kStages;
constexpr uint32_t kTmemCols = 256;
static_assert(kSfbCol + 8 * kMaxSlots <= kTmemCols, "TMEM columns");
constexpr long long kWaitCycles = 2000000000LL;  // ~1 s: far above any legitimate wait
constexpr int kSfbBytes = 2 * 64 * 4;            // scale words of a column slot

struct TcParams {
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* codes;
    int64_t ldc;
    const uint8_t* scales;
    int64_t lds;
    uint16_t* y;
    int64_t ldy;
    int M, N, chunks;
    int cols;   // MMA columns: 4 M rounded up to 16
    int slots;  // of the column ring
    int pdl;
};

constexpr int kMiscBytes = 512;  // barriers, TMEM address, flags
__host__ __device__ inline int tc_bytes(int cols, int slots) {
    return kStages * kStageBytes + slots * (2 * cols * 128 + kSfbBytes) + kMiscBytes;
}

// Bounded wait for a barrier phase; false (and the abort flag) when it expires.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
    const long long t0 = clock64();
    while (!ptx::mbar_test(bar, parity)) {
        if (*abort_flag || clock64() - t0 > kWaitCycles) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
    return ptx::mbar_test(bar, parity) || wait_slow(bar, parity, abort_flag);
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t v) {
    asm volatile("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tst.shared.b8 [%0], h;\n\t}" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Instruction descriptor: A e2m1 (format 5), B e4m3 (0), e8m0 scales, both
// K-major; byte k of the scale words.
__device__ __forceinline__ uint32_t idesc_e2m1_e4m3(uint32_t n, uint32_t k) {
    return (k << 4) | (5u << 7) | ((n >> 3) << 17) | (1u << 23) | ((kRowsBlock >> 4) << 24) | (k << 29);
}

// Plain sum of one row and token over [k0, k1), for tokens with infinities or NaN.
__device__ __noinline__ float plain_sum(const TcParams& p, int row, int m, int k0, int k1) {
    const uint8_t* c = p.codes + row * p.ldc;
    const uint8_t* s = p.scales + row * p.lds;
    const uint16_t* x = p.x + m * p.ldx;
    float v = 0.0f;
    for (int k = k0; k < k1; k += 32) {
        float part = 0.0f;
        for (int i = 0; i < 32; i += 2) {
            uint32_t two;
            asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
                : "=r"(two)
                : "r"(static_cast<uint32_t>(c[(k + i) / 2])));
            const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&two));
            part = fmaf(w.x, bf16_bits_to_float(x[k + i]), part);
            part = fmaf(w.y, bf16_bits_to_float(x[k + i + 1]), part);
        }
        v = fmaf(part, e8m0_to_float(s[k / 32]), v);
    }
    return v;
}

__global__ void __launch_bounds__(kThreads, 1) gemv_w4_tc_kernel(const __grid_constant__ TcParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int block = blockIdx.x / ranks;
    const int first = rank * p.chunks / ranks, last = (rank + 1) * p.chunks / ranks, nc = last - first;
    const int stages = (nc + 1) / 2;
    const int slot_bytes = 2 * p.cols * 128;
    uint8_t* cols = smem + kStages * kStageBytes;  // [slots][2 chunks][cols][128]
    uint8_t* sfb = cols + p.slots * slot_bytes;    // [slots][2][64] words
    uint64_t* bars = reinterpret_cast<uint64_t*>(sfb + p.slots * kSfbBytes);
    uint64_t *code_free = bars, *col_full = bars + kStages, *col_free = col_full + kMaxSlots, *done = col_free + kMaxSlots;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(done + 1);  // TMEM address, abort flag
    uint32_t* bad = reinterpret_cast<uint32_t*>(done + 2);                     // [16] tokens to sum plainly

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) ptx::mbar_init(&code_free[i], 1);
        for (int i = 0; i < p.slots; ++i) ptx::mbar_init(&col_full[i], 4), ptx::mbar_init(&col_free[i], 1);
        ptx::mbar_init(done, 1);
        misc[1] = 0;
        ptx::fence_mbar_init();
    }
    if (tid < FP8BS_W4_MAX_M) bad[tid] = 0;
    if (warp == 0) {
        ptx::tmem_alloc(const_cast<uint32_t*>(&misc[0]), kTmemCols);
        ptx::tmem_relinquish();
    }
    // columns past 4 M stay zero with scale 1
    for (int i = tid; i < p.slots * slot_bytes / 16; i += kThreads) reinterpret_cast<uint4*>(cols)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < p.slots * kSfbBytes / 4; i += kThreads) reinterpret_cast<uint32_t*>(sfb)[i] = 0x7F7F7F7Fu;
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp < 4) {
        // ---- codes, weight scales, MMAs --------------------------------------------
        const int row0 = block * kRowsBlock;
        const int t16 = tid & 15, r8 = tid >> 4;  // 8 bytes of a row's 128; rows r8 + 8 j
        const int unit = t16 & 7;
        const uint32_t to = ptx::smem_addr(smem) + (t16 >> 3) * kChunkBytes + r8 * 128 + ((unit ^ r8) << 4);
        const uint8_t* src = p.codes + first * 64 + t16 * 8;
        const uint8_t* ssrc = p.scales + static_cast<int64_t>(min(row0 + tid, p.N - 1)) * p.lds + first * 4;
        const bool whole = row0 + kRowsBlock <= p.N;
        uint2 raw[kStages - 1];
        auto issue = [&](int s, uint2& words) {
            const int nch = min(nc - 2 * s, 2);
            const uint32_t dst = to + (s % kStages) * kStageBytes;
            if ((t16 >> 3) < nch) {
                const uint8_t* from = src + s * 128;
                if (whole) {
                    from += static_cast<int64_t>(row0 + r8) * p.ldc;
#pragma unroll
                    for (int j = 0; j < 16; ++j) cp_async8(dst + j * 1024, at(from, static_cast<uint32_t>(p.ldc), 8 * j));
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) cp_async8(dst + j * 1024, from + static_cast<int64_t>(min(row0 + r8 + 8 * j, p.N - 1)) * p.ldc);
                }
            }
            words.x = __ldg(reinterpret_cast<const uint32_t*>(ssrc + s * 8));
            words.y = nch > 1 ? __ldg(reinterpret_cast<const uint32_t*>(ssrc + s * 8 + 4)) : 0x7F7F7F7Fu;
        };
        if (!p.pdl) ptx::griddep_wait();
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (s < stages) issue(s, raw[s]);
            cp_async_commit();
        }
        if (p.pdl) ptx::griddep_wait();
        ptx::griddep_launch_dependents();
        bool ok = true;
        for (int s = 0; s < stages; ++s) {
            const uint2 words = raw[0];
#pragma unroll
            for (int i = 0; i + 2 < kStages; ++i) raw[i] = raw[i + 1];
            const int ahead = s + kStages - 1;
            if (ahead < stages) {
                if (ahead >= kStages) ok = ok && wait_bar(&code_free[ahead % kStages], (ahead / kStages - 1) & 1, misc + 1);
                issue(ahead, raw[kStages - 2]);
            }
            cp_async_commit();
            cp_async_wait<kStages - 1>();
            ptx::fence_proxy_async_smem();
            // row 32 q + lane: its scale words, column q of the chunk's four
            const uint32_t sfa = tmem + kSfaCol + 8 * (s % kStages);
            ptx::tmem_st_32x32b_x1(sfa + (static_cast<uint32_t>(warp * 32) << 16) + warp, words.x);
            ptx::tmem_st_32x32b_x1(sfa + (static_cast<uint32_t>(warp * 32) << 16) + 4 + warp, words.y);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::named_sync(1, 128);
            if (warp == 0) {
                const int slot = s % p.slots;
                uint32_t go = 1;
                if (lane == 0) go = wait_bar(&col_full[slot], (s / p.slots) & 1, misc + 1) ? 1u : 0u;
                go = __shfl_sync(0xFFFFFFFFu, go, 0);
                ptx::tc_fence_after();
                if (go) {
                    const uint32_t a = ptx::smem_addr(smem) + (s % kStages) * kStageBytes;
                    const uint32_t b = ptx::smem_addr(cols) + slot * slot_bytes;
                    const int nch = min(nc - 2 * s, 2);
                    for (int c = 0; c < nch; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_mxf8f6f4_bs_warp(tmem, ptx::smem_desc_sw128(a + c * kChunkBytes + 32 * k),
                                                      ptx::smem_desc_sw128(b + c * p.cols * 128 + 32 * k),
                                                      idesc_e2m1_e4m3(p.cols, k), sfa + 4 * c, tmem + kSfbCol + 8 * slot + 4 * c,
                                                      s > 0 || c > 0 || k > 0 ? 1u : 0u);
                }
                ptx::mma_commit_warp(&code_free[s % kStages]);
                ptx::mma_commit_warp(&col_free[slot]);
                if (s == stages - 1) ptx::mma_commit_warp(done);
                __syncwarp();
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ---- x as columns -------------------------------------------------------------
        const int w = warp - 4, sub = lane & 3;
        ptx::griddep_wait();
        const uint32_t cols_at = ptx::smem_addr(cols), sfb_at = ptx::smem_addr(sfb);
        bool ok = true;
        for (int s = 0; s < stages; ++s) {
            const int slot = s % p.slots, groups = 4 * min(nc - 2 * s, 2);
            if (s >= p.slots) ok = ok && wait_bar(&col_free[slot], (s / p.slots - 1) & 1, misc + 1);
            // 8 (token, group) pairs a warp and pass, 4 lanes each, 8 k a lane
            const int pairs = p.M * groups;
            uint4 raw[4];
            for (int base = 0; base < pairs; base += 128) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int q = base + 32 * i + w * 8 + (lane >> 2);
                    raw[i] = make_uint4(0, 0, 0, 0);
                    if (q < pairs) {
                        const int m = q / groups, g = q - m * groups;
                        raw[i] = *reinterpret_cast<const uint4*>(p.x + m * p.ldx + (first + 2 * s) * kChunk + g * 32 + sub * 8);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (base + 32 * i + w * 8 >= pairs) break;
                    const int q = base + 32 * i + w * 8 + (lane >> 2);
                    const int m = q / groups, g = q - m * groups;
                    float r[8];
                    unpack8(raw[i], r);
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(r[j]) & 0x7FFFFFFFu);
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const int ef = static_cast<int>(top >> 23);
                    if (ef == 255) {
                        if (q < pairs) bad[m] = 1;
#pragma unroll
                        for (int j = 0; j < 8; ++j) r[j] = 0.0f;
                    }
                    // column t's row is 4 m + t: row n at (n / 8) 1024 + (n % 8) 128 of its chunk
                    const int c16 = (g & 3) * 2 + (sub >> 1);
                    const uint32_t chunk_at = cols_at + slot * slot_bytes + (g >> 2) * p.cols * 128 + (sub & 1) * 8;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        constexpr int kShift[4] = {0, 5, 22, 27};
                        // the biased exponent of the column's scale, at least 2^-127
                        const int sc = max(ef == 255 ? 127 : ef - 7 - kShift[t], 0);
                        uint32_t lo = 0, hi = 0;
                        bool any = true;
                        if (t == 2) {
                            bool rest = false;
#pragma unroll
                            for (int j = 0; j < 8; ++j) rest |= r[j] != 0.0f;
                            any = __any_sync(0xFFFFFFFFu, rest);
                        }
                        if (t == 3) {
                            bool rest = false;
#pragma unroll
                            for (int j = 0; j < 8; ++j) rest |= r[j] != 0.0f;
                            any = __any_sync(0xFFFFFFFFu, rest);
                        }
                        if (any) {
                            const float s2 = e8m0_to_float(sc), up = e8m0_to_float(254 - sc);
                            uint32_t h[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t code = e4m3x2(r[2 * j] * up, r[2 * j + 1] * up);
                                h[j] = code;
                                uint32_t two;
                                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(code)));
                                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&two));
                                r[2 * j] = fmaf(-v.x, s2, r[2 * j]);
                                r[2 * j + 1] = fmaf(-v.y, s2, r[2 * j + 1]);
                            }
                            lo = h[0] | h[1] << 16;
                            hi = h[2] | h[3] << 16;
                        }
                        if (q < pairs) {
                            const int n = 4 * m + t;
                            sts64(chunk_at + (n >> 3) * 1024 + (n & 7) * 128 + ((c16 ^ (n & 7)) << 4), lo, hi);
                            if (sub == 0) sts8(sfb_at + slot * kSfbBytes + ((g >> 2) * 64 + n) * 4 + (g & 3), static_cast<uint32_t>(sc));
                        }
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::named_sync(2, 128);
            // every quadrant holds column n's scale word in lane n % 32, column n / 32
            const uint32_t* words = reinterpret_cast<const uint32_t*>(sfb + slot * kSfbBytes);
            const uint32_t sf = tmem + (static_cast<uint32_t>(w * 32) << 16) + kSfbCol + 8 * slot;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                ptx::tmem_st_32x32b_x1(sf + 4 * c, words[c * 64 + lane]);
                if (p.cols > 32) ptx::tmem_st_32x32b_x1(sf + 4 * c + 1, words[c * 64 + 32 + lane]);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&col_full[slot]);
        }
    }

    // ---- sums ---------------------------------------------------------------------------
    __syncwarp();
    if (lane == 0) wait_bar(done, 0, misc + 1);
    __syncwarp();
    __syncthreads();
    ptx::tc_fence_after();
    const bool failed = misc[1] != 0;
    float* red = reinterpret_cast<float*>(smem);  // [M][128], in the place of the codes
    if (warp < 4) {
        const int row = min(block * kRowsBlock + tid, p.N - 1);
        for (int h = 0; h < p.cols / 16; ++h) {
            uint32_t v[16];
            ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 16 * h, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = 4 * h + i;
                if (m < p.M) {
                    float sum = (__uint_as_float(v[4 * i]) + __uint_as_float(v[4 * i + 1])) +
                                (__uint_as_float(v[4 * i + 2]) + __uint_as_float(v[4 * i + 3]));
                    if (bad[m]) sum = plain_sum(p, row, m, first * kChunk, last * kChunk);
                    red[m * kRowsBlock + tid] = failed ? __uint_as_float(0x7FC00000u) : sum;
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (ranks > 1)
        cluster_sync();
    else
        __syncthreads();
    const int rows = kRowsBlock / ranks, r0 = rank * rows;
    const uint32_t red_at = ptx::smem_addr(red);
    for (int o = tid; o < p.M * rows; o += kThreads) {
        const int m = o / rows, r = r0 + o - m * rows;
        const int64_t row = static_cast<int64_t>(block) * kRowsBlock + r;
        float v = 0.0f;
        if (ranks > 1)
            for (int k = 0; k < ranks; ++k) v += ld_cluster(red_at + (m * kRowsBlock + r) * 4, k);
        else
            v = red[m * kRowsBlock + r];
        if (row < p.N) p.y[m * p.ldy + row] = to_bf16(v);
    }
    __syncwarp();
    if (ranks > 1) cluster_sync();  // a block's sums stay until its peers have read them
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

bool gemv_w4_tc_serves(const GemvW4Args& a) { return a.format == FP8BS_W4_MXFP4; }

cudaError_t launch_gemv_w4_tc(const GemvW4Args& a, cudaStream_t stream) {
    TcParams p;
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
    p.cols = (4 * a.M + 15) / 16 * 16;
    p.slots = min(kMaxSlots, (kMaxBlockShared - kStages * kStageBytes - kMiscBytes) / (2 * p.cols * 128 + kSfbBytes));
    p.pdl = a.pdl;
    // K over a cluster while its blocks still fit the machine together
    const int blocks = (a.N + kRowsBlock - 1) / kRowsBlock;
    int ranks = 1;
    while (ranks < 8 && 2 * ranks * blocks <= a.sm_count && 4 * ranks <= p.chunks) ranks *= 2;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(gemv_w4_tc_kernel, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(tc_bytes(p.cols, p.slots));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gemv_w4_tc_kernel, p);
}

}  // namespace fp8bs
