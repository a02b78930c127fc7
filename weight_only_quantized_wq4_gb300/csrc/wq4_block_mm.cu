// Product of 8-bit float operands with block scales, sm_103a:
//
//     Y[m][n] = sum_b sx[b][m] sw[n / 128][b] P_b[m][n],   P_b[m][n] = sum_{k in block b} xq[m][k] wq[n][k]
//
// with e4m3 codes xq, wq and blocks of 128 along K. P_b runs on the tensor core (tcgen05, kind::f8f6f4,
// fp32 accumulation; products of e4m3 codes are exact in fp32); its scales differ from block to
// block, so every P_b lands in a buffer of tensor memory of its own and is added to Y's
// accumulators, which the fold warps hold in registers: acc += (sx sw) P_b, in fp32.
//
// One operand's rows are the MMA's 128 lanes, the other's its columns:
//   tokens on the lanes     (many tokens) a fold thread holds one token: its factor sx sw is one number
//                           per block, as a tile's columns lie in whole blocks of 128 weight rows.
//   weight rows on the lanes (few tokens) the columns are the tokens, padded to the tile's width
//                           only, so that a tile's cost is its weights' bytes.
//
// Warp roles (one CTA per SM, persistent over tiles):
//   warps 0, 2   copies: per block of K, one operand's 128-byte row pieces each as a 2-D tensor copy with
//                the 128-byte swizzle (rows and K past the end read as zero), into a ring of stages. A
//                thread alone cannot issue both operands' copies as fast as a block is used.
//   warps 1, 3   MMAs: one thread each, taking blocks in turn; four MMAs (K = 32) a block, then a commit
//                to the fold warps. A thread issues an MMA in 46 cycles and needs some 75 for each wait
//                and commit besides, longer than the tensor core takes for narrow tiles; two overlap.
//   warps 4+     fold: read P_b, add it in, at a tile's end round once and store
// With fewer tiles than SMs, a cluster of CTAs shares each tile, cut along K; the parts are sent
// through distributed shared memory to the CTA that joins them, which adds them in rank order.
//
// What bounds it, and measured device times (passes back to back, replayed from a graph, weights not in L2):
//   few tokens    the weights' bytes, and some 4 us of launch, first copies and last stores: 16 x 14336 x 4096 bf16
//                 13.4 us (4.4 TB/s; a kernel that only copies as many bytes takes 12.1), 1 x 4096 x 4096 6.4 us
//   middle sizes  the same 4 us, then 480 to 600 cycles a block: 333 x 4100 x 2064 fp16 10.3 us
//   large sizes   the fold: 650 to 810 cycles per block of 256 columns for tcgen05.ld and 128 FMAs a thread,
//                 against the MMAs' 515: 4096 x 4096 x 14336 bf16 184 us (2.6 PFLOP/s; the MMAs alone are 72% of
//                 it), 199 in calls from Python, where the board's power limit tells. A third buffer of tensor memory would
//                 hide the fold's latency; two of 256 columns fill it.
//
// Every wait is bounded, as in wq4_gemm.cuh: one that runs out is recorded in the status word and the
// CTA drains its copies and MMAs, frees its tensor memory and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdio>
#include <type_traits>

#include "wq4_device.cuh"
#include "wq4_runtime.h"

namespace wq4 {
namespace {

constexpr int kBmBlock = 128;                  // K elements (bytes) of a block
constexpr int kBmLanes = 128;                  // rows of the lane operand per tile
constexpr int kBmMaxSmem = 232448;

struct BmArgs {
    CUtensorMap lane_map, col_map;             // e4m3 codes [rows][K], box 128 K x tile rows
    CUtensorMap sx_map;                        // tokens on the lanes: token scales [blocks][M], box 128 tokens x 8 blocks
    const float *sx, *sw;                      // token scales, row b, column m; weight scales, row n / 128, column b
    void* y;
    long long ldsx, ldsw, ldy;
    int M, N, kb;                              // kb: blocks of K
    int lane_tiles, tiles;                     // tile t: lane tile t % lane_tiles, column tile t / lane_tiles
    int split;                                 // CTAs per cluster, each with a part of K (1: none)
    int stages;                                // of the ring: an even number
    int share;                                 // split: columns that a rank joins (weights on the lanes), or columns of
                                               // every fold thread (tokens on the lanes, a multiple of 8)
    int dtype;
    int unit;                                  // bytes that a row of Y is stored by: 16, or what its start allows
    unsigned int* status;
    long long timeout_cycles;
    int test_stall;
};

// NT: columns of a tile; TOK_LANES: tokens on the lanes (else weight rows); PAIR: two CTAs of a cluster
// share each tile of 256 lanes, 128 lanes and half the columns' copies each (cta_group::2).
template <int NT, bool TOK_LANES, bool PAIR>
struct BmCfg {
    static constexpr int kAhead = 4;                            // blocks whose scales are loaded together, one such group ahead
    static constexpr int kFW = TOK_LANES ? 8 : 4;               // fold warps
    static constexpr int kParts = kFW / 4;                      // fold warps per lane quarter
    static constexpr int kNC = NT / kParts;                     // columns of a fold thread
    static constexpr int kThreads = 128 + 32 * kFW;
    static constexpr int kLaneBytes = kBmLanes * kBmBlock;
    static constexpr int kColRows = PAIR ? NT / 2 : NT;         // rows of the column operand a CTA copies
    static constexpr int kColBytes = kColRows * kBmBlock;
    static constexpr int kTokens = TOK_LANES ? kBmLanes : NT;
    static constexpr int kStageBytes = kLaneBytes + kColBytes;
    static constexpr int kBarBytes = 1024;
    // per fold warp: rows of an output chunk on their way to coalesced stores, 32 of 64 + 16 bytes (tokens on
    // the lanes), or the factors of a block's tokens, twice
    static constexpr int kWarpBytes = TOK_LANES ? 32 * 80 : 2 * NT * 4;
    // tokens on the lanes: the tokens' scales of 8 blocks at a time come as one copy, in a ring of their own
    static constexpr int kScBlocks = 8, kScRing = TOK_LANES ? 3 : 0, kScBytes = kScBlocks * kBmLanes * 4;
    // An even number of stages (fit) and of P buffers: the MMA warps take alternate blocks, so each walks
    // every phase of its own ones (a parity wait is unambiguous one phase ahead only).
    // Shared memory before the stages, and the most that the parts other CTAs of a cluster send may take
    static constexpr int kHeadBytes = 128 + 1024 + kBarBytes + kScRing * kScBytes + kFW * kWarpBytes;
    static constexpr int kRedBytes = PAIR ? 0 : TOK_LANES ? NT * kBmLanes * 4 : (NT + 8) * kBmLanes * 4;
    static constexpr int fit(int red) { return ((kBmMaxSmem - kHeadBytes - red) / kStageBytes > 12 ? 12 : (kBmMaxSmem - kHeadBytes - red) / kStageBytes) & ~1; }
    static constexpr int kHalfStages = ((115712 - kHeadBytes) / kStageBytes) & ~1;   // two CTAs of an SM: that many bytes each
    static constexpr int kPBufs = NT <= 128 ? 4 : 2;
    static constexpr int kTmemCols = NT * kPBufs > 256 ? 512 : NT * kPBufs;
    // 128 fp32 accumulators per fold thread want more registers than an even share: 384 threads
    // launched with 168 each (64512 in all), of which the copy and MMA warps keep 56 and the fold
    // warps take 224 (128 x 56 + 256 x 224 = 64512).
    static constexpr bool kRegSplit = kNC > 64;
    static constexpr int kLaunchRegs = 168, kRegWg0 = 56, kRegFold = 224;
    static_assert(!kRegSplit || 128 * kRegWg0 + 32 * kFW * kRegFold <= kThreads * kLaunchRegs, "register split");
    static_assert(fit(kRedBytes) >= 4 && fit(0) <= 16 && kTmemCols <= 512, "tile");
    static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
    static_assert(!PAIR || (TOK_LANES && kPBufs == 2), "pairs");
};

template <bool PAIR>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}

// The instructions of wq4_device.cuh as a pair of CTAs uses them: both allocate and free, a commit
// arrives on the barrier of that offset in each, and a barrier of the leader's (rank 0) takes arrivals
// from both.
template <bool PAIR>
__device__ __forceinline__ void bm_tmem_alloc(uint32_t dst, uint32_t cols) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    }
}
template <bool PAIR>
__device__ __forceinline__ void bm_tmem_dealloc(uint32_t taddr, uint32_t cols) {
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
    else tmem_dealloc(taddr, cols);
}
template <bool PAIR>
__device__ __forceinline__ void bm_commit(uint32_t bar) {
    if constexpr (PAIR) {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    } else {
        mma_commit(bar);
    }
}
// One value to shared memory of a CTA of the cluster; its bytes count on that CTA's barrier.
__device__ __forceinline__ void st_async(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_async4(uint32_t addr, const float* v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive_leader(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(bar, 0)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {   // (does not wait)
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// mbar_wait of wq4_device.cuh for a barrier with arrivals from the other CTA of the pair.
__device__ __forceinline__ bool mbar_wait_pair(uint32_t bar, uint32_t parity, const WaitCtl& ctl) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*ctl.abort_flag) return false;
        if (clock64() - t0 > ctl.limit) {
            *ctl.abort_flag = 1;
            atomicOr(ctl.status, kStatusTimeout);
            return false;
        }
    }
}

// kind::f8f6f4: D fp32, A and B e4m3 (format code 0), both K-major, M x N.
__device__ constexpr uint32_t f8_idesc(uint32_t M, uint32_t N) { return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24); }

// (d0, d1) += (f0, f1) * (v0, v1), one packed fp32 FMA.
__device__ __forceinline__ void fma_pair(float& d0, float& d1, float f0, float f1, uint32_t v0, uint32_t v1) {
    uint64_t d, f, v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(d0), "f"(d1));
    asm("mov.b64 %0, {%1, %2};" : "=l"(f) : "f"(f0), "f"(f1));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(f), "l"(v));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(d));
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int dtype) {
    uint32_t u;
    if (dtype == WQ4_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    return u;
}

// UNIT bytes from shared to global memory.
template <int UNIT>
__device__ __forceinline__ void copy_unit(void* to, uint32_t from) {
    if constexpr (UNIT == 16) {
        *static_cast<uint4*>(to) = lds128(from);
    } else if constexpr (UNIT == 8) {
        uint2 u;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(from));
        *static_cast<uint2*>(to) = u;
    } else if constexpr (UNIT == 4) {
        uint32_t u;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(from));
        *static_cast<uint32_t*>(to) = u;
    } else {
        uint16_t u;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(u) : "r"(from));
        *static_cast<uint16_t*>(to) = u;
    }
}

// The 32 rows of CNT columns in `buf` (80 bytes a row) to rows m0.. of Y, columns n..: runs of a row
// by neighbouring lanes, UNIT bytes each (what the rows of Y start on), SIZE bytes a value.
template <int SIZE, int UNIT, int CNT>
__device__ __forceinline__ void copy_rows(const BmArgs& a, uint32_t buf, int lane, int m0, int n) {
    constexpr int kPerRow = CNT * SIZE / UNIT, kRows = 32 / kPerRow, kIn = UNIT / SIZE;
    const int c = lane % kPerRow * kIn, r0 = lane / kPerRow;
    const int cols = a.N - n - c, rows = a.M - m0;   // what exists from here on
    if (!WQ4_CHECK(n >= 0 && m0 >= 0 && m0 < (a.M + 255) / 256 * 256, a.status, nullptr, check::kSiteBlockOut, n, m0, a.N)) return;
    uint8_t* to = static_cast<uint8_t*>(a.y) + ((m0 + r0) * a.ldy + n + c) * SIZE;
    const long long step = a.ldy * (kRows * SIZE);
    const uint32_t from = buf + r0 * 80 + c * SIZE;
    if (rows >= 32 && a.N - n >= CNT) {              // all of it exists
#pragma unroll
        for (int p = 0; p < 32 / kRows; ++p) copy_unit<UNIT>(to + p * step, from + p * kRows * 80);
        return;
    }
#pragma unroll 1
    for (int p = 0; p < 32 / kRows; ++p, to += step) {
        if (r0 + p * kRows >= rows) break;
        if (cols >= kIn) {
            copy_unit<UNIT>(to, from + p * kRows * 80);
        } else {                                     // the row ends inside the unit
            for (int j = 0; j < cols; ++j) copy_unit<SIZE>(to + j * SIZE, from + p * kRows * 80 + j * SIZE);
        }
    }
}

// A warp's 32 rows from m0, one per lane, CNT columns from n, through `buf` in shared memory: stored by
// their lanes directly, rows would touch 32 lines with every instruction.
template <int CNT>
__device__ __forceinline__ void store_rows(const BmArgs& a, uint32_t buf, int lane, int m0, int n, const float* v) {
    const uint32_t mine = buf + lane * 80;
    constexpr int kChunk = CNT < 32 ? CNT : 32, kWide = CNT < 16 ? CNT : 16;   // columns of 16, 32 bits at a time
    if (a.dtype == WQ4_FP32) {
#pragma unroll
        for (int c = 0; c < CNT; c += kWide) {
#pragma unroll
            for (int j = 0; j < kWide; j += 4)
                sts128(mine + 4 * j, __float_as_uint(v[c + j]), __float_as_uint(v[c + j + 1]),
                       __float_as_uint(v[c + j + 2]), __float_as_uint(v[c + j + 3]));
            __syncwarp();
            if (a.unit == 16) copy_rows<4, 16, kWide>(a, buf, lane, m0, n + c);
            else copy_rows<4, 4, kWide>(a, buf, lane, m0, n + c);
            __syncwarp();
        }
    } else {
#pragma unroll
        for (int c = 0; c < CNT; c += kChunk) {
#pragma unroll
            for (int j = 0; j < kChunk; j += 8)
                sts128(mine + 2 * j, pack16(v[c + j], v[c + j + 1], a.dtype), pack16(v[c + j + 2], v[c + j + 3], a.dtype),
                       pack16(v[c + j + 4], v[c + j + 5], a.dtype), pack16(v[c + j + 6], v[c + j + 7], a.dtype));
            __syncwarp();
            if (a.unit == 16) copy_rows<2, 16, kChunk>(a, buf, lane, m0, n + c);
            else if (a.unit == 8) copy_rows<2, 8, kChunk>(a, buf, lane, m0, n + c);
            else if (a.unit == 4) copy_rows<2, 4, kChunk>(a, buf, lane, m0, n + c);
            else copy_rows<2, 2, kChunk>(a, buf, lane, m0, n + c);
            __syncwarp();
        }
    }
}

// One column n of Y per lane, `rows` tokens (CNT at most) from m: neighbouring lanes' columns are neighbours
// in memory.
template <int CNT>
__device__ __forceinline__ void store_cols(const BmArgs& a, int m, int rows, int n, const float* v) {
    if (n >= a.N) return;
    if (!WQ4_CHECK(n >= 0 && m >= 0 && m < a.M + CNT, a.status, nullptr, check::kSiteBlockOut, n, m, a.N)) return;
    const long long at = m * a.ldy + n;
    if (a.dtype == WQ4_FP32) {
        float* y = static_cast<float*>(a.y) + at;
#pragma unroll
        for (int j = 0; j < CNT; ++j, y += a.ldy)
            if (j < rows) *y = v[j];
    } else {
        uint16_t* y = static_cast<uint16_t*>(a.y) + at;
#pragma unroll
        for (int j = 0; j < CNT; ++j, y += a.ldy)
            if (j < rows) *y = static_cast<uint16_t>(pack16(v[j], 0.f, a.dtype));
    }
}

// The tiles of one CTA, in order, and the part of K it takes of each.
struct BmSched {
    int t, step, kb0, kb1;
    __device__ BmSched(const BmArgs& a, int rank, bool pair) {
        if (pair) {
            t = blockIdx.x / 2;
            step = gridDim.x / 2;
            kb0 = 0;
            kb1 = a.kb;
            return;
        }
        t = blockIdx.x / a.split;
        step = gridDim.x / a.split;
        kb0 = static_cast<int>(static_cast<long long>(a.kb) * rank / a.split);
        kb1 = static_cast<int>(static_cast<long long>(a.kb) * (rank + 1) / a.split);
    }
};

template <int NT, bool TOK_LANES, bool PAIR>
__global__ void __launch_bounds__(BmCfg<NT, TOK_LANES, PAIR>::kThreads, !TOK_LANES && NT <= 32 ? 2 : 1)
    block_mm_kernel(const __grid_constant__ BmArgs a) {
    using C = BmCfg<NT, TOK_LANES, PAIR>;
    constexpr int kTileLanes = PAIR ? 2 * kBmLanes : kBmLanes, kAhead = C::kAhead;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t s_bar = (raw_s + 127u) & ~127u;
    const uint32_t s_sc = s_bar + C::kBarBytes;                       // token scales
    const uint32_t s_warp = s_sc + C::kScRing * C::kScBytes;          // the fold warps' buffers
    const uint32_t s_ring = (s_warp + C::kFW * C::kWarpBytes + 1023u) & ~1023u;
    const uint32_t s_red = s_ring + a.stages * C::kStageBytes;        // parts from the cluster's CTAs
    auto full_bar = [&](int s) { return s_bar + 8u * s; };
    auto empty_bar = [&](int s) { return s_bar + 8u * (16 + s); };
    auto pfull_bar = [&](int b) { return s_bar + 8u * (32 + b); };
    auto pempty_bar = [&](int b) { return s_bar + 8u * (36 + b); };
    auto scfull_bar = [&](int c) { return s_bar + 8u * (40 + c); };
    auto scempty_bar = [&](int c) { return s_bar + 8u * (44 + c); };
    const uint32_t drain_bar = s_bar + 8u * 48, stall_bar = s_bar + 8u * 49, red_bar = s_bar + 8u * 50;
    uint8_t* const gmisc = smem_raw + (s_bar - raw_s) + 8 * 56;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gmisc);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(gmisc + 4);
    volatile int* const issued_by = reinterpret_cast<volatile int*>(gmisc + 8);   // stages the two copy threads filled
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR || a.split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int lane0 = PAIR ? rank * kBmLanes : 0;    // this CTA's first lane of a tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full_bar(s), PAIR && rank == 0 ? 3 : 2);   // both operands' copies (and the other CTA's)
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < C::kPBufs; ++b) {
            mbar_init(pfull_bar(b), 1);
            mbar_init(pempty_bar(b), PAIR ? 2 * C::kFW : C::kFW);
        }
        for (int c = 0; c < C::kScRing; ++c) {
            mbar_init(scfull_bar(c), 1);
            mbar_init(scempty_bar(c), C::kFW);
        }
        mbar_init(drain_bar, 2);                     // one commit from each MMA warp
        mbar_init(stall_bar, 1);
        if (!PAIR && a.split > 1) {                  // the bytes of the parts of this CTA's columns
            mbar_init(red_bar, 1);
            const int own = min(max((TOK_LANES ? C::kNC : a.M) - rank * a.share, 0), a.share);
            mbar_arrive_expect_tx(red_bar, own * kBmLanes * 4 * (TOK_LANES ? (a.split - 1) * C::kParts : a.split));
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&a.lane_map);
        prefetch_tensormap(&a.col_map);
        if constexpr (TOK_LANES) prefetch_tensormap(&a.sx_map);
    }
    if (warp == 1) {
        bm_tmem_alloc<PAIR>(smem_u32(tmem_slot), C::kTmemCols);
    }
    tc_fence_before();
    if (PAIR || a.split > 1) {
        __syncwarp();
        cluster_sync();                              // (the other CTAs' barriers are set up too)
    } else {
        __syncthreads();
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const WaitCtl ctl{abort_flag, a.status, a.timeout_cycles};
    int issued = 0, sc_issued = 0;                   // stages a copy thread has filled, scale copies

    if (warp < 4) {
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegWg0));
        if (warp == 0 || warp == 2) {
            if (lane == 0) {
                // an operand that only one tile along its side reads streams through L2
                const bool lanes = warp == 0, once = lanes ? a.tiles == a.lane_tiles : a.lane_tiles == 1;
                const uint64_t policy = once ? policy_evict_first() : policy_evict_last();
                const CUtensorMap* map = lanes ? &a.lane_map : &a.col_map;
                // rows of this operand's tiles (the last may be partly past its end)
                [[maybe_unused]] const int row_end = lanes ? a.lane_tiles * kTileLanes : a.tiles / a.lane_tiles * NT;
                const uint32_t dst = s_ring + (lanes ? 0 : C::kLaneBytes), bytes = lanes ? C::kLaneBytes : C::kColBytes;
                bool ok = true;
                int st = 0, i = 0, sc = 0;
                uint32_t phase = 1, sc_phase = 1;
                for (BmSched s(a, rank, PAIR); s.t < a.tiles && ok; s.t += s.step) {
                    const int row = lanes ? s.t % a.lane_tiles * kTileLanes + lane0
                                          : s.t / a.lane_tiles * NT + (PAIR ? rank * C::kColRows : 0);
                    for (int b = s.kb0; b < s.kb1; ++b, ++i) {
                        if (TOK_LANES && warp == 2 && (b - s.kb0) % C::kScBlocks == 0) {
                            if (!mbar_wait(scempty_bar(sc), sc_phase, ctl)) { ok = false; break; }
                            mbar_arrive_expect_tx(scfull_bar(sc), C::kScBytes);
                            tma_load_2d(s_sc + sc * C::kScBytes, &a.sx_map, scfull_bar(sc),
                                        s.t % a.lane_tiles * kTileLanes + lane0, b, policy_evict_last());
                            ++sc_issued;
                            if (++sc == C::kScRing) { sc = 0; sc_phase ^= 1; }
                        }
                        if (!mbar_wait(empty_bar(st), phase, ctl)) { ok = false; break; }
                        mbar_arrive_expect_tx(full_bar(st), bytes);
                        int x = b * kBmBlock, y = row;       // (a failed check reads the tensor's origin instead)
                        if (!WQ4_CHECK(check::block_copy_ok(b, a.kb, row, row_end) && check::tma_x_ok(x, 1, 0, x), a.status,
                                       abort_flag, check::kSiteBlockCopy, b, row, a.kb)) x = y = 0;
                        tma_load_2d(dst + st * C::kStageBytes, map, full_bar(st), x, y, policy);
                        if (++st == a.stages) { st = 0; phase ^= 1; }
                    }
                }
                issued = i;
            }
            __syncwarp();
        } else if (PAIR && rank != 0) {
            // The leader's MMAs read both CTAs' stages: warp 1 tells it of this one's.
            if (warp == 1 && lane == 0) {
                int st = 0;
                uint32_t full = 0;
                bool ok = true;
                for (BmSched s(a, rank, PAIR); s.t < a.tiles && ok; s.t += s.step) {
                    for (int b = s.kb0; b < s.kb1; ++b) {
                        if (!mbar_wait(full_bar(st), full, ctl)) { ok = false; break; }
                        mbar_arrive_leader(full_bar(st));
                        if (++st == a.stages) { st = 0; full ^= 1; }
                    }
                }
            }
            __syncwarp();
        } else {
            if (lane == 0) {
                constexpr uint32_t idesc = f8_idesc(kTileLanes, NT);
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    return PAIR ? mbar_wait_pair(bar, parity, ctl) : mbar_wait(bar, parity, ctl);
                };
                const int mine = warp >> 1;          // this thread's blocks: the even or the odd ones
                bool ok = !(a.test_stall && mine == 0) || mbar_wait(stall_bar, 0, ctl);
                const uint64_t desc0 = make_sdesc_sw128(s_ring);
                int st = mine, p = mine, skip = mine;
                uint32_t full = 0, free = 1;         // phase parities
                for (BmSched s(a, rank, PAIR); s.t < a.tiles && ok; s.t += s.step) {
                    int b = s.kb0 + skip;
                    for (; b < s.kb1; b += 2) {
                        if (!wait(full_bar(st), full)) { ok = false; break; }
                        if (!wait(pempty_bar(p), free)) { ok = false; break; }
                        tc_fence_after();
                        const uint64_t desc = desc0 + static_cast<uint32_t>(st * (C::kStageBytes >> 4));
                        const uint32_t d = tmem + p * NT;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8<PAIR>(d, desc + 2 * k, desc + (C::kLaneBytes >> 4) + 2 * k, idesc, k > 0);
                        bm_commit<PAIR>(pfull_bar(p));
                        bm_commit<PAIR>(empty_bar(st));
                        if ((st += 2) >= a.stages) { st = mine; full ^= 1; }
                        if ((p += 2) >= C::kPBufs) { p = mine; free ^= 1; }
                    }
                    skip = b - s.kb1;                // (the turns go on over the tiles' ends)
                }
                bm_commit<PAIR>(drain_bar);               // every MMA is done before the tensor memory goes
                mbar_wait_plain(drain_bar, 0, drain_limit(a.timeout_cycles));
            }
            __syncwarp();
        }
    } else {
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegFold));
        float acc[C::kNC] = {};
        const int quarter = warp & 3, part = (warp - 4) >> 2;
        const int r = 32 * quarter + lane;           // this thread's lane of the tile
        const int col0 = part * C::kNC;              // and its first column
        const uint32_t t_addr = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + col0;
        const uint32_t buf = s_warp + (warp - 4) * C::kWarpBytes;
        const int sw_rows = (a.N + 127) / 128;
        bool ok = true;
        int p = 0, sc = 0;
        uint32_t phase = 0, sc_phase = 0;
        for (BmSched s(a, rank, PAIR); s.t < a.tiles && ok; s.t += s.step) {
            const int l0 = s.t % a.lane_tiles * kTileLanes + lane0, c0 = s.t / a.lane_tiles * NT;
            const float* sw = a.sw + min((TOK_LANES ? c0 + col0 : l0) / 128, sw_rows - 1) * a.ldsw;
            if constexpr (TOK_LANES) {
                // A token per thread: its factor of a block is its scale (from the ring; 0 past the last token)
                // times the weight's, of which the warp's lanes load 32 blocks at a time. While one piece of P is added
                // in, the next is read.
                constexpr int kCols = 16, kPieces = C::kNC / kCols;
                const int nb = s.kb1 - s.kb0;
                float w32 = lane < nb ? sw[s.kb0 + lane] : 0.f;
#pragma unroll
                for (int j = 0; j < C::kNC; ++j) acc[j] = 0.f;
                uint32_t v[2][kCols];
#pragma unroll 1
                for (int b = 0; b < nb; ++b) {
                    if (b % C::kScBlocks == 0) {
                        if (b % 32 == 0 && b) w32 = b + lane < nb ? sw[s.kb0 + b + lane] : 0.f;
                        if (!mbar_wait(scfull_bar(sc), sc_phase, ctl)) { ok = false; break; }
                    }
                    const float f = lds_f32(s_sc + sc * C::kScBytes + (b % C::kScBlocks) * (kBmLanes * 4) + 4 * r) *
                                    __shfl_sync(0xffffffffu, w32, b % 32);
                    const uint32_t from = t_addr + p * NT, freed = pempty_bar(p);
                    if (!mbar_wait(pfull_bar(p), phase, ctl)) { ok = false; break; }
                    tc_fence_after();
                    tmem_ld16(from, v[0]);
                    if (++p == C::kPBufs) { p = 0; phase ^= 1; }
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        tmem_ld_wait();
                        if (c + 1 < kPieces) {
                            tmem_ld16(from + (c + 1) * kCols, v[(c + 1) & 1]);
                        } else {                     // all of the block's P is in registers: the buffer is free
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                if constexpr (PAIR) mbar_arrive_leader(freed);
                                else mbar_arrive(freed);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < kCols; q += 2)
                            fma_pair(acc[c * kCols + q], acc[c * kCols + q + 1], f, f, v[c & 1][q], v[c & 1][q + 1]);
                    }
                    if (b % C::kScBlocks == C::kScBlocks - 1 || b + 1 == nb) {
                        __syncwarp();                // (every lane has its last factor)
                        if (lane == 0) mbar_arrive(scempty_bar(sc));
                        if (++sc == C::kScRing) { sc = 0; sc_phase ^= 1; }
                    }
                }
            } else {
                // A lane loads the scales of one token (two at NT = 64; none past the last token, whose values are
                // not stored), kAhead blocks at a time and one such group ahead; they are multiplied only
                // when their turn comes, so that nothing waits for a load just issued. A block's factors
                // then go to shared memory, where every lane reads all of them.
                constexpr int kCols = 16, kPieces = NT / kCols, kPer = (NT + 31) / 32;
                const bool loads = c0 + lane < a.M && lane < NT, loads2 = kPer > 1 && c0 + lane + 32 < a.M;
                const float *px = a.sx + (c0 + lane) + s.kb0 * a.ldsx, *pw = sw + s.kb0;
                float nsx[kAhead * kPer] = {}, nsw[kAhead] = {};
                auto load_scales = [&](int n) {      // of the next n blocks (kAhead at most)
#pragma unroll
                    for (int j = 0; j < kAhead; ++j, px += a.ldsx) {
                        if (j >= n) break;
                        nsw[j] = pw[j];
                        if (loads) nsx[j * kPer] = *px;
                        if constexpr (kPer > 1)
                            if (loads2) nsx[j * kPer + 1] = px[32];
                    }
                    pw += kAhead;
                };
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[j] = 0.f;
                uint32_t v[2][kCols];
                load_scales(s.kb1 - s.kb0);
                __syncwarp();                        // (no lane still reads the last tile's factors)
                for (int b0 = s.kb0; b0 < s.kb1 && ok; b0 += kAhead) {
                    float f[kAhead * kPer];
#pragma unroll
                    for (int j = 0; j < kAhead * kPer; ++j) f[j] = nsx[j] * nsw[j / kPer];
                    load_scales(s.kb1 - b0 - kAhead);
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        if (b0 + j >= s.kb1) break;
                        const uint32_t factors = buf + (j & 1) * (NT * 4);
#pragma unroll
                        for (int q = 0; q < kPer; ++q)
                            if (lane + 32 * q < NT)
                                asm volatile("st.shared.f32 [%0], %1;" ::"r"(factors + (lane + 32 * q) * 4), "f"(f[j * kPer + q])
                                             : "memory");
                        __syncwarp();
                        if (!mbar_wait(pfull_bar(p), phase, ctl)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t from = t_addr + p * NT, freed = pempty_bar(p);
                        if (++p == C::kPBufs) { p = 0; phase ^= 1; }
                        tmem_ld16(from, v[0]);
#pragma unroll
                        for (int c = 0; c < kPieces; ++c) {
                            tmem_ld_wait();
                            if (c + 1 < kPieces) {
                                tmem_ld16(from + (c + 1) * kCols, v[(c + 1) & 1]);
                            } else {                 // all of the block's P is in registers: the buffer is free
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(freed);
                            }
#pragma unroll
                            for (int q = 0; q < kCols; q += 4) {
                                const uint4 w = lds128(factors + (c * kCols + q) * 4);
                                float* d = acc + c * kCols + q;
                                const uint32_t* x = v[c & 1] + q;
                                fma_pair(d[0], d[1], __uint_as_float(w.x), __uint_as_float(w.y), x[0], x[1]);
                                fma_pair(d[2], d[3], __uint_as_float(w.z), __uint_as_float(w.w), x[2], x[3]);
                            }
                        }
                    }
                }
            }
            if (!ok) break;
            if (!PAIR && a.split > 1) continue;               // (one tile per cluster: the loop ends here)
            if constexpr (TOK_LANES) {
                store_rows<C::kNC>(a, buf, lane, l0 + 32 * quarter, c0 + col0, acc);
            } else {
                store_cols<C::kNC>(a, c0 + col0, a.M - c0 - col0, l0 + r, acc);
            }
        }
        if (!PAIR && a.split > 1) {
            // Every CTA sends its part of each column to the CTA that joins it, which adds the ranks' parts in order
            // once all their bytes have come. (A CTA that gave up sends what it has.)
            const BmSched s(a, rank, PAIR);          // (one tile per cluster)
            const int l0 = s.t % a.lane_tiles * kBmLanes, c0 = s.t / a.lane_tiles * NT;
            if constexpr (TOK_LANES) {
                // Each rank joins `share` of every fold thread's columns, so that the thread that holds a column's
                // part here joins it there: [source][fold part][four columns][lane]. Its own part waits where the
                // ring's stages were: every MMA that read them has ended.
                const int quads = a.share / 4, mine = rank * a.share, own = min(C::kNC - mine, a.share);
                const uint32_t at = (part * quads * kBmLanes + r) * 16, step = C::kParts * quads * kBmLanes * 16;
                int owner = 0, q = 0;
#pragma unroll
                for (int j = 0; j < C::kNC; j += 4) {
                    const uint32_t off = at + q * (kBmLanes * 16);
                    if (owner == rank)
                        sts128(s_ring + off, __float_as_uint(acc[j]), __float_as_uint(acc[j + 1]),
                               __float_as_uint(acc[j + 2]), __float_as_uint(acc[j + 3]));
                    else
                        st_async4(map_to_rank(s_red + off + (rank - (rank > owner)) * step, owner), acc + j,
                                  map_to_rank(red_bar, owner));
                    if (++q == quads) q = 0, ++owner;
                }
                if (own > 0 && mbar_wait(red_bar, 0, ctl)) {
                    int done = 0;                    // columns
                    auto join = [&](auto columns) {
                        constexpr int kCnt = decltype(columns)::value;
                        float v[kCnt];
#pragma unroll
                        for (int i = 0; i < kCnt; ++i) v[i] = 0.f;
                        for (int o = 0; o < a.split; ++o) {
                            const uint32_t from = (o == rank ? s_ring : s_red + (o - (o > rank)) * step) + at +
                                                  done / 4 * (kBmLanes * 16);
#pragma unroll
                            for (int i = 0; i < kCnt / 4; ++i) {
                                const uint4 x = lds128(from + i * (kBmLanes * 16));
                                v[4 * i] += __uint_as_float(x.x), v[4 * i + 1] += __uint_as_float(x.y);
                                v[4 * i + 2] += __uint_as_float(x.z), v[4 * i + 3] += __uint_as_float(x.w);
                            }
                        }
                        store_rows<kCnt>(a, buf, lane, l0 + r - lane, c0 + part * C::kNC + mine + done, v);
                        done += kCnt;
                    };
                    if (own & 32) join(std::integral_constant<int, 32>());
                    if (own & 16) join(std::integral_constant<int, 16>());
                    if (own & 8) join(std::integral_constant<int, 8>());
                }
            } else {
                int owner = 0, at = 0;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (j >= a.M) break;
                    st_async(map_to_rank(s_red + ((rank * a.share + at) * kBmLanes + r) * 4, owner), acc[j],
                             map_to_rank(red_bar, owner));
                    if (++at == a.share) at = 0, ++owner;
                }
                const int first = rank * a.share, own = min(a.M - first, a.share);
                if (own > 0 && mbar_wait(red_bar, 0, ctl)) {
                    constexpr int kCnt = 4;
                    for (int c = 0; c < own; c += kCnt) {
                        float v[kCnt];
#pragma unroll
                        for (int q = 0; q < kCnt; ++q) v[q] = 0.f;
                        for (int o = 0; o < a.split; ++o) {
                            const uint32_t from = s_red + ((o * a.share + c) * kBmLanes + r) * 4;
#pragma unroll
                            for (int q = 0; q < kCnt; ++q)
                                if (c + q < own) v[q] += lds_f32(from + q * (kBmLanes * 4));
                        }
                        store_cols<kCnt>(a, c0 + first + c, own - c, l0 + r, v);
                    }
                }
            }
        }
    }
    if ((warp == 0 || warp == 2) && lane == 0) issued_by[warp >> 1] = issued;
    tc_fence_before();
    if constexpr (PAIR) {
        __syncwarp();
        cluster_sync();                              // the leader's MMAs are done, and every arrival on its barriers
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        bm_tmem_dealloc<PAIR>(tmem, C::kTmemCols);
    }
    // A CTA whose parts all came is sent nothing more. One that gave up stays until what the others send (they do
    // so in any case) is here, and until they, which may still send, have gone or given up too.
    if (!PAIR && a.split > 1 && *abort_flag) {
        if (threadIdx.x == 0) mbar_wait_plain(red_bar, 0, drain_limit(a.timeout_cycles));
        __syncwarp();
        cluster_sync();
    }
    if constexpr (TOK_LANES) {
        if (warp == 2 && lane == 0 && *abort_flag)
            for (int j = sc_issued > C::kScRing ? sc_issued - C::kScRing : 0; j < sc_issued; ++j)
                mbar_wait_plain(scfull_bar(j % C::kScRing), (j / C::kScRing) & 1, drain_limit(a.timeout_cycles));
    }
    // A CTA that gave up lets every copy in flight land before it goes. Where one copy thread stopped ahead
    // of the other, its arrivals are made up for first, so that the other's stages complete.
    if (warp == 0 && lane == 0 && *abort_flag) {
        const int less = min(issued_by[0], issued_by[1]), more = max(issued_by[0], issued_by[1]);
        for (int j = less; j < more; ++j) mbar_arrive(full_bar(j % a.stages));
        if (PAIR && rank == 0)                       // (nor can it be told whether the other CTA's arrivals came)
            for (int j = more > a.stages ? more - a.stages : 0; j < more; ++j)
                if (!mbar_test(full_bar(j % a.stages), (j / a.stages) & 1)) mbar_arrive(full_bar(j % a.stages));
        for (int j = more > a.stages ? more - a.stages : 0; j < more; ++j)
            mbar_wait_plain(full_bar(j % a.stages), (j / a.stages) & 1, drain_limit(a.timeout_cycles));
    }
}

bool encode_2d(EncodeTiledFn fn, CUtensorMap* map, CUtensorMapDataType type, const void* p, long long inner,
               long long rows, long long row_bytes, int box_inner, int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t one[2] = {1, 1};
    return fn(map, type, 2, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct BmCall {
    const void *X, *W;
    long long ldx, ldw;
    int K;
};

template <int NT, bool TOK_LANES, bool PAIR>
int go_block_mm(const Runtime& rt, const BmCall& c, BmArgs& a, wq4_stream_t st) {
    using C = BmCfg<NT, TOK_LANES, PAIR>;
    auto kern = block_mm_kernel<NT, TOK_LANES, PAIR>;
    // A kernel's shared memory is granted by device, as its occupancy below is a device's own.
    static PerDevice ready;
    const int regs = ready.get(rt.device, [&]() -> int {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBmMaxSmem) != cudaSuccess) {
            cudaGetLastError();
            return -1;
        }
        return fa.numRegs;
    });
    if (regs <= 0) return WQ4_ERR_CUDA;
    // the fold warps' share counts on the registers of the launch; with fewer their request would wait
    if (C::kRegSplit && regs != C::kLaunchRegs) return WQ4_ERR_CUDA;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto sw128 = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap *xmap = TOK_LANES ? &a.lane_map : &a.col_map, *wmap = TOK_LANES ? &a.col_map : &a.lane_map;
    if (!encode_2d(rt.encode, xmap, u8, c.X, c.K, a.M, c.ldx, kBmBlock, C::kTokens, sw128) ||
        !encode_2d(rt.encode, wmap, u8, c.W, c.K, a.N, c.ldw, kBmBlock, TOK_LANES ? C::kColRows : kBmLanes, sw128) ||
        (TOK_LANES && !encode_2d(rt.encode, &a.sx_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.sx, a.M, a.kb, a.ldsx * 4, kBmLanes,
                                 C::kScBlocks, CU_TENSOR_MAP_SWIZZLE_NONE)))
        return WQ4_ERR_CUDA;
    const int lanes = TOK_LANES ? a.M : a.N, cols = TOK_LANES ? a.N : a.M;
    constexpr int kTileLanes = PAIR ? 2 * kBmLanes : kBmLanes;
    a.lane_tiles = (lanes + kTileLanes - 1) / kTileLanes;
    const long long tiles = static_cast<long long>(a.lane_tiles) * ((cols + NT - 1) / NT);
    if (tiles > (1 << 30)) return WQ4_ERR_UNSUPPORTED;
    a.tiles = static_cast<int>(tiles);
    // CTAs per tile: what leaves each the fewest blocks of K, and of those the fewest. Clusters of s lie within
    // groups of SMs, so that fewer than sm_count / s run at a time: the occupancy calculation says how many
    // (95 x 2432 x 2176, 19 tiles: 13.9 us with 8 CTAs each, in two waves; 8.1 with 5).
    a.split = 1;
    for (int s = 2; !PAIR && s <= 8 && s <= a.kb && s * tiles <= rt.sm_count; ++s) {
        if (TOK_LANES && (s == 6 || s == 7)) continue;      // (their parts leave the ring fewer than four stages)
        if ((a.kb + s - 1) / s >= (a.kb + a.split - 1) / a.split) continue;
        static PerDevice resident[9];                // of clusters of s, and one more
        const int room = resident[s].get(rt.device, [&]() -> int {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(s);
            cfg.blockDim = dim3(C::kThreads);
            cfg.dynamicSmemBytes = kBmMaxSmem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = s;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
                cudaGetLastError();
                return -1;
            }
            return n + 1;
        });
        if (room <= 0) return WQ4_ERR_CUDA;
        if (tiles < room) a.split = s;
    }
    // More narrow tiles than SMs (and no whole number of waves of them): rings of half the size, two CTAs per SM
    // (4 x 28672 x 4096: 21.1 us; one CTA with the whole ring 23.6).
    constexpr bool kHalf = !TOK_LANES && NT <= 32;
    const bool half = kHalf && tiles > rt.sm_count;
    const int most = PAIR ? rt.sm_count / 2 : half ? 2 * rt.sm_count : rt.sm_count;   // tiles at a time
    const int grid = PAIR ? 2 * (a.tiles < most ? a.tiles : most) : a.split > 1 ? a.tiles * a.split : a.tiles < most ? a.tiles : most;
    // no more stages than a CTA has blocks: with few, the next launch's CTAs fit beside this one's
    a.share = TOK_LANES ? 8 * ((C::kNC / 8 + a.split - 1) / a.split) : (a.M + a.split - 1) / a.split;
    const int red = a.split == 1 ? 0 : kBmLanes * 4 * a.share * (TOK_LANES ? (a.split - 1) * C::kParts : a.split);
    const int blocks = (a.kb + a.split - 1) / a.split;
    a.stages = half ? C::kHalfStages : C::fit(red);
    if (a.split > 1 && blocks < a.stages) a.stages = blocks < 4 ? 4 : (blocks + 1) & ~1;
    const int smem = C::kHeadBytes + a.stages * C::kStageBytes + red;
    if (rt.trace)
        std::fprintf(stderr, "wq4: block_mm M=%d N=%d K=%d lanes=%s columns=%d pair=%d grid=%d split=%d\n", a.M, a.N, c.K,
                     TOK_LANES ? "tokens" : "weights", NT, PAIR ? 1 : 0, grid, a.split);
    return launch(rt, kern, dim3(grid), C::kThreads, smem, PAIR ? 2 : a.split, st, a);
}

}  // namespace
}  // namespace wq4

using namespace wq4;

extern "C" int wq4_block_mm(const void* X, long long ldx, const float* x_scales, long long ldsx, const void* W,
                            long long ldw, const float* w_scales, long long ldsw, void* Y, long long ldy, int M, int N,
                            int K, int dtype, wq4_stream_t stream) {
    if (M < 0 || N < 1 || K < 1) return WQ4_ERR_INVALID;
    if (dtype != WQ4_BF16 && dtype != WQ4_FP16 && dtype != WQ4_FP32) return WQ4_ERR_INVALID;
    const int kb = K / kBmBlock + (K % kBmBlock ? 1 : 0);
    if (K % 16) return WQ4_ERR_UNSUPPORTED;
    if (M == 0) return WQ4_OK;
    if (ldx < K || ldw < K || ldsx < M || ldsw < kb || ldy < N) return WQ4_ERR_INVALID;
    if (!X || !x_scales || !W || !w_scales || !Y) return WQ4_ERR_INVALID;
    const int size = dtype == WQ4_FP32 ? 4 : 2;
    if (!aligned_to(X, 16) || !aligned_to(W, 16) || !aligned_to(x_scales, 16) || ldx % 16 || ldw % 16 || ldsx % 4 ||
        !aligned_to(w_scales, 4) || !aligned_to(Y, size))
        return WQ4_ERR_ALIGN;
    // a tensor map's row stride is below 2^40 bytes
    if (ldx >= (1LL << 40) || ldw >= (1LL << 40) || ldsx >= (1LL << 38)) return WQ4_ERR_UNSUPPORTED;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    const BmCall c{X, W, ldx, ldw, K};
    BmArgs a{};
    a.sx = x_scales;
    a.sw = w_scales;
    a.ldsx = ldsx;
    a.y = Y;
    a.ldy = ldy;
    a.ldsw = ldsw;
    a.M = M;
    a.N = N;
    a.kb = kb;
    a.dtype = dtype;
    a.unit = 16;
    while (a.unit > size && !(aligned_to(Y, a.unit) && ldy * size % a.unit == 0)) a.unit /= 2;
    if (dtype == WQ4_FP32 && a.unit == 8) a.unit = 4;
    a.status = rt.status;
    a.timeout_cycles = rt.timeout_cycles;
    a.test_stall = rt.test_stall;
    if (M <= 16) return go_block_mm<16, false, false>(rt, c, a, stream);
    if (M <= 32) return go_block_mm<32, false, false>(rt, c, a, stream);
    if (M <= 64) return go_block_mm<64, false, false>(rt, c, a, stream);
    // A wave of pair tiles takes 1.5 times as long as one of 128-column tiles, and covers twice as much of Y
    // (1109 x 3840 x 7168: 26.9 us in one wave of pairs, 34.3 in two of the others; 877 x 10019 x 4736: 55.2
    // in three of pairs, 49.3 in four of the others).
    const long long rows = (M + 127) / 128, cols = (N + 127) / 128, one = rt.sm_count, pairs = rt.sm_count / 2;
    const long long w128 = (rows * cols + one - 1) / one, w256 = ((rows + 1) / 2 * ((cols + 1) / 2) + pairs - 1) / pairs;
    if (3 * w256 <= 2 * w128) return go_block_mm<256, true, true>(rt, c, a, stream);
    return go_block_mm<128, true, false>(rt, c, a, stream);
}
