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
//   warp 0   copies: per block of K, both operands' 128-byte row pieces as 2-D tensor copies with the
//            128-byte swizzle (rows and K past the end read as zero) and the tokens' scales, into a
//            ring of stages
//   warp 1   MMAs: one thread issues the block's four (K = 32 each), commits to the fold warps
//   warps 4+ fold: read P_b, add it in, at a tile's end round once and store
// With fewer tiles than SMs, a cluster of CTAs shares each tile, cut along K; the parts are added in
// rank order through distributed shared memory.
//
// Every wait is bounded, as in wq4_gemm.cuh: one that runs out is recorded in the status word and the
// CTA drains its copies and MMAs, frees its tensor memory and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdio>

#include "wq4_device.cuh"
#include "wq4_runtime.h"

namespace wq4 {
namespace {

constexpr int kBmBlock = 128;                  // K elements (bytes) of a block
constexpr int kBmLanes = 128;                  // rows of the lane operand per tile
constexpr int kBmMaxSmem = 232448;

struct BmArgs {
    CUtensorMap lane_map, col_map;             // e4m3 codes [rows][K], box 128 K x tile rows
    CUtensorMap sx_map;                        // token scales [blocks][M], box tokens of a tile x 1
    const float* sw;                           // weight scales, row n / 128, column b
    void* y;
    long long ldy, ldsw;
    int M, N, kb;                              // kb: blocks of K
    int lane_tiles, tiles;                     // tile t: lane tile t % lane_tiles, column tile t / lane_tiles
    int split;                                 // CTAs per cluster, each with a part of K (1: none)
    int dtype;
    int vec_store;                             // rows of Y start on 16-byte boundaries
    unsigned int* status;
    long long timeout_cycles;
    int test_stall;
};

// NT: columns of a tile; TOK_LANES: tokens on the lanes (else weight rows).
template <int NT, bool TOK_LANES>
struct BmCfg {
    static constexpr int kFW = TOK_LANES ? 8 : 4;               // fold warps
    static constexpr int kParts = kFW / 4;                      // fold warps per lane quarter
    static constexpr int kNC = NT / kParts;                     // columns of a fold thread
    static constexpr int kThreads = 128 + 32 * kFW;
    static constexpr int kLaneBytes = kBmLanes * kBmBlock;
    static constexpr int kColBytes = NT * kBmBlock;
    static constexpr int kTokens = TOK_LANES ? kBmLanes : NT;
    static constexpr int kScaleBytes = kTokens * 4;
    static constexpr int kStageBytes = kLaneBytes + kColBytes + 1024;   // scales in the last KB
    static constexpr int kBarBytes = 1024;
    static constexpr int kFit = (kBmMaxSmem - 1024 - kBarBytes) / kStageBytes;
    static constexpr int kStages = kFit > 12 ? 12 : kFit;
    static constexpr int kPBufs = NT <= 128 ? 4 : 2;
    static constexpr int kTmemCols = NT * kPBufs < 32 ? 32 : NT * kPBufs;
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kBarBytes;
    // 128 fp32 accumulators per fold thread want more registers than an even share: 384 threads
    // launched with 168 each (64512 in all), of which the copy and MMA warps keep 72 and the fold
    // warps take 216 (128 x 72 + 256 x 216 = 64512).
    static constexpr bool kRegSplit = kNC > 64;
    static constexpr int kLaunchRegs = 168, kRegWg0 = 72, kRegFold = 216;
    static_assert(!kRegSplit || 128 * kRegWg0 + 32 * kFW * kRegFold <= kThreads * kLaunchRegs, "register split");
    static_assert(kStages >= 3 && kTmemCols <= 512 && kSmemBytes <= kBmMaxSmem, "tile");
    static_assert(kStages * kStageBytes >= kBmLanes * NT * 4, "cluster reduction buffer");
};

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// kind::f8f6f4: D fp32, A and B e4m3 (format code 0), both K-major, M x N.
__device__ constexpr uint32_t f8_idesc(uint32_t M, uint32_t N) { return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24); }

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

// One value in the output type (dtype is the same for the whole launch).
__device__ __forceinline__ void store_y(void* y, long long at, float v, int dtype) {
    if (dtype == WQ4_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else if (dtype == WQ4_FP16) static_cast<__half*>(y)[at] = __float2half_rn(v);
    else static_cast<float*>(y)[at] = v;
}

// Columns [n, n + 8) of row m, of which those below N exist.
__device__ __forceinline__ void store_row8(const BmArgs& a, int m, int n, const float* v) {
    const long long at = m * a.ldy + n;
    if (a.vec_store && n + 8 <= a.N) {
        if (a.dtype == WQ4_FP32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.y) + at);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
            return;
        }
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (a.dtype == WQ4_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
            else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + at) = make_uint4(u[0], u[1], u[2], u[3]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (n + j < a.N) store_y(a.y, at + j, v[j], a.dtype);
}

// The tiles of one CTA, in order, and the part of K it takes of each.
struct BmSched {
    int t, step, kb0, kb1;
    __device__ BmSched(const BmArgs& a, int rank) {
        t = blockIdx.x / a.split;
        step = gridDim.x / a.split;
        kb0 = static_cast<int>(static_cast<long long>(a.kb) * rank / a.split);
        kb1 = static_cast<int>(static_cast<long long>(a.kb) * (rank + 1) / a.split);
    }
};

template <int NT, bool TOK_LANES>
__global__ void __launch_bounds__(BmCfg<NT, TOK_LANES>::kThreads, 1) block_mm_kernel(const __grid_constant__ BmArgs a) {
    using C = BmCfg<NT, TOK_LANES>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t s_ring = (raw_s + 1023u) & ~1023u;
    const uint32_t s_bar = s_ring + C::kStages * C::kStageBytes;
    auto full_bar = [&](int s) { return s_bar + 8u * s; };
    auto empty_bar = [&](int s) { return s_bar + 8u * (16 + s); };
    auto pfull_bar = [&](int b) { return s_bar + 8u * (32 + b); };
    auto pempty_bar = [&](int b) { return s_bar + 8u * (36 + b); };
    const uint32_t drain_bar = s_bar + 8u * 40, stall_bar = s_bar + 8u * 41;
    uint8_t* const gmisc = smem_raw + (s_bar - raw_s) + 8 * 48;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gmisc);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(gmisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.split > 1 ? static_cast<int>(cluster_rank()) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1 + C::kFW);     // the MMAs' commit, and the fold warps done with the scales
        }
        for (int b = 0; b < C::kPBufs; ++b) {
            mbar_init(pfull_bar(b), 1);
            mbar_init(pempty_bar(b), C::kFW);
        }
        mbar_init(drain_bar, 1);
        mbar_init(stall_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&a.lane_map);
        prefetch_tensormap(&a.col_map);
        prefetch_tensormap(&a.sx_map);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const WaitCtl ctl{abort_flag, a.status, a.timeout_cycles};
    int issued = 0;                                  // stages the copy thread has filled

    if (warp < 4) {
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegWg0));
        if (warp == 0) {
            if (lane == 0) {
                // an operand that only one tile along its side reads streams through L2
                const uint64_t first = policy_evict_first(), last = policy_evict_last();
                const bool cols_once = a.lane_tiles == 1, lanes_once = a.tiles == a.lane_tiles;
                bool ok = true;
                int i = 0;
                for (BmSched s(a, rank); s.t < a.tiles && ok; s.t += s.step) {
                    const int l0 = s.t % a.lane_tiles * kBmLanes, c0 = s.t / a.lane_tiles * NT;
                    for (int b = s.kb0; b < s.kb1; ++b, ++i) {
                        const int st = i % C::kStages;
                        if (!mbar_wait(empty_bar(st), ((i / C::kStages) & 1) ^ 1, ctl)) { ok = false; break; }
                        const uint32_t stage = s_ring + st * C::kStageBytes;
                        mbar_arrive_expect_tx(full_bar(st), C::kLaneBytes + C::kColBytes + C::kScaleBytes);
                        tma_load_2d(stage, &a.lane_map, full_bar(st), b * kBmBlock, l0, lanes_once ? first : last);
                        tma_load_2d(stage + C::kLaneBytes, &a.col_map, full_bar(st), b * kBmBlock, c0, cols_once ? first : last);
                        tma_load_2d(stage + C::kLaneBytes + C::kColBytes, &a.sx_map, full_bar(st), TOK_LANES ? l0 : c0, b, last);
                    }
                }
                issued = i;
            }
            __syncwarp();
        } else if (warp == 1) {
            if (lane == 0) {
                constexpr uint32_t idesc = f8_idesc(kBmLanes, NT);
                bool ok = !a.test_stall || mbar_wait(stall_bar, 0, ctl);
                int i = 0;
                for (BmSched s(a, rank); s.t < a.tiles && ok; s.t += s.step) {
                    for (int b = s.kb0; b < s.kb1; ++b, ++i) {
                        const int st = i % C::kStages, p = i % C::kPBufs;
                        if (!mbar_wait(full_bar(st), (i / C::kStages) & 1, ctl)) { ok = false; break; }
                        if (!mbar_wait(pempty_bar(p), ((i / C::kPBufs) & 1) ^ 1, ctl)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t stage = s_ring + st * C::kStageBytes;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8(tmem + p * NT, make_sdesc_sw128(stage + 32 * k),
                                   make_sdesc_sw128(stage + C::kLaneBytes + 32 * k), idesc, k > 0);
                        mma_commit(pfull_bar(p));
                        mma_commit(empty_bar(st));
                    }
                }
                mma_commit(drain_bar);               // every MMA is done before the tensor memory goes
                mbar_wait_plain(drain_bar, 0, drain_limit(a.timeout_cycles));
            }
            __syncwarp();
        }
    } else {
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegFold));
        const int quarter = warp & 3, part = (warp - 4) >> 2;
        const int r = 32 * quarter + lane;           // this thread's lane of the tile
        const int col0 = part * C::kNC;              // and its first column
        const uint32_t t_addr = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + col0;
        const int sw_rows = (a.N + 127) / 128;
        float acc[C::kNC] = {};
        bool ok = true;
        int i = 0;
        for (BmSched s(a, rank); s.t < a.tiles && ok; s.t += s.step) {
            const int l0 = s.t % a.lane_tiles * kBmLanes, c0 = s.t / a.lane_tiles * NT;
            const int wrow = min((TOK_LANES ? c0 + col0 : l0) / 128, sw_rows - 1);
            const float* sw = a.sw + wrow * a.ldsw;
#pragma unroll
            for (int j = 0; j < C::kNC; ++j) acc[j] = 0.f;
            float w = s.kb0 < s.kb1 ? __ldg(sw + s.kb0) : 0.f;
            for (int b = s.kb0; b < s.kb1; ++b, ++i) {
                const int st = i % C::kStages, p = i % C::kPBufs;
                const float w_next = b + 1 < s.kb1 ? __ldg(sw + b + 1) : 0.f;
                if (!mbar_wait(pfull_bar(p), (i / C::kPBufs) & 1, ctl)) { ok = false; break; }
                // (the stage's copies had landed before its MMAs were issued; this wait, which passes at
                // once, makes the scales among them visible here)
                if (!mbar_wait(full_bar(st), (i / C::kStages) & 1, ctl)) { ok = false; break; }
                tc_fence_after();
                const uint32_t s_sx = s_ring + st * C::kStageBytes + C::kLaneBytes + C::kColBytes;
                if constexpr (TOK_LANES) {
                    const float f = lds_f32(s_sx + 4 * r) * w;
#pragma unroll
                    for (int j = 0; j < C::kNC; j += 32) {
                        uint32_t v[32];
                        tmem_ld32(t_addr + p * NT + j, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 32; ++q) acc[j + q] = fmaf(f, __uint_as_float(v[q]), acc[j + q]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < C::kNC; j += 8) {
                        uint32_t v[8];
                        tmem_ld8(t_addr + p * NT + j, v);
                        const uint4 f0 = lds128(s_sx + 4 * j), f1 = lds128(s_sx + 4 * j + 16);
                        const uint32_t f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            acc[j + q] = fmaf(__uint_as_float(f[q]) * w, __uint_as_float(v[q]), acc[j + q]);
                    }
                }
                w = w_next;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(pempty_bar(p));
                    mbar_arrive(empty_bar(st));
                }
            }
            if (!ok) break;
            if (a.split > 1) continue;               // (one tile per cluster: the loop ends here)
            if constexpr (TOK_LANES) {
                if (l0 + r < a.M) {
#pragma unroll
                    for (int j = 0; j < C::kNC; j += 8) store_row8(a, l0 + r, c0 + col0 + j, acc + j);
                }
            } else if (l0 + r < a.N) {
#pragma unroll
                for (int j = 0; j < C::kNC; ++j)
                    if (c0 + col0 + j < a.M) store_y(a.y, (c0 + col0 + j) * a.ldy + l0 + r, acc[j], a.dtype);
            }
        }
        if (a.split > 1) {
            // This CTA's part, [column][lane], over the ring: its MMAs and with them its copies are done,
            // and after the barrier no fold warp reads scales from it. (Of a CTA that gave up the parts
            // are undefined, as its outputs are; its copies still land in its own shared memory.)
            asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kFW) : "memory");
#pragma unroll
            for (int j = 0; j < C::kNC; ++j)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(s_ring + ((col0 + j) * kBmLanes + r) * 4), "f"(acc[j])
                             : "memory");
        }
    }
    if (a.split > 1) {
        __syncwarp();
        cluster_sync();                              // every part of the tile is in its CTA's shared memory
        if (warp >= 4) {
            const int t = blockIdx.x / a.split;      // (one tile per cluster)
            const int l0 = t % a.lane_tiles * kBmLanes, c0 = t / a.lane_tiles * NT;
            const int r = 32 * (warp & 3) + lane;
            // eight columns at a time, dealt out over the ranks and their warps
            for (int j = (rank * C::kParts + ((warp - 4) >> 2)) * 8; j < NT; j += a.split * C::kParts * 8) {
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = 0.f;
                for (int o = 0; o < a.split; ++o) {
                    const uint32_t base = map_to_rank(s_ring, o);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] += ld_cluster_f32(base + ((j + q) * kBmLanes + r) * 4);
                }
                if constexpr (TOK_LANES) {
                    if (l0 + r < a.M) store_row8(a, l0 + r, c0 + j, v);
                } else if (l0 + r < a.N) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (c0 + j + q < a.M) store_y(a.y, (c0 + j + q) * a.ldy + l0 + r, v[q], a.dtype);
                }
            }
        }
        __syncwarp();
        cluster_sync();                              // no CTA leaves while another reads its part
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    // a CTA that gave up lets every copy in flight land before it goes
    if (warp == 0 && lane == 0 && *abort_flag)
        for (int j = issued > C::kStages ? issued - C::kStages : 0; j < issued; ++j)
            mbar_wait_plain(full_bar(j % C::kStages), (j / C::kStages) & 1, drain_limit(a.timeout_cycles));
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
    const float* sx;
    long long ldx, ldw, ldsx;
    int K;
};

template <int NT, bool TOK_LANES>
int go_block_mm(const Runtime& rt, const BmCall& c, BmArgs& a, wq4_stream_t st) {
    using C = BmCfg<NT, TOK_LANES>;
    auto kern = block_mm_kernel<NT, TOK_LANES>;
    static int regs = -1;                            // (one value per kernel, whoever writes it)
    if (regs < 0) {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
            return WQ4_ERR_CUDA;
        regs = fa.numRegs;
    }
    // the fold warps' share counts on the registers of the launch; with fewer their request would wait
    if (C::kRegSplit && regs != C::kLaunchRegs) return WQ4_ERR_CUDA;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto sw128 = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap *xmap = TOK_LANES ? &a.lane_map : &a.col_map, *wmap = TOK_LANES ? &a.col_map : &a.lane_map;
    if (!encode_2d(rt.encode, xmap, u8, c.X, c.K, a.M, c.ldx, kBmBlock, C::kTokens, sw128) ||
        !encode_2d(rt.encode, wmap, u8, c.W, c.K, a.N, c.ldw, kBmBlock, TOK_LANES ? NT : kBmLanes, sw128) ||
        !encode_2d(rt.encode, &a.sx_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, c.sx, a.M, a.kb, c.ldsx * 4, C::kTokens, 1,
                   CU_TENSOR_MAP_SWIZZLE_NONE))
        return WQ4_ERR_CUDA;
    const int lanes = TOK_LANES ? a.M : a.N, cols = TOK_LANES ? a.N : a.M;
    a.lane_tiles = (lanes + kBmLanes - 1) / kBmLanes;
    const long long tiles = static_cast<long long>(a.lane_tiles) * ((cols + NT - 1) / NT);
    if (tiles > (1 << 30)) return WQ4_ERR_UNSUPPORTED;
    a.tiles = static_cast<int>(tiles);
    a.split = 1;
    while (a.split < 8 && 2 * a.split * tiles <= rt.sm_count && 2 * a.split <= a.kb) a.split *= 2;
    const int grid = a.split > 1 ? a.tiles * a.split : (a.tiles < rt.sm_count ? a.tiles : rt.sm_count);
    if (rt.trace)
        std::fprintf(stderr, "wq4: block_mm M=%d N=%d K=%d lanes=%s columns=%d grid=%d split=%d\n", a.M, a.N, c.K,
                     TOK_LANES ? "tokens" : "weights", NT, grid, a.split);
    return launch(rt, kern, dim3(grid), C::kThreads, C::kSmemBytes, a.split, st, a);
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
    const BmCall c{X, W, x_scales, ldx, ldw, ldsx, K};
    BmArgs a{};
    a.sw = w_scales;
    a.y = Y;
    a.ldy = ldy;
    a.ldsw = ldsw;
    a.M = M;
    a.N = N;
    a.kb = kb;
    a.dtype = dtype;
    a.vec_store = aligned_to(Y, 16) && ldy * size % 16 == 0;
    a.status = rt.status;
    a.timeout_cycles = rt.timeout_cycles;
    a.test_stall = rt.test_stall;
    if (M <= 16) return go_block_mm<16, false>(rt, c, a, stream);
    if (M <= 32) return go_block_mm<32, false>(rt, c, a, stream);
    if (M <= 64) return go_block_mm<64, false>(rt, c, a, stream);
    const long long wide = static_cast<long long>((M + 127) / 128) * ((N + 255) / 256);
    if (2 * wide > rt.sm_count) return go_block_mm<256, true>(rt, c, a, stream);
    return go_block_mm<128, true>(rt, c, a, stream);
}
