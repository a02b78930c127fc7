// Rows in 8-bit float for the block-scaled product (wq4_block_mm.cu): RMS norm with the residual's
// addition, and the gated activation. Both end alike. A row's values y, in fp32, are cut into
// blocks of 128; block b of token t gets the scale
//     s[b][t] = max(max |y| / 448, 2^-126)
// and the codes q = e4m3(y / s), every quotient rounded to fp32 and the code to nearest even; 448 is e4m3's largest value, and the
// lower bound keeps the quotient defined for a block of zeros. A NaN stays one in its own code and
// does not touch its block's scale; a block with an infinity has an infinite scale, so that every
// value read back from it (q s) is NaN.
//
// Both are bound by memory: each element is read and written once, in 16-byte vectors of 8 elements
// (across boundaries where rows do not start on one), and everything in between stays in registers. 16
// neighbouring lanes hold one block of 128, so a block's maximum takes four shuffles and no shared
// memory. Passes back to back: norm with residual, 4096 x 4096 bf16, 20.6 us (5.7 TB/s); gated,
// 4096 x 14336 bf16, 44.8 us (6.6 TB/s); 1 x 4096 and 16 x 14336 take 1.6 and 1.4 us, a launch and one
// trip to memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "wq4_device.cuh"
#include "wq4_runtime.h"

namespace wq4 {
namespace {

constexpr int kVec = 8;                 // elements a thread handles together
constexpr int kRowBlock = 128;          // elements that share a scale
constexpr float kE4m3Max = 448.f;

template <bool BF16>
__device__ __forceinline__ float to_f32(uint32_t b16) {
    if constexpr (BF16) return __uint_as_float(b16 << 16);
    else return __half2float(__ushort_as_half(static_cast<uint16_t>(b16)));
}

// Two values rounded to the 16-bit type, `lo` in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t u;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    return u;
}

// Two fp32 operations in one instruction each: at the rate of HBM an SM has some 20 instructions for
// 32 elements, and these kernels' arithmetic is most of what they issue.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ void add8(float (&a)[kVec], const float (&b)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; j += 2) {
        uint64_t d;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])));
        unpair(d, a[j], a[j + 1]);
    }
}
__device__ __forceinline__ void mul8(float (&a)[kVec], const float (&b)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; j += 2) {
        uint64_t d;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])));
        unpair(d, a[j], a[j + 1]);
    }
}
__device__ __forceinline__ void mul8(float (&a)[kVec], float b) {
    const float v[kVec] = {b, b, b, b, b, b, b, b};
    mul8(a, v);
}
// sum of the squares, added to the two halves of s
__device__ __forceinline__ void squares8(const float (&a)[kVec], uint64_t& s) {
#pragma unroll
    for (int j = 0; j < kVec; j += 2) {
        const uint64_t x = pair(a[j], a[j + 1]);
        asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(s) : "l"(x));
    }
}
// 1 / x to an ulp or so (0 for infinity and for x > 2^126)
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// -a / b of each, rounded to nearest, from r, the reciprocal of b rounded to nearest: q = -a r is within an ulp or so of it, and
// q - r (q b + a), two fused operations more, then is it (P. Markstein, Computation of elementary functions on the IBM
// RISC System/6000 processor, 1990), as long as nothing underflows. (So and not with a / b, a zero keeps its sign.)
__device__ __forceinline__ void minus_div8(float (&a)[kVec], float b, float r) {
    const uint64_t bb = pair(b, b), minus_r = pair(-r, -r);
#pragma unroll
    for (int j = 0; j < kVec; j += 2) {
        const uint64_t x = pair(a[j], a[j + 1]);
        uint64_t q, rest;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(minus_r));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rest) : "l"(q), "l"(bb), "l"(x));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q) : "l"(rest), "l"(minus_r));
        unpair(q, a[j], a[j + 1]);
    }
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint32_t (&u)[4], float (&v)[kVec]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = to_f32<BF16>(u[j] & 0xffffu);
        v[2 * j + 1] = to_f32<BF16>(u[j] >> 16);
    }
}

// Four words from byte `at` (a multiple of 2, at most 16) of the eight in c.
__device__ __forceinline__ void words_from(const uint32_t (&c)[8], uint32_t at, uint32_t (&d)[4]) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c[j];
#pragma unroll
    for (int step = 4; step; step >>= 1)
        if (at & (4 * step)) {
#pragma unroll
            for (int j = 0; j + step < 8; ++j) w[j] = w[j + step];
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = at & 2 ? __funnelshift_r(w[j], w[j + 1], 16) : w[j];
}

// Eight elements from column `col` (a multiple of 8) of a row of D, zeros past its end, in two steps, so that
// a thread's loads are all under way before the first is used. VEC: the row starts and ends on
// 16-byte boundaries, one load. Otherwise two aligned loads that the eight lie across, where both are
// inside the row, and single elements at its ends (in the second step).
template <bool VEC>
struct Raw8 {
    uint4 lo, hi;
};
template <bool VEC>
__device__ __forceinline__ bool inside(uint32_t off, int col, int D) {
    return VEC ? col < D : off ? col > 0 && col + 2 * kVec <= D : col + kVec <= D;
}
__device__ __forceinline__ uint32_t row_off(const uint16_t* row) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
}
template <bool VEC>
__device__ __forceinline__ Raw8<VEC> begin8(const uint16_t* row, int col, int D) {
    Raw8<VEC> r;
    r.lo = r.hi = make_uint4(0, 0, 0, 0);
    const uint32_t off = VEC ? 0 : row_off(row);
    const bool in = inside<VEC>(off, col, D);
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row + col) - off);
    if (in) r.lo = p[0];
    if (!VEC && in && off) r.hi = p[1];
    return r;
}
template <bool BF16, bool VEC>
__device__ __forceinline__ void end8(const Raw8<VEC>& r, const uint16_t* row, int col, int D, float (&v)[kVec]) {
    if constexpr (VEC) {
        const uint32_t u[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
        unpack8<BF16>(u, v);
    } else {
        const uint32_t off = row_off(row), c[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
        uint32_t u[4];
        words_from(c, off, u);
        unpack8<BF16>(u, v);
        if (!inside<VEC>(off, col, D) && col < D) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = col + j < D ? to_f32<BF16>(row[col + j]) : 0.f;
        }
    }
}
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const uint16_t* row, int col, int D, float (&v)[kVec]) {
    end8<BF16, VEC>(begin8<VEC>(row, col, D), row, col, D, v);
}

// The reverse, for a warp whose lanes hold neighbouring eights: off a boundary, each lane stores the aligned
// sixteen bytes that end inside its eight, of which the first come from the lane below, and what
// has no lane below or above in the warp goes in single elements. Every lane of the warp calls it.
template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(uint16_t* row, int col, int D, const float (&v)[kVec]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = pack2<BF16>(v[2 * j], v[2 * j + 1]);
    if constexpr (VEC) {
        if (col < D) *reinterpret_cast<uint4*>(row + col) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
        const int lane = threadIdx.x & 31, back = off / 2;       // elements of the lane below
        uint32_t c[8], w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = __shfl_up_sync(0xffffffffu, u[j], 1);
            c[4 + j] = u[j];
        }
        words_from(c, 16 - off, w);
        const int first = col - back;                            // the column w starts with
        if ((lane || !off) && first + kVec <= D) {
            *reinterpret_cast<uint4*>(row + first) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if ((lane || j >= back) && first + j < D)
                    row[first + j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
        }
        if (lane == 31) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (j >= kVec - back && col + j < D) row[col + j] = static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)));
        }
    }
}

// Two fp32 to two e4m3 codes (nearest even; past 448: 448; NaN stays NaN), `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// The codes of -y, eight values of a row (the thread's 16 lanes hold the block of 128 they are in), and, from the
// first of those lanes, the block's scale. Every lane of the warp calls it.
template <bool VEC>
__device__ __forceinline__ void quantise8(float (&y)[kVec], int col, int D, uint8_t* q_row, float* scale) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) m = fmaxf(m, fabsf(y[j]));      // (fmaxf passes NaN over)
#pragma unroll
    for (int d = 8; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    // m / 448 and the quotients rounded to nearest, by reciprocals and remainders: divisions one by one took
    // longer (4096 x 4096 norm 21.4 us), products with the reciprocals alone less (20.3), but their codes can be a
    // step off at a rounding boundary.
    float s = m;
    if (m <= FLT_MAX) {
        const float s0 = m * (1.f / kE4m3Max);
        s = fmaxf(fmaf(fmaf(-kE4m3Max, s0, m), 1.f / kE4m3Max, s0), FLT_MIN);
        const float r = rcp(s);
        minus_div8(y, s, fmaf(r, fmaf(-s, r, 1.f), r));
    } else {
        mul8(y, -0.f);                               // (y / s is 0, or NaN; branches: 4096 x 14336 46.8 us with selects)
    }
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = e4m3x2(y[2 * j], y[2 * j + 1]);
    if (col < D) {                                   // (rows of codes start on 16-byte boundaries)
        if (VEC || col + kVec <= D) {
            *reinterpret_cast<uint2*>(q_row + col) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (col + j < D) q_row[col + j] = static_cast<uint8_t>(c[j >> 1] >> (8 * (j & 1)));
        }
        if ((threadIdx.x & 15) == 0) *scale = s;
    }
}

// ------------------------------------------------------------------------------ RMS norm
struct NormArgs {
    const uint16_t *x, *r, *w;          // r: null without a residual
    uint16_t *r_out, *y;                // null where not asked for
    uint8_t* q;                         // null where not asked for
    float* scales;
    long long ldx, ldr, ldro, ldy, ldq, lds;
    int T, D;
    float eps, one_over_D;
};

// A thread holds VPT vectors of a row in registers, so the row is read once although its norm has to be known
// before the first value can be scaled. WARP: one warp per row, kNormRows rows per CTA; else one CTA per
// row. With one vector per thread (few rows: the time is the latency of one row) the weight is loaded ahead
// of the sum; with more its registers are better spent on more rows per SM.
constexpr int kNormRows = 4;

// CTAs of the largest size that an SM holds, by their registers.
constexpr int norm_ctas(bool vec, int vpt) { return vpt == 1 ? (vec ? 2 : 1) : vpt == 2 ? (vec ? 3 : 2) : vec && vpt == 4 ? 2 : 1; }

template <bool BF16, bool VEC, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kNormRows : VPT > 1 ? 512 : 1024, WARP ? (VEC ? 16 : 8) : norm_ctas(VEC, VPT))
    norm_kernel(const NormArgs a) {
    __shared__ float part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tid = WARP ? lane : threadIdx.x, n = WARP ? 32 : blockDim.x;
    const long long t = WARP ? static_cast<long long>(blockIdx.x) * kNormRows + warp : blockIdx.x;
    const int D = a.D;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (WARP && t >= a.T) return;

    float h[VPT][kVec], w0[kVec];
    uint64_t ss2 = 0;
    auto col_of = [&](int i) { return (i * n + tid) * kVec; };
    if constexpr (VEC || VPT > 4) {
        if constexpr (VPT == 1) load8<BF16, VEC>(a.w, col_of(0), D, w0);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            load8<BF16, VEC>(a.x + t * a.ldx, col_of(i), D, h[i]);
            if (a.r) {
                float r[kVec];
                load8<BF16, VEC>(a.r + t * a.ldr, col_of(i), D, r);
                add8(h[i], r);
            }
        }
    } else {                                         // (single elements only after every vector is under way)
        Raw8<VEC> x[VPT], r[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            x[i] = begin8<VEC>(a.x + t * a.ldx, col_of(i), D);
            if (a.r) r[i] = begin8<VEC>(a.r + t * a.ldr, col_of(i), D);
        }
        if constexpr (VPT == 1) load8<BF16, VEC>(a.w, col_of(0), D, w0);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            end8<BF16, VEC>(x[i], a.x + t * a.ldx, col_of(i), D, h[i]);
            if (a.r) {
                float v[kVec];
                end8<BF16, VEC>(r[i], a.r + t * a.ldr, col_of(i), D, v);
                add8(h[i], v);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        squares8(h[i], ss2);
        // the sum in the 16-bit type is for the next layer; the norm goes by the unrounded one
        if (a.r_out) store8<BF16, VEC>(a.r_out + t * a.ldro, col_of(i), D, h[i]);
    }
    float ss, odd;
    unpair(ss2, ss, odd);
    ss += odd;
#pragma unroll
    for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if constexpr (!WARP) {
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        ss = lane < (n >> 5) ? part[lane] : 0.f;
#pragma unroll
        for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    }
    const float rstd = rsqrtf(fmaf(ss, a.one_over_D, a.eps));     // (2 ulp)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int col = col_of(i);
        float w[kVec];
        if constexpr (VPT > 1) load8<BF16, VEC>(a.w, col, D, w);
        mul8(h[i], -rstd);                           // (-y from here on)
        if constexpr (VPT == 1) mul8(h[i], w0);
        else mul8(h[i], w);
        if (a.y) {
            float y[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) y[j] = -h[i][j];
            store8<BF16, VEC>(a.y + t * a.ldy, col, D, y);
        }
        if (a.q) quantise8<VEC>(h[i], col, D, a.q + t * a.ldq, a.scales + (col / kRowBlock) * a.lds + t);
    }
}

template <bool BF16, bool VEC>
int go_norm(const Runtime& rt, const NormArgs& a, wq4_stream_t st) {
    const int nv = (a.D + kVec - 1) / kVec;
    const bool many = a.T > 4 * rt.sm_count;
    // Many short rows: a warp each (8192 x 256 bf16: 4.2 us against 8.6 with a CTA each).
    if (many && nv <= 64) {
        const dim3 grid((static_cast<unsigned>(a.T) + kNormRows - 1) / kNormRows);
        if (nv <= 32) return launch(rt, norm_kernel<BF16, VEC, 1, true>, grid, 32 * kNormRows, 0, 1, st, a);
        return launch(rt, norm_kernel<BF16, VEC, 2, true>, grid, 32 * kNormRows, 0, 1, st, a);
    }
    // Vectors per thread: one, two or four. Measured with the residual, bf16: 4096 x 4096, 24.2 / 21.0 / 22.1 us;
    // 2000 x 8192, 26.7 / 21.1 / 22.1; 1 x 4096, 1.7 / 2.0 / 2.7; 4096 x 1024, 7.2 / 8.7 / 9.5; 517 x 2064
    // without it, 2.2 / 3.1 / 3.4. (Two: at most 40 registers, three CTAs of 512.)
    const int vpt = nv > 2048 ? 8 : nv > 1024 ? 4 : many && nv > 256 ? 2 : 1;
    const int threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
    switch (vpt) {
        case 1: return launch(rt, norm_kernel<BF16, VEC, 1, false>, dim3(a.T), threads, 0, 1, st, a);
        case 2: return launch(rt, norm_kernel<BF16, VEC, 2, false>, dim3(a.T), threads, 0, 1, st, a);
        case 4: return launch(rt, norm_kernel<BF16, VEC, 4, false>, dim3(a.T), threads, 0, 1, st, a);
        default: return launch(rt, norm_kernel<BF16, VEC, 8, false>, dim3(a.T), threads, 0, 1, st, a);
    }
}

constexpr int kNormMaxD = 512 * 8 * kVec;

// ------------------------------------------------------------------------------ gated activation
struct GatedArgs {
    const uint16_t* x;                  // [T][2 D]: gate, then up
    uint8_t* q;
    float* scales;
    long long ldx, ldq, lds;
    int D, chunks;                      // chunks: CTAs per row
    int blocks, groups;                 // short rows: blocks of 128 per row, and in all
};

constexpr int kGatedVecs = 256;         // vectors of each half that a CTA takes: 2048 columns of one row

// VPT vectors of each half per thread, all loaded before the first is used. SHORT: each sixteen lanes take the
// next block of 128, of whichever row, so that rows shorter than a CTA's columns leave no lanes idle.
template <bool BF16, bool VEC, int VPT, bool SHORT>
__global__ void __launch_bounds__(kGatedVecs / VPT) gated_kernel(const GatedArgs a) {
    constexpr int kThreads = kGatedVecs / VPT;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int D = a.D;
    long long t[VPT];
    int col[VPT];
    Raw8<VEC> rg[VPT], ru[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (SHORT) {
            const unsigned g = (blockIdx.x * VPT + i) * (kThreads / 16u) + threadIdx.x / 16u;
            const unsigned r = g / static_cast<unsigned>(a.blocks);
            t[i] = r;
            col[i] = (g - r * a.blocks) * kRowBlock + threadIdx.x % 16 * kVec;
            if (g >= static_cast<unsigned>(a.groups)) t[i] = 0, col[i] = a.blocks * kRowBlock;   // (past every row's end)
        } else {
            t[i] = blockIdx.x / a.chunks;
            col[i] = ((blockIdx.x % a.chunks) * kGatedVecs + i * kThreads + threadIdx.x) * kVec;
        }
        const uint16_t* row = a.x + t[i] * a.ldx;
        rg[i] = begin8<VEC>(row, col[i], D);
        ru[i] = begin8<VEC>(row + D, col[i], D);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const uint16_t* row = a.x + t[i] * a.ldx;
        float g[kVec], u[kVec];
        end8<BF16, VEC>(rg[i], row, col[i], D, g);
        end8<BF16, VEC>(ru[i], row + D, col[i], D, u);
        // silu(g) = g / (1 + exp(-g)); where exp(-g) is beyond 2^126 (g < -87.3) the quotient is taken for its limit, 0
        float e[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) e[j] = rcp(-1.f - __expf(-g[j]));
        mul8(g, e);                                  // (-silu(g); before u: g u may overflow where silu(g) u does not)
        mul8(g, u);
        quantise8<VEC>(g, col[i], D, a.q + t[i] * a.ldq, a.scales + (col[i] / kRowBlock) * a.lds + t[i]);
    }
}

// Rows shorter than a CTA's columns share CTAs (16384 x 128 bf16: 3.3 us, a CTA per row 21.9; 4096 x 1408:
// 7.0 against 8.1), and so do rows off 16-byte boundaries while a row's last CTA can be a good part of it
// (2000 x 4101: 11.5 against 13.7; 4096 x 14335: 66.7 against 63.7). Otherwise, with more CTAs than the
// SMs hold at once, 64 threads with four vectors each keep more loads under way (4096 x 14336 bf16:
// 44.8 us; 128 with two 50.3, 256 with one 52.4); with fewer, one vector each is sooner done
// (16 x 14336: 1.4 us against 1.6 with two).
template <bool BF16, bool VEC>
int go_gated(const Runtime& rt, const GatedArgs& a, int T, wq4_stream_t st) {
    const long long ctas = static_cast<long long>(T) * a.chunks, groups = static_cast<long long>(T) * a.blocks;
    constexpr int kPerCta = kGatedVecs * kVec / kRowBlock;
    if (a.blocks < (VEC ? 1 : 4) * kPerCta && groups < (1LL << 31) - kPerCta) {
        GatedArgs s = a;
        s.groups = static_cast<int>(groups);
        const dim3 grid(static_cast<unsigned>((groups + kPerCta - 1) / kPerCta));
        return launch(rt, gated_kernel<BF16, VEC, 1, true>, grid, kGatedVecs, 0, 1, st, s);
    }
    if (ctas > 8LL * rt.sm_count)
        return launch(rt, gated_kernel<BF16, VEC, 4, false>, dim3(static_cast<unsigned>(ctas)), kGatedVecs / 4, 0, 1, st, a);
    return launch(rt, gated_kernel<BF16, VEC, 1, false>, dim3(static_cast<unsigned>(ctas)), kGatedVecs, 0, 1, st, a);
}

// The quantised rows an operator writes and the product reads: rows of codes on 16-byte boundaries,
// a scale row per block of 128, also on 16-byte boundaries (both are copied as tensors).
int check_rows(const void* Q, long long ldq, const void* scales, long long lds, int T, int D) {
    if (!Q || !scales || ldq < D || lds < T) return WQ4_ERR_INVALID;
    if (!aligned_to(Q, 16) || !aligned_to(scales, 16) || ldq % 16 || lds % 4) return WQ4_ERR_ALIGN;
    return WQ4_OK;
}

bool vec_ok(const void* p, long long ld) { return !p || (aligned_to(p, 16) && ld % kVec == 0); }

}  // namespace
}  // namespace wq4

using namespace wq4;

extern "C" {

int wq4_add_rmsnorm_quant(const void* X, long long ldx, const void* R, long long ldr, const void* weight, int T, int D,
                          float eps, int dtype, void* R_out, long long ldro, void* Y, long long ldy, void* Q,
                          long long ldq, float* scales, long long lds, wq4_stream_t stream) {
    if (T < 0 || D < 1 || (dtype != WQ4_BF16 && dtype != WQ4_FP16) || !(eps >= 0.f) || std::isinf(eps))
        return WQ4_ERR_INVALID;
    if (D > kNormMaxD) return WQ4_ERR_UNSUPPORTED;
    if (T == 0) return WQ4_OK;
    if (!X || !weight || (R_out && !R) || (!Y && !Q) || (!Q != !scales)) return WQ4_ERR_INVALID;
    if (ldx < D || (R && ldr < D) || (R_out && ldro < D) || (Y && ldy < D)) return WQ4_ERR_INVALID;
    if (!aligned_to(X, 2) || !aligned_to(R, 2) || !aligned_to(weight, 2) || !aligned_to(R_out, 2) || !aligned_to(Y, 2))
        return WQ4_ERR_ALIGN;
    if (Q)
        if (const int rc = check_rows(Q, ldq, scales, lds, T, D)) return rc;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    const NormArgs a{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(R),
                     static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(R_out), static_cast<uint16_t*>(Y),
                     static_cast<uint8_t*>(Q), scales, ldx, ldr, ldro, ldy, ldq, lds, T, D, eps, 1.f / static_cast<float>(D)};
    const bool vec = D % kVec == 0 && vec_ok(X, ldx) && vec_ok(R, ldr) && vec_ok(weight, 0) && vec_ok(R_out, ldro) &&
                     vec_ok(Y, ldy);
    if (dtype == WQ4_BF16) return vec ? go_norm<true, true>(rt, a, stream) : go_norm<true, false>(rt, a, stream);
    return vec ? go_norm<false, true>(rt, a, stream) : go_norm<false, false>(rt, a, stream);
}

int wq4_silu_mul_quant(const void* X, long long ldx, int T, int D, int dtype, void* Q, long long ldq, float* scales,
                       long long lds, wq4_stream_t stream) {
    if (T < 0 || D < 1 || (dtype != WQ4_BF16 && dtype != WQ4_FP16)) return WQ4_ERR_INVALID;
    if (D > (1 << 24)) return WQ4_ERR_UNSUPPORTED;
    if (T == 0) return WQ4_OK;
    if (!X || ldx < 2LL * D) return WQ4_ERR_INVALID;
    if (!aligned_to(X, 2)) return WQ4_ERR_ALIGN;
    if (const int rc = check_rows(Q, ldq, scales, lds, T, D)) return rc;
    const int chunks = (D + kGatedVecs * kVec - 1) / (kGatedVecs * kVec);
    if (static_cast<long long>(T) * chunks > 0x7fffffffLL) return WQ4_ERR_UNSUPPORTED;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    const GatedArgs a{static_cast<const uint16_t*>(X), static_cast<uint8_t*>(Q), scales, ldx, ldq, lds, D, chunks,
                      (D + kRowBlock - 1) / kRowBlock, 0};
    const bool vec = D % kVec == 0 && vec_ok(X, ldx);
    if (dtype == WQ4_BF16) return vec ? go_gated<true, true>(rt, a, T, stream) : go_gated<true, false>(rt, a, T, stream);
    return vec ? go_gated<false, true>(rt, a, T, stream) : go_gated<false, false>(rt, a, T, stream);
}

}  // extern "C"
