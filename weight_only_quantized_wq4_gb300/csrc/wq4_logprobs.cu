// Log probabilities of given tokens, the entropy of each row and its most likely tokens, in one pass
// over the logits.
//
// For a row x of V logits, with m = max x, t_i = (x_i - m) log2(e), z = sum 2^t_i, s = sum t_i 2^t_i:
//     log p_i = x_i - m - ln z            H = -sum p_i log p_i = ln z - ln(2) s / z
// The pass keeps (m, z, s) of what a thread has seen, in fp32; when its m grows by D / log2(e), z and s
// become 2^-D z and 2^-D (s - D z), and parts are joined by the same rule. What limits the pass is
// instructions per logit (at the rate of HBM an SM sees 12 bf16 logits a cycle, and has 4 issue slots of
// 32 lanes), so two logits share each packed operation:
//   clamp  a 16-bit maximum with a large negative number: -inf (and the type's lowest value) then
//          add 0 and not 0 * inf; NaN passes and makes the row NaN
//   t      one packed fp32 FMA, x log2(e) - R with R = m log2(e) rounded. Every term is then 2^r too large,
//          r = m log2(e) - R: z and s are moved from one m to the next with the change of r, and the last r is
//          taken out once per thread at the end
//   2^t    one exponential each; then one packed addition and one packed FMA
// Where |m| is so large that r would be (beyond 2^20; half an ulp of R is below 2^-4 up to there), or m is near
// the clamp (fp16), a thread subtracts and multiplies instead.
//
// The k most likely tokens need no second pass over the row. A thread remembers the largest vector
// it saw (its maximum and where, the first among equals). 64 groups of threads make 64 such bests (a
// group's threads are 64 apart, so that logits next to one another fall to different groups); the
// k-th largest of them, tau, is a bound that at least k elements reach, so only threads whose own
// best reaches it can hold an answer, about k of them. Their vectors (a 512th, 256th or 128th of the row each,
// by the CTA's threads) are read again by whole warps; the elements that reach tau, a few dozen, are ranked by counting. An
// element's order is one 64-bit key: the float as an unsigned integer of the same order, then the
// complement of its index, so that equal logits rank by the lower index and no two keys are equal.
//
// Bound by the latency of loads for many rows (each logit is read once; an SM holds 1024 threads, half of what it
// could, issues in 54 % of its cycles and waits for loads most): 2048 x 131072 bf16 109 us (4.9 TB/s), of which the
// steps after the pass, some 850 instructions a warp, are a tenth: a CTA loads nothing meanwhile. For few
// rows a cluster of CTAs shares a row; each sends its statistics and list to the first through
// distributed shared memory. That is a chain of latencies: 1 x 131072 fp32 6.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "wq4_device.cuh"
#include "wq4_runtime.h"

namespace wq4 {
namespace {

constexpr int kLpThreads = 512;               // of a CTA (128 or 256 where there are many rows)
constexpr int kLpGroups = 64;                 // bests that bound the k-th largest
constexpr int kLpMaxTop = 32;
constexpr int kLpMaxCluster = 8;
constexpr int kLpUnroll = 4;                  // vectors of a thread in flight
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFar = 150.f;                 // exp(-150) is below the smallest fp32
constexpr float kNegInf = -INFINITY;
constexpr float kFine = 1048576.f;            // 2^20: up to here m log2(e) in fp32 is within 2^-4

static_assert(kLpMaxCluster * kLpMaxTop <= kLpThreads / 2, "two threads to a key");

enum : int { kLpBf16 = 0, kLpFp16 = 1, kLpFp32 = 2 };   // the header's dtype codes

struct LpArgs {
    const void* logits;
    const long long* tokens;                  // null where not asked for, like the outputs
    float *logprobs, *entropy, *top_logprobs;
    int* top_ids;
    long long ld;
    int V, k, cluster;
    unsigned int* status;
    long long timeout_cycles;
    int test_stall;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// One 16-byte vector of logits: kN of them, the maximum that passes NaN over, and element j as fp32.
template <int DT>
struct LpVec {
    static constexpr int kN = DT == kLpFp32 ? 4 : 8;
    static constexpr int kSize = 16 / kN;
    __device__ static float at(const uint4& v, int j) {
        const uint32_t w = DT == kLpFp32 ? (j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w)
                                         : (j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w);
        if constexpr (DT == kLpFp32) return __uint_as_float(w);
        else if constexpr (DT == kLpBf16) return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
        else return __half2float(__ushort_as_half(static_cast<uint16_t>(j & 1 ? w >> 16 : w & 0xffffu)));
    }
    __device__ static float max(const uint4& v) {
        if constexpr (DT == kLpFp32) {
            return fmaxf(fmaxf(at(v, 0), at(v, 1)), fmaxf(at(v, 2), at(v, 3)));
        } else {
            uint32_t a, b, c;
            if constexpr (DT == kLpBf16) {
                asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
                asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
                asm("max.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
            } else {
                asm("max.f16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
                asm("max.f16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
                asm("max.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
            }
            const uint4 p = make_uint4(c, 0, 0, 0);
            return fmaxf(at(p, 0), at(p, 1));
        }
    }
    // all elements -inf
    __device__ static uint4 none() {
        const uint32_t w = DT == kLpFp32 ? 0xff800000u : DT == kLpBf16 ? 0xff80ff80u : 0xfc00fc00u;
        return make_uint4(w, w, w, w);
    }
};

// The order of the floats as unsigned integers (+0 and -0 alike; x is not NaN), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned long long key_of(float x, int index) {
    return (static_cast<unsigned long long>(order_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(index));
}

// A row cut into 16-byte vectors on 16-byte boundaries: vector v holds elements v kN - head + j; the
// first and the last may be partly outside the row, and what is outside is not read.
template <int DT>
struct LpRow {
    const char* base;       // vector 0 (its address may lie before the row's first element)
    int head, V, nv;
    __device__ LpRow(const void* logits, long long ld, long long t, int V_) : V(V_) {
        const char* p = static_cast<const char*>(logits) + t * ld * LpVec<DT>::kSize;
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
        head = off / LpVec<DT>::kSize;
        base = p - off;
        nv = (V + head + LpVec<DT>::kN - 1) / LpVec<DT>::kN;
    }
    __device__ bool whole(int v) const { return v * LpVec<DT>::kN >= head && (v + 1) * LpVec<DT>::kN <= V + head; }
    __device__ uint4 load(int v) const { return reinterpret_cast<const uint4*>(base)[v]; }
    __device__ uint4 load_edge(int v) const {
        if (whole(v)) return load(v);
        uint4 r = LpVec<DT>::none();
        uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < LpVec<DT>::kN; ++j) {
            const int i = v * LpVec<DT>::kN - head + j;
            if (i < 0 || i >= V) continue;
            if constexpr (DT == kLpFp32) {
                w[j] = reinterpret_cast<const uint32_t*>(base)[v * 4 + j];
            } else {
                const uint32_t b = reinterpret_cast<const uint16_t*>(base)[v * 8 + j];
                w[j >> 1] = j & 1 ? (w[j >> 1] & 0xffffu) | (b << 16) : (w[j >> 1] & 0xffff0000u) | b;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two logits of word w of a vector (fp32: of words w and w + 1), at least the clamp.
template <int DT>
__device__ __forceinline__ uint64_t clamped_pair(const uint32_t (&u)[4], int i) {
    if constexpr (DT == kLpFp32) {
        return pair(max_nan(__uint_as_float(u[2 * i]), -1e30f), max_nan(__uint_as_float(u[2 * i + 1]), -1e30f));
    } else if constexpr (DT == kLpBf16) {
        uint32_t w;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(u[i]), "r"(0xf149f149u));       // -1e30
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        uint32_t w;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(w) : "r"(u[i]), "r"(0xfbfffbffu));        // -65504
        return pair(__half2float(__ushort_as_half(static_cast<uint16_t>(w & 0xffffu))),
                    __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16))));
    }
}

// Softmax statistics of a set of logits; m = -inf: nothing but -inf (and NaN) so far.
struct LpStat {
    float m, z, s;
    // to a reference n >= m; dr: how much larger n's r is than m's
    __device__ void move(float n, float dr = 0.f) {
        if (n > m) {
            const float d = fmaf(fmaxf(m - n, -kFar), kLog2e, dr);     // (m = -inf: z and s are 0, or NaN)
            const float f = ex2(d);
            s = f * fmaf(d, z, s);
            z = f * z;
            m = n;
        }
    }
};

// A thread's statistics as the pass builds them: even and odd elements' sums apart.
template <int DT>
struct LpAcc {
    float m = kNegInf;
    uint64_t z = 0, s = 0;
    // whether R = m log2(e) is too coarse for a reference, or (fp16) m is not well above the clamp
    __device__ bool slow() const {
        if constexpr (DT == kLpFp16) return (m < -6e4f && m != kNegInf) || m == INFINITY;
        else return fabsf(m) > kFine && m != kNegInf;
    }
    __device__ float ref() const { return m == kNegInf ? 0.f : m * kLog2e; }
    // r, by which the exponents of the terms so far are too large
    __device__ float rest() const { return m == kNegInf || slow() ? 0.f : fmaf(m, kLog2e, -ref()); }
    __device__ void move(float n) {
        float z0, z1, s0, s1;
        unpair(z, z0, z1);
        unpair(s, s0, s1);
        LpStat a{m, z0, s0}, b{m, z1, s1};
        const float r = rest();
        m = n;
        const float dr = rest() - r;
        a.move(n, dr);
        b.move(n, dr);
        z = pair(a.z, b.z);
        s = pair(a.s, b.s);
    }
    __device__ void add_slow(const uint4& v) {
        float z0, z1, s0, s1;
        unpair(z, z0, z1);
        unpair(s, s0, s1);
#pragma unroll
        for (int j = 0; j < LpVec<DT>::kN; ++j) {
            const float t = max_nan(LpVec<DT>::at(v, j) - m, -kFar) * kLog2e, e = ex2(t);
            z0 += e;
            s0 = fmaf(t, e, s0);
        }
        z = pair(z0, z1);
        s = pair(s0, s1);
    }
    // vectors that m already covers
    template <int U>
    __device__ void add(const uint4 (&v)[U]) {
        if (slow()) {
#pragma unroll
            for (int u = 0; u < U; ++u) add_slow(v[u]);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) add_fast(v[u]);
        }
    }
    __device__ void add_fast(const uint4& v) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        const uint64_t minus_r = pair(-ref(), -ref()), l2e = pair(kLog2e, kLog2e);
#pragma unroll
        for (int i = 0; i < LpVec<DT>::kN / 2; ++i) {
            const uint64_t t = fma2(clamped_pair<DT>(u, i), l2e, minus_r);
            float t0, t1;
            unpair(t, t0, t1);
            const uint64_t e = pair(ex2(t0), ex2(t1));
            z = add2(z, e);
            s = fma2(t, e, s);
        }
    }
    // The whole, with m itself as the reference: t was r too large.
    __device__ LpStat done() const {
        float z0, z1, s0, s1;
        unpair(z, z0, z1);
        unpair(s, s0, s1);
        const float r = rest(), f = ex2(-r), zz = (z0 + z1) * f;
        return LpStat{m, zz, fmaf(-r, zz, (s0 + s1) * f)};
    }
};

// To shared memory of a CTA of the cluster; the bytes count on that CTA's barrier.
__device__ __forceinline__ void st_async(uint32_t addr, unsigned long long v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(addr), "l"(v), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_async(uint32_t addr, const LpStat& v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.s)), "r"(0), "r"(bar)
                 : "memory");
}

template <int THREADS>
struct LpShared {
    float2 stat[THREADS / 32];                       // warps' z and s, with the CTA's m
    LpStat total;
    unsigned long long best[kLpGroups];
    int above[kLpGroups];                            // bests above each
    int n, flagged;
    uint16_t flag[THREADS];                          // threads whose best reaches tau
    static constexpr int kCand = THREADS < 256 ? 256 : THREADS;
    unsigned long long cand[kCand];                // its room is an ordered list of every warp's
    int rank[kLpMaxCluster * kLpMaxTop];             // of the clusters' lists
    // what rank 0 is sent by the cluster's CTAs: their statistics and their lists
    float4 part_stat[kLpMaxCluster];
    unsigned long long part_top[kLpMaxCluster * kLpMaxTop];
    unsigned long long part_bar, stall_bar;
    int abort;
    unsigned long long top[kLpMaxTop];               // this CTA's best, in order, 0 where there are fewer
};

// THREADS: of a CTA, which takes a row or, in a cluster (of kLpThreads only), a part of one.
template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprobs_kernel(const LpArgs a) {
    using Vec = LpVec<DT>;
    constexpr int kWarps = THREADS / 32, kParts = THREADS / kLpGroups;
    __shared__ LpShared<THREADS> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = THREADS == kLpThreads ? a.cluster : 1, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const long long t = C > 1 ? blockIdx.x / C : blockIdx.x;
    if (C > 1) {
        if (tid == 0) {
            mbar_init(smem_u32(&sh.part_bar), 1);
            mbar_init(smem_u32(&sh.stall_bar), 1);
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.part_bar), C * (16 + 8 * a.k));
            sh.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        cluster_sync();                              // rank 0's barrier is set up before anything is sent to it
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const LpRow<DT> row(a.logits, a.ld, t, a.V);
    const int v0 = C > 1 ? static_cast<int>(static_cast<long long>(row.nv) * rank / C) : 0;
    const int v1 = C > 1 ? static_cast<int>(static_cast<long long>(row.nv) * (rank + 1) / C) : row.nv;

    // the asked token's logit, on its way while the row is read (NaN: no such token)
    float asked = NAN;
    if (tid == 64 && rank == 0 && a.logprobs) {
        const long long id = a.tokens[t];
        if (id >= 0 && id < a.V) {
            const char* p = static_cast<const char*>(a.logits) + (t * a.ld + id) * Vec::kSize;
            const uint32_t u = DT == kLpFp32 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
            asked = Vec::at(make_uint4(u, 0, 0, 0), 0);
        }
    }
    LpAcc<DT> acc;
    int bv = -1;                                     // the vector of this thread's maximum, acc.m
    int v = v0 + tid;
    // the row's first and last vector, where they are partly outside it, are taken at the end
    const bool head = v == 0 && v < v1 && !row.whole(0);
    if (head) v += THREADS;
    const int last = v1 == row.nv && !row.whole(v1 - 1) ? v1 - 1 : v1;   // whole vectors end here
    uint4 x[kLpUnroll];
    bool more = v + (kLpUnroll - 1) * THREADS < last;
    if (more)
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) x[u] = row.load(v + u * THREADS);
    // vectors from `at` on; the thread's maximum is its first of equal ones
    auto take = [&](const auto& y, int at) {
        constexpr int kY = sizeof(y) / sizeof(uint4);
        float n = acc.m;
#pragma unroll
        for (int u = 0; u < kY; ++u) {
            const float vm = Vec::max(y[u]);
            if (vm > n) {
                n = vm;
                bv = at + u * THREADS;
            }
        }
        if (n > acc.m) acc.move(n);
        acc.add(y);
    };
    while (more) {
        uint4 y[kLpUnroll];
        const int at = v;
        v += kLpUnroll * THREADS;
        more = v + (kLpUnroll - 1) * THREADS < last;
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) y[u] = x[u];
        if (more)                                    // the next batch is on its way while this one is added in
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) x[u] = row.load(v + u * THREADS);
        take(y, at);
    }
    // What is left, fewer whole vectors than a batch and the edges, on its way together as well.
    const bool tail = last < v1 && tid == (last - v0) % THREADS && !(head && last == 0);
    if (v < last || head || tail) {
        uint4 y[kLpUnroll - 1], one[1], e[1];
        const bool some = v + THREADS < last;        // (most short rows leave one)
        if (some) {
#pragma unroll
            for (int u = 0; u < kLpUnroll - 1; ++u) y[u] = v + u * THREADS < last ? row.load(v + u * THREADS) : Vec::none();
        } else if (v < last) {
            one[0] = row.load(v);
        }
        if (head || tail) e[0] = row.load_edge(head ? 0 : last);
        if (some) take(y, v);
        else if (v < last) take(one, v);
        if (head) {                                  // (before the others in the row: it wins among equals)
            const float n = Vec::max(e[0]);
            if (n >= acc.m && n > kNegInf) bv = 0;
            if (n > acc.m) acc.move(n);
            acc.add(e);
            if (tail) e[0] = row.load_edge(last);
        }
        if (tail) take(e, last);
    }
    // this thread's best as a bound for elements: its value and its vector's last index
    const unsigned long long best =
        bv < 0 ? 0ull : key_of(acc.m, min(bv * Vec::kN + Vec::kN - 1 - row.head, a.V - 1));
    sh.cand[tid] = best;
    if (tid == 0) {
        sh.n = 0;
        sh.flagged = 0;
    }
    if (tid < kLpMaxTop) sh.top[tid] = 0;
    __syncthreads();
    if (tid < kLpGroups) {                           // a group's threads are kLpGroups apart
        unsigned long long g = sh.cand[tid];
#pragma unroll
        for (int i = 1; i < kParts; ++i) g = max(g, sh.cand[tid + i * kLpGroups]);
        sh.best[tid] = g;
        sh.above[tid] = 0;
    }
    __syncthreads();

    // ---- the CTA's m, every thread's sums with it, and tau
    const uint32_t top_order = __reduce_max_sync(
        0xffffffffu, max(static_cast<uint32_t>(sh.best[lane] >> 32), static_cast<uint32_t>(sh.best[lane + 32] >> 32)));
    LpStat st = acc.done();
    const float m = top_order ? value_of(top_order) : kNegInf;
    st.move(m);
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        st.z += __shfl_xor_sync(0xffffffffu, st.z, d);
        st.s += __shfl_xor_sync(0xffffffffu, st.s, d);
    }
    if (lane == 0) sh.stat[warp] = make_float2(st.z, st.s);
    if (a.k > 0) {                                   // how many bests are above each: a kParts-th of them per thread
        const unsigned long long mine = sh.best[tid % kLpGroups];
        int above = 0;
#pragma unroll
        for (int i = 0; i < kLpGroups / kParts; ++i)
            above += sh.best[tid / kLpGroups * (kLpGroups / kParts) + i] > mine ? 1 : 0;
        if (above) atomicAdd(&sh.above[tid % kLpGroups], above);
    }
    __syncthreads();
    if (warp == kWarps - 1) {
        float2 w = lane < kWarps ? sh.stat[lane] : make_float2(0.f, 0.f);
#pragma unroll
        for (int d = kWarps / 2; d; d >>= 1) {
            w.x += __shfl_xor_sync(0xffffffffu, w.x, d);
            w.y += __shfl_xor_sync(0xffffffffu, w.y, d);
        }
        if (lane == 0) sh.total = LpStat{m, w.x, w.y};
    }

    // ---- the CTA's k best: the flagged threads' vectors once more
    if (a.k > 0) {
        // tau: the best with k - 1 above it (none, so 0, where fewer than k groups have one)
        const unsigned long long b0 = sh.above[lane] == a.k - 1 ? sh.best[lane] : 0,
                                 b1 = sh.above[lane + 32] == a.k - 1 ? sh.best[lane + 32] : 0;
        const unsigned int h0 = __ballot_sync(0xffffffffu, b0 != 0), h1 = __ballot_sync(0xffffffffu, b1 != 0);
        const unsigned long long tau = h0   ? __shfl_sync(0xffffffffu, b0, __ffs(h0) - 1)
                                       : h1 ? __shfl_sync(0xffffffffu, b1, __ffs(h1) - 1)
                                            : 0;
        const unsigned int mine = __ballot_sync(0xffffffffu, best != 0 && best >= tau);
        if (mine) {
            int at = 0;
            if (lane == 0) at = atomicAdd(&sh.flagged, __popc(mine));
            at = __shfl_sync(0xffffffffu, at, 0);
            if (mine >> lane & 1) sh.flag[at + __popc(mine & ((1u << lane) - 1))] = static_cast<uint16_t>(tid);
        }
        __syncthreads();
        const uint32_t tau_order = static_cast<uint32_t>(tau >> 32);
        // The flagged threads' vectors, dealt out over the warps in units of 32: a thread has `per`, and as many
        // threads as fit share a unit. A warp's loads are under way together, kUnits at a time.
        const int per = (v1 - v0 + THREADS - 1) / THREADS;
        const int shift = per <= 1 ? 0 : per >= 32 ? 5 : 32 - __clz(per - 1);
        const int rounds = (per + 31) >> 5, flagged = sh.flagged;
        const int units = (flagged << shift) + 31 >> 5;
        constexpr int kUnits = 4;
        auto second_look = [&](auto&& offer) {
            for (int r = 0; r < rounds; ++r) {
                for (int u0 = warp; u0 < units; u0 += kUnits * kWarps) {
                    uint4 y[kUnits];
                    int w[kUnits];
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) {
                        const int slot = (u0 + i * kWarps) * 32 + lane;     // of the flagged threads' vectors
                        const int who = slot >> shift;
                        w[i] = who < flagged ? v0 + sh.flag[who] + (r * 32 + (slot & ((1 << shift) - 1))) * THREADS : v1;
                        y[i] = w[i] < v1 ? row.load_edge(w[i]) : Vec::none();
                    }
#pragma unroll
                    for (int i = 0; i < kUnits; ++i)
                        if (u0 + i * kWarps < units) offer(y[i], w[i]);
                }
            }
        };
        // A vector per lane, vector index w: what reaches tau is noted, a few dozen elements in all.
        const unsigned long long floor0 = tau ? tau - 1 : 0;     // what an element has to be above
        second_look([&](const uint4& x, int w) {
            const float most = Vec::max(x);
            if (most > kNegInf && order_of(most) >= tau_order) {
#pragma unroll
                for (int j = 0; j < Vec::kN; ++j) {
                    const float f = Vec::at(x, j);
                    const unsigned long long key = f > kNegInf ? key_of(f, w * Vec::kN - row.head + j) : 0ull;
                    if (key > floor0) {
                        const int at = atomicAdd(&sh.n, 1);
                        if (at < sh.kCand) sh.cand[at] = key;
                    }
                }
            }
        });
        __syncthreads();
        if (sh.n > sh.kCand) {                       // (the same for every thread)
            __syncthreads();
            if (tid == 0) sh.n = 0;
            __syncthreads();
            unsigned long long list = 0;                 // lane i: the warp's i-th best so far
            unsigned long long floor = floor0;
            // More than fit (equal or steadily larger logits in one thread's share): each warp keeps the best k of
            // what it sees in order, one per lane; the elements of a vector that reaches tau go one to a lane.
            auto keep = [&](const uint4& x, int w) {
                const float most = Vec::max(x);
                unsigned int hit = __ballot_sync(0xffffffffu, most > kNegInf && order_of(most) >= tau_order);
                while (hit) {
                    const int from = __ffs(hit) - 1;
                    hit &= hit - 1;
                    const uint32_t u0 = __shfl_sync(0xffffffffu, x.x, from), u1 = __shfl_sync(0xffffffffu, x.y, from),
                                   u2 = __shfl_sync(0xffffffffu, x.z, from), u3 = __shfl_sync(0xffffffffu, x.w, from);
                    const int at_w = __shfl_sync(0xffffffffu, w, from);
                    const int j = lane & (Vec::kN - 1), word = DT == kLpFp32 ? j : j >> 1;
                    const uint32_t u = word == 0 ? u0 : word == 1 ? u1 : word == 2 ? u2 : u3;
                    // (its logit in the low half: element 0 of a vector of it)
                    const float f = Vec::at(make_uint4(DT != kLpFp32 && (j & 1) ? u >> 16 : u, 0, 0, 0), 0);
                    const unsigned long long key =
                        lane < Vec::kN && f > kNegInf ? key_of(f, at_w * Vec::kN - row.head + j) : 0ull;
                    unsigned int in = __ballot_sync(0xffffffffu, key > floor);
                    while (in) {
                        const unsigned long long c = __shfl_sync(0xffffffffu, key, __ffs(in) - 1);
                        in &= in - 1;
                        if (c <= floor) continue;
                        const int at = __popc(__ballot_sync(0xffffffffu, list > c));
                        const unsigned long long up = __shfl_up_sync(0xffffffffu, list, 1);
                        if (lane == at) list = c;
                        else if (lane > at) list = up;
                        const unsigned long long kth = __shfl_sync(0xffffffffu, list, a.k - 1);
                        if (kth > floor) floor = kth;
                    }
                }
            };
            second_look(keep);
            const int have = min(__popc(__ballot_sync(0xffffffffu, list != 0)), a.k);
            if (have) {
                int at = 0;
                if (lane == 0) at = atomicAdd(&sh.n, have);
                at = __shfl_sync(0xffffffffu, at, 0);
                if (lane < have) sh.cand[at + lane] = list;
            }
            __syncthreads();
        }
        const int n = sh.n;
        for (int at = tid; at < n; at += THREADS) {
            const unsigned long long mine = sh.cand[at];
            int above = 0;
#pragma unroll 8
            for (int i = 0; i < n; ++i) above += sh.cand[i] > mine ? 1 : 0;
            if (above < a.k) sh.top[above] = mine;
        }
    }
    __syncthreads();

    // ---- the row's, from its CTAs'
    if (C > 1) {
        // Every CTA sends rank 0 its statistics and its list (its own too) and is done; their bytes count on rank
        // 0's barrier.
        if (tid < 32) {
            const uint32_t bar = map_to_rank(smem_u32(&sh.part_bar), 0);
            if (tid < a.k) st_async(map_to_rank(smem_u32(&sh.part_top[rank * a.k + tid]), 0), sh.top[tid], bar);
            if (tid == 0) st_async(map_to_rank(smem_u32(&sh.part_stat[rank]), 0), sh.total, bar);
        }
        if (rank != 0) return;
        const WaitCtl ctl{&sh.abort, a.status, a.timeout_cycles};
        // one thread's answer holds for all
        if (tid == 0 && (!a.test_stall || mbar_wait(smem_u32(&sh.stall_bar), 0, ctl))) mbar_wait(smem_u32(&sh.part_bar), 0, ctl);
        __syncthreads();
        if (sh.abort) {                              // (not before what the others sent is here, and they are gone)
            if (tid == 0) mbar_wait_plain(smem_u32(&sh.part_bar), 0, drain_limit(a.timeout_cycles));
            __syncwarp();
            cluster_sync();
            return;
        }
        if (warp == 0) {
            const float4 x = lane < C ? sh.part_stat[lane] : make_float4(kNegInf, 0.f, 0.f, 0.f);
            LpStat w{x.x, x.y, x.z};
            float n = w.m;
#pragma unroll
            for (int d = kLpMaxCluster / 2; d; d >>= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
            w.move(n);
#pragma unroll
            for (int d = kLpMaxCluster / 2; d; d >>= 1) {
                w.z += __shfl_xor_sync(0xffffffffu, w.z, d);
                w.s += __shfl_xor_sync(0xffffffffu, w.s, d);
            }
            if (lane == 0) sh.total = LpStat{n, w.z, w.s};
        }
        for (int i = tid; i < C * kLpMaxTop; i += THREADS) sh.rank[i] = 0;
        if (tid < kLpMaxTop) sh.top[tid] = 0;
        __syncthreads();
        if (a.k > 0) {                               // ranked by counting, two threads to a key
            const int keys = C * a.k, i = tid & (THREADS / 2 - 1), from = tid < THREADS / 2 ? 0 : keys / 2;
            const int to = tid < THREADS / 2 ? keys / 2 : keys;
            const unsigned long long mine = i < keys ? sh.part_top[i] : 0;
            if (mine) {
                int above = 0;
#pragma unroll 8
                for (int q = from; q < to; ++q) above += sh.part_top[q] > mine ? 1 : 0;
                if (above) atomicAdd(&sh.rank[i], above);
            }
            __syncthreads();
            if (tid < keys && mine && sh.rank[tid] < a.k) sh.top[sh.rank[tid]] = mine;
        }
        __syncthreads();
    }

    const LpStat all = sh.total;
    const float logz = all.m == kNegInf ? 0.f : logf(all.z);   // z is NaN where the row holds a NaN
    const bool nothing = all.m == kNegInf && all.z == 0.f;
    auto logp = [&](float x) { return nothing ? kNegInf : (x == kNegInf ? x + 0.f * all.z : x - all.m) - logz; };
    if (tid < a.k) {
        const unsigned long long key = sh.top[tid];
        a.top_ids[t * a.k + tid] = key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
        a.top_logprobs[t * a.k + tid] = logp(key ? value_of(static_cast<uint32_t>(key >> 32)) : kNegInf);
    }
    if (tid == 32 && a.entropy) a.entropy[t] = nothing ? 0.f : logz - kLn2 * (all.s / all.z);
    if (tid == 64 && a.logprobs) a.logprobs[t] = asked == asked ? logp(asked) : asked;
}

template <int DT>
int go_logprobs(const Runtime& rt, const LpArgs& a, int threads, dim3 grid, wq4_stream_t st) {
    if (threads == 128) return launch(rt, logprobs_kernel<DT, 128>, grid, 128, 0, 1, st, a);
    if (threads == 256) return launch(rt, logprobs_kernel<DT, 256>, grid, 256, 0, 1, st, a);
    return launch(rt, logprobs_kernel<DT, kLpThreads>, grid, kLpThreads, 0, a.cluster, st, a);
}

}  // namespace
}  // namespace wq4

using namespace wq4;

extern "C" int wq4_token_logprobs(const void* logits, long long ld, const long long* tokens, int T, int V, int dtype,
                                  int top_k, float* logprobs, float* entropy, int* top_ids, float* top_logprobs,
                                  wq4_stream_t stream) {
    if (T < 0 || V < 1 || top_k < 0 || top_k > V) return WQ4_ERR_INVALID;
    if (dtype != WQ4_BF16 && dtype != WQ4_FP16 && dtype != WQ4_FP32) return WQ4_ERR_INVALID;
    if (top_k > kLpMaxTop || V > (1 << 30)) return WQ4_ERR_UNSUPPORTED;
    if (T == 0) return WQ4_OK;
    if (!logits || ld < V || !tokens != !logprobs) return WQ4_ERR_INVALID;
    if ((top_k > 0) != (top_ids != nullptr) || (top_k > 0) != (top_logprobs != nullptr)) return WQ4_ERR_INVALID;
    if (!logprobs && !entropy && top_k == 0) return WQ4_ERR_INVALID;
    if (!aligned_to(logits, dtype == WQ4_FP32 ? 4 : 2) || !aligned_to(tokens, 8) || !aligned_to(logprobs, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(top_ids, 4) || !aligned_to(top_logprobs, 4))
        return WQ4_ERR_ALIGN;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    // Few rows: a cluster per row, as long as the CTAs still fit the GPU twice over and a CTA's share
    // is a batch of loads for every thread.
    int C = 1;
    const int vec = dtype == WQ4_FP32 ? 4 : 8;
    while (C < kLpMaxCluster && 2LL * C * T <= 2LL * rt.sm_count && V / (2 * C) >= kLpThreads * vec) C *= 2;
    if (static_cast<long long>(T) * C > 0x7fffffffLL) return WQ4_ERR_UNSUPPORTED;
    const LpArgs a{logits, tokens, logprobs, entropy, top_logprobs, top_ids, ld, V, top_k, C, rt.status, rt.timeout_cycles,
                   rt.test_stall};
    const dim3 grid(static_cast<unsigned>(T) * C);
    // Many rows: fewer threads per row, so that more rows share what the steps after the pass cost each of them
    // (2048 x 8192 bf16, top 8: 14.7 us with 128 threads, 21.0 with 256, 38.3 with 512), unless the waves or the
    // length say otherwise (700 x 128256: 45.1 us with 512, 54.0 with 256, 61.2 with 128; 2048 x 131072:
    // 109, 116, 149). An SM holds 1024 threads; a wave takes as long as a thread needs for its share of
    // a row, and the steps after the pass are worth some 200 bytes of that. Fewer threads per row also
    // leave more of the last wave empty, as CTAs do not end together: an eighth, three eighths on top.
    int threads = kLpThreads;
    if (C == 1) {
        const long long bytes = static_cast<long long>(V) * (16 / vec);
        auto cost = [&](int th) {
            const long long at_once = static_cast<long long>(rt.sm_count) * (1024 / th);
            return (T + at_once - 1) / at_once * (200 + bytes * (th == 128 ? 11 : th == 256 ? 9 : 8) / (8 * th));
        };
        for (const int th : {256, 128})
            if (cost(th) < cost(threads)) threads = th;
    }
    return dtype == WQ4_BF16   ? go_logprobs<kLpBf16>(rt, a, threads, grid, stream)
           : dtype == WQ4_FP16 ? go_logprobs<kLpFp16>(rt, a, threads, grid, stream)
                               : go_logprobs<kLpFp32>(rt, a, threads, grid, stream);
}
