// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// A walk over a sequence's tree holds the weights w of the node it is at, w_i = exp(x_i - max x) of the scaled logits, and
// their sum z: p = w / z. A draft c is kept if u q(c) z < w_c. One that is not kept leaves w_i = max(w_i / z - q_i, 0), or
// w_c = 0 where drafts come without probabilities, with a new sum. The next token is the first whose running sum of
// w exceeds u z.
//
// A cluster of CTAs walks a sequence, each with its share of the vocabulary in shared memory: a row's logits as they lie in
// memory, which decide on a node's first draft unless it is near to its border, and, where it is or is not kept or there
// is none, the weights as fp32. So a row is read once however many children are tried. Each step ends with one exchange: every CTA
// tells the others its part of the sum and, if it has it, the weight of the draft that is tried next; all of them then come
// to the same decision. Decisions hang on sums over the whole vocabulary next to a random border, so sums are kept as a pair of
// floats (the rounding of each addition is carried along; some fifty of them leave 2^-37 of a sum at worst); the weights
// themselves are rounded as fp32 operations round them, one by one.
//
// Bound by the latency of these steps, one after another: a visited row costs a load, two or three barriers and one exchange across the
// cluster (about 5000 cycles with the row on its way ahead of time), the end of a walk a pass of exponentials, one over the draft's
// row and a search (some 20000). One chain of 5 over 32001 tokens, fp32: 17.3 us; 32 trees of 16 over 131072, bf16: 32; 192
// chains of 6: 108, 1.9 TB/s of the rows that are visited. Sums in 64-bit arithmetic took five times as long (650 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdio>

#include "wq4_cache.cuh"

namespace wq4 {
namespace {

constexpr int kMaxThreads = 512;        // of a CTA, with few sequences; 256 with many
constexpr int kMaxCluster = 8;
constexpr int kBlock = 1024;            // weights whose sums are held while the next token is searched
constexpr int kMaxShare = 50 * 1024;    // weights of a CTA: 200 KB
constexpr int kVerifyMaxV = 400000;

struct VerifyArgs {
    const void* logits;
    const long long* tokens;
    const int *parents, *starts;
    const float *draft_probs, *temperature, *uniforms, *final_uniforms;
    int *accepted, *path;
    long long* next_tokens;
    long long ld, ldp;
    int B, T, max_tokens, V, ld_path;
    int cluster, share;                 // CTAs of a sequence; weights of each, a multiple of kBlock
    int ahead;                          // whether there is room for the row ahead
    unsigned int* status;
};

// A sum and what its additions rounded off (D. E. Knuth, The art of computer programming 2, 4.2.2: the error of
// s = a + b is (a - (s - t)) + (b - t) with t = s - a, exactly).
struct Sum {
    float s, c;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(s, x), y = __fsub_rn(t, s);
        c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, y)), __fsub_rn(x, y)));
        s = t;
    }
    __device__ __forceinline__ void add(const Sum& o) {
        add(o.s);
        c = __fadd_rn(c, o.c);
    }
    // hi + lo with hi the sum rounded
    __device__ __forceinline__ Sum normal() const {
        const float hi = __fadd_rn(s, c);
        return Sum{hi, __fadd_rn(__fsub_rn(s, hi), c)};
    }
    __device__ __forceinline__ bool exceeds(const Sum& o) const {
        const Sum x = normal(), y = o.normal();
        return x.s > y.s || (x.s == y.s && x.c > y.c);
    }
};
// Two sums beside each other, two operations to an instruction.
struct Sum2 {
    uint64_t s = 0, c = 0;
    static __device__ __forceinline__ uint64_t plus(uint64_t a, uint64_t b) {
        uint64_t d;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
        return d;
    }
    static __device__ __forceinline__ uint64_t minus(uint64_t a, uint64_t b) {
        uint64_t d;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(b), "l"(0xbf800000bf800000ull), "l"(a));   // a - 1 b
        return d;
    }
    __device__ __forceinline__ void add(float x0, float x1) {
        uint64_t x;
        asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
        const uint64_t t = plus(s, x), y = minus(t, s);
        c = plus(c, plus(minus(s, minus(t, y)), minus(x, y)));
        s = t;
    }
    __device__ __forceinline__ Sum sum() const {
        Sum a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a.s), "=f"(b.s) : "l"(s));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a.c), "=f"(b.c) : "l"(c));
        a.add(b);
        return a;
    }
};
__device__ __forceinline__ Sum warp_sum(Sum x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        Sum o;
        o.s = __shfl_xor_sync(0xffffffffu, x.s, d);
        o.c = __shfl_xor_sync(0xffffffffu, x.c, d);
        x.add(o);
    }
    x.s = __shfl_sync(0xffffffffu, x.s, 0);          // (lanes may differ in the last bits, and all decide alike)
    x.c = __shfl_sync(0xffffffffu, x.c, 0);
    return x;
}
// 1 / x, rounded to nearest (but for ties within 2^-24 of a step): one step of Newton's method from the reciprocal of x.s.
__device__ __forceinline__ float reciprocal(const Sum& x) {
    const float hi = __fadd_rn(x.s, x.c), lo = __fadd_rn(__fsub_rn(x.s, hi), x.c), r = __frcp_rn(hi);
    return __fmaf_rn(r, __fmaf_rn(-lo, r, __fmaf_rn(-hi, r, 1.f)), r);
}

// What a CTA tells the others at the end of a step. Of a row's logits: its largest, the sum of exp against that (greedy: the
// largest one's place) and the logit of the draft that is tried, -inf where it is another CTA's. Of weights: their sum, as
// a pair, and the weight of the draft that is tried next, -1 where it is another CTA's, by the new weights and by the old.
struct Part {
    float a, b, c, d;
};

constexpr int kHeld = 128;              // drafts of a sequence whose parents, tokens and numbers are kept at hand

struct Shared {
    Part part[2][kMaxCluster];          // [turn][CTA]: written by the others
    float top[kMaxThreads / 32], sum[kMaxThreads / 32];
    int top_at;
    Sum block[kMaxShare / kBlock];
    long long tokens[kHeld];
    int parents[kHeld];
    float uniforms[kHeld];
};

__device__ __forceinline__ void st_cluster(uint32_t addr, const Part& p) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(p.a), "f"(p.b), "f"(p.c), "f"(p.d) : "memory");
}

// The kinds of logits: eight of them as they lie in memory, their values, and the larger of each, NaN where there is one.
template <int DT>
struct Kind {
    static constexpr int kSize = DT == WQ4_FP32 ? 4 : 2, kWords = DT == WQ4_FP32 ? 8 : 4;
    struct Eight {
        uint32_t u[kWords];
    };
    static __device__ __forceinline__ uint32_t minus_inf() { return DT == WQ4_FP32 ? 0xff800000u : DT == WQ4_BF16 ? 0xff80ff80u : 0xfc00fc00u; }
    // from column i of a row that holds n; aligned: its columns lie on 16-byte boundaries in eights
    static __device__ __forceinline__ Eight load(const void* p, int i, int n, bool aligned) {
        Eight e;
        if (aligned && i + 8 <= n) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + static_cast<long long>(i) * kSize);
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k) {
                const uint4 x = q[k];
                e.u[4 * k] = x.x, e.u[4 * k + 1] = x.y, e.u[4 * k + 2] = x.z, e.u[4 * k + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                e.u[k] = minus_inf();
                if constexpr (DT == WQ4_FP32) {
                    if (i + k < n) e.u[k] = static_cast<const uint32_t*>(p)[i + k];
                } else {
                    const uint16_t* q = static_cast<const uint16_t*>(p) + i + 2 * k;
                    if (i + 2 * k < n) e.u[k] = (e.u[k] & 0xffff0000u) | q[0];
                    if (i + 2 * k + 1 < n) e.u[k] = (e.u[k] & 0x0000ffffu) | static_cast<uint32_t>(q[1]) << 16;
                }
            }
        }
        return e;
    }
    // eight in a row in shared memory, filled to whole eights
    static __device__ __forceinline__ Eight held(const char* raw, int i) {
        Eight e;
        const uint4* q = reinterpret_cast<const uint4*>(raw + i * kSize);
#pragma unroll
        for (int k = 0; k < kWords / 4; ++k) {
            const uint4 x = q[k];
            e.u[4 * k] = x.x, e.u[4 * k + 1] = x.y, e.u[4 * k + 2] = x.z, e.u[4 * k + 3] = x.w;
        }
        return e;
    }
    static __device__ __forceinline__ void values(const Eight& e, float (&v)[8]) {
        if constexpr (DT == WQ4_FP32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(e.u[k]);
        } else {
            unpack8<DT == WQ4_BF16>(make_uint4(e.u[0], e.u[1], e.u[2], e.u[3]), v);
        }
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t d;
        if constexpr (DT == WQ4_FP32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else if constexpr (DT == WQ4_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // the largest in m, +inf for NaN
    static __device__ __forceinline__ float largest(uint32_t m) {
        float x;
        if constexpr (DT == WQ4_FP32) {
            x = __uint_as_float(m);
        } else {
            const float lo = to_f32<DT == WQ4_BF16>(m & 0xffffu), hi = to_f32<DT == WQ4_BF16>(m >> 16);
            x = isnan(lo) || isnan(hi) ? INFINITY : fmaxf(lo, hi);
        }
        return isnan(x) ? INFINITY : x;
    }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kMaxThreads ? 2 : 3) verify_kernel(const VerifyArgs a) {
    constexpr int kThreads = THREADS, kWarps = kThreads / 32;
    using K = Kind<DT>;
    // Two buffers of this CTA's logits as they lie in memory: of the node's row, and of the row the walk goes on with if it keeps the
    // node's first draft, which is on its way meanwhile. The weights come where both are (16 bits) or where the row is.
    extern __shared__ float4 buffers[];
    auto buffer = [&](int i) { return reinterpret_cast<char*>(buffers) + i * a.share * K::kSize; };
    int cur = 0;                                     // the node's row
    char* raw = buffer(0);
    float4* w4 = buffers;
    float* w = reinterpret_cast<float*>(buffers);
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.cluster, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0, b = blockIdx.x / C;
    const int v0 = rank * a.share, mine = max(0, min(a.share, a.V - v0));   // vocabulary [v0, v0 + mine)
    const int blocks = (mine + kBlock - 1) / kBlock;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s0 = a.starts[b], s1 = a.starts[b + 1];
    int n = static_cast<int>(static_cast<unsigned>(s1) - static_cast<unsigned>(s0));
    if (s0 < 0 || s1 < s0 || s1 > a.T || n > a.max_tokens) {
        if (tid == 0) atomicOr(a.status, kStatusBadIndex);
        n = 0;
    }
    if (tid < kHeld && tid < n) {
        sh.parents[tid] = a.parents[s0 + tid];
        sh.tokens[tid] = a.tokens[s0 + tid];
        sh.uniforms[tid] = a.uniforms[s0 + tid];
    }
    const float heat = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = heat == 0.f;
    const float inv_heat = greedy ? 1.f : __frcp_rn(heat);
    bool fine = n > 0 && heat >= 0.f && !isinf(heat);
    // (every CTA is there before anything is sent to it)
    if (C > 1) cluster_sync();
    else __syncthreads();
    int turn = 0;
    // Sends this CTA's part to all, waits for theirs.
    auto exchange = [&](const Part& p) {
        if (tid < C) {
            if (C > 1) st_cluster(map_to_rank(smem_u32(&sh.part[turn][rank]), tid), p);
            else sh.part[turn][0] = p;
        }
        __syncwarp();
        if (C > 1) cluster_sync();
        else __syncthreads();
        turn ^= 1;                                   // (a CTA may send its next part while another reads these)
        return turn ^ 1;
    };
    int* path = a.path + static_cast<long long>(b) * a.ld_path;
    int node = 0, kept = 0, j = 0;                   // j: the last draft tried
    // The next draft to try after j: a child of the node whose token exists.
    long long draft = -1;
    float draft_q = 1.f;
    auto next_draft = [&] {
        while (++j < n) {
            if ((j < kHeld ? sh.parents[j] : a.parents[s0 + j]) != node) continue;
            draft = j < kHeld ? sh.tokens[j] : a.tokens[s0 + j];
            if (draft >= 0 && draft < a.V) {
                if (a.draft_probs) draft_q = a.draft_probs[(s0 + node) * a.ldp + draft];
                return;
            }
        }
        draft = -1;
    };
    auto number = [&] { return j < kHeld ? sh.uniforms[j] : a.uniforms[s0 + j]; };
    // Whether the draft is kept, its weight and the weights' sum given. (The products are held as pairs too: what each rounds off is
    // what the fused operation finds.)
    auto keeps = [&](float weight, const Sum& sum) {
        const Sum z = sum.normal();
        const float u = number(), uq = __fmul_rn(u, draft_q), uq_off = __fmaf_rn(u, draft_q, -uq), x = __fmul_rn(uq, z.s);
        return Sum{weight, 0.f}.exceeds(Sum{x, __fmaf_rn(uq, z.s, -x) + (uq * z.c + uq_off * z.s)});
    };
    auto scaled = [&](int i) {                       // a logit
        float x;
        if constexpr (DT == WQ4_FP32) x = reinterpret_cast<const float*>(raw)[i];
        else x = to_f32<DT == WQ4_BF16>(reinterpret_cast<const uint16_t*>(raw)[i]);
        return __fmul_rn(x, inv_heat);
    };
    auto here = [&](long long t) { return t >= v0 && t < v0 + mine; };
    auto sum_blocks = [&] {                          // in warp 0
        Sum all{0.f, 0.f};
        if (warp == 0) {
            for (int k = lane; k < blocks; k += 32) all.add(sh.block[k]);
            all = warp_sum(all);
        }
        return all;
    };
    // f of each of the CTA's weights and of the same place of another row (null: 0): the sums of blocks of 1024 go to sh.block, f
    // itself, if it is to, into the weights' place. Returns the sum of all, in warp 0.
    auto weigh = [&](const float* other, bool write, auto f) {
        const bool vec = (reinterpret_cast<uintptr_t>(other) & 15u) == 0;
        for (int k = warp; k < blocks; k += kWarps) {
            Sum s{0.f, 0.f};
            Sum2 s2;
            const int from = k * kBlock + lane * 4;
            if (vec && k * kBlock + kBlock <= mine) {
                float4 o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = other ? *reinterpret_cast<const float4*>(other + from + 128 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = from + 128 * i;
                    float4 x = w4[at / 4];
                    x.x = f(at, x.x, o[i].x), x.y = f(at + 1, x.y, o[i].y), x.z = f(at + 2, x.z, o[i].z), x.w = f(at + 3, x.w, o[i].w);
                    if (write) w4[at / 4] = x;
                    s2.add(x.x, x.y), s2.add(x.z, x.w);
                }
                s = s2.sum();
            } else {
                for (int i0 = 0; i0 < kBlock; i0 += 256) {
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = k * kBlock + i0 + 32 * i + lane;
                        o[i] = other && at < mine ? other[at] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = k * kBlock + i0 + 32 * i + lane;
                        if (at < mine) {
                            const float x = f(at, w[at], o[i]);
                            if (write) w[at] = x;
                            s.add(x);
                        }
                    }
                }
            }
            s = warp_sum(s);
            if (lane == 0) sh.block[k] = s;
        }
        __syncthreads();
        return sum_blocks();
    };
    // The sum that the CTAs told, in every thread of the cluster to the same bits.
    auto sum_of = [&](int was) {
        Sum t{0.f, 0.f};
        if (lane < C) t = Sum{sh.part[was][lane].a, sh.part[was][lane].b};
        return warp_sum(t);
    };

    // The largest of the lanes' values, and the lowest place of it.
    auto largest = [&](float& x, int& at, int from) {
        for (int d = from; d; d >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, x, d);
            const int o_at = __shfl_xor_sync(0xffffffffu, at, d);
            if (o > x || (o == x && o_at < at)) at = o_at;
            x = fmaxf(x, o);
        }
    };
    // Brings this CTA's part of a row to a buffer: on its way when the call returns, there after arrived(). Returns false, with nothing
    // done, for the row ahead where it cannot be copied in words.
    bool ready = false;
    auto bring = [&](int i, int buf) {
        const char* const from = static_cast<const char*>(a.logits) + ((s0 + i) * a.ld + v0) * K::kSize;
        char* const to = buffer(buf);
        const bool aligned = (reinterpret_cast<uintptr_t>(from) & 15u) == 0;
        if (!aligned && K::kSize == 2 && buf != cur) return false;
        for (int c = tid * 8; c < a.share; c += kThreads * 8) {
            if ((aligned || K::kSize == 4) && c + 8 <= mine) {
                const uint32_t at = smem_u32(to + c * K::kSize);
                const char* const p = from + static_cast<long long>(c) * K::kSize;
                if (aligned) {
#pragma unroll
                    for (int k = 0; k < K::kSize / 2; ++k)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + 16 * k), "l"(p + 16 * k) : "memory");
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + 4 * k), "l"(p + 4 * k) : "memory");
                }
            } else {
                const typename K::Eight e = K::load(from, c, mine, aligned);
#pragma unroll
                for (int k = 0; k < K::kWords; k += 4)
                    *reinterpret_cast<uint4*>(to + c * K::kSize + 4 * k) = make_uint4(e.u[k], e.u[k + 1], e.u[k + 2], e.u[k + 3]);
            }
        }
        return true;
    };
    auto arrived = [&] {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    };
    float top = 0.f;
    int top_at = 0, was = 0;
    // a draft that was not kept: its row, 1 / sum of the weights it is taken from, its place among the CTA's
    const float* q_row = nullptr;
    float inv = 0.f;
    long long tried = -1;
    bool pending = false;                            // whether it is still to be taken
    float gone = 0.f;
    auto take_off = [&](int, float x, float q) { return fmaxf(__fsub_rn(__fmul_rn(x, inv), q), 0.f); };
    auto left = [&](int i) { return a.draft_probs ? take_off(i, w[i], q_row[i]) : w[i]; };
    auto block_sum = [&](int k) {                    // (a warp)
        Sum2 s2;
        for (int i = lane * 2; i < kBlock; i += 64) s2.add(w[k * kBlock + i], w[k * kBlock + i + 1]);
        return warp_sum(s2.sum());
    };
    while (fine) {
        // ---- the node's row: its logits, scaled, in shared memory; their maximum
        if (!ready) bring(node, cur);
        arrived();
        raw = buffer(cur);
        if constexpr (K::kSize == 4) w4 = reinterpret_cast<float4*>(raw), w = reinterpret_cast<float*>(raw);
        next_draft();
        ready = false;
        if (j < n && a.ahead) ready = bring(j, cur ^ 1);
        uint32_t most = K::minus_inf();
        for (int i = tid * 8; i < a.share; i += kThreads * 8) {
            const typename K::Eight e = K::held(raw, i);
#pragma unroll
            for (int c = 0; c < K::kWords; ++c) most = K::larger(most, e.u[c]);
        }
        float m_raw = K::largest(most);
#pragma unroll
        for (int d = 16; d; d >>= 1) m_raw = fmaxf(m_raw, __shfl_xor_sync(0xffffffffu, m_raw, d));
        if (lane == 0) sh.top[warp] = m_raw;
        if (tid == 0) sh.top_at = 0x7fffffff;
        __syncthreads();
        m_raw = sh.top[lane % kWarps];
#pragma unroll
        for (int d = kWarps / 2; d; d >>= 1) m_raw = fmaxf(m_raw, __shfl_xor_sync(0xffffffffu, m_raw, d));
        float m = __fmul_rn(m_raw, inv_heat);        // (rounding keeps the order)
        if (isnan(m)) m = INFINITY;
        if (greedy) {                                // its place
            for (int i = tid * 8; i < mine; i += kThreads * 8) {
                float x[8];
                K::values(K::held(raw, i), x);
#pragma unroll
                for (int c = 7; c >= 0; --c)
                    if (x[c] == m && i + c < mine) atomicMin(&sh.top_at, v0 + i + c);
            }
            __syncthreads();
        }
        // ---- their sum, against the CTA's maximum. It decides on the first draft where the draft is not near to its border.
        float s = 0.f;
        if (!greedy && j < n && !isinf(m)) {
            // (differences first: where x and the maximum are near, they are exact)
            const float to2 = 1.44269504f * inv_heat;
            float s2 = 0.f;
            for (int i = tid * 8; i < a.share; i += kThreads * 8) {
                float x[8];
                K::values(K::held(raw, i), x);
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    s += exp2_fast((x[c] - m_raw) * to2);
                    s2 += exp2_fast((x[c + 1] - m_raw) * to2);
                }
            }
            s += s2;
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane == 0) sh.sum[warp] = s;
            __syncthreads();
            s = sh.sum[lane % kWarps];
#pragma unroll
            for (int d = kWarps / 2; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        }
        was = exchange(Part{m, greedy ? __int_as_float(sh.top_at) : s, j < n && here(draft) ? scaled(static_cast<int>(draft - v0)) : -INFINITY, 0.f});
        const Part told = sh.part[was][lane & (C - 1)];
        float draft_x = told.c;
        top = told.a, top_at = __float_as_int(told.b);
        largest(top, top_at, kMaxCluster / 2);
#pragma unroll
        for (int d = kMaxCluster / 2; d; d >>= 1) draft_x = fmaxf(draft_x, __shfl_xor_sync(0xffffffffu, draft_x, d));
        if (isinf(top)) {                            // (either way; NaN as +inf)
            fine = false;
            break;
        }
        // ---- the first draft: by approximations, unless it lies as near to its border as they may be off: a hundred and some additions of
        // 2^-24 each, exponentials to 2^-22 with arguments to 2^-24 of up to 20 (smaller weights do not tell), and of the
        // logits that x / temperature is rounded to for the weights themselves. Then the weights decide: a sequence's
        // tokens do not hang on how many threads and CTAs the batch gives it.
        bool near = false;
        if (j < n) {
            float draft_w = draft == top_at ? 1.f : 0.f;
            bool keep = greedy && keeps(draft_w, Sum{1.f, 0.f});
            if (!greedy) {
                draft_w = expf(__fsub_rn(draft_x, top));
                float z = lane < C ? told.b * expf(__fsub_rn(told.a, top)) : 0.f;
#pragma unroll
                for (int d = kMaxCluster / 2; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
                z = __shfl_sync(0xffffffffu, z, 0);
                const float border = __fmul_rn(__fmul_rn(number(), draft_q), z);
                // (or there is no sum: 1.44 / temperature may overflow where 1 / temperature does not)
                near = !(fabsf(border - draft_w) > (0x1p-16f + 0x1p-21f * fabsf(top)) * fmaxf(border, draft_w));
                keep = !near && border < draft_w;
            }
            if (keep) {
                if (rank == 0 && tid == 0) path[kept] = j;
                ++kept;
                node = j;
                if (ready) cur ^= 1;
                __syncthreads();                     // (the logits, and sh.top, are written again)
                continue;
            }
        }
        // ---- the weights themselves, and their sum
        // (A round of blocks is read by all before it is written, and 16-bit logits in the second buffer are ahead of the weights
        // that replace them if the first round comes first, those in the first buffer if the last one does.)
        arrived();
        ready = false;
        const int rounds = (a.share / kBlock + kWarps - 1) / kWarps;
        for (int round = 0; round < rounds; ++round) {
            const int k = (cur ? round : rounds - 1 - round) * kWarps + warp;
            typename K::Eight e[4];
            if (k * kBlock < mine) {
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = K::held(raw, k * kBlock + (32 * i + lane) * 8);
            }
            __syncthreads();
            if (k * kBlock < mine) {
                Sum2 s2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = k * kBlock + (32 * i + lane) * 8;
                    float x[8];
                    K::values(e[i], x);
                    if (greedy) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) x[c] = v0 + at + c == top_at ? 1.f : 0.f;
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c) x[c] = expf(__fsub_rn(__fmul_rn(x[c], inv_heat), top));   // (rounded one by one)
                    }
#pragma unroll
                    for (int c = 0; c < 8; c += 2) s2.add(x[c], x[c + 1]);
                    w4[at / 4] = make_float4(x[0], x[1], x[2], x[3]);
                    w4[at / 4 + 1] = make_float4(x[4], x[5], x[6], x[7]);
                }
                const Sum s = warp_sum(s2.sum());
                if (lane == 0) sh.block[k] = s;
            }
            __syncthreads();
        }
        Sum all = sum_blocks();
        was = exchange(Part{all.s, all.c, near && here(draft) ? w[draft - v0] : -1.f, 0.f});
        if (j >= n) break;
        // Whether the draft that is tried is kept by what the CTAs told: the walk goes on from it.
        auto moves = [&] {
            float draft_w = -1.f;
            for (int i = 0; i < C; ++i) draft_w = fmaxf(draft_w, sh.part[was][i].c);
            if (!keeps(draft_w, sum_of(was))) return false;
            if (rank == 0 && tid == 0) path[kept] = j;
            ++kept;
            node = j;
            __syncthreads();                         // (the weights are written over)
            return true;
        };
        if (near && moves()) continue;
        // ---- what each draft that is not kept leaves of them
        bool moved = false;
        for (;;) {
            inv = reciprocal(sum_of(was));
            q_row = a.draft_probs ? a.draft_probs + (s0 + node) * a.ldp + v0 : nullptr;
            tried = draft - v0;
            if (a.draft_probs) {
                all = weigh(q_row, false, take_off);
            } else {                                 // one weight is gone, and its block's sum is another
                if (here(draft) && warp == 0) {
                    const int i = static_cast<int>(tried), k = i / kBlock;
                    gone = w[i];
                    __syncwarp();
                    if (lane == 0) w[i] = 0.f;
                    __syncwarp();
                    const Sum s = block_sum(k);
                    if (lane == 0) sh.block[k] = s;
                }
                __syncthreads();
                all = sum_blocks();
            }
            next_draft();
            const int at = j < n && here(draft) ? static_cast<int>(draft - v0) : -1;
            was = exchange(Part{all.s, all.c, at < 0 ? -1.f : left(at), 0.f});
            const bool some = sum_of(was).s > 0.f;
            if (!some) {                             // nothing is left: the weights stay
                if (!a.draft_probs && tried >= 0 && tried < mine && tid == 0) w[tried] = gone;
                __syncthreads();
                all = weigh(nullptr, false, [](int, float x, float) { return x; });
                was = exchange(Part{all.s, all.c, at < 0 ? -1.f : w[at], 0.f});
            }
            if (j >= n) {
                pending = some && a.draft_probs;     // (the search below takes what is left from the weights)
                break;
            }
            if (some && a.draft_probs) {
                weigh(q_row, true, take_off);
                __syncthreads();
            }
            if ((moved = moves())) break;
        }
        if (!moved) break;
    }
    if (rank == 0) {
        for (int i = kept + tid; i < max(1, a.max_tokens - 1); i += kThreads) path[i] = -1;
        if (tid == 0) a.accepted[b] = kept;
    }
    if (!fine) {
        if (rank == 0 && tid == 0) a.next_tokens[b] = -1;
        return;
    }
    // ---- the next token: the CTA, its block of 1024, of the block's 32 pieces and of the piece's 32 weights the first at which the
    // running sum exceeds the aim
    if (warp != 0) return;
    // The first lane at which the running sum of x, from `upto` on, exceeds the aim, or -1; upto: the sum ahead of it. any: the last with
    // a weight.
    auto first_over = [&](const Sum& x, const Sum& aim, Sum& upto, bool any) {
        Sum run = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            Sum o;
            o.s = __shfl_up_sync(0xffffffffu, run.s, d);
            o.c = __shfl_up_sync(0xffffffffu, run.c, d);
            if (lane >= d) {
                o.add(run);
                run = o;
            }
        }
        Sum with = upto;
        with.add(run);
        const unsigned over = any ? 0u : __ballot_sync(0xffffffffu, with.exceeds(aim)), some = __ballot_sync(0xffffffffu, x.s > 0.f);
        const int at = over ? __ffs(over) - 1 : any && some ? 31 - __clz(some) : -1;
        if (at != 0) {
            upto.s = __shfl_sync(0xffffffffu, with.s, at < 0 ? 31 : at - 1);
            upto.c = __shfl_sync(0xffffffffu, with.c, at < 0 ? 31 : at - 1);
        }
        return at;
    };
    const Sum part = lane < C ? Sum{sh.part[was][lane].a, sh.part[was][lane].b} : Sum{0.f, 0.f};
    // u z as a pair: the product's rounding is what the fused operation finds
    const Sum z = warp_sum(part).normal();
    const float u = a.final_uniforms[b];
    Sum aim{__fmul_rn(u, z.s), 0.f};
    aim.c = __fmaf_rn(u, z.c, __fmaf_rn(u, z.s, -aim.s));
    Sum upto{0.f, 0.f};
    int owner = first_over(part, aim, upto, false);
    bool end = owner < 0;                            // (u z rounded up to all of z): the last token with a weight
    if (end) owner = first_over(part, aim, upto, true);
    if (owner != rank) return;
    int k = -1;
    for (int at = 0; at < blocks && k < 0 && !end; at += 32) {
        const Sum x = at + lane < blocks ? sh.block[at + lane] : Sum{0.f, 0.f};
        const int f = first_over(x, aim, upto, false);
        if (f >= 0) k = at + f;
    }
    // (where the blocks' sums and the CTA's do not agree to the last bit, the last one with a weight)
    if (k < 0) {
        end = true;
        for (int at = 0; at < blocks; at += 32) {
            const unsigned some = __ballot_sync(0xffffffffu, at + lane < blocks && sh.block[at + lane].s > 0.f);
            if (some) k = at + 31 - __clz(some);
        }
        k = max(k, 0);
    }
    auto weight = [&](int at) { return at >= mine ? 0.f : pending ? left(at) : w[at]; };
    auto pick = [&](const Sum& x) {                  // the lane
        Sum before = upto;
        int at = end ? -1 : first_over(x, aim, before, false);
        if (at < 0) {
            end = true;
            at = max(0, first_over(x, aim, before, true));
        }
        upto = before;
        return at;
    };
    Sum mine_of_32{0.f, 0.f};
    if (pending) {                          // (a row in global memory: read along it, a piece at a time)
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = weight(k * kBlock + 32 * i + lane);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const Sum s = warp_sum(Sum{x[i], 0.f});
            if (lane == i) mine_of_32 = s;
        }
    } else {                                         // each lane's reads askew, so that the lanes lie in different banks
        for (int i = 0; i < 32; ++i) mine_of_32.add(weight(k * kBlock + lane * 32 + ((i + lane) & 31)));
    }
    const int piece = pick(mine_of_32);
    const int from = k * kBlock + piece * 32;
    const int at = pick(Sum{weight(from + lane), 0.f});
    if (lane == 0) a.next_tokens[b] = v0 + from + at;
}

template <int DT, int THREADS>
int go_verify(const Runtime& rt, const VerifyArgs& a, wq4_stream_t st) {
    auto kern = verify_kernel<DT, THREADS>;
    static PerDevice ready;
    const int ok = ready.get(rt.device, [&]() -> int {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShare * 4) == cudaSuccess) return 1;
        cudaGetLastError();
        return -1;
    });
    if (ok <= 0) return WQ4_ERR_CUDA;
    const int smem = a.share * (DT == WQ4_FP32 && a.ahead ? 8 : 4);
    return launch(rt, kern, dim3(static_cast<unsigned>(a.B) * a.cluster), THREADS, smem, a.cluster, st, a);
}
// As long as two CTAs of 512 threads to an SM hold all sequences at once, a walk over large shares is soonest done by them; else three of
// 256 walk more of them at a time, or meet sooner (32 trees of 16 over 131072: 32.7 us with 512 threads, 36.4 with 256; 192 chains of
// 6: 148 and 114; one chain of 5 over 32001, shares of 4096: 20.5 and 17.9).
template <int DT>
int go_verify(const Runtime& rt, const VerifyArgs& a, wq4_stream_t st) {
    const bool few = static_cast<long long>(a.B) * a.cluster <= 2 * rt.sm_count && a.share > 8192;
    return few ? go_verify<DT, kMaxThreads>(rt, a, st) : go_verify<DT, kMaxThreads / 2>(rt, a, st);
}

}  // namespace
}  // namespace wq4

using namespace wq4;

extern "C" int wq4_verify_drafts(const void* logits, long long ld, const long long* tokens, const int* parents, const int* starts,
                                 int B, int T, int max_tokens, int V, int dtype, const float* draft_probs, long long ldp,
                                 const float* temperature, const float* uniforms, const float* final_uniforms, int* accepted,
                                 int* path, int ld_path, long long* next_tokens, wq4_stream_t stream) {
    if (B < 0 || T < 0 || max_tokens < 1 || V < 1 || (dtype != WQ4_BF16 && dtype != WQ4_FP16 && dtype != WQ4_FP32))
        return WQ4_ERR_INVALID;
    if (V > kVerifyMaxV || B > (1 << 27) || max_tokens > (1 << 20)) return WQ4_ERR_UNSUPPORTED;
    if (B == 0) return WQ4_OK;
    if (!starts || !accepted || !path || !next_tokens || !final_uniforms || ld_path < (max_tokens > 1 ? max_tokens - 1 : 1)) return WQ4_ERR_INVALID;
    if (T > 0 && (!logits || !tokens || !parents || !uniforms || ld < V || (draft_probs && ldp < V))) return WQ4_ERR_INVALID;
    if (ld > (1LL << 40) || (draft_probs && ldp > (1LL << 40))) return WQ4_ERR_INVALID;
    if (!aligned_to(logits, dtype == WQ4_FP32 ? 4 : 2) || !aligned_to(tokens, 8) || !aligned_to(next_tokens, 8)) return WQ4_ERR_ALIGN;
    for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(starts), static_cast<const void*>(draft_probs),
                          static_cast<const void*>(temperature), static_cast<const void*>(uniforms), static_cast<const void*>(final_uniforms),
                          static_cast<const void*>(accepted), static_cast<const void*>(path)})
        if (!aligned_to(p, 4)) return WQ4_ERR_ALIGN;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    VerifyArgs a{logits, tokens, parents, starts, draft_probs, temperature, uniforms, final_uniforms, accepted, path, next_tokens,
                 ld, ldp, B, T, max_tokens, V, ld_path, 1, 0, 0, rt.status};
    while (a.cluster < kMaxCluster && (V > 16 * kBlock * a.cluster || (2LL * a.cluster * B <= rt.sm_count && V > 2 * kBlock * a.cluster)))
        a.cluster *= 2;
    a.share = ((V + a.cluster - 1) / a.cluster + kBlock - 1) / kBlock * kBlock;
    a.ahead = dtype != WQ4_FP32 || a.share <= kMaxShare / 2;
    if (rt.trace) std::fprintf(stderr, "wq4: verify_drafts B=%d tokens=%d V=%d cluster=%d\n", B, max_tokens, V, a.cluster);
    if (dtype == WQ4_BF16) return go_verify<WQ4_BF16>(rt, a, stream);
    if (dtype == WQ4_FP16) return go_verify<WQ4_FP16>(rt, a, stream);
    return go_verify<WQ4_FP32>(rt, a, stream);
}
