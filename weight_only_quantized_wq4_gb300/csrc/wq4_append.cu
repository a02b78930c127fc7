// Queries, keys and values of new tokens on their way into attention: RMS norm of each query and key head, rotation by the
// token's position, the queries written out and keys and values written to their slots of a paged cache, in one pass.
//
// Rotation: the first R features of a head are R / 2 pairs, (i, i + R / 2) or (2 i, 2 i + 1); pair i of a token at
// position p is turned by the angle p f_i. In turns that is p f_i / 2 pi, of which only the fraction counts, so the
// frequency is held as F = f_i / 2 pi in units of 2^-128 turns and p F is taken modulo 2^128: what the multiplication
// drops is whole turns. F is exact to a unit (f_i units above 1), so the angle is off by |p| 2^-128 turns, 2^-65 at the farthest
// position of 64 bits, where p f_i in fp32 would be off by 2^-25 of its value: 0.004 rad at position 131072, half a step of
// bf16 (2^-8).
//
// Each element is read and written once, 16 elements per thread in two 16-byte vectors, chosen so that both halves of each pair
// are the same thread's. 8192 tokens of 32 + 8 heads of 128, bf16: 45.5 us (4.4 TB/s, 65 % of the copy rate). Too few bytes are under way
// beside some 320 instructions per thread and token (issue slots 63 % busy, 47 % of the warps an SM could hold): one token per CTA
// took 56 us, with conflicts in shared memory 59, the next token's loads ahead of the last one's end 48 (registers spill), four
// CTAs of fewer registers 48. One token takes 2.8 us, a launch and two trips to memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "wq4_cache.cuh"

namespace wq4 {
namespace {

struct AppendArgs {
    const uint16_t *q, *k, *v;          // q: null without query heads
    const uint16_t *q_weight, *k_weight;   // null without norms
    const long long *positions, *slots;
    const float* inv_freq;
    uint16_t* q_out;
    CacheArgs cache;
    long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs;
    int T, Hq, Hk, D, R;
    int per_head;                       // threads of a head, a power of two
    int beside, steps;                  // tokens of a CTA: beside each other, one after the other
    float eps, one_over_D;
    unsigned int* status;
};

// 2^128 / 2 pi
constexpr unsigned long long kTurnHi = 0x28be60db9391054aull, kTurnLo = 0x7f09d5f47d4d3770ull;

struct Turns {                          // in units of 2^-128
    unsigned long long hi, lo;
};

// The frequency f (radians per position), modulo a turn: mantissa times 2^128 / 2 pi, three words, shifted by the exponent.
__device__ __forceinline__ Turns turns_of(float f) {
    const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255u;
    const unsigned long long m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
    unsigned long long x0 = m * kTurnLo, x1 = m * kTurnHi + __umul64hi(m, kTurnLo);
    unsigned long long x2 = __umul64hi(m, kTurnHi) + (x1 < __umul64hi(m, kTurnLo));
    int sh = 150 - static_cast<int>(e ? e : 1u);     // f = m 2^-sh
    if (sh < 0) {                                    // (a frequency of 2^24 and more: whole words first, as below)
        if (sh <= -64) x1 = x0, x0 = 0, sh += 64;
        const int up = -sh;
        x2 = 0;
        if (up) x1 = x1 << up | x0 >> (64 - up), x0 <<= up;
        sh = 0;
    }
    if (sh >= 64) x0 = x1, x1 = x2, x2 = 0, sh -= 64;
    if (sh >= 64) x0 = x1, x1 = 0, sh -= 64;
    Turns F{x1, x0};
    if (sh) F.lo = x0 >> sh | x1 << (64 - sh), F.hi = x1 >> sh | x2 << (64 - sh);
    if (u >> 31) F.lo = 0ull - F.lo, F.hi = ~F.hi + (F.lo == 0);
    return F;
}

// cos and sin of p F turns
__device__ __forceinline__ float2 turned(long long p, const Turns& F, float f) {
    // (the upper half of the product modulo 2^128; a negative p is 2^64 less than what is multiplied)
    const unsigned long long up = static_cast<unsigned long long>(p);
    const unsigned long long a = up * F.hi + __umul64hi(up, F.lo) - (p < 0 ? F.lo : 0ull);
    const float half = static_cast<float>(static_cast<int>(a >> 32)) * 0x1p-31f;     // in half turns, [-1, 1]
    float2 cs;
    sincospif(half, &cs.y, &cs.x);
    if (!isfinite(f)) cs.x = cs.y = __int_as_float(0x7fc00000);
    return cs;
}

constexpr int kAppendMaxD = 1024, kAppendThreads = 384;

// Two fp32 to an instruction.
__device__ __forceinline__ uint64_t both(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& x, uint64_t (&v)[4]) {
    float f[8];
    wq4::unpack8<BF16>(x, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = both(f[2 * j], f[2 * j + 1]);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("mov.b64 {%0, %1}, %2;" : "=f"(f[2 * j]), "=f"(f[2 * j + 1]) : "l"(v[j]));
    return wq4::pack8<BF16>(f);
}

// A thread has two vectors of one head and goes through `steps` tokens with it, so that the head's place, its weights' loads and what
// depends on them are found once; the angles of all the CTA's tokens and their places in the cache are found first, by
// all its threads, while the first token's loads are under way.
// ROTATE: 0 none, 1 pairs (i, i + R / 2), 2 pairs (2 i, 2 i + 1).
template <bool BF16, int ROTATE, bool NORM>
__global__ void __launch_bounds__(kAppendThreads, 3) append_kernel(const AppendArgs a) {
    // [token] a slot, -1 where there is none to write; then [token][4][lane] cos and sin, each lane's 16 bytes beside the next one's:
    // two of a lane's pairs (cos, cos, sin, sin) with ROTATE 1, (cos, sin) of each with 2
    extern __shared__ float4 shared4[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int heads = a.Hq + 2 * a.Hk, D = a.D, P = a.per_head;
    const int lane = threadIdx.x % P, group = threadIdx.x / P, groups = blockDim.x / P;
    const int beside = a.beside, tok0 = beside > 1 ? group / heads : 0;          // tokens beside each other, this thread's first
    const long long t0 = static_cast<long long>(blockIdx.x) * (beside * a.steps);
    const int most = beside * a.steps, tokens = static_cast<int>(min(static_cast<long long>(most), a.T - t0));
    int* const slots = reinterpret_cast<int*>(shared4);
    float4* const turns = shared4 + (most + 3) / 4;
    const int r16 = a.R / 16;                        // lanes whose features are all rotated
    // this thread's two vectors of a head
    int c0 = lane * 16, c1 = c0 + 8;
    const bool rot = ROTATE != 0 && lane < r16;
    if (ROTATE == 1 && rot) c0 = lane * 8, c1 = c0 + a.R / 2;
    int head = group - tok0 * heads;
    const int last = beside > 1 ? head + 1 : (heads + groups - 1) / groups * groups;   // (all of a warp's lanes take as many rounds)
    bool found = false;
    for (; head < last; head += groups) {
        const bool in = c0 < D && head < heads && tok0 < beside;
        const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hk;
        const int hk = is_v ? head - a.Hq - a.Hk : head - a.Hq;
        const long long ts = is_q ? a.q_ts : is_v ? a.v_ts : a.k_ts;
        const uint16_t* p = (is_q ? a.q + head * a.q_hs : is_v ? a.v + hk * a.v_hs : a.k + hk * a.k_hs) + (t0 + tok0) * ts;
        const long long step_in = beside * ts;
        int left = in ? tokens - tok0 : 0;           // of this thread's tokens, counted in the CTA's
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
        if (left > 0) {
            x0 = *reinterpret_cast<const uint4*>(p + c0);
            x1 = *reinterpret_cast<const uint4*>(p + c1);
        }
        if (!found) {
            found = true;
            if constexpr (ROTATE != 0) {
                const int half = a.R / 2;
                float* const t = reinterpret_cast<float*>(turns);
                for (int i = threadIdx.x; i < tokens * half; i += blockDim.x) {
                    const int tok = i / half, pair = i - tok * half;
                    const float f = a.inv_freq[pair];
                    const float2 cs = turned(a.positions[t0 + tok], turns_of(f), f);
                    float* at = t + (((tok * 4 + (pair >> 1 & 3)) * r16 + (pair >> 3)) << 2);
                    at[ROTATE == 1 ? pair & 1 : 2 * (pair & 1)] = cs.x;
                    at[ROTATE == 1 ? 2 + (pair & 1) : 2 * (pair & 1) + 1] = cs.y;
                }
            }
            for (int i = threadIdx.x; i < tokens; i += blockDim.x) {
                const long long slot = a.slots[t0 + i];
                const bool past = slot >= static_cast<long long>(a.cache.pages) * a.cache.page_size;
                if (past) atomicOr(a.status, kStatusBadIndex);
                slots[i] = slot < 0 || past ? -1 : static_cast<int>(slot);       // (a negative one is a padded token)
            }
            __syncthreads();
        }
        uint16_t* q_out = a.q_out + (t0 + tok0) * a.qo_ts + head * a.qo_hs;      // (of a query head)
        // (as many rounds for lanes without a head: they take part in the others' exchanges)
        for (int round = 0, tok = tok0; round < a.steps; ++round, tok += beside, left -= beside) {
            if (round != 0 && left > 0) {
                p += step_in;
                x0 = *reinterpret_cast<const uint4*>(p + c0);
                x1 = *reinterpret_cast<const uint4*>(p + c1);
            }
            if (!is_v || NORM) {                     // (with a norm: every lane of the warp, whatever its head is)
                uint64_t v0[4], v1[4];
                unpack8<BF16>(x0, v0);
                unpack8<BF16>(x1, v1);
                if constexpr (NORM) {
                    uint64_t s2 = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) s2 = fma2(v0[j], v0[j], fma2(v1[j], v1[j], s2));
                    float ss, odd;
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(ss), "=f"(odd) : "l"(s2));
                    ss += odd;
                    for (int d = P / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
                    const float r = rsqrtf(fmaf(ss, a.one_over_D, a.eps));
                    const uint64_t rr = both(r, r);
                    if (left > 0 && !is_v) {
                        const uint16_t* weight = is_q ? a.q_weight : a.k_weight;     // (in L1 after the first token)
                        uint64_t w[4];
                        unpack8<BF16>(*reinterpret_cast<const uint4*>(weight + c0), w);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v0[j] = mul2(mul2(v0[j], rr), w[j]);
                        unpack8<BF16>(*reinterpret_cast<const uint4*>(weight + c1), w);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v1[j] = mul2(mul2(v1[j], rr), w[j]);
                    }
                }
                if (ROTATE != 0 && rot && left > 0) {
                    const float4* cs = turns + tok * 4 * r16 + lane;
                    if constexpr (ROTATE == 1) {
                        const uint64_t minus = both(-1.f, -1.f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 t = cs[j * r16];
                            const uint64_t c = both(t.x, t.y), s = both(t.z, t.w), x = v0[j], y = v1[j];
                            v0[j] = fma2(mul2(y, minus), s, mul2(x, c));
                            v1[j] = fma2(x, s, mul2(y, c));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 t = cs[j * r16];                 // of pairs 2 j and 2 j + 1 of the lane's eight
                            const float c[2] = {t.x, t.z}, s[2] = {t.y, t.w};
                            uint64_t(&v)[4] = j < 2 ? v0 : v1;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x, y;
                                asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v[2 * (j & 1) + e]));
                                v[2 * (j & 1) + e] = both(x * c[e] - y * s[e], y * c[e] + x * s[e]);
                            }
                        }
                    }
                }
                if (!is_v) {
                    x0 = pack8<BF16>(v0);
                    x1 = pack8<BF16>(v1);
                }
            }
            if (left > 0) {
                uint16_t* out = q_out;
                if (!is_q) {
                    const int slot = slots[tok];
                    out = slot < 0 ? nullptr : is_v ? a.cache.v_at(slot, hk) : a.cache.k_at(slot, hk);
                }
                if (out) {
                    *reinterpret_cast<uint4*>(out + c0) = x0;
                    *reinterpret_cast<uint4*>(out + c1) = x1;
                }
            }
            q_out += beside * a.qo_ts;
        }
    }
}

// Heads whose sizes or addresses are not multiples of 16 elements or 16 bytes: a warp per head, the row held in shared
// memory as fp32 so that it may be written where it was read.
constexpr int kOddWarps = 4;
template <bool BF16, int ROTATE, bool NORM>
__global__ void __launch_bounds__(32 * kOddWarps) append_odd_kernel(const AppendArgs a) {
    extern __shared__ float rows[];                  // [warps][D]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int heads = a.Hq + 2 * a.Hk, D = a.D, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const long long item = static_cast<long long>(blockIdx.x) * kOddWarps + warp;
    const long long t = item / heads;
    if (t >= a.T) return;
    const int head = static_cast<int>(item - t * heads);
    const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hk;
    const int hk = is_v ? head - a.Hq - a.Hk : head - a.Hq;
    const uint16_t* p = is_q ? a.q + t * a.q_ts + head * a.q_hs : is_v ? a.v + t * a.v_ts + hk * a.v_hs : a.k + t * a.k_ts + hk * a.k_hs;
    uint16_t* out = nullptr;
    if (is_q) {
        out = a.q_out + t * a.qo_ts + head * a.qo_hs;
    } else {
        const long long slot = a.slots[t];
        if (slot < 0) return;
        if (slot >= static_cast<long long>(a.cache.pages) * a.cache.page_size) {
            if (lane == 0) atomicOr(a.status, kStatusBadIndex);
            return;
        }
        out = is_v ? a.cache.v_at(static_cast<unsigned>(slot), hk) : a.cache.k_at(static_cast<unsigned>(slot), hk);
    }
    if (is_v) {
        for (int d = lane; d < D; d += 32) out[d] = p[d];
        return;
    }
    float* row = rows + warp * D;
    float ss = 0.f;
    for (int d = lane; d < D; d += 32) {
        const float x = to_f32<BF16>(p[d]);
        row[d] = x;
        ss = fmaf(x, x, ss);
    }
    __syncwarp();
    float r = 1.f;
    if constexpr (NORM) {
#pragma unroll
        for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        r = rsqrtf(fmaf(ss, a.one_over_D, a.eps));
    }
    const uint16_t* w = is_q ? a.q_weight : a.k_weight;
    auto value = [&](int d) { return NORM ? row[d] * (r * to_f32<BF16>(w[d])) : row[d]; };
    const int half = ROTATE ? a.R / 2 : 0;
    for (int i = lane; i < half; i += 32) {
        const float f = a.inv_freq[i];
        const float2 cs = turned(a.positions[t], turns_of(f), f);
        const int d0 = ROTATE == 1 ? i : 2 * i, d1 = ROTATE == 1 ? i + half : 2 * i + 1;
        const float x = value(d0), y = value(d1);
        out[d0] = to_16<BF16>(x * cs.x - y * cs.y);
        out[d1] = to_16<BF16>(y * cs.x + x * cs.y);
    }
    for (int d = 2 * half + lane; d < D; d += 32) out[d] = to_16<BF16>(value(d));
}

template <bool BF16, int ROTATE, bool NORM>
int go_append(const Runtime& rt, AppendArgs& a, bool vec, wq4_stream_t st) {
    const int heads = a.Hq + 2 * a.Hk;
    if (!vec) {
        const long long ctas = (static_cast<long long>(a.T) * heads + kOddWarps - 1) / kOddWarps;
        if (ctas > 0x7fffffffLL) return WQ4_ERR_UNSUPPORTED;
        return launch(rt, append_odd_kernel<BF16, ROTATE, NORM>, dim3(static_cast<unsigned>(ctas)), 32 * kOddWarps,
                      kOddWarps * a.D * 4, 1, st, a);
    }
    a.per_head = 1;
    while (a.per_head < a.D / 16) a.per_head *= 2;
    // A CTA takes one token's heads side by side, as many tokens as its threads hold where the heads are few; and, with more than
    // a few waves of CTAs, up to four tokens one after the other.
    const int all = heads * a.per_head;              // threads of a token
    a.beside = all >= kAppendThreads ? 1 : std::max(1, std::min(256 / all, a.T));
    const int threads = all >= kAppendThreads ? kAppendThreads : (all * a.beside + 31) / 32 * 32;
    const int waves = static_cast<int>(a.T / (static_cast<long long>(a.beside) * rt.sm_count * 4));
    a.steps = std::max(1, std::min(4, waves));
    const int tokens = a.beside * a.steps;
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.T) + tokens - 1) / tokens);
    return launch(rt, append_kernel<BF16, ROTATE, NORM>, dim3(grid), threads, (tokens + 3) / 4 * 16 + (ROTATE ? tokens * a.R * 4 : 0), 1, st, a);
}

template <bool BF16>
int go_append(const Runtime& rt, AppendArgs& a, int rotate, bool norm, bool vec, wq4_stream_t st) {
    if (norm) {
        if (rotate == 0) return go_append<BF16, 0, true>(rt, a, vec, st);
        return rotate == 1 ? go_append<BF16, 1, true>(rt, a, vec, st) : go_append<BF16, 2, true>(rt, a, vec, st);
    }
    if (rotate == 0) return go_append<BF16, 0, false>(rt, a, vec, st);
    return rotate == 1 ? go_append<BF16, 1, false>(rt, a, vec, st) : go_append<BF16, 2, false>(rt, a, vec, st);
}

}  // namespace
}  // namespace wq4

using namespace wq4;

extern "C" int wq4_rope_append(const void* Q, long long q_ts, long long q_hs, const void* K, long long k_ts, long long k_hs,
                               const void* V, long long v_ts, long long v_hs, int T, int q_heads, int kv_heads, int D,
                               int dtype, const void* q_weight, const void* k_weight, float eps, const long long* positions,
                               const float* inv_freq, int rot_dim, int interleaved, void* Q_out, long long qo_ts,
                               long long qo_hs, const wq4_kv_cache* kv_cache, const long long* slots, wq4_stream_t stream) {
    if (T < 0 || q_heads < 0 || kv_heads < 1 || D < 1 || (dtype != WQ4_BF16 && dtype != WQ4_FP16) || rot_dim < 0 ||
        rot_dim > D || rot_dim % 2 || (interleaved != 0 && interleaved != 1) || !kv_cache)
        return WQ4_ERR_INVALID;
    const bool norm = k_weight != nullptr;
    if (norm && (!(eps >= 0.f) || std::isinf(eps))) return WQ4_ERR_INVALID;
    if ((q_weight != nullptr) != (norm && q_heads > 0)) return WQ4_ERR_INVALID;
    if (q_heads > 65536 || kv_heads > 65536) return WQ4_ERR_INVALID;
    if (D > kAppendMaxD) return WQ4_ERR_UNSUPPORTED;
    wq4_kv_cache cache = *kv_cache;
    if (const int rc = check_cache(cache, kv_heads, D)) return rc;
    if (T == 0) return WQ4_OK;
    if (!K || !V || !slots || (rot_dim && (!positions || !inv_freq)) || (q_heads && (!Q || !Q_out))) return WQ4_ERR_INVALID;
    unused_stride(q_ts, T, D), unused_stride(k_ts, T, D), unused_stride(v_ts, T, D), unused_stride(qo_ts, T, D);
    unused_stride(q_hs, q_heads, D), unused_stride(k_hs, kv_heads, D), unused_stride(v_hs, kv_heads, D);
    unused_stride(qo_hs, q_heads, D);
    if (!strides_ok(q_ts, q_hs, T, q_heads, D) || !strides_ok(k_ts, k_hs, T, kv_heads, D) || !strides_ok(v_ts, v_hs, T, kv_heads, D) ||
        !strides_ok(qo_ts, qo_hs, T, q_heads, D))
        return WQ4_ERR_INVALID;
    for (const void* p : {Q, K, V, q_weight, k_weight, static_cast<const void*>(Q_out)})
        if (!aligned_to(p, 2)) return WQ4_ERR_ALIGN;
    if (!aligned_to(positions, 8) || !aligned_to(slots, 8) || !aligned_to(inv_freq, 4)) return WQ4_ERR_ALIGN;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    AppendArgs a{};
    a.q = static_cast<const uint16_t*>(Q);
    a.k = static_cast<const uint16_t*>(K);
    a.v = static_cast<const uint16_t*>(V);
    a.q_weight = static_cast<const uint16_t*>(q_weight);
    a.k_weight = static_cast<const uint16_t*>(k_weight);
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.q_out = static_cast<uint16_t*>(Q_out);
    a.cache = CacheArgs(cache);
    a.q_ts = q_ts, a.q_hs = q_hs, a.k_ts = k_ts, a.k_hs = k_hs, a.v_ts = v_ts, a.v_hs = v_hs, a.qo_ts = qo_ts, a.qo_hs = qo_hs;
    a.T = T, a.Hq = q_heads, a.Hk = kv_heads, a.D = D, a.R = rot_dim;
    a.eps = eps, a.one_over_D = 1.f / static_cast<float>(D);
    a.status = rt.status;
    const int rotate = rot_dim == 0 ? 0 : interleaved ? 2 : 1;
    bool vec = D % 16 == 0 && D <= 512 && rot_dim % 16 == 0;   // (32 threads a head at most)
    for (const void* p : {Q, K, V, q_weight, k_weight, static_cast<const void*>(Q_out), static_cast<const void*>(cache.k),
                          static_cast<const void*>(cache.v)})
        vec = vec && aligned_to(p, 16);
    for (const long long s : {q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs}) vec = vec && s % 8 == 0;
    for (const long long s : {a.cache.k_page, a.cache.k_token, a.cache.k_head, a.cache.v_page, a.cache.v_token, a.cache.v_head})
        vec = vec && s % 8 == 0;
    if (dtype == WQ4_BF16) return go_append<true>(rt, a, rotate, norm, vec, stream);
    return go_append<false>(rt, a, rotate, norm, vec, stream);
}
