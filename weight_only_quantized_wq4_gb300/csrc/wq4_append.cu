// Queries, keys and values of new tokens on their way into attention: RMS norm of each query and key head, rotation by the
// token's position, the queries written out and keys and values written to their slots of a paged cache, in one pass.
//
// Rotation: the first R features of a head are R / 2 pairs, (i, i + R / 2) or (2 i, 2 i + 1); pair i of a token at
// position p is turned by the angle p f_i. In turns that is p f_i / 2 pi, of which only the fraction counts, so the
// frequency is held as F = f_i / 2 pi in units of 2^-64 turns and p F is taken modulo 2^64: what the multiplication
// drops is whole turns. F is exact to a unit, so the angle is off by p 2^-64 turns, at any position, where p f_i in
// fp32 would be off by 2^-25 of its value: 0.004 rad at position 131072, half a step of bf16 (2^-8).
//
// Bound by memory: each element is read and written once, 16 elements per thread in two 16-byte vectors, chosen so that both
// halves of each pair are the same thread's.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
    int tokens;                         // of a CTA
    float eps, one_over_D;
    unsigned int* status;
};

// 2^64 / 2 pi
constexpr unsigned long long kTurn = 0x28be60db9391054aull;

// The frequency f (radians per position) in units of 2^-64 turns, modulo a turn: mantissa times kTurn, shifted by the exponent.
__device__ __forceinline__ unsigned long long turns_of(float f) {
    const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255u;
    const unsigned long long m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
    const unsigned long long lo = m * kTurn, hi = __umul64hi(m, kTurn);
    const int sh = 150 - static_cast<int>(e ? e : 1u);          // f = m 2^-sh
    unsigned long long F;
    if (sh >= 128) F = 0;
    else if (sh >= 64) F = hi >> (sh - 64);
    else if (sh > 0) F = (lo >> sh) | (hi << (64 - sh));
    else F = sh > -64 ? lo << -sh : 0;
    return u >> 31 ? 0ull - F : F;
}

// cos and sin of p F turns
__device__ __forceinline__ float2 turned(long long p, unsigned long long F, float f) {
    const unsigned long long a = static_cast<unsigned long long>(p) * F;
    const float half = static_cast<float>(static_cast<int>(a >> 32)) * 0x1p-31f;     // in half turns, [-1, 1]
    float2 cs;
    sincospif(half, &cs.y, &cs.x);
    if (!isfinite(f)) cs.x = cs.y = __int_as_float(0x7fc00000);
    return cs;
}

constexpr int kAppendMaxD = 1024;

// ROTATE: 0 none, 1 pairs (i, i + R / 2), 2 pairs (2 i, 2 i + 1).
template <bool BF16, int ROTATE, bool NORM>
__global__ void __launch_bounds__(1024) append_kernel(const AppendArgs a) {
    extern __shared__ float4 turns[];                // [tokens][R / 2] (cos, sin)
    float2* const turn = reinterpret_cast<float2*>(turns);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int heads = a.Hq + 2 * a.Hk, D = a.D, P = a.per_head;
    const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
    const int tokens = static_cast<int>(min(static_cast<long long>(a.tokens), a.T - t0));
    const int lane = threadIdx.x % P, groups = blockDim.x / P;
    // this thread's two vectors of a head
    int c0 = lane * 16, c1 = c0 + 8;
    bool rot = ROTATE == 2 ? c0 < a.R : false, rot1 = ROTATE == 2 ? c1 < a.R : false;
    if (ROTATE == 1) {
        if (lane < a.R / 16) c0 = lane * 8, c1 = c0 + a.R / 2, rot = true;
    }
    const bool in = c0 < D;
    const int all = tokens * heads;
    // One head of one token: where it lies, what is read of it.
    struct Item {
        long long t, slot;
        int tok, head, hk;
        bool live, is_q, is_v;
        uint4 x0, x1;
    };
    auto load = [&](int item) {
        Item m;
        m.tok = item / heads, m.head = item - m.tok * heads;
        m.live = in && item < all;
        m.t = t0 + m.tok;
        m.is_q = m.head < a.Hq, m.is_v = m.head >= a.Hq + a.Hk;
        m.hk = m.is_v ? m.head - a.Hq - a.Hk : m.head - a.Hq;
        m.x0 = m.x1 = make_uint4(0, 0, 0, 0);
        m.slot = -1;
        if (m.live) {
            const uint16_t* p = m.is_q ? a.q + m.t * a.q_ts + m.head * a.q_hs : m.is_v ? a.v + m.t * a.v_ts + m.hk * a.v_hs
                                                                                   : a.k + m.t * a.k_ts + m.hk * a.k_hs;
            m.x0 = *reinterpret_cast<const uint4*>(p + c0);
            m.x1 = *reinterpret_cast<const uint4*>(p + c1);
            if (!m.is_q) m.slot = a.slots[m.t];
        }
        return m;
    };
    auto finish = [&](Item& m) {
        float v0[8], v1[8];
        unpack8<BF16>(m.x0, v0);
        unpack8<BF16>(m.x1, v1);
        float ss = 0.f;
        if constexpr (NORM) {                        // (every lane of the warp, whatever its head is)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v0[j], v0[j], fmaf(v1[j], v1[j], ss));
            for (int d = P / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        }
        if (!m.live) return;
        if (!m.is_v) {
            if constexpr (NORM) {
                const float r = rsqrtf(fmaf(ss, a.one_over_D, a.eps));
                float w0[8], w1[8];
                const uint16_t* w = m.is_q ? a.q_weight : a.k_weight;
                unpack8<BF16>(*reinterpret_cast<const uint4*>(w + c0), w0);
                unpack8<BF16>(*reinterpret_cast<const uint4*>(w + c1), w1);
#pragma unroll
                for (int j = 0; j < 8; ++j) v0[j] *= r * w0[j], v1[j] *= r * w1[j];
            }
            if (ROTATE == 1 && rot) {
                const float4* cs = reinterpret_cast<const float4*>(turn + m.tok * (a.R / 2) + c0);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 c = cs[j / 2];
                    const float x = v0[j], y = v1[j], x2 = v0[j + 1], y2 = v1[j + 1];
                    v0[j] = x * c.x - y * c.y;
                    v1[j] = y * c.x + x * c.y;
                    v0[j + 1] = x2 * c.z - y2 * c.w;
                    v1[j + 1] = y2 * c.z + x2 * c.w;
                }
            }
            if (ROTATE == 2) {
                auto rotate = [&](float(&v)[8], const float2* cs) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = v[2 * j], y = v[2 * j + 1];
                        v[2 * j] = x * cs[j].x - y * cs[j].y;
                        v[2 * j + 1] = y * cs[j].x + x * cs[j].y;
                    }
                };
                const float2* cs = turn + m.tok * (a.R / 2) + c0 / 2;
                if (rot) rotate(v0, cs);
                if (rot1) rotate(v1, cs + 4);
            }
            m.x0 = pack8<BF16>(v0);
            m.x1 = pack8<BF16>(v1);
        }
        uint16_t* out = nullptr;
        if (m.is_q) {
            out = a.q_out + m.t * a.qo_ts + m.head * a.qo_hs;
        } else if (m.slot >= 0) {                    // (a negative one is a padded token)
            if (m.slot < static_cast<long long>(a.cache.pages) * a.cache.page_size) {
                out = m.is_v ? a.cache.v_at(static_cast<unsigned>(m.slot), m.hk) : a.cache.k_at(static_cast<unsigned>(m.slot), m.hk);
            } else {
                atomicOr(a.status, kStatusBadIndex);
            }
        }
        if (out) {
            *reinterpret_cast<uint4*>(out + c0) = m.x0;
            *reinterpret_cast<uint4*>(out + c1) = m.x1;
        }
    };
    int item = threadIdx.x / P;
    Item next = load(item);                          // (under way while the angles are found)
    if constexpr (ROTATE != 0) {
        const int half = a.R / 2;
        for (int i = threadIdx.x; i < tokens * half; i += blockDim.x) {
            const int tok = i / half, pair = i - tok * half;
            const float f = a.inv_freq[pair];
            turn[i] = turned(a.positions[t0 + tok], turns_of(f), f);
        }
        __syncthreads();
    }
    for (const int rounds = (all + groups - 1) / groups * groups; item < rounds;) {
        Item now = next;
        item += groups;
        if (item < rounds) next = load(item);
        finish(now);
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
    const int all = heads * a.per_head;              // threads of a token
    a.tokens = 1;
    const int threads = all > 512 ? 512 : (all + 31) / 32 * 32;
    const unsigned grid = static_cast<unsigned>((a.T + a.tokens - 1) / a.tokens);
    return launch(rt, append_kernel<BF16, ROTATE, NORM>, dim3(grid), threads, ROTATE ? a.tokens * (a.R / 2) * 8 : 0, 1, st, a);
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
