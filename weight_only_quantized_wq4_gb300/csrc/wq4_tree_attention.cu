// Attention of a few tokens per sequence over a paged cache: a decode step's single tokens, chains and trees of drafts.
//
// The heads of a query group read the same keys, so the rows of one problem are (token i, head g of the group), r = i G + g,
// and a problem's unit of work is (sequence, kv head, 16 rows). One pass over the keys and values with the running maximum
// and sum of the softmax; S = Q K^T and O = P V by warp-level MMA with Q, P and O in registers.
//
// Work is split over the caches' lengths: all units' tiles of 64 places lie one after the other, and each CTA takes an
// equal share of them, whichever units they belong to. A unit that several CTAs share is joined by
// the CTA that finishes last, from (maximum, sum, O) of each, in the order of the tiles.
//
// Bound by memory where there is much to read: 64 single tokens of 32 heads over 8 of 128, 500 to 16000 places, bf16: 331 us in pages of
// 64 (6.5 TB/s, 96 % of the copy rate) and 353 in pages of 16, a copy for each of which takes the copy engine longer (410 with
// each page looked up only when its turn came). Few tokens over short contexts are a chain of latencies: one token over
// 600 places takes 9.4 us, of which 5.7 are there with 60 places too, and the join of the CTAs' parts most of the rest.
#include <algorithm>
#include <cstdio>

#include "wq4_attention.cuh"

namespace wq4 {
namespace {

constexpr int kTile = 64;               // places of a tile
constexpr int kLeast = 2;               // tiles worth a CTA (one sequence over 600 places: 9.5 us, with 1 9.7, with 4 12.9)
constexpr int kRows = 16;               // rows of a unit
constexpr int kWarps = 4;               // that compute: 16 places of each tile each
constexpr int kThreads = 32 * (kWarps + 1);

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NC: 64-wide panels of a row.
template <int NC>
struct Cfg {
    static constexpr int kDp = 64 * NC;
    static constexpr int kHalf = kTile * kDp * 2;            // bytes of a tile's keys, or values
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = NC == 1 ? 8 : NC == 2 ? 6 : NC == 3 ? 4 : 3;
    static constexpr int kRed = 2 * kRows * kDp * 4;         // two warps' O
    static constexpr int kHead = 1024;
    static constexpr int kSmem = kHead + kStages * kStage + kRed + 1024;   // (and up to 1008 bytes before the first stage)
};

template <bool BF16, int NC>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<NC>;
    constexpr int kDp = C::kDp;
    constexpr float kRoom = BF16 ? 0.f : kMostLog2;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t s_base = smem_u32(smem_raw);
    const uint32_t s_full = s_base, s_empty = s_base + 8 * C::kStages, s_stall = s_base + 16 * C::kStages;
    int* shared_i = reinterpret_cast<int*>(smem_raw + 256);            // [0] abort, [1] last to finish
    volatile int* abort_flag = shared_i;
    float* s_ml = reinterpret_cast<float*>(smem_raw + 512);            // [warps][rows]: maxima, then sums (512 bytes)
    const uint32_t s_ring = (s_base + C::kHead + 1023) & ~1023u;
    float* s_red = reinterpret_cast<float*>(smem_raw + (s_ring - s_base) + C::kStages * C::kStage);
    __shared__ Scan scan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_empty + 8 * i, kWarps);
        }
        mbar_init(s_stall, 1);
        fence_mbar_init();
    }
    if (warp == kWarps && lane == 0) {
        prefetch_tensormap(&a.k_map);
        prefetch_tensormap(&a.v_map);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // This CTA's share of all the tiles.
    Walk w(a, kTile, kRows, kLeast);
    if (!w.begin(scan, tid, kThreads)) return;                          // (all threads of the CTA alike)
    int issued = 0;
    const WaitCtl ctl{abort_flag, a.status, a.timeout_cycles};

    if (warp == kWarps) {
        // ---------------------------------------------------------------- copies
        const uint64_t pol = policy_evict_first();
        int slot = 0;
        uint32_t phase = 1;
        bool ok = true;
        const int boxes = kTile / a.box, nj = boxes * 2 * a.copies;
        const int part = lane % (2 * a.copies), box = lane / (2 * a.copies);     // lane: (box, panel, keys or values) of a tile
        const bool values = part & 1;
        while (ok && w.next()) {
            // The page of this lane's places, looked up a tile ahead.
            auto there = [&](int t) { return lane < nj && t < w.t1 && t * kTile + box * a.box < w.len; };
            auto find = [&](int t) {
                return there(t) ? a.table[static_cast<long long>(w.b) * a.ld_table + (t * kTile + box * a.box) / a.cache.page_size] : 0;
            };
            int ahead = find(w.t0);
            for (int t = w.t0; t < w.t1 && ok; ++t) {
                int page = ahead;
                ahead = find(t + 1);
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.cache.pages)) atomicOr(a.status, kStatusBadIndex), page = a.cache.pages;
                if (!there(t)) page = a.cache.pages;         // past the last place: outside the tensor, zeros
                if (lane == 0) ok = mbar_wait(s_empty + 8 * slot, phase, ctl);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const uint32_t bar = s_full + 8 * slot;
                if (lane == 0) mbar_arrive_expect_tx(bar, C::kStage);
                __syncwarp();
                if (lane < nj) {
                    const int panel = part >> 1;
                    const uint32_t dst = s_ring + slot * C::kStage + (values ? C::kHalf : 0) + box * a.box * kDp * 2 +
                                         panel * a.box * 128;
                    tma_load_5d(dst, values ? &a.v_map : &a.k_map, bar, 64 * panel, (t * kTile + box * a.box) % a.cache.page_size, 0, w.h, page, pol);
                }
                ++issued;
                if (++slot == C::kStages) slot = 0, phase ^= 1;
            }
        }
    } else {
    // -------------------------------------------------------------------- products
    int slot = 0;
    uint32_t phase = 0;
    if (a.test_stall && tid == 0) mbar_wait(s_stall, 0, ctl);           // (tests: nothing arrives there)
    const int row_lo = lane >> 2, quad = lane & 3;
    // ldmatrix: this lane's row within the warp's 16 places, and which 16-byte half
    const int lm_row_k = (lane & 7) + ((lane >> 4) << 3), lm_half_k = (lane >> 3) & 1;
    const int lm_row_v = (lane & 7) + (((lane >> 3) & 1) << 3), lm_half_v = lane >> 4;
    const int box_in = warp * 16 / a.box, row_in = warp * 16 % a.box;   // where the warp's places lie in a tile
    const uint32_t tile_off = box_in * a.box * kDp * 2 + row_in * 128, panel_step = a.box * 128;
    const uint32_t off_k = tile_off + lm_row_k * 128, off_v = tile_off + lm_row_v * 128;
    const uint32_t sw_k = lm_row_k & 7, sw_v = lm_row_v & 7;
    while (w.next()) {
        const int first = a.starts[w.b];
        uint32_t q[4 * NC][4];
        int token[2];
        bool live[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = w.row0 + row_lo + 8 * e;
            live[e] = r < w.rows;
            token[e] = live[e] ? r / a.G : 0;
            const uint16_t* p = a.q + (first + token[e]) * a.q_ts + (w.h * a.G + (live[e] ? r - token[e] * a.G : 0)) * a.q_hs;
#pragma unroll
            for (int ks = 0; ks < 4 * NC; ++ks)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int d = ks * 16 + f * 8 + quad * 2;
                    q[ks][e + 2 * f] = live[e] && d < a.D ? *reinterpret_cast<const uint32_t*>(p + d) : 0u;
                }
        }
        float o[8 * NC][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < 8 * NC; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j] = 0.f;
        for (int t = w.t0; t < w.t1; ++t) {
            const bool ok = mbar_wait(s_full + 8 * slot, phase, ctl);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t sk = s_ring + slot * C::kStage, sv = sk + C::kHalf;
            const int place0 = t * kTile + warp * 16;
            if (place0 < w.len) {
                float s[2][4] = {};
#pragma unroll
                for (int ks = 0; ks < 4 * NC; ++ks) {
                    uint32_t b[4];
                    ldsm4(sk + off_k + (ks >> 2) * panel_step + (((2 * (ks & 3) + lm_half_k) ^ sw_k) << 4), b);
                    mma16816<BF16>(s[0], q[ks], b[0], b[1]);
                    mma16816<BF16>(s[1], q[ks], b[2], b[3]);
                }
                const bool drafted = place0 + 16 > w.context;
                uint32_t seen[2] = {0xffu, 0xffu};   // bit 4 n + 2 pair... of this thread's places: n * 2 + j
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[n][j] *= a.scale_log2;
                if (drafted) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        seen[e] = 0;
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const bool sees = live[e] && a.sees(first + token[e], token[e], place0 + n * 8 + quad * 2 + j, w.context, w.count);
                                if (sees) seen[e] |= 1u << (2 * n + j);
                                else s[n][2 * e + j] = -INFINITY;
                            }
                    }
                }
                uint32_t p[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float now = fmaxf(m[e], top - kRoom), ref = now == -INFINITY ? 0.f : now;
                    const float keep = exp2_approx(m[e] - ref);
                    m[e] = now;
                    l[e] *= keep;
                    if (keep != 1.f) {
#pragma unroll
                        for (int n = 0; n < 8 * NC; ++n) o[n][2 * e] *= keep, o[n][2 * e + 1] *= keep;
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float x = exp2_approx(s[n][2 * e] - ref), y = exp2_approx(s[n][2 * e + 1] - ref);
                        l[e] += x + y;
                        p[e + 2 * n] = pack2<BF16>(x, y);
                    }
                }
                if (!drafted) {
#pragma unroll
                    for (int n = 0; n < 4 * NC; ++n) {
                        uint32_t b[4];
                        ldsm4_t(sv + off_v + (n >> 2) * panel_step + (((2 * (n & 3) + lm_half_v) ^ sw_v) << 4), b);
                        mma16816<BF16>(o[2 * n], p, b[0], b[1]);
                        mma16816<BF16>(o[2 * n + 1], p, b[2], b[3]);
                    }
                } else {
                    // Places past the last hold whatever the page held: they become zeros. A drafted token's value that is
                    // not finite becomes zero too, as 0 times it would not be, and is added where it is seen.
                    const uint32_t keep0 = pair_mask(place0 + quad * 2, w.len), keep1 = pair_mask(place0 + 8 + quad * 2, w.len);
                    uint32_t vis[4];                 // 1 where seen, as P is laid out
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int n = 0; n < 2; ++n) vis[e + 2 * n] = ones<BF16>(seen[e] >> (2 * n));
#pragma unroll
                    for (int n = 0; n < 4 * NC; ++n) {
                        uint32_t b[4];
                        ldsm4_t(sv + off_v + (n >> 2) * panel_step + (((2 * (n & 3) + lm_half_v) ^ sw_v) << 4), b);
                        b[0] &= keep0, b[1] &= keep1, b[2] &= keep0, b[3] &= keep1;
                        uint32_t bad = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) bad |= not_finite<BF16>(b[j]);
                        if (__any_sync(0xffffffffu, bad != 0)) {
                            uint32_t up[4], down[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) split_bad<BF16>(b[j], up[j], down[j]);
                            float cu[2][4] = {}, cd[2][4] = {};
                            mma16816<BF16>(cu[0], vis, up[0], up[1]);
                            mma16816<BF16>(cu[1], vis, up[2], up[3]);
                            mma16816<BF16>(cd[0], vis, down[0], down[1]);
                            mma16816<BF16>(cd[1], vis, down[2], down[3]);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    if (cu[k][j] > 0.f) o[2 * n + k][j] += INFINITY;
                                    if (cd[k][j] > 0.f) o[2 * n + k][j] -= INFINITY;
                                }
                        }
                        mma16816<BF16>(o[2 * n], p, b[0], b[1]);
                        mma16816<BF16>(o[2 * n + 1], p, b[2], b[3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(s_empty + 8 * slot);
            if (++slot == C::kStages) slot = 0, phase ^= 1;
        }
        // (A warp that gave up goes on to the unit's end, as the others may.)
        // ---------------------------------------------------------------- the warps' parts, then the CTAs'
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (quad == 0) {
                s_ml[warp * kRows + row_lo + 8 * e] = m[e];
                s_ml[(kWarps + warp) * kRows + row_lo + 8 * e] = l[e];
            }
        }
        if (tid == 0) shared_i[2] = *abort_flag;     // (up already where one of these warps gave up in this unit or before)
        bar_sync(1, 32 * kWarps);
        const bool gave_up = shared_i[2];
        float M[2], L[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row_lo + 8 * e;
            M[e] = -INFINITY;
            L[e] = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) M[e] = fmaxf(M[e], s_ml[i * kRows + r]);
            const float ref = M[e] == -INFINITY ? 0.f : M[e];
#pragma unroll
            for (int i = 0; i < kWarps; ++i) L[e] += s_ml[(kWarps + i) * kRows + r] * exp2_approx(s_ml[i * kRows + r] - ref);
            const float f = exp2_approx(m[e] - ref);
#pragma unroll
            for (int n = 0; n < 8 * NC; ++n) o[n][2 * e] *= f, o[n][2 * e + 1] *= f;
        }
        // halves: warps 2, 3 to 0, 1, then 1 to 0
#pragma unroll
        for (int step = kWarps / 2; step; step >>= 1) {
            if (warp >= step && warp < 2 * step) {
                float4* to = reinterpret_cast<float4*>(s_red + (warp - step) * kRows * kDp) + lane;
#pragma unroll
                for (int n = 0; n < 8 * NC; ++n) to[n * 32] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
            }
            bar_sync(1, 32 * kWarps);
            if (warp < step) {
                const float4* from = reinterpret_cast<const float4*>(s_red + warp * kRows * kDp) + lane;
#pragma unroll
                for (int n = 0; n < 8 * NC; ++n) {
                    const float4 x = from[n * 32];
                    o[n][0] += x.x, o[n][1] += x.y, o[n][2] += x.z, o[n][3] += x.w;
                }
            }
            bar_sync(1, 32 * kWarps);
        }
        if (gave_up) break;
        if (w.pieces == 1) {
            if (warp == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!live[e]) continue;
                    const int head = w.h * a.G + (w.row0 + row_lo + 8 * e - token[e] * a.G);
                    const float inv = L[e] == 0.f ? 0.f : 1.f / L[e];
                    uint16_t* p = a.out + (first + token[e]) * a.o_ts + head * a.o_hs;
#pragma unroll
                    for (int n = 0; n < 8 * NC; ++n) {
                        const int d = n * 8 + quad * 2;
                        if (d < a.D) *reinterpret_cast<uint32_t*>(p + d) = pack2<BF16>(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
                    }
                    if (a.lse && quad == 0) a.lse[static_cast<long long>(first + token[e]) * a.Hq + head] = lse_of(M[e], L[e]);
                }
            }
            continue;
        }
        if (warp == 0) {
            float4* to = reinterpret_cast<float4*>(a.parts + static_cast<long long>(w.part) * kRows * kDp) + lane;
#pragma unroll
            for (int n = 0; n < 8 * NC; ++n) __stcg(to + n * 32, make_float4(o[n][0], o[n][1], o[n][2], o[n][3]));
            if (quad == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    __stcg(a.stats + static_cast<long long>(w.part) * kRows + row_lo + 8 * e, make_float2(M[e], L[e]));
            }
            __syncwarp();
            if (lane == 0) {
                __threadfence();                     // (what the warp wrote ahead of its barrier goes with it)
                const int before = atomic_add_acq_rel_gpu(a.counters + w.first_cta, 1);
                const bool last = before == w.pieces - 1;
                if (last) st_relaxed_gpu(a.counters + w.first_cta, 0);     // as the next call finds it
                shared_i[1] = last;
            }
        }
        bar_sync(1, 32 * kWarps);
        const bool last = shared_i[1];
        if (last) {
            // every piece is there: each warp joins its part of the columns
            float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
            for (int i = 0; i < w.pieces; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    top[e] = fmaxf(top[e], __ldcg(a.stats + static_cast<long long>(w.part_of(i)) * kRows + row_lo + 8 * e).x);
            constexpr int kN = 8 * NC / kWarps;
            float4 acc[kN];
#pragma unroll
            for (int n = 0; n < kN; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = 0; i < w.pieces; ++i) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 s = __ldcg(a.stats + static_cast<long long>(w.part_of(i)) * kRows + row_lo + 8 * e);
                    f[e] = exp2_approx(s.x - (top[e] == -INFINITY ? 0.f : top[e]));
                    sum[e] = fmaf(s.y, f[e], sum[e]);
                }
                const float4* from = reinterpret_cast<const float4*>(a.parts + static_cast<long long>(w.part_of(i)) * kRows * kDp) + lane;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const float4 x = __ldcg(from + (warp * kN + n) * 32);
                    acc[n].x = fmaf(x.x, f[0], acc[n].x), acc[n].y = fmaf(x.y, f[0], acc[n].y);
                    acc[n].z = fmaf(x.z, f[1], acc[n].z), acc[n].w = fmaf(x.w, f[1], acc[n].w);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!live[e]) continue;
                const int head = w.h * a.G + (w.row0 + row_lo + 8 * e - token[e] * a.G);
                const float inv = sum[e] == 0.f ? 0.f : 1.f / sum[e];
                uint16_t* p = a.out + (first + token[e]) * a.o_ts + head * a.o_hs;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const int d = (warp * kN + n) * 8 + quad * 2;
                    const float x = e ? acc[n].z : acc[n].x, y = e ? acc[n].w : acc[n].y;
                    if (d < a.D) *reinterpret_cast<uint32_t*>(p + d) = pack2<BF16>(x * inv, y * inv);
                }
                if (a.lse && warp == 0 && quad == 0)
                    a.lse[static_cast<long long>(first + token[e]) * a.Hq + head] = lse_of(top[e], sum[e]);
            }
        }
        bar_sync(1, 32 * kWarps);                    // (shared_i[1] is written again)
    }
    }
    __syncthreads();
    // where a wait ran out, copies in flight land before the CTA goes
    if (warp == kWarps && lane == 0 && *abort_flag)
        for (int j = issued > C::kStages ? issued - C::kStages : 0; j < issued; ++j)
            mbar_wait_plain(s_full + 8 * (j % C::kStages), (j / C::kStages) & 1, drain_limit(a.timeout_cycles));
}

template <bool BF16, int NC>
int go_attention(const Runtime& rt, AttnArgs& a, wq4_stream_t st) {
    using C = Cfg<NC>;
    auto kern = attention_kernel<BF16, NC>;
    static PerDevice ready;
    const int ok = ready.get(rt.device, [&]() -> int {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) == cudaSuccess) return 1;
        cudaGetLastError();
        return -1;
    });
    if (ok <= 0) return WQ4_ERR_CUDA;
    return launch(rt, kern, dim3(a.grid), kThreads, C::kSmem, 1, st, a);
}

// Bytes of a workspace: arrival counters, (maximum, sum) and O of two parts per CTA.
struct Space {
    size_t stats, parts, bytes;
};
Space space_of(int grid, int D, int rows) {
    const size_t parts = 2 * static_cast<size_t>(grid), dp = (D + 63) / 64 * 64;
    Space s;
    s.stats = (4 * static_cast<size_t>(grid) + 255) / 256 * 256;
    s.parts = s.stats + parts * rows * 8;
    s.bytes = s.parts + parts * rows * dp * 4;
    return s;
}

// Whether the kernel with tiles of 128 rows applies: where the rows of a kv head fill more than one of 16 (rows of 16 read the keys and
// values again for each 16).
bool can_tile(int max_tokens, int group, int D) { return static_cast<long long>(max_tokens) * group > kRows && D <= 128; }

// And whether it is the sooner done: but where there are few units of 16 rows, over contexts that L2 holds, their latency counts and not
// what is read (8 tokens, 32 heads over 8: 12.5 us over 2000 places by rows of 16, 19.2 by tiles, 22 and 36 over 8000; 16
// tokens over 2000: 17.6 and 19.5; eight sequences of 8: 35 and 30). Contexts are in device memory; the table's width bounds them.
bool should_tile(const AttnArgs& a) {
    const long long units = static_cast<long long>(a.B) * a.Hk * ((static_cast<long long>(a.max_tokens) * a.G + kRows - 1) / kRows);
    return units > 32 || static_cast<long long>(a.table_width) * a.cache.page_size > 16384;
}

int check_heads(int B, int max_tokens, int q_heads, int kv_heads, int D) {
    if (B < 0 || max_tokens < 1 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads || D < 1) return WQ4_ERR_INVALID;
    if (D % 8 || D > 256 || q_heads > 65536 || max_tokens > (1 << 20) || static_cast<long long>(max_tokens) * (q_heads / kv_heads) > (1 << 30))
        return WQ4_ERR_UNSUPPORTED;
    return WQ4_OK;
}

}  // namespace
}  // namespace wq4

using namespace wq4;

extern "C" {

int wq4_tree_attention_workspace_bytes(int B, int max_tokens, int q_heads, int kv_heads, int D, size_t* bytes) {
    if (!bytes) return WQ4_ERR_INVALID;
    if (const int rc = check_heads(B, max_tokens, q_heads, kv_heads, D)) return rc;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    *bytes = space_of(rt.sm_count, D, can_tile(max_tokens, q_heads / kv_heads, D) ? tiles_rows() : kRows).bytes;
    return WQ4_OK;
}

int wq4_tree_attention(const void* Q, long long q_ts, long long q_hs, const wq4_kv_cache* kv_cache, const int* page_table,
                       int ld_table, int table_width, const int* starts, const int* context, int B, int T,
                       int max_tokens, int q_heads, int kv_heads, int D, int dtype, float scale,
                       const unsigned long long* mask, int mask_words, void* out, long long o_ts, long long o_hs,
                       float* lse, void* workspace, size_t workspace_bytes, wq4_stream_t stream) {
    if (T < 0 || (dtype != WQ4_BF16 && dtype != WQ4_FP16) || !std::isfinite(scale) || !kv_cache) return WQ4_ERR_INVALID;
    if (const int rc = check_heads(B, max_tokens, q_heads, kv_heads, D)) return rc;
    wq4_kv_cache cache = *kv_cache;
    if (const int rc = check_cache(cache, kv_heads, D)) return rc;
    if (table_width < 1 || ld_table < table_width || (mask && static_cast<long long>(mask_words) * 64 < max_tokens)) return WQ4_ERR_INVALID;
    if (cache.page_size % 16) return WQ4_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return WQ4_OK;
    if (!Q || !page_table || !starts || !context || !out) return WQ4_ERR_INVALID;
    unused_stride(q_ts, T, D), unused_stride(q_hs, q_heads, D), unused_stride(o_ts, T, D), unused_stride(o_hs, q_heads, D);
    if (!strides_ok(q_ts, q_hs, T, q_heads, D) || !strides_ok(o_ts, o_hs, T, q_heads, D)) return WQ4_ERR_INVALID;
    for (const void* p : {Q, static_cast<const void*>(out), static_cast<const void*>(cache.k), static_cast<const void*>(cache.v),
                          static_cast<const void*>(workspace)})
        if (!aligned_to(p, 16)) return WQ4_ERR_ALIGN;
    for (const long long s : {q_ts, q_hs, o_ts, o_hs, cache.k_page, cache.k_token, cache.k_head, cache.v_page, cache.v_token, cache.v_head})
        if (s % 8) return WQ4_ERR_ALIGN;
    if (!aligned_to(page_table, 4) || !aligned_to(starts, 4) || !aligned_to(context, 4) || !aligned_to(mask, 8) || !aligned_to(lse, 4))
        return WQ4_ERR_ALIGN;
    // a tensor map's strides are below 2^40 bytes
    for (const long long s : {cache.k_page, cache.k_token, cache.k_head, cache.v_page, cache.v_token, cache.v_head})
        if (s >= (1LL << 39)) return WQ4_ERR_UNSUPPORTED;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    AttnArgs a{};
    a.grid = rt.sm_count;
    a.q = static_cast<const uint16_t*>(Q);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.table = page_table;
    a.starts = starts;
    a.context = context;
    a.mask = mask;
    a.q_ts = q_ts, a.q_hs = q_hs, a.o_ts = o_ts, a.o_hs = o_hs;
    a.cache = CacheArgs(cache);
    a.ld_table = ld_table, a.table_width = table_width, a.mask_words = mask_words;
    a.B = B, a.T = T, a.max_tokens = max_tokens, a.Hq = q_heads, a.Hk = kv_heads, a.G = q_heads / kv_heads, a.D = D;
    a.max_rows = static_cast<int>(std::min(static_cast<long long>(max_tokens) * a.G, 1LL << 20));
    a.scale_log2 = scale * 1.4426950408889634f;
    a.test_stall = rt.test_stall;
    // (the tiles' softmax takes maxima ahead of the scale; the other kernel, whose parts are smaller, after it)
    const bool can = can_tile(max_tokens, q_heads / kv_heads, D);
    const bool tiles = can && scale > 1e-30f && should_tile(a) && attention_tiles_fit(rt, dtype, D);
    if (!workspace || workspace_bytes < space_of(a.grid, D, can ? tiles_rows() : kRows).bytes) return WQ4_ERR_WORKSPACE;
    const Space sp = space_of(a.grid, D, tiles ? tiles_rows() : kRows);
    a.counters = static_cast<int*>(workspace);
    a.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + sp.stats);
    a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.parts);
    a.status = rt.status;
    a.timeout_cycles = rt.timeout_cycles;
    a.box = 16;                                      // the places of one copy: they lie in one page
    while (a.box < (tiles ? tiles_places() : kTile) && cache.page_size % (2 * a.box) == 0) a.box *= 2;
    const int panels = (D + 63) / 64;
    const bool whole = D % 64 == 0 && !tiles;        // all panels in one copy, or (D cuts one, or they lie apart) a copy each
    a.copies = whole ? 1 : panels;
    if (!encode_cache(rt.encode, &a.k_map, dtype, cache.k, D, cache.k_token, cache.k_head, cache.k_page, cache, kv_heads, a.box, whole ? panels : 1) ||
        !encode_cache(rt.encode, &a.v_map, dtype, cache.v, D, cache.v_token, cache.v_head, cache.v_page, cache, kv_heads, a.box, whole ? panels : 1))
        return WQ4_ERR_CUDA;
    if (rt.trace)
        std::fprintf(stderr, "wq4: tree_attention B=%d tokens=%d heads=%d/%d D=%d box=%d grid=%d rows=%d\n", B, max_tokens, q_heads, kv_heads, D, a.box, a.grid, tiles ? tiles_rows() : kRows);
    if (tiles) return launch_attention_tiles(rt, a, dtype, stream);
    if (dtype == WQ4_BF16) {
        switch (panels) {
            case 1: return go_attention<true, 1>(rt, a, stream);
            case 2: return go_attention<true, 2>(rt, a, stream);
            case 3: return go_attention<true, 3>(rt, a, stream);
            default: return go_attention<true, 4>(rt, a, stream);
        }
    }
    switch (panels) {
        case 1: return go_attention<false, 1>(rt, a, stream);
        case 2: return go_attention<false, 2>(rt, a, stream);
        case 3: return go_attention<false, 3>(rt, a, stream);
        default: return go_attention<false, 4>(rt, a, stream);
    }
}

}  // extern "C"
