// Attention over a paged cache for many rows per kv head (trees of drafts, many queries to a key): the products on the tensor
// cores' own path. A row is (token i, head g of the group), r = i G + g; S = Q K^T and O += P V are tcgen05 MMAs of 128 rows
// by 128 places, with S, P (where S was) and O in tensor memory; one thread of 128 owns a row of S, so the softmax
// needs no exchange between threads.
//
// Two streams of S tiles keep the tensor cores and the softmax warps busy in turn. A unit of more than 128 rows gives each stream
// 128 rows of its own and the same places (each tile of keys and values is read once for 256 rows); a
// unit of fewer gives both the same rows and every other tile of places, and the streams' O, maxima and sums are joined at
// the end. A row's maximum is taken over when it has grown by more than 2^8 (any reference will do for the softmax as
// long as nothing overflows), so that O is rarely scaled.
//
// Work is cut as in wq4_tree_attention.cu: equal shares of all the units' tiles, and the CTA that finishes last joins a unit.
#include "wq4_attention.cuh"

namespace wq4 {
namespace {

constexpr int kTile = 128;              // places of a tile
constexpr int kLanes = 128;             // rows of a stream's tile
constexpr int kUnitRows = 2 * kLanes;
constexpr int kSoftmaxWarp = 4;         // the first of eight; before them: copies, MMAs, two that look at drafted values
constexpr int kThreads = 32 * (kSoftmaxWarp + 8);
constexpr int kMaxSlots = 16;
constexpr float kSlack = 8.f;           // log2 of what a probability may exceed 1 by

template <int NC>
struct Cfg {
    static constexpr int kDp = 64 * NC;
    static constexpr int kSlot = kTile * kDp * 2;            // a tile's keys, or values
    static constexpr int kQ = kLanes * kDp * 2;
    static constexpr int kHead = 4096;                       // barriers, statistics
    static constexpr int kMaxSmem = 232448;                  // 227 KB
    static constexpr int kSlots = (kMaxSmem - 1024 - kHead - 2 * kQ) / kSlot < kMaxSlots ? (kMaxSmem - 1024 - kHead - 2 * kQ) / kSlot : kMaxSlots;
    static constexpr int kSmem = 1024 + kHead + 2 * kQ + kSlots * kSlot;
    static constexpr int kO = 2 * kTile;                     // tensor memory: S of both streams, then O of both
    static constexpr uint32_t kTmemCols = 2 * kTile + 2 * kDp > 256 ? 512 : 256;
};

// Registers: 128 x 88 + 256 x 208 are those of the launch, 384 x 168.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Values as the B operand of O = P V: 64 features by 8 places are the swizzle's atom, so the features are the leading
// dimension; `panel` bytes from one 64 features to the next.
__device__ __forceinline__ uint64_t values_desc(uint32_t saddr, uint32_t panel) {
    uint64_t d = make_sdesc_sw128(saddr);
    d &= ~(static_cast<uint64_t>(0x3fff) << 16);
    return d | static_cast<uint64_t>(panel >> 4) << 16;
}

// The items of a unit's ring in order: values of tile j - lag, then keys of tile j.
struct Ring {
    uint32_t it = 0;
    int slots;
    __device__ explicit Ring(int n) : slots(n) {}
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step() {
        ++it;
        if (++slot == slots) slot = 0, phase ^= 1;
    }
};

// Which of 32 places from j0 on (in drafted tokens: j < 0 is the context) token i sees.
__device__ __forceinline__ uint32_t seen32(const AttnArgs& a, int t, int i, int j0, int count) {
    if (j0 <= -32) return 0xffffffffu;
    const uint32_t ctx = j0 < 0 ? (1u << -j0) - 1u : 0u;
    const int from = j0 < 0 ? 0 : j0, shift = from - j0;             // drafted tokens [from, j0 + 32)
    uint64_t bits = 0;
    if (from < count) {
        if (a.mask) {
            const unsigned long long* m = a.mask + static_cast<long long>(t) * a.mask_words;
            const int w = from >> 6, s = from & 63;
            bits = m[w] >> s;
            if (s > 32 && w + 1 < a.mask_words) bits |= m[w + 1] << (64 - s);
        } else {
            bits = i >= from ? (i - from >= 31 ? 0xffffffffu : (2u << (i - from)) - 1u) : 0u;
        }
        if (count - from < 32) bits &= (1u << (count - from)) - 1u;
    }
    return ctx | static_cast<uint32_t>(bits << shift);
}

template <bool BF16, int NC>
__global__ void __launch_bounds__(kThreads, 1) attention_tiles_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<NC>;
    constexpr int kDp = C::kDp, kPanel = kTile * 128;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t s_base = (smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* base = smem_raw + (s_base - smem_u32(smem_raw));
    // barriers
    const uint32_t s_full = s_base, s_empty = s_base + 8 * kMaxSlots, s_vok = s_base + 16 * kMaxSlots;
    const uint32_t s_sfull = s_base + 24 * kMaxSlots, s_pfull = s_sfull + 16, s_ofull = s_sfull + 32, s_qfull = s_sfull + 40,
                   s_drain = s_sfull + 48, s_stall = s_sfull + 56;
    int* ctl_i = reinterpret_cast<int*>(base + 512);         // [0] abort, [1] last to finish, [2] gave up, [3] tensor memory, [4] values not finite
    volatile int* abort_flag = ctl_i;
    volatile int* bad_slot = ctl_i + 8;                      // [slots] a drafted value that is not finite was taken out
    float2* s_stat = reinterpret_cast<float2*>(base + 1024); // [2][lanes] (maximum, sum)
    const uint32_t s_q = s_base + C::kHead, s_ring = s_q + 2 * C::kQ;
    __shared__ Scan scan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 16; ++i) ctl_i[i] = 0;
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_empty + 8 * i, 3);           // the MMAs that read it, and the two warps that look at drafted values
            mbar_init(s_vok + 8 * i, 2);
            bad_slot[i] = 0;
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_sfull + 8 * s, 1);
            mbar_init(s_pfull + 8 * s, 4);
        }
        mbar_init(s_ofull, 2);
        mbar_init(s_qfull, 8);
        mbar_init(s_drain, 1);
        mbar_init(s_stall, 1);
        fence_mbar_init();
        prefetch_tensormap(&a.k_map);
        prefetch_tensormap(&a.v_map);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(ctl_i + 3), C::kTmemCols);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(ctl_i[3]);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Walk w(a, kTile, kUnitRows);
    const bool work = w.begin(scan, tid, kThreads);          // (all threads of the CTA alike)
    const WaitCtl ctl{abort_flag, a.status, a.timeout_cycles};
    Ring ring(C::kSlots);
    // A unit's tiles: lag of the values behind the keys, and whether both streams have rows of their own.
    auto two = [&] { return w.rows - w.row0 > kLanes; };

    if (warp < kSoftmaxWarp) {
        fewer_registers<88>();
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            const uint64_t pol = policy_evict_first();
            const int per_box = NC, panel = lane % NC, box = lane / NC;
            const bool mine = lane < kTile / a.box * per_box;
            bool ok = work;
            while (ok && w.next()) {
                const int n = w.t1 - w.t0, lag = two() ? 1 : 2;
                for (int j = 0; j < n + lag && ok; ++j) {
                    for (int kind = 0; kind < 2 && ok; ++kind) {         // 0: values of j - lag, 1: keys of j
                        const int tile = kind ? j : j - lag;
                        if (tile < 0 || tile >= n) continue;
                        const int place = (w.t0 + tile) * kTile + box * a.box;
                        int page = a.cache.pages, at = 0;                // past the last place: outside the tensor, zeros
                        if (mine && place < w.len) {
                            const int i = place / a.cache.page_size;
                            page = a.table[static_cast<long long>(w.b) * a.ld_table + i];
                            at = place - i * a.cache.page_size;
                            if (page < 0 || page >= a.cache.pages) {
                                atomicOr(a.status, kStatusBadIndex);
                                page = a.cache.pages;
                            }
                        }
                        if (lane == 0) ok = mbar_wait(s_empty + 8 * ring.slot, ring.phase ^ 1, ctl);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        const uint32_t bar = s_full + 8 * ring.slot;
                        if (lane == 0) mbar_arrive_expect_tx(bar, C::kSlot);
                        __syncwarp();
                        if (mine)
                            tma_load_5d(s_ring + ring.slot * C::kSlot + panel * kPanel + box * a.box * 128, kind ? &a.k_map : &a.v_map, bar,
                                        64 * panel, at, 0, w.h, page, pol);
                        ring.step();
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMAs
            if (lane == 0) {
                constexpr uint32_t kIdescS = make_idesc(BF16, kLanes, kTile);
                constexpr uint32_t kIdescO = make_idesc(BF16, kLanes, kDp) | (1u << 16);    // values: features lead
                const int ksteps = (a.D + 15) / 16;
                uint32_t vok_phase = 0, p_phase[2] = {0, 0}, q_phase = 0;
                bool ok = work, any = false;
                while (ok && w.next()) {
                    const bool pair = two();
                    const int n = w.t1 - w.t0, lag = pair ? 1 : 2;
                    if (!(ok = mbar_wait(s_qfull, q_phase, ctl))) break;
                    q_phase ^= 1;
                    tc_fence_after();
                    ctl_i[4] = 0;
                    uint32_t begun = 0;                      // streams whose O has begun
                    for (int j = 0; j < n + lag && ok; ++j) {
                        const int v = j - lag;
                        int v_slot = -1, k_slot = -1;
                        if (v >= 0) {
                            v_slot = ring.slot;
                            if (!(ok = mbar_wait(s_full + 8 * v_slot, ring.phase, ctl))) break;
                            if ((w.t0 + v + 1) * kTile > w.context) {     // (looked at, and mended, by the warps beside)
                                if (!(ok = mbar_wait(s_vok + 8 * v_slot, vok_phase >> v_slot & 1u, ctl))) break;
                                vok_phase ^= 1u << v_slot;
                                if (bad_slot[v_slot]) ctl_i[4] = 1, bad_slot[v_slot] = 0;
                            }
                            ring.step();
                        }
                        if (j < n) {
                            k_slot = ring.slot;
                            if (!(ok = mbar_wait(s_full + 8 * k_slot, ring.phase, ctl))) break;
                            ring.step();
                        }
                        for (int s = 0; s < 2; ++s) {
                            if (v >= 0 && (pair || (v & 1) == s)) {
                                if (!(ok = mbar_wait(s_pfull + 8 * s, p_phase[s], ctl))) break;
                                p_phase[s] ^= 1;
                                tc_fence_after();
                                const uint32_t from = s_ring + v_slot * C::kSlot;
#pragma unroll
                                for (int k = 0; k < kTile / 16; ++k)
                                    mma_ts(tmem + C::kO + s * kDp, tmem + s * kTile + k * 8, values_desc(from + k * 2048, kPanel), kIdescO,
                                           (begun >> s & 1u) | (k > 0));
                                begun |= 1u << s;
                            }
                            if (j < n && (pair || (j & 1) == s)) {
                                const uint32_t q = s_q + (pair ? s * C::kQ : 0), from = s_ring + k_slot * C::kSlot;
                                for (int k = 0; k < ksteps; ++k) {
                                    const uint32_t off = (k >> 2) * kPanel + (k & 3) * 32;
                                    mma_ss(tmem + s * kTile, make_sdesc_sw128(q + off), make_sdesc_sw128(from + off), kIdescS, k > 0);
                                }
                                mma_commit(s_sfull + 8 * s);
                            }
                        }
                        any = true;
                        if (!ok) break;
                        if (v >= 0) mma_commit(s_empty + 8 * v_slot);
                        if (k_slot >= 0) mma_commit(s_empty + 8 * k_slot);
                    }
                    if (!ok) break;
                    mma_commit(s_ofull);
                    mbar_arrive(s_ofull);                    // (with what ctl_i[4] says)
                }
                if (any && !ok) {                            // what was begun ends before the CTA goes
                    mma_commit(s_drain);
                    mbar_wait_plain(s_drain, 0, drain_limit(a.timeout_cycles));
                }
            }
        } else {
            // ------------------------------------------------------------ drafted tokens' values
            // Rows past the last place hold whatever the page held: they become zeros. A value of a drafted token that is not
            // finite becomes zero too, as 0 times it would not be; the rows that see it add it at the end.
            // (They see every slot filled, so that a slot is never filled twice between two looks at its barrier.)
            bool ok = work;
            while (ok && w.next()) {
                const int n = w.t1 - w.t0, lag = two() ? 1 : 2;
                for (int j = 0; j < n + lag && ok; ++j) {
                    for (int kind = 0; kind < 2; ++kind) {
                        const int tile = kind ? j : j - lag;
                        if (tile < 0 || tile >= n) continue;
                        ok = mbar_wait(s_full + 8 * ring.slot, ring.phase, ctl);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        const int place0 = (w.t0 + tile) * kTile;
                        if (kind == 0 && place0 + kTile > w.context) {
                            const int first = max(0, w.context - place0), last = w.len - place0;    // drafted rows
                            uint8_t* slot = base + (s_ring - s_base) + ring.slot * C::kSlot;
                            constexpr int kChunks = NC * 8;              // 16 bytes each, of a row
                            for (int i = first * kChunks + (warp - 2) * 32 + lane; i < kTile * kChunks; i += 64) {
                                const int row = i / kChunks, c = i % kChunks;
                                uint4* p = reinterpret_cast<uint4*>(slot + (c >> 3) * kPanel + row * 128 + (((c & 7) ^ (row & 7)) << 4));
                                if (row >= last) {
                                    *p = make_uint4(0, 0, 0, 0);
                                    continue;
                                }
                                uint4 x = *p;
                                uint32_t u[4] = {x.x, x.y, x.z, x.w}, f = 0;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t nf = not_finite<BF16>(u[k]);
                                    f |= nf;
                                    if (nf & 1u) u[k] &= 0xffff0000u;
                                    if (nf & 2u) u[k] &= 0x0000ffffu;
                                }
                                if (f) {
                                    *p = make_uint4(u[0], u[1], u[2], u[3]);
                                    bad_slot[ring.slot] = 1;
                                }
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(s_vok + 8 * ring.slot);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_empty + 8 * ring.slot);
                        ring.step();
                    }
                }
            }
        }
    } else {
        more_registers<208>();
        // ---------------------------------------------------------------- softmax
        const int s = (warp - kSoftmaxWarp) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t t_lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_s = t_lanes + s * kTile;
        uint32_t s_phase = 0, o_phase = 0;
        bool dead = false;
        if (a.test_stall && work && tid == 32 * kSoftmaxWarp) mbar_wait(s_stall, 0, ctl);   // (tests: nothing arrives there)
        while (work && w.next()) {
            const bool pair = two();
            const int n = w.t1 - w.t0, first = a.starts[w.b];
            const int r = w.row0 + (pair ? s * kLanes : 0) + row;        // of the problem
            const bool live = r < w.rows;
            const bool idle = __all_sync(0xffffffffu, !live);
            const int token = live ? r / a.G : 0, head = w.h * a.G + (live ? r - token * a.G : 0);
            // ---- this stream's rows of Q (each stream half of them where they are shared)
            {
                const uint16_t* from = a.q + static_cast<long long>(first + token) * a.q_ts + head * a.q_hs;
                const uint32_t to = s_q + (pair ? s * C::kQ : 0) + row * 128;
                const int c0 = pair ? 0 : s * (NC * 4), c1 = pair ? NC * 8 : c0 + NC * 4;
#pragma unroll 8
                for (int c = c0; c < c1; ++c) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (live && c * 8 < a.D) x = *reinterpret_cast<const uint4*>(from + c * 8);
                    sts128(to + (c >> 3) * (kLanes * 128) + (((c & 7) ^ (row & 7)) << 4), x.x, x.y, x.z, x.w);
                }
                fence_proxy_async_smem();
                tc_fence_before();                           // (and the last unit's O has been read)
                __syncwarp();
                if (lane == 0) mbar_arrive(s_qfull);
            }
            float ref = -INFINITY, l = 0.f;
            bool begun = false;
            for (int j = pair ? 0 : s; j < n; j += pair ? 1 : 2) {
                if (!dead) {
                    const bool ok = mbar_wait(s_sfull + 8 * s, s_phase, ctl);
                    dead = !__all_sync(0xffffffffu, ok);
                }
                if (dead) break;
                s_phase ^= 1;
                tc_fence_after();
                if (!idle) {
                    uint32_t x[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld32(t_s + 32 * k, x[k]);
                    tmem_ld_wait();
                    const int place0 = (w.t0 + j) * kTile;
                    if (place0 + kTile > w.context) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t seen = seen32(a, first + token, token, place0 + 32 * k - w.context, w.count);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen >> c & 1u)) x[k][c] = 0xff800000u;
                        }
                    }
                    float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            top = max3(top, __uint_as_float(x[k][c]), __uint_as_float(x[k][c + 1]));
                            top2 = max3(top2, __uint_as_float(x[k][c + 2]), __uint_as_float(x[k][c + 3]));
                        }
                    top = fmaxf(top, top2) * a.scale_log2;
                    const bool grows = top > ref + kSlack || (ref == -INFINITY && top > ref);
                    if (__any_sync(0xffffffffu, grows)) {
                        const float now = grows ? top : ref;
                        const float keep = ref == -INFINITY ? 0.f : exp2_approx(ref - now);
                        ref = now;
                        l *= keep;
                        if (begun) {                         // (the MMAs of the tiles before have ended: S came after them)
#pragma unroll
                            for (int k = 0; k < kDp / 32; ++k) {
                                uint32_t o[32];
                                tmem_ld32(t_lanes + C::kO + s * kDp + 32 * k, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * keep);
                                tmem_st16(t_lanes + C::kO + s * kDp + 32 * k, reinterpret_cast<const uint32_t(&)[16]>(o[0]));
                                tmem_st16(t_lanes + C::kO + s * kDp + 32 * k + 16, reinterpret_cast<const uint32_t(&)[16]>(o[16]));
                            }
                        }
                    }
                    const float minus = ref == -INFINITY ? 0.f : -ref;
                    float l2[2] = {0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t p[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const float e0 = exp2_approx(fmaf(__uint_as_float(x[k][c]), a.scale_log2, minus));
                            const float e1 = exp2_approx(fmaf(__uint_as_float(x[k][c + 1]), a.scale_log2, minus));
                            l2[0] += e0;
                            l2[1] += e1;
                            p[c / 2] = pack2<BF16>(e0, e1);
                        }
                        tmem_st16(t_s + 16 * k, p);
                    }
                    l += l2[0] + l2[1];
                    tmem_st_wait();
                }
                begun = true;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_pfull + 8 * s);
            }
            if (!dead) {
                const bool ok = mbar_wait(s_ofull, o_phase, ctl);
                dead = !__all_sync(0xffffffffu, ok);
            }
            o_phase ^= 1;
            tc_fence_after();
            s_stat[s * kLanes + row] = make_float2(ref, l);
            if (tid == 32 * kSoftmaxWarp) ctl_i[2] = *abort_flag;
            bar_sync(1, 256);
            if (ctl_i[2]) break;                             // (all 256 threads alike)
            // ---- join the streams where they share rows; each then has half of the columns
            float M = ref, L = l, f0 = 1.f, f1 = 1.f;
            if (!pair) {
                const float2 p = s_stat[row], q = s_stat[kLanes + row];
                M = fmaxf(p.x, q.x);
                const float at = M == -INFINITY ? 0.f : M;
                f0 = exp2_approx(p.x - at);
                f1 = exp2_approx(q.x - at);
                L = p.y * f0 + q.y * f1;
            }
            const bool bad = ctl_i[4];
            const bool whole = w.pieces == 1;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            constexpr int kCh = kDp / 32;
            const int k0 = pair ? 0 : s * (kCh / 2), k1 = pair ? kCh : k0 + kCh / 2;
            const int unit_row = (pair ? s * kLanes : 0) + row;
            if (!idle) {
                for (int k = k0; k < k1; ++k) {
                    uint32_t o[32];
                    tmem_ld32(t_lanes + C::kO + (pair ? s * kDp : 0) + 32 * k, o);
                    if (!pair && n > 1) {
                        uint32_t o1[32];
                        tmem_ld32(t_lanes + C::kO + kDp + 32 * k, o1);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o[c] = __float_as_uint(__uint_as_float(o[c]) * f0 + __uint_as_float(o1[c]) * f1);
                    } else {
                        tmem_ld_wait();
                    }
                    if (bad && live) {
                        const int lo = max(0, w.t0 * kTile - w.context), hi = min(w.count, w.t1 * kTile - w.context);
                        for (int j = lo; j < hi; ++j) {
                            const int place = w.context + j, i = place / a.cache.page_size;
                            if (!a.sees(first + token, token, place, w.context, w.count)) continue;
                            const int page = a.table[static_cast<long long>(w.b) * a.ld_table + i];
                            if (page < 0 || page >= a.cache.pages) continue;
                            const uint16_t* v = a.cache.v + page * a.cache.v_page + (place - i * a.cache.page_size) * a.cache.v_token +
                                                w.h * a.cache.v_head + 32 * k;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (32 * k + c < a.D && not_finite<BF16>(v[c]) & 1u) o[c] = __float_as_uint(__uint_as_float(o[c]) + to_f32<BF16>(v[c]));
                        }
                    }
                    if (whole) {
                        if (live) {
                            uint16_t* to = a.out + static_cast<long long>(first + token) * a.o_ts + head * a.o_hs + 32 * k;
#pragma unroll
                            for (int c = 0; c < 32; c += 8) {
                                if (32 * k + c >= a.D) break;
                                float y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[c + e]) * inv;
                                *reinterpret_cast<uint4*>(to + c) = pack8<BF16>(y);
                            }
                        }
                    } else {
                        float4* to = reinterpret_cast<float4*>(a.parts) + (static_cast<long long>(w.part) * (kDp / 4) + 8 * k) * kUnitRows + unit_row;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            __stcg(to + c * kUnitRows, make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                                                   __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3])));
                    }
                }
            }
            if (whole) {
                if (live && a.lse && (pair || s == 0)) a.lse[static_cast<long long>(first + token) * a.Hq + head] = lse_of(M, L);
                bar_sync(1, 256);                            // (s_stat and ctl_i[2] are written again)
                continue;
            }
            if (pair || s == 0) __stcg(a.stats + static_cast<long long>(w.part) * kUnitRows + unit_row, make_float2(M, L));
            __threadfence();
            bar_sync(1, 256);
            if (tid == 32 * kSoftmaxWarp) {
                const int before = atomic_add_acq_rel_gpu(a.counters + w.first_cta, 1);
                const bool last = before == w.pieces - 1;
                if (last) st_relaxed_gpu(a.counters + w.first_cta, 0);   // as the next call finds it
                ctl_i[1] = last;
            }
            bar_sync(1, 256);
            if (ctl_i[1] && !idle) {
                __threadfence();
                float most = -INFINITY, sum = 0.f;
                for (int i = 0; i < w.pieces; ++i) most = fmaxf(most, __ldcg(a.stats + static_cast<long long>(w.part_of(i)) * kUnitRows + unit_row).x);
                const float at = most == -INFINITY ? 0.f : most;
                for (int k = k0; k < k1; ++k) {
                    float y[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) y[c] = 0.f;
                    sum = 0.f;
                    for (int i = 0; i < w.pieces; ++i) {
                        const int part = w.part_of(i);
                        const float2 st = __ldcg(a.stats + static_cast<long long>(part) * kUnitRows + unit_row);
                        const float f = exp2_approx(st.x - at);
                        sum = fmaf(st.y, f, sum);
                        const float4* from = reinterpret_cast<const float4*>(a.parts) + (static_cast<long long>(part) * (kDp / 4) + 8 * k) * kUnitRows + unit_row;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float4 v = __ldcg(from + c * kUnitRows);
                            y[4 * c] = fmaf(v.x, f, y[4 * c]), y[4 * c + 1] = fmaf(v.y, f, y[4 * c + 1]);
                            y[4 * c + 2] = fmaf(v.z, f, y[4 * c + 2]), y[4 * c + 3] = fmaf(v.w, f, y[4 * c + 3]);
                        }
                    }
                    if (!live) continue;
                    const float by = sum == 0.f ? 0.f : 1.f / sum;
                    uint16_t* to = a.out + static_cast<long long>(first + token) * a.o_ts + head * a.o_hs + 32 * k;
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        if (32 * k + c >= a.D) break;
                        float z[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e] = y[c + e] * by;
                        *reinterpret_cast<uint4*>(to + c) = pack8<BF16>(z);
                    }
                }
                if (live && a.lse && (pair || s == 0)) a.lse[static_cast<long long>(first + token) * a.Hq + head] = lse_of(most, sum);
            }
            bar_sync(1, 256);                                // (ctl_i[1] is written again)
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    // where a wait ran out, copies in flight land before the CTA goes
    if (warp == 0 && lane == 0 && *abort_flag)
        for (uint32_t i = ring.it > C::kSlots ? ring.it - C::kSlots : 0; i < ring.it; ++i)
            mbar_wait_plain(s_full + 8 * (i % C::kSlots), (i / C::kSlots) & 1, drain_limit(a.timeout_cycles));
}

template <bool BF16, int NC>
int go(const Runtime& rt, const AttnArgs& a, wq4_stream_t st) {
    using C = Cfg<NC>;
    auto kern = attention_tiles_kernel<BF16, NC>;
    static PerDevice ready;
    const int regs = ready.get(rt.device, [&]() -> int {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) == cudaSuccess &&
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) == cudaSuccess)
            return fa.numRegs;
        cudaGetLastError();
        return -1;
    });
    if (regs != 168) return WQ4_ERR_CUDA;            // the warps' shares count on the registers of the launch; with fewer they would wait
    return launch(rt, kern, dim3(a.grid), kThreads, C::kSmem, 1, st, a);
}

}  // namespace

int tiles_rows() { return kUnitRows; }
int tiles_places() { return kTile; }

int launch_attention_tiles(const Runtime& rt, const AttnArgs& a, int dtype, wq4_stream_t st) {
    if (dtype == WQ4_BF16) return a.D <= 64 ? go<true, 1>(rt, a, st) : go<true, 2>(rt, a, st);
    return a.D <= 64 ? go<false, 1>(rt, a, st) : go<false, 2>(rt, a, st);
}

}  // namespace wq4
