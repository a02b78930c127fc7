// Attention over a paged cache for many rows per kv head (trees of drafts, many queries to a key): the products on the tensor
// cores' own path. A row is (token i, head g of the group), r = i G + g; S = Q K^T and O += P V are tcgen05 MMAs of 128 rows
// by 128 places, with S, P (where S was) and O in tensor memory. Two threads own a row of S, 64 places each; all they tell each
// other are their maxima.
//
// Two streams of S tiles keep the tensor cores and the softmax warps busy in turn. A unit of more than 128 rows gives each stream
// 128 rows of its own and the same places (each tile of keys and values is read once for 256 rows); a
// unit of fewer gives both the same rows and every other tile of places, and the streams' O, maxima and sums are joined at
// the end. A row's maximum is taken over when it has grown by more than 2^8, 2^2 in fp16 (any reference will do for the softmax as
// long as nothing overflows), so that O is rarely scaled.
//
// Work is cut as in wq4_tree_attention.cu: equal shares of all the units' tiles, and the CTA that finishes last joins a unit.
//
// 16 trees of 32 tokens over 1000 to 8000 places, 32 heads over 8 of 128: 79 us (3.9 TB/s; memory's floor 45): a tile of 64 KB takes 2950
// cycles where memory would take 2800, and about 25 us go by before the first tile, at the joins and at the end. One
// tree of 64 tokens, 64 heads over 8, over 131000 places: 275 us (1.00 PFLOP/s, 51 % of the MMAs' rate): per stream, the
// softmax (some 1350 cycles from S to P, 700 of them exponentials) is longer than the other stream's MMAs (1040). One thread per row
// took 298 us; a thread that issues the MMAs of each stream, in place of one for both, 304; descriptors built for each MMA 300.
#include <new>

#include "wq4_attention.cuh"

namespace wq4 {
namespace {

constexpr int kTile = 128;              // places of a tile
constexpr int kLeast = 4;               // tiles worth a CTA (8 tokens over 2000 places: 19 us, with 1 26)
constexpr int kLanes = 128;             // rows of a stream's tile
constexpr int kUnitRows = 2 * kLanes;
constexpr int kSoftmaxWarp = 4;         // the first of sixteen; before them: copies, MMAs, two that look at drafted values
constexpr int kSoftmax = 512;           // their threads
constexpr int kThreads = 32 * kSoftmaxWarp + kSoftmax;
constexpr int kMaxSlots = 16;

template <int NC>
struct Cfg {
    static constexpr int kDp = 64 * NC;
    static constexpr int kSlot = kTile * kDp * 2;            // a tile's keys, or values
    static constexpr int kQ = kLanes * kDp * 2;
    static constexpr int kHead = 3 * 1024;                   // barriers, maxima
    static constexpr int kMaxSmem = 232448;                  // 227 KB
    // Ring slots beside one or two streams' Q.
    __host__ __device__ static constexpr int slots(int q) {
        const int n = (kMaxSmem - kHead - q * kQ) / kSlot;
        return n < kMaxSlots ? n : kMaxSlots;
    }
    __host__ __device__ static constexpr int smem(int q) { return kHead + q * kQ + slots(q) * kSlot; }
    static constexpr int kO = 2 * kTile;                     // tensor memory: S of both streams, then O of both
    static constexpr uint32_t kTmemCols = 512;
};

// Registers: 128 x 64 + 512 x 104 are those of the launch, 640 x 96 (a compiler that gives the kernel fewer: it does not fit).
constexpr int kFewRegs = 64, kManyRegs = 104;
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint64_t both(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
// Scores of places that are not seen.
__device__ __forceinline__ void hide(uint32_t (&x)[32], uint32_t seen) {
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (!(seen >> c & 1u)) x[c] = 0xff800000u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Operands in shared memory are named by descriptors whose upper word is the same for all of them (eight rows of 128 bytes to a
// swizzle atom, as make_sdesc_sw128 says) and whose lower word is the address in units of 16 bytes, so that the thread that
// issues the MMAs adds constants: built anew for each, they took longer than the MMAs (112 cycles each against 65).
// Values are the B operand of O = P V with the features leading: 64 features by 8 places are the atom, and the lower word also
// holds the distance from one 64 features to the next.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t rows_lo(uint32_t saddr) { return saddr >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t values_lo(uint32_t saddr, uint32_t panel) { return saddr >> 4 | panel >> 4 << 16; }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kDescHi));
    return d;
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

// A unit as the softmax warps see it: in shared memory, as their registers hold S.
struct Unit {
    int more;                                                // whether there is one
    int b, h, row0, rows, context, count, t0, n, first;      // n: tiles; first: the sequence's first row
    int pieces, first_cta, part;
    __device__ __forceinline__ bool two() const volatile { return rows - row0 > kLanes; }
    __device__ __forceinline__ int part_of(int i) const volatile { return 2 * (first_cta + i) + (i == 0 ? 1 : 0); }
};

template <bool BF16, int NC>
__global__ void __launch_bounds__(kThreads, 1) attention_tiles_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<NC>;
    constexpr int kDp = C::kDp, kPanel = kTile * 128;
    constexpr float kSlack = BF16 ? 8.f : 2.f;               // log2 of what a row's maximum may grow by before it is taken over
    constexpr float kRoom = BF16 ? 0.f : kMostLog2 - kSlack;
    // (nothing else is in shared memory, so that it starts on a swizzle's boundary: checked below)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t s_base = smem_u32(smem_raw);
    const int queries = a.max_rows > kLanes ? 2 : 1, slots = C::slots(queries);
    // the ring and Q first, on 1024-byte boundaries
    const uint32_t s_q = s_base, s_ring = s_base + queries * C::kQ;
    uint8_t* const head = smem_raw + queries * C::kQ + slots * C::kSlot;
    const uint32_t s_head = smem_u32(head);
    // barriers
    const uint32_t s_full = s_head, s_empty = s_head + 8 * kMaxSlots, s_vok = s_head + 16 * kMaxSlots;
    const uint32_t s_sfull = s_head + 24 * kMaxSlots, s_pfull = s_sfull + 16, s_ofull = s_sfull + 32, s_qfull = s_sfull + 40,
                   s_drain = s_sfull + 48, s_stall = s_sfull + 56;
    int* ctl_i = reinterpret_cast<int*>(head + 512);         // [0] abort, [1] last to finish, [2] gave up, [3] tensor memory, [4] values not finite
    volatile int* abort_flag = ctl_i;
    volatile int* bad_slot = ctl_i + 8;                      // [slots] a drafted value that is not finite was taken out
    Walk* const walk = reinterpret_cast<Walk*>(head + 640);  // (the softmax warps' own)
    Unit* const units = reinterpret_cast<Unit*>(head + 832); // [2] the unit at hand and the next
    static_assert(sizeof(Walk) <= 192 && 2 * sizeof(Unit) <= 192, "fit ahead of the maxima");
    float* s_max = reinterpret_cast<float*>(head + 1024);    // [stream][half of the places][lane]
    // at times when Q is not there: the schedule's sums, and at a unit's end [stream][half][lane] (maximum, sum)
    Scan& scan = *reinterpret_cast<Scan*>(smem_raw);
    float2* s_stat = reinterpret_cast<float2*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 32; ++i) ctl_i[i] = 0;
        for (int i = 0; i < slots; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_empty + 8 * i, 3);           // the MMAs that read it, and the two warps that look at drafted values
            mbar_init(s_vok + 8 * i, 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_sfull + 8 * s, 1);
            mbar_init(s_pfull + 8 * s, 8);
        }
        mbar_init(s_ofull, 2);
        mbar_init(s_qfull, 16);
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
    Walk w(a, kTile, kUnitRows, kLeast);
    bool work = w.begin(scan, tid, kThreads);                // (all threads of the CTA alike)
    if (s_base & 1023u) {
        if (tid == 0) atomicOr(a.status, kStatusPlacement);
        work = false;
    }
    __syncthreads();                                         // (Q comes where the schedule's sums were)
    const WaitCtl ctl{abort_flag, a.status, a.timeout_cycles};
    Ring ring(slots);
    // A unit's tiles: lag of the values behind the keys, and whether both streams have rows of their own.
    auto two = [&] { return w.rows - w.row0 > kLanes; };

    if (warp < kSoftmaxWarp) {
        fewer_registers<kFewRegs>();
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            const uint64_t pol = policy_evict_first();
            const int panel = lane % NC, box = lane / NC;
            const bool mine = lane < kTile / a.box * NC;
            bool ok = work;
            while (ok && w.next()) {
                const int n = w.t1 - w.t0, lag = two() ? 1 : 2;
                // The page of this lane's places of a tile: looked up a tile ahead of its keys and kept for its values.
                auto place_of = [&](int tile) { return (w.t0 + tile) * kTile + box * a.box; };
                auto there = [&](int tile) { return mine && tile < n && place_of(tile) < w.len; };
                auto find = [&](int tile) {
                    return there(tile) ? a.table[static_cast<long long>(w.b) * a.ld_table + place_of(tile) / a.cache.page_size] : 0;
                };
                int ahead = find(0), page[3] = {};           // of tile j + 1; of j, j - 1, j - 2
                for (int j = 0; j < n + lag && ok; ++j) {
                    page[2] = page[1], page[1] = page[0], page[0] = ahead;
                    ahead = find(j + 1);
                    if (static_cast<unsigned>(page[0]) >= static_cast<unsigned>(a.cache.pages)) atomicOr(a.status, kStatusBadIndex), page[0] = a.cache.pages;
                    if (!there(j)) page[0] = a.cache.pages;  // past the last place: outside the tensor, zeros
                    for (int kind = 0; kind < 2; ++kind) {               // 0: values of j - lag, 1: keys of j
                        if (kind ? j >= n : j < lag) continue;
                        if (lane == 0) ok = mbar_wait(s_empty + 8 * ring.slot, ring.phase ^ 1, ctl);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        const uint32_t bar = s_full + 8 * ring.slot;
                        if (lane == 0) mbar_arrive_expect_tx(bar, C::kSlot);
                        __syncwarp();
                        if (mine)
                            tma_load_5d(s_ring + ring.slot * C::kSlot + panel * kPanel + box * a.box * 128, kind ? &a.k_map : &a.v_map, bar,
                                        64 * panel, place_of(kind ? j : j - lag) % a.cache.page_size, 0, w.h,
                                        kind ? page[0] : lag == 1 ? page[1] : page[2], pol);
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
                const uint32_t k_lo = rows_lo(s_ring), v_lo = values_lo(s_ring, kPanel), q_lo = rows_lo(s_q);
                uint32_t vok_phase = 0, p_phase = 0, q_phase = 0;   // p_phase: bit s
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
#pragma unroll 1
                        for (int s = 0; s < 2; ++s) {
                            if (v >= 0 && (pair || (v & 1) == s)) {
                                if (!(ok = mbar_wait(s_pfull + 8 * s, p_phase >> s & 1u, ctl))) break;
                                p_phase ^= 1u << s;
                                tc_fence_after();
                                uint32_t from = v_lo + v_slot * (C::kSlot >> 4);
                                asm volatile("" : "+r"(from));           // (the sums below are not worth registers)
#pragma unroll
                                for (int k = 0; k < kTile / 16; ++k)
                                    mma_ts(tmem + C::kO + s * kDp, tmem + s * kTile + (k >> 2) * 64 + (k & 3) * 8, desc_of(from + k * (2048 >> 4)),
                                           kIdescO, k > 0 ? 1u : begun >> s & 1u);
                                begun |= 1u << s;
                            }
                            if (j < n && (pair || (j & 1) == s)) {
                                uint32_t q = q_lo + (pair ? s * (C::kQ >> 4) : 0), from = k_lo + k_slot * (C::kSlot >> 4);
                                asm volatile("" : "+r"(q), "+r"(from));
#pragma unroll
                                for (int k = 0; k < 4 * NC; ++k) {
                                    constexpr int kStep = kPanel >> 4;
                                    if (k < ksteps)
                                        mma_ss(tmem + s * kTile, desc_of(q + (k >> 2) * kStep + (k & 3) * 2), desc_of(from + (k >> 2) * kStep + (k & 3) * 2),
                                               kIdescS, k > 0);
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
                            uint8_t* slot = smem_raw + (s_ring - s_base) + ring.slot * C::kSlot;
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
        more_registers<kManyRegs>();
        // ---------------------------------------------------------------- softmax
        // Two threads to a row of S, each with 64 places; they tell each other their maxima.
        const int s = (warp - kSoftmaxWarp) >> 3, half = warp >> 2 & 1, row = (warp & 3) * 32 + lane;
        const uint32_t t_lanes = tmem + (static_cast<uint32_t>(row & ~31) << 16);
        const uint32_t max_at = smem_u32(s_max) + ((s * 2 + half) * kLanes + row) * 4;       // (the other's: 4 kLanes bytes across)
        uint32_t s_phase = 0, o_phase = 0;
        bool dead = false;
        if (a.test_stall && work && tid == 32 * kSoftmaxWarp) mbar_wait(s_stall, 0, ctl);   // (tests: nothing arrives there)
        // This thread's row of a unit's problem (past its rows: the last one's token and head, for loads alone), found anew where it is
        // needed: the registers are S's.
        auto row_of = [&](const volatile Unit* u) {
            int at = row;
            asm volatile("" : "+r"(at));
            return u->row0 + (u->two() ? s * kLanes : 0) + at;
        };
        auto token_of = [&](const volatile Unit* u) { return min(row_of(u), u->rows - 1) / a.G; };
        auto head_of = [&](const volatile Unit* u, int token) { return u->h * a.G + min(row_of(u), u->rows - 1) - token * a.G; };
        const bool leads = tid == 32 * kSoftmaxWarp;
        auto describe = [&](Unit& u) {                       // (the leading thread)
            Walk& v = *walk;
            u.more = v.next();
            if (!u.more) return;
            u.b = v.b, u.h = v.h, u.row0 = v.row0, u.rows = v.rows, u.context = v.context, u.count = v.count;
            u.t0 = v.t0, u.n = v.t1 - v.t0, u.first = a.starts[v.b];
            u.pieces = v.pieces, u.first_cta = v.first_cta, u.part = v.part;
        };
        if (leads) {
            units[0].more = 0;
            if (work) {
                new (walk) Walk(w);
                describe(units[0]);
            }
        }
        bar_sync(1, kSoftmax);
        for (const volatile Unit* u = units; u->more; u = u == units ? units + 1 : units) {
            const bool pair = u->two();
            const bool idle = u->row0 + (pair ? s * kLanes : 0) + (row & ~31) >= u->rows;
            // ---- this thread's part of its row of Q: a half, a quarter where the streams share rows
            {
                const bool live = row_of(u) < u->rows;
                const int token = token_of(u), head = head_of(u, token);
                const uint16_t* from = a.q + static_cast<long long>(u->first + token) * a.q_ts + head * a.q_hs;
                const uint32_t to = s_q + (pair ? s * C::kQ : 0) + row * 128;
                constexpr int kAll = NC * 8;                 // 16-byte pieces of a row
                const int c0 = pair ? half * (kAll / 2) : (2 * s + half) * (kAll / 4), c1 = c0 + (pair ? kAll / 2 : kAll / 4);
#pragma unroll 4
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
            if (leads) describe(units[u == units]);          // (the next one, seen by all after the barriers below)
            float ref = -INFINITY, l = 0.f;
            bool begun = false;
            for (int j = pair ? 0 : s; j < u->n; j += pair ? 1 : 2) {
                if (!dead) {
                    const bool ok = mbar_wait(s_sfull + 8 * s, s_phase, ctl);
                    dead = !__all_sync(0xffffffffu, ok);
                }
                s_phase ^= 1;
                if (!idle) {                                 // (a warp that gave up goes on, as the one it meets may)
                    tc_fence_after();
                    // S is read twice, 32 places at a time: for the maxima and for the probabilities. (Held in registers in between, it pushes
                    // others out to local memory, whose loads miss the small L1 beside 227 KB of shared memory: 7000 cycles a tile.)
                    const uint32_t t_s = t_lanes + s * kTile + 64 * half;
                    const int place0 = (u->t0 + j) * kTile + 64 * half;
                    const bool tail = place0 + 64 > u->context;
                    uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
                    if (tail) {
                        const int tok = token_of(u);
#pragma unroll
                        for (int k = 0; k < 2; ++k) seen[k] = seen32(a, u->first + tok, tok, place0 + 32 * k - u->context, u->count);
                    }
                    float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t x[32];
                        tmem_ld32(t_s + 32 * k, x);
                        tmem_ld_wait();
                        if (tail) hide(x, seen[k]);
#pragma unroll
                        for (int c = 0; c < 32; c += 8) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) top4[e] = max3(top4[e], __uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]));
                        }
                    }
                    float top = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]) * a.scale_log2;
                    // (read by the other warp before this stream's next S is there)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(max_at), "f"(top) : "memory");
                    bar_sync(2 + s * 4 + (warp & 3), 64);
                    float other;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(max_at ^ (4 * kLanes)) : "memory");
                    top = fmaxf(top, other) - kRoom;
                    const bool grows = top > ref + kSlack || (ref == -INFINITY && top > ref);
                    if (__any_sync(0xffffffffu, grows)) {
                        const float now = grows ? top : ref;
                        const float keep = ref == -INFINITY ? 0.f : exp2_approx(ref - now);
                        ref = now;
                        l *= keep;
                        if (begun) {                         // (the MMAs of the tiles before have ended: S came after them)
#pragma unroll 1
                            for (int k = 0; k < kDp / 64; ++k) {
                                const uint32_t at = t_lanes + C::kO + s * kDp + half * (kDp / 2) + 32 * k;
                                uint32_t o[32];
                                tmem_ld32(at, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * keep);
                                tmem_st16(at, reinterpret_cast<const uint32_t(&)[16]>(o[0]));
                                tmem_st16(at + 16, reinterpret_cast<const uint32_t(&)[16]>(o[16]));
                            }
                        }
                    }
                    const float minus = ref == -INFINITY ? 0.f : -ref;
                    const uint64_t scale2 = both(a.scale_log2, a.scale_log2), minus2 = both(minus, minus);
                    uint64_t sum2[2] = {0, 0};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t x[32], p[16];
                        tmem_ld32(t_s + 32 * k, x);
                        tmem_ld_wait();
                        if (tail) hide(x, seen[k]);
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            uint64_t d;
                            asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(both(__uint_as_float(x[c]), __uint_as_float(x[c + 1]))), "l"(scale2), "l"(minus2));
                            float e0, e1;
                            asm("mov.b64 {%0, %1}, %2;" : "=f"(e0), "=f"(e1) : "l"(d));
                            e0 = exp2_approx(e0), e1 = exp2_approx(e1);
                            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum2[c >> 1 & 1]) : "l"(both(e0, e1)));
                            p[c / 2] = pack2<BF16>(e0, e1);
                        }
                        tmem_st16(t_s + 16 * k, p);          // (where S has been read)
                    }
                    float l4[4];
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(l4[0]), "=f"(l4[1]) : "l"(sum2[0]));
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(l4[2]), "=f"(l4[3]) : "l"(sum2[1]));
                    l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
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
            s_stat[(s * 2 + half) * kLanes + row] = make_float2(ref, l);         // (Q has been read: O is there)
            if (tid == 32 * kSoftmaxWarp) ctl_i[2] = *abort_flag;
            bar_sync(1, kSoftmax);
            if (ctl_i[2]) break;                             // (all these threads alike)
            // ---- join the halves' sums, and the streams where they share rows; each thread then has a part of the row's columns
            const float2 h0 = s_stat[(pair ? s * 2 : 0) * kLanes + row], h1 = s_stat[((pair ? s * 2 : 0) + 1) * kLanes + row];
            float M = h0.x, L = h0.y + h1.y, f0 = 1.f, f1 = 1.f;
            if (!pair) {
                const float2 g0 = s_stat[2 * kLanes + row], g1 = s_stat[3 * kLanes + row];
                M = fmaxf(h0.x, g0.x);
                const float at = M == -INFINITY ? 0.f : M;
                f0 = exp2_approx(h0.x - at);
                f1 = exp2_approx(g0.x - at);
                L = L * f0 + (g0.y + g1.y) * f1;
            }
            const bool live = row_of(u) < u->rows;
            const int token = token_of(u), head = head_of(u, token);
            const bool bad = ctl_i[4], whole = u->pieces == 1;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int k0 = pair ? half * (kDp / 32) : (2 * s + half) * (kDp / 64), k1 = k0 + (pair ? kDp / 32 : kDp / 64);     // in sixteens
            const int unit_row = (pair ? s * kLanes : 0) + row;
            const bool tells = half == 0 && (pair || s == 0);            // of the threads with a row, the one that writes its lse
            uint16_t* const out = a.out + static_cast<long long>(u->first + token) * a.o_ts + head * a.o_hs;
            auto store16 = [&](int k, const float (&y)[16], float by) {
#pragma unroll
                for (int c = 0; c < 16; c += 8) {
                    if (16 * k + c >= a.D) break;
                    float z[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] = y[c + e] * by;
                    *reinterpret_cast<uint4*>(out + 16 * k + c) = pack8<BF16>(z);
                }
            };
            if (!idle) {
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {
                    uint32_t o[16];
                    float y[16];
                    tmem_ld16(t_lanes + C::kO + (pair ? s * kDp : 0) + 16 * k, o);
                    if (!pair && u->n > 1) {
                        uint32_t o1[16];
                        tmem_ld16(t_lanes + C::kO + kDp + 16 * k, o1);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 16; ++c) y[c] = __uint_as_float(o[c]) * f0 + __uint_as_float(o1[c]) * f1;
                    } else {
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 16; ++c) y[c] = __uint_as_float(o[c]);
                    }
                    if (bad && live) {
                        const int lo = max(0, u->t0 * kTile - u->context), hi = min(u->count, (u->t0 + u->n) * kTile - u->context);
#pragma unroll 1
                        for (int j = lo; j < hi; ++j) {
                            const int place = u->context + j, i = place / a.cache.page_size;
                            if (!a.sees(u->first + token, token, place, u->context, u->count)) continue;
                            const int page = a.table[static_cast<long long>(u->b) * a.ld_table + i];
                            if (page < 0 || page >= a.cache.pages) continue;
                            const uint16_t* v = a.cache.v + page * a.cache.v_page + (place - i * a.cache.page_size) * a.cache.v_token +
                                                u->h * a.cache.v_head + 16 * k;
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (16 * k + c < a.D && not_finite<BF16>(v[c]) & 1u) y[c] += to_f32<BF16>(v[c]);
                        }
                    }
                    if (whole) {
                        if (live) store16(k, y, inv);
                    } else {
                        float4* to = reinterpret_cast<float4*>(a.parts) + (static_cast<long long>(u->part) * (kDp / 4) + 4 * k) * kUnitRows + unit_row;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            __stcg(to + c * kUnitRows, make_float4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]));
                    }
                }
            }
            if (whole) {
                if (live && a.lse && tells) a.lse[static_cast<long long>(u->first + token) * a.Hq + head] = lse_of(M, L);
                bar_sync(1, kSoftmax);                       // (s_stat, where Q comes, and ctl_i[2] are written again)
                continue;
            }
            if (tells) __stcg(a.stats + static_cast<long long>(u->part) * kUnitRows + unit_row, make_float2(M, L));
            bar_sync(1, kSoftmax);
            if (tid == 32 * kSoftmaxWarp) {
                __threadfence();                             // (what the others wrote ahead of the barrier goes with it)
                const int before = atomic_add_acq_rel_gpu(a.counters + u->first_cta, 1);
                const bool last = before == u->pieces - 1;
                if (last) st_relaxed_gpu(a.counters + u->first_cta, 0);   // as the next call finds it
                ctl_i[1] = last;
            }
            bar_sync(1, kSoftmax);
            if (ctl_i[1] && !idle) {
                float most = -INFINITY, sum = 0.f;
#pragma unroll 4
                for (int i = 0; i < u->pieces; ++i) most = fmaxf(most, __ldcg(a.stats + static_cast<long long>(u->part_of(i)) * kUnitRows + unit_row).x);
                const float at = most == -INFINITY ? 0.f : most;
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {
                    float y[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) y[c] = 0.f;
                    sum = 0.f;
#pragma unroll 2
                    for (int i = 0; i < u->pieces; ++i) {
                        const int part = u->part_of(i);
                        const float2 st = __ldcg(a.stats + static_cast<long long>(part) * kUnitRows + unit_row);
                        const float4* from = reinterpret_cast<const float4*>(a.parts) + (static_cast<long long>(part) * (kDp / 4) + 4 * k) * kUnitRows + unit_row;
                        float4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[c] = __ldcg(from + c * kUnitRows);
                        const float f = exp2_approx(st.x - at);
                        sum = fmaf(st.y, f, sum);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            y[4 * c] = fmaf(v[c].x, f, y[4 * c]), y[4 * c + 1] = fmaf(v[c].y, f, y[4 * c + 1]);
                            y[4 * c + 2] = fmaf(v[c].z, f, y[4 * c + 2]), y[4 * c + 3] = fmaf(v[c].w, f, y[4 * c + 3]);
                        }
                    }
                    if (live) store16(k, y, sum == 0.f ? 0.f : 1.f / sum);
                }
                if (live && a.lse && tells) a.lse[static_cast<long long>(u->first + token) * a.Hq + head] = lse_of(most, sum);
            }
            bar_sync(1, kSoftmax);                           // (ctl_i[1] is written again)
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
        for (uint32_t i = ring.it > static_cast<uint32_t>(slots) ? ring.it - slots : 0; i < ring.it; ++i)
            mbar_wait_plain(s_full + 8 * (i % slots), (i / slots) & 1, drain_limit(a.timeout_cycles));
}

// Whether the kernel can run: its warps' shares count on the registers of the launch, with fewer they would wait.
template <bool BF16, int NC>
bool fits(const Runtime& rt) {
    auto kern = attention_tiles_kernel<BF16, NC>;
    static PerDevice ready;
    return ready.get(rt.device, [&]() -> int {       // 1: it can, 2: it cannot
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) == cudaSuccess &&
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NC>::kMaxSmem) == cudaSuccess)
            return check::registers_cover(fa.numRegs, kThreads, 32 * kSoftmaxWarp * kFewRegs + kSoftmax * kManyRegs) ? 1 : 2;
        cudaGetLastError();
        return -1;
    }) == 1;
}

template <bool BF16, int NC>
int go(const Runtime& rt, const AttnArgs& a, wq4_stream_t st) {
    return launch(rt, attention_tiles_kernel<BF16, NC>, dim3(a.grid), kThreads, Cfg<NC>::smem(a.max_rows > kLanes ? 2 : 1), 1, st, a);
}

}  // namespace

int tiles_rows() { return kUnitRows; }
int tiles_places() { return kTile; }

bool attention_tiles_fit(const Runtime& rt, int dtype, int D) {
    if (dtype == WQ4_BF16) return D <= 64 ? fits<true, 1>(rt) : fits<true, 2>(rt);
    return D <= 64 ? fits<false, 1>(rt) : fits<false, 2>(rt);
}

int launch_attention_tiles(const Runtime& rt, const AttnArgs& a, int dtype, wq4_stream_t st) {
    if (dtype == WQ4_BF16) return a.D <= 64 ? go<true, 1>(rt, a, st) : go<true, 2>(rt, a, st);
    return a.D <= 64 ? go<false, 1>(rt, a, st) : go<false, 2>(rt, a, st);
}

}  // namespace wq4
