// What the attention kernels share: their arguments, how the work is cut, copies of cache tiles, and small pieces of arithmetic.
#pragma once

#include <cmath>

#include "wq4_cache.cuh"

namespace wq4 {

struct AttnArgs {
    CUtensorMap k_map, v_map;           // (feature, place in the page, panel of 64 features, head, page)
    const uint16_t* q;
    uint16_t* out;
    float* lse;                         // null where not asked for
    const int *table, *starts, *context;
    const unsigned long long* mask;     // null: each token sees those before it and itself
    CacheArgs cache;
    long long q_ts, q_hs, o_ts, o_hs;
    int ld_table, table_width, mask_words;
    int B, T, max_tokens, Hq, Hk, G, D;
    int max_rows;                       // max_tokens G, or as many as matter
    int box, copies;                    // places of one copy; copies of a box's panels
    int grid;                           // CTAs
    float scale_log2;
    int* counters;                      // [grid] parts that have come, of the unit whose first part is the CTA's
    float2* stats;                      // [2 grid][rows] (maximum, sum)
    float* parts;                       // [2 grid][rows x padded D]
    unsigned int* status;
    long long timeout_cycles;
    int test_stall;

    // Whether token `i` of a sequence (row t of the arrays) sees a place.
    __device__ __forceinline__ bool sees(int t, int i, int place, int ctx, int count) const {
        const int j = place - ctx;
        if (j < 0) return true;
        if (j >= count) return false;
        return mask ? mask[static_cast<long long>(t) * mask_words + (j >> 6)] >> (j & 63) & 1u : j <= i;
    }
};

// Probabilities are rounded to the values' type, as the tensor cores' products read both operands in one type (an fp32 P would
// take two products each; its half step is what the result's own rounding has too). Their sum is taken ahead of that, in fp32. fp16
// has 2^-14 as its least normal number, and a long context may put much of a row's weight on places below that: the
// softmax's reference lies so far below the row's maximum that P reaches 2^15 at most, 2^13 at least, and sum and O carry the
// same factor. (P of the maximum itself is a power of two, as it is without: where one place has nearly all of the weight, its
// rounding is nearly all of the error.) What lies 2^-27 and more below the row's largest loses bits, 2^-38 below it vanishes.
// bf16 has fp32's range and needs no room.
constexpr float kMostLog2 = 15.f;

constexpr int kMostPlaces = 1 << 30;    // of a sequence: sums of a place and a tile stay in 32 bits

struct Scan {
    unsigned long long sum[32], part[32], before;
    int longest[32], b;
};

// The work in order: sequence, kv head, tile of `rows` rows, tile of `places` places. A CTA walks over its share, unit by unit
// (one sequence, kv head and tile of rows); every role of the CTA does so by itself, from the same start.
struct Walk {
    const AttnArgs& a;
    const int places, unit_rows, least;              // least: tiles that are worth a CTA, where a unit has as many
    // the unit at hand
    int b, h, row0, rows, context, count, len;       // rows: of the whole problem (count G); len: places
    int t0, t1;                                      // this CTA's tiles of it
    int pieces, first_cta, part;                     // CTAs that share it, the first of them, where this one's part goes
    // the walk
    unsigned pos, end, chunk, base, work;            // base, work: of the sequence at hand
    int tiles, row_tiles, cta;

    __device__ Walk(const AttnArgs& args, int places_, int rows_, int least_) : a(args), places(places_), unit_rows(rows_), least(least_) {}

    // Sequence i's lengths; its number of tiles, 0 where there is nothing to do or the lengths cannot be.
    __device__ __forceinline__ unsigned long long load(int i, int& n, int& c) const {
        const int s0 = a.starts[i], s1 = a.starts[i + 1];
        c = a.context[i];
        n = static_cast<int>(static_cast<unsigned>(s1) - static_cast<unsigned>(s0));
        if (s0 < 0 || s1 < s0 || s1 > a.T || n > a.max_tokens || c < 0 ||
            (n > 0 && (c > kMostPlaces - n || c + n > static_cast<long long>(a.table_width) * a.cache.page_size))) {
            atomicOr(a.status, kStatusBadIndex);
            n = 0;
        }
        if (n == 0) return 0;
        const unsigned long long rt = (static_cast<long long>(n) * a.G + unit_rows - 1) / unit_rows;
        return rt * a.Hk * ((static_cast<unsigned>(c) + n + places - 1) / places);
    }

    // Finds this CTA's share; false where there is none. Every thread of the CTA calls it.
    __device__ bool begin(Scan& sc, int tid, int threads) {
        const int lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
        int n, c;
        auto scan = [&](unsigned long long x) {      // up to and with this lane's
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            return x;
        };
        // the sum of what each thread loads of all sequences; with no more of those than threads, their running sum too
        unsigned long long own = 0, mine = 0;
        int longest = 0;                             // tiles of a unit
        for (int i = tid; i < a.B; i += threads) {
            own = load(i, n, c);
            mine += own;
            if (own) longest = max(longest, static_cast<int>((static_cast<unsigned>(c) + n + places - 1) / places));
        }
        const unsigned long long upto = scan(mine);
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 31) sc.sum[warp] = upto, sc.longest[warp] = longest;
        __syncthreads();
        unsigned long long total = 0, ahead = 0;
        for (int i = 0; i < warps; ++i) {
            if (i == warp) ahead = total;
            total += sc.sum[i];
            longest = max(longest, sc.longest[i]);
        }
        if (total > 0x7fffffffull) {
            if (tid == 0) atomicOr(a.status, kStatusBadIndex);
            return false;
        }
        cta = blockIdx.x;
        chunk = max((static_cast<unsigned>(total) + a.grid - 1) / a.grid, static_cast<unsigned>(min(least, longest)));
        const unsigned long long lo = static_cast<unsigned long long>(cta) * chunk;
        if (lo >= total) return false;
        if (a.B <= threads) {
            if (ahead + upto - own <= lo && lo < ahead + upto) {
                sc.b = tid;
                sc.before = ahead + upto - own;
            }
        } else {
            unsigned long long carry = 0;
            for (int at = 0; at < a.B && carry <= lo; at += threads) {
                const unsigned long long x = at + tid < a.B ? load(at + tid, n, c) : 0, up = scan(x);
                if (lane == 31) sc.part[warp] = up;
                __syncthreads();
                unsigned long long before = carry;
                for (int i = 0; i < warps; ++i) {
                    if (i < warp) before += sc.part[i];
                    carry += sc.part[i];
                }
                if (before + up - x <= lo && lo < before + up) {
                    sc.b = at + tid;
                    sc.before = before + up - x;
                }
                __syncthreads();
            }
        }
        __syncthreads();
        pos = static_cast<unsigned>(lo);
        end = static_cast<unsigned>(min(total, lo + chunk));
        base = static_cast<unsigned>(sc.before);
        enter(sc.b);
        return true;
    }

    __device__ __forceinline__ void enter(int i) {
        b = i;
        work = static_cast<unsigned>(load(i, count, context));
        rows = count * a.G;
        len = context + count;
        tiles = (len + places - 1) / places;
        row_tiles = (rows + unit_rows - 1) / unit_rows;
    }

    // The next unit, or false at the end of the share.
    __device__ bool next() {
        if (pos >= end) return false;
        while (pos - base >= work) {
            base += work;
            enter(b + 1);
        }
        const unsigned off = pos - base, u = off / tiles;
        t0 = static_cast<int>(off - u * tiles);
        t1 = min(tiles, t0 + static_cast<int>(end - pos));
        h = static_cast<int>(u / row_tiles);
        row0 = static_cast<int>(u - h * row_tiles) * unit_rows;
        const unsigned from = pos - t0;
        first_cta = static_cast<int>(from / chunk);
        pieces = static_cast<int>((from + tiles - 1) / chunk) - first_cta + 1;
        part = 2 * cta + (cta == first_cta ? 1 : 0);
        pos += t1 - t0;
        return true;
    }

    // Where piece i of the unit lies. A CTA has two places: of the unit that it begins, and of the one it goes on with.
    __device__ __forceinline__ int part_of(int i) const { return 2 * (first_cta + i) + (i == 0 ? 1 : 0); }
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x0, int x1, int x2, int x3,
                                            int x4, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(x4), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// 2^x to 2^-22 (0 for -inf)
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log sum exp from the maximum of the scaled scores (base 2) and the sum
__device__ __forceinline__ float lse_of(float M, float L) {
    return L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// All bits of each half of a pair of places' values where the place is below len.
__device__ __forceinline__ uint32_t pair_mask(int place, int len) {
    return (place < len ? 0xffffu : 0u) | (place + 1 < len ? 0xffff0000u : 0u);
}

// 1.0 in the low and high half by bits 0 and 1.
template <bool BF16>
__device__ __forceinline__ uint32_t ones(uint32_t bits) {
    constexpr uint32_t one = BF16 ? 0x3f80u : 0x3c00u;
    return (bits & 1u ? one : 0u) | (bits & 2u ? one << 16 : 0u);
}

// Non-zero where a half is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t u) {
    constexpr uint32_t top = BF16 ? 0x7f80u : 0x7c00u;
    return ((u & top) == top ? 1u : 0u) | ((u & top << 16) == top << 16 ? 2u : 0u);
}

// Takes what is not finite out of a pair of values: 1.0 into `up` for +inf, into `down` for -inf, into both for NaN.
template <bool BF16>
__device__ __forceinline__ void split_bad(uint32_t& u, uint32_t& up, uint32_t& down) {
    constexpr uint32_t top = BF16 ? 0x7f80u : 0x7c00u, one = BF16 ? 0x3f80u : 0x3c00u;
    up = down = 0;
#pragma unroll
    for (int s = 0; s < 32; s += 16) {
        const uint32_t x = (u >> s) & 0xffffu;
        if ((x & top) != top) continue;
        const bool nan = (x & 0x7fffu) != top;
        if (nan || !(x & 0x8000u)) up |= one << s;
        if (nan || (x & 0x8000u)) down |= one << s;
        u &= ~(0xffffu << s);
    }
}

// The tensor map of a cache's keys or values: boxes of `box` places by `panels` panels of 64 features, swizzled
// by 128 bytes. One panel: boxes start at any multiple of 64 features and read zeros past D.
inline bool encode_cache(EncodeTiledFn fn, CUtensorMap* map, int dtype, void* p, int D, long long token, long long head,
                         long long page, const wq4_kv_cache& c, int heads, int box, int panels) {
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(panels > 1 ? 64 : D), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(panels), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[4] = {static_cast<cuuint64_t>(token) * 2, 128, static_cast<cuuint64_t>(head) * 2,
                                   static_cast<cuuint64_t>(page) * 2};
    const cuuint32_t boxes[5] = {64, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(panels), 1, 1};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return fn(map, dtype == WQ4_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, p, dims, strides,
              boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel for many rows per kv head (wq4_attention_tiles.cu): D <= 128, scale above 0.
int tiles_rows();                       // rows of a unit
int tiles_places();                     // places of a tile
bool attention_tiles_fit(const Runtime& rt, int dtype, int D);   // whether it can be launched; ahead of the call below
int launch_attention_tiles(const Runtime& rt, const AttnArgs& a, int dtype, wq4_stream_t st);

}  // namespace wq4
