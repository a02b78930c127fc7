// What the operators round attention share: the paged cache as the kernels see it, 16-bit vectors, and argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "wq4_device.cuh"
#include "wq4_runtime.h"

namespace wq4 {

// 16-bit elements to fp32 and back (nearest even).
template <bool BF16>
__device__ __forceinline__ float to_f32(uint32_t b16) {
    if constexpr (BF16) return __uint_as_float(b16 << 16);
    else return __half2float(__ushort_as_half(static_cast<uint16_t>(b16)));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t u;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    return u;
}
template <bool BF16>
__device__ __forceinline__ uint16_t to_16(float x) {
    return static_cast<uint16_t>(pack2<BF16>(x, 0.f));
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& x, float (&v)[8]) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = to_f32<BF16>(u[j] & 0xffffu);
        v[2 * j + 1] = BF16 ? __uint_as_float(u[j] & 0xffff0000u) : to_f32<BF16>(u[j] >> 16);
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
}

// A wq4_kv_cache in a kernel. A slot is page * page_size + the token's place in the page.
struct CacheArgs {
    uint16_t *k, *v;
    long long k_page, k_token, k_head, v_page, v_token, v_head;
    int pages, page_size;

    CacheArgs() = default;
    explicit CacheArgs(const wq4_kv_cache& c)
        : k(static_cast<uint16_t*>(c.k)), v(static_cast<uint16_t*>(c.v)), k_page(c.k_page), k_token(c.k_token),
          k_head(c.k_head), v_page(c.v_page), v_token(c.v_token), v_head(c.v_head), pages(c.pages), page_size(c.page_size) {}
    __device__ __forceinline__ uint16_t* k_at(unsigned slot, int head) const {
        const unsigned page = slot / static_cast<unsigned>(page_size), at = slot - page * page_size;
        return k + page * k_page + at * k_token + head * k_head;
    }
    __device__ __forceinline__ uint16_t* v_at(unsigned slot, int head) const {
        const unsigned page = slot / static_cast<unsigned>(page_size), at = slot - page * page_size;
        return v + page * v_page + at * v_token + head * v_head;
    }
};

// Strides in elements of `rows` x `heads` rows of D elements, none of which may lie across another.
inline bool strides_ok(long long token, long long head, int rows, int heads, int D) {
    constexpr long long kMost = 1LL << 40;           // (products of a stride and an index stay in 64 bits)
    if (token > kMost || head > kMost) return false;
    return heads == 0 || (token >= D && head >= D);
}

// A stride of a dimension of one is never used: it becomes that of a padded row, which every rule allows.
inline void unused_stride(long long& stride, long long size, int D) {
    if (size <= 1) stride = (D + 7) / 8 * 8;
}

// Checks a cache of heads of D elements; strides that are never used are replaced.
inline int check_cache(wq4_kv_cache& c, int heads, int D) {
    unused_stride(c.k_page, c.pages, D), unused_stride(c.k_token, c.page_size, D), unused_stride(c.k_head, heads, D);
    unused_stride(c.v_page, c.pages, D), unused_stride(c.v_token, c.page_size, D), unused_stride(c.v_head, heads, D);
    if (!c.k || !c.v || c.pages < 1 || c.page_size < 1) return WQ4_ERR_INVALID;
    if (static_cast<long long>(c.pages) * c.page_size > 0x7fffffffLL) return WQ4_ERR_UNSUPPORTED;
    if (!strides_ok(c.k_token, c.k_head, c.page_size, heads, D) || !strides_ok(c.v_token, c.v_head, c.page_size, heads, D) ||
        !strides_ok(c.k_page, c.v_page, c.pages, c.pages, D))
        return WQ4_ERR_INVALID;
    if (!aligned_to(c.k, 2) || !aligned_to(c.v, 2)) return WQ4_ERR_ALIGN;
    return WQ4_OK;
}

}  // namespace wq4
