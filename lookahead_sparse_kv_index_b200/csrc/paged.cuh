// Shared pieces of the paged-cache operators (attention over pages, the append of a step's heads, the pages' books).
#pragma once

#include "lsa_internal.cuh"

namespace lsa {
namespace paged {

// What the kernels need of an lsa_page_cache: strides in bytes.
struct CacheView {
    uint8_t *k, *v;
    float *ks, *vs;          // e4m3 row scales, else null
    int64_t page_stride, slot_stride, head_stride;
    int64_t n_pages;
    int32_t page_size, Hkv, D;
};

inline CacheView view_of(const lsa_page_cache &c) {
    const int64_t e = int64_t(elem_size(c.dtype));
    return CacheView{static_cast<uint8_t *>(c.k), static_cast<uint8_t *>(c.v), c.k_scale, c.v_scale,
                     c.page_stride * e, c.slot_stride * e, c.head_stride * e, c.n_pages,
                     c.page_size, c.Hkv, c.D};
}

// a / b for a, b >= 0.  Counts of work fit 32 bits in all but the largest calls, and a 64-bit division is a hundred
// instructions that every CTA would fetch before its first load.
__device__ __noinline__ inline int64_t div64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t div_units(int64_t a, int64_t b) {
    return uint64_t(a | b) >> 32 ? div64(a, b) : int64_t(uint32_t(a) / uint32_t(b));
}

// Validates a cache descriptor on the host (`who`: the entry point, for the message).
lsa_status check_cache(const lsa_page_cache *c, const char *who);

}  // namespace paged
}  // namespace lsa
