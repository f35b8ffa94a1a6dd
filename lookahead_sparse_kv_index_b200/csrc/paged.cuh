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

// Memory that a call reads or writes, for the checks on the host that refuse outputs over other operands.
struct Span {
    const void *p;
    int64_t bytes;
    const char *name;
};
inline bool meet(const Span &a, const Span &b) {
    const int64_t x = int64_t(reinterpret_cast<uintptr_t>(a.p)), y = int64_t(reinterpret_cast<uintptr_t>(b.p));
    return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
// The bytes from a cache's first row to its last, of K as of V, and of its scales.
inline int64_t row_span(const lsa_page_cache &c) {
    return ((c.n_pages - 1) * c.page_stride + (c.page_size - 1) * c.slot_stride + (c.Hkv - 1) * c.head_stride + c.D) *
           int64_t(elem_size(c.dtype));
}
// The bytes from a table's first row to its last (more than any memory has: 2^60).
inline int64_t table_span(int64_t rows, int64_t stride, int64_t width) {
    const int64_t most = int64_t(1) << 60;
    return rows - 1 > most / 4 / stride ? most : ((rows - 1) * stride + width) * 4;
}
inline int64_t scale_span(const lsa_page_cache &c) { return c.n_pages * c.page_size * c.Hkv * 4; }

// Validates a cache descriptor on the host (`who`: the entry point, for the message).
lsa_status check_cache(const lsa_page_cache *c, const char *who);

}  // namespace paged
}  // namespace lsa
