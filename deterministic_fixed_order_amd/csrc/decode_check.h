// decode_check.h -- what the host checks of the decode-step operators share:
// limits, what plans go by, alignment, the extents of strided buffers and whether two meet.
// Host only; nothing here touches the device.
#ifndef DETFOLD_DECODE_CHECK_H
#define DETFOLD_DECODE_CHECK_H

#include <cstdint>

#include "decode.h"
#include "internal.h"

namespace detfold_impl {

constexpr int64_t kMaxCount = (int64_t)1 << 31;   // counts that the kernels hold in 32 bits
constexpr int64_t kMaxElems = (int64_t)1 << 46;   // extent of one buffer, in elements
constexpr int32_t kMaxHeads = 1 << 16;

// What the plans of the attention go by.
constexpr int64_t kWavesPerCu = 8;                // of the attention, resident
constexpr int64_t kShortRow = 512;                // tokens that are not worth cutting where rows fill the device
// Of the cache, read in a step of 64 tokens: with less, or with products in
// float32 from narrower values, a compute unit takes 8 waves instead of 4 (heads
// of 64 bfloat16 27.7 us instead of 28.3; bfloat16 to float32 194 instead of 230).
constexpr int64_t kStepBytes = 32768;
constexpr int64_t kMaxEven = 4096;                // rows that every workgroup adds up the lengths of
constexpr int64_t kLongPart = 8192;               // tokens of a part where there are more rows

inline bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// The elements a strided [n0][n1]...[last] buffer spans, or -1 where a stride
// is negative or the span passes kMaxElems.  n >= 1 each.
inline int64_t span(const int64_t (*dims)[2], int count, int64_t last)
{
    int64_t e = last;
    for (int i = 0; i < count; ++i) {
        const int64_t n = dims[i][0], s = dims[i][1];
        if (s < 0 || (n > 1 && s > kMaxElems / (n - 1)))
            return -1;
        e += (n - 1) * s;
        if (e > kMaxElems)
            return -1;
    }
    return e;
}

inline int64_t span2(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t last)
{
    const int64_t d[2][2] = {{n0, s0}, {n1, s1}};
    return span(d, 2, last);
}

// Whether a written [n0][n1][last] buffer has no element twice.
inline bool distinct(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t last)
{
    if (n0 > 1 && n1 > 1)
        return s0 >= s1 ? s1 >= last && s0 >= (n1 - 1) * s1 + last : s0 >= last && s1 >= (n0 - 1) * s0 + last;
    return n1 > 1 ? s1 >= last : n0 <= 1 || s0 >= last;
}

struct Range {
    uintptr_t p;
    uint64_t bytes;
};

inline Range range(const void *p, int64_t elems, int size) { return {(uintptr_t)p, p ? (uint64_t)elems * (uint64_t)size : 0}; }
inline bool meet(const Range &a, const Range &b) { return ranges_overlap(a.p, a.bytes, b.p, b.bytes); }

inline int64_t cache_span(const detfold_paged_cache &c, bool values)
{
    const int64_t d[3][2] = {{c.pages, values ? c.v_page : c.k_page},
                             {c.page, values ? c.v_token : c.k_token},
                             {c.heads, values ? c.v_head : c.k_head}};
    return span(d, 3, values ? c.v_dim : c.dim);
}

inline Range cache_range(const detfold_paged_cache &c, bool values)
{
    return range(values ? c.v : c.k, cache_span(c, values), elem_size(c.type));
}

}  // namespace detfold_impl

#endif  // DETFOLD_DECODE_CHECK_H
