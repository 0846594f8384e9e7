// tl_spans.h - host checks of the calls over row-strided matrices: element types, alignment, and
// which memory a call touches.
#pragma once

#include <cstdint>

#include "../../include/tl.h"

namespace tl {

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool float_type(int dt) { return dt == TL_F32 || dt == TL_BF16 || dt == TL_F16; }
inline int64_t type_bytes(int dt) { return dt == TL_F32 ? 4 : 2; }

// Element offsets stay far from 2^63: rows < 2^31, ld < 2^40 would reach 2^71, so
// the product is bounded too.
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr int64_t kMaxSpan = int64_t(1) << 56;
// Elements of a matrix: more than any device holds, and every kernel's grid is below 2^31 CTAs up to there (of at
// least 1,024 elements each, or of whole rows).
constexpr int64_t kMaxElements = int64_t(1) << 40;
inline bool too_many(int64_t rows, int64_t cols) { return rows > 0 && cols > kMaxElements / rows; }

// The memory a call touches: no output may share bytes with anything else.
struct Spans {
    struct One {
        uintptr_t lo, hi;
        bool out;
    } v[16];
    int n = 0;
    void add(const void* p, int64_t bytes, bool out) {
        if (p == nullptr || bytes <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        v[n++] = {lo, lo + uintptr_t(bytes), out};
    }
    bool clash() const {
        for (int i = 0; i < n; ++i)
            for (int j = i + 1; j < n; ++j)
                if ((v[i].out || v[j].out) && v[i].lo < v[j].hi && v[j].lo < v[i].hi) return true;
        return false;
    }
};

inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t size) {
    return rows < 1 || cols < 1 ? 0 : ((rows - 1) * ld + cols) * size;
}

// Whether two row-strided matrices of one shape share an element without being the same one: equal strides
// interleave when their columns stay apart, others are held to disjoint spans.  The stride of a single row is
// not used (and may be anything).
inline bool rows_clash(const void* x, int64_t ldx, const void* d, int64_t ldd, int64_t rows, int64_t cols, int64_t size) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(d);
    const uintptr_t ahi = a + uintptr_t(span_bytes(rows, cols, ldx, size));
    const uintptr_t bhi = b + uintptr_t(span_bytes(rows, cols, ldd, size));
    if (a >= bhi || b >= ahi) return false;
    if (rows == 1) return a != b;
    if (ldx != ldd) return true;
    if (a == b) return false;   // in place
    const uintptr_t stride = uintptr_t(ldx * size), width = uintptr_t(cols * size);
    const uintptr_t off = (a < b ? b - a : a - b) % stride;
    return off < width || off + width > stride;
}

}  // namespace tl
