// ndq_overlap.h -- which memory of a call's arguments overlaps, for the host
// checks.  Not part of the public ABI.
#pragma once

#include <cstdint>

namespace ndq {

// `rows` pieces of `bytes` each, one every `stride` bytes.
struct Rows {
    const void* p;
    int64_t bytes;
    int64_t rows = 1;
    int64_t stride = 0;
};

namespace overlap_detail {
using Wide = __int128;  // (strides of 2^42 bytes times 2^31 rows)

inline Wide floor_div(Wide a, Wide b) { return a >= 0 ? a / b : -((-a + b - 1) / b); }

// Rows a + i s (i < n, la bytes) and b + j s (j < m, lb bytes), d = a - b: with
// k = i - j they overlap where -la < d + k s < lb.
inline bool same_stride(Wide d, Wide s, int64_t n, int64_t la, int64_t m, int64_t lb) {
    Wide k = s > 0 ? floor_div(-la - d, s) + 1 : 0;  // the first above -la
    if (k < 1 - Wide(m)) k = 1 - Wide(m);
    return k <= Wide(n) - 1 && d + k * s < lb && d + k * s > -la;
}
}  // namespace overlap_detail

// Rows whose extents meet.
inline bool rows_meet(const Rows& a, const Rows& b) {
    using namespace overlap_detail;
    const Wide x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (a.rows == 1 || b.rows == 1 || a.stride == b.stride)
        return same_stride(x - y, a.rows == 1 ? b.stride : a.stride, a.rows, a.bytes, b.rows, b.bytes);
    // strides apart: the rows of one against all of the other, from where they meet
    const bool swap = a.rows > b.rows;
    const Rows &u = swap ? b : a, &v = swap ? a : b;
    const Wide u0 = swap ? y : x, v0 = swap ? x : y, v1 = v0 + Wide(v.rows - 1) * v.stride + v.bytes;
    Wide i = u0 + u.bytes > v0 ? 0 : floor_div(v0 - u0 - u.bytes, u.stride) + 1;
    for (; i < u.rows && u0 + i * u.stride < v1; ++i)
        if (same_stride(u0 + i * u.stride - v0, v.stride, 1, u.bytes, v.rows, v.bytes)) return true;
    return false;
}

// The first byte behind the rows (the largest address, where it would be beyond).
inline uintptr_t rows_end(const Rows& a) {
    uint64_t span, end;
    if (__builtin_mul_overflow(static_cast<uint64_t>(a.rows - 1), static_cast<uint64_t>(a.stride), &span) ||
        __builtin_add_overflow(span, static_cast<uint64_t>(a.bytes), &span) ||
        __builtin_add_overflow(span, static_cast<uint64_t>(reinterpret_cast<uintptr_t>(a.p)), &end))
        return UINTPTR_MAX;
    return end;
}

// Does a byte of a lie in b?  (Rows in one another's gaps do not.)  Most
// arguments lie apart as a whole, which costs a nanosecond or two a pair.
inline bool overlap(const Rows& a, const Rows& b) {
    if (a.bytes <= 0 || b.bytes <= 0 || a.rows <= 0 || b.rows <= 0) return false;
    if (rows_end(a) <= reinterpret_cast<uintptr_t>(b.p) || rows_end(b) <= reinterpret_cast<uintptr_t>(a.p)) return false;
    return rows_meet(a, b);
}

}  // namespace ndq
