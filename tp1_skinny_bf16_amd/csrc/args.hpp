// args.hpp -- host-side argument checks shared by the layer entry points.
#pragma once

#include <cstddef>
#include <cstdint>

namespace tp1 {

inline bool is_aligned(const void *p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// The bytes [lo, hi) a strided operand spans; empty for a null pointer.
struct Span {
    uintptr_t lo = 0, hi = 0;
    Span(const void *p, size_t bytes) {
        if (p && bytes) {
            lo = reinterpret_cast<uintptr_t>(p);
            hi = lo + bytes;
        }
    }
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// Bytes spanned by `rows` rows of `width` bytes, `pitch` bytes apart.
inline size_t span_bytes(size_t rows, size_t width, size_t pitch) {
    return rows ? (rows - 1) * pitch + width : 0;
}

}  // namespace tp1
