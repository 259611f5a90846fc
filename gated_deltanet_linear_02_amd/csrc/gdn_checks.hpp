// gdn_checks.hpp -- argument checks that the C entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

inline bool valid_head(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

inline bool valid_dtype(int32_t t) { return t == GDN_BF16 || t == GDN_F32; }
inline size_t dtype_bytes(int32_t t) { return t == GDN_BF16 ? 2 : 4; }

struct Range {
    uintptr_t lo, hi;
};
inline Range span(const void *p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}
// Tensors the kernels read or write in 16-byte pieces must start on a
// 16-byte boundary (their rows are then aligned too: d >= 16).
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline bool overlaps(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

}  // namespace gdn
