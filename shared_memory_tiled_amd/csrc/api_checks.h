// api_checks.h -- argument checks shared by the entry points' translation
// units (host only; not part of the public interface).
#pragma once

#include <stdint.h>

namespace gemmf32 {
namespace {

inline bool misaligned(const void* ptr) { return ((uintptr_t)ptr & 3u) != 0; }

// (rows - 1) * ld + cols must be addressable with 64-bit element offsets.
inline bool extent_fits(int64_t rows, int64_t cols, int64_t ld) {
    if (rows == 0 || cols == 0) return true;
    int64_t last;
    if (__builtin_mul_overflow(rows - 1, ld, &last)) return false;
    return !__builtin_add_overflow(last, cols, &last);
}

}  // namespace
}  // namespace gemmf32
