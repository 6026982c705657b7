// Host-side argument checks shared by the C ABI's translation units.
#pragma once

#include <stdint.h>

namespace {

inline bool mul(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

inline int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

struct Range {
    uintptr_t lo, hi;  // [lo, hi); empty when the pointer is NULL
};

inline Range span(const void* p, int64_t bytes)
{
    if (!p) return {0, 0};
    return {reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(bytes)};
}

inline bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline bool aligned(const void* p, uintptr_t al) { return (reinterpret_cast<uintptr_t>(p) % al) == 0; }

}  // namespace
