// rad_check.h -- argument checks shared by the files of the C ABI (host only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/rad.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};
// [p, p + bytes), the end clamped to the top of the address space (no real
// buffer wraps; the clamp only keeps the comparison below meaningful).
Span span(const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    const uintptr_t n = static_cast<uintptr_t>(bytes);
    return Span{lo, n > UINTPTR_MAX - lo ? UINTPTR_MAX : lo + n};
}
bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

constexpr int64_t kI32Max = 2147483647;
// Product of non-negative sizes, or -1 when it does not fit int64 (no buffer
// is that large, so such sizes are out of range).
int64_t checked_mul(std::initializer_list<int64_t> xs) {
    int64_t r = 1;
    for (int64_t x : xs)
        if (__builtin_mul_overflow(r, x, &r)) return -1;
    return r;
}
int hip_status(hipError_t e) { return e == hipSuccess ? RAD_OK : RAD_E_HIP; }

}  // namespace
