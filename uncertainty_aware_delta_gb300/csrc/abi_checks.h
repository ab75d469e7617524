// Argument checks shared by the C ABI's translation units (host side).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kStatusBytes = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    const void* p;
    size_t n;
};

inline bool overlaps(Range a, Range b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

}  // namespace
