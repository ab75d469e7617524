// Argument checks shared by the C ABI's translation units (host side).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "attention.h"
#include "kdn.h"

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

// Counts up to here: what loops and grids add to them (steps of a block's or a grid's threads, row tiles) stays in 32 bits.
constexpr int kMostRows = 0x7fffffff - (1 << 25);

// Strides of a [rows, heads, d] operand: positive multiples of 16 bytes that keep rows and
// heads apart.  An axis of length one has no stride to check.
inline kdn_status check_strided(kdn::Strided* x, long long rows, int heads, int d, size_t esz) {
    if (heads <= 1) x->head = d;
    if (rows <= 1) x->row = (long long)heads * d;
    if (x->head < d || x->row < d) return KDN_ERR_SHAPE;
    // one axis steps over the whole of the other
    if (rows > 1 && heads > 1 && x->row < (heads - 1) * x->head + d && x->head < (rows - 1) * x->row + d)
        return KDN_ERR_SHAPE;
    if (x->head * esz % 16 || x->row * esz % 16) return KDN_ERR_ALIGN;
    if (x->row > (1ll << 36) || x->head > (1ll << 36)) return KDN_ERR_SHAPE;
    return KDN_OK;
}

inline Range range_of(const kdn::Strided& x, long long rows, int heads, int d, size_t esz) {
    if (rows <= 0 || heads <= 0) return Range{nullptr, 0};
    return Range{x.p, (size_t)((rows - 1) * x.row + (heads - 1) * x.head + d) * esz};
}

template <int N, int M> kdn_status check_alias(const Range (&out)[N], const Range (&in)[M]) {
    for (int i = 0; i < N; ++i) {
        for (int j = i + 1; j < N; ++j)
            if (overlaps(out[i], out[j])) return KDN_ERR_ALIAS;
        for (int j = 0; j < M; ++j)
            if (overlaps(out[i], in[j])) return KDN_ERR_ALIAS;
    }
    return KDN_OK;
}

template <int N> bool all_aligned(const void* const (&p)[N]) {
    for (const void* x : p)
        if (x && !aligned16(x)) return false;
    return true;
}

inline kdn_status done(cudaError_t e) { return e == cudaSuccess ? KDN_OK : KDN_ERR_CUDA; }

}  // namespace
