// Device helpers of the paths of the decayed memory.
#pragma once

#include <math.h>

#include "decay.h"

namespace kdn {

// exp(l n) for a whole n >= 0: 1 for n = 0 whatever l is.
__device__ __forceinline__ float power(float l, int n) { return n == 0 ? 1.f : expf(l * static_cast<float>(n)); }

// exp(l n) as a sum of two fp32 numbers: the states of thousands of chunks are multiplied by it one after another, and the
// rounding of one number close to 1 would add up (2e-5 over 800 chunks of 64 tokens at l = -1e-4).
__device__ __forceinline__ float2 power2(float l, int n) {
    const float e = n == 0 ? 0.f : expm1f(l * static_cast<float>(n)), hi = 1.f + e, lo = e - (hi - 1.f);
    return make_float2(hi, fabsf(lo) < INFINITY ? lo : 0.f);
}

// Tokens of sequence b: first row and length; false where its bounds run backwards or outside.
__device__ __forceinline__ bool sequence(const DecayParams& P, int b, int& row, int& len) {
    if (!P.cu) {
        len = P.n_tok / P.n_seq;
        row = b * len;
        return true;
    }
    const int x = P.cu[b], y = P.cu[b + 1];
    row = x;
    len = y - x;
    if (x >= 0 && y >= x && y <= P.n_tok) return true;
    row = len = 0;
    return false;
}

}  // namespace kdn
