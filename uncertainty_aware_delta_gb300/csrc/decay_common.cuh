// Device helpers of the paths of the decayed memory.
#pragma once

#include <math.h>

#include "common.cuh"
#include "decay.h"

namespace kdn {

// exp(l n) for a whole n >= 0: 1 for n = 0 whatever l is.
__device__ __forceinline__ float power(float l, int n) { return n == 0 ? 1.f : expf(l * static_cast<float>(n)); }

// exp(l n), by which the states of thousands of chunks, or of hundreds of segments, are multiplied one after another: the rounding
// of one number close to 1 would add up (2e-5 over 800 chunks of 64 tokens at l = -1e-4).  It is held as a sum of two, and next() gives the nearest
// number to what is left to multiply by, so that the product of any chunks' factors stays within a rounding of the power.
// Where the power is small it has more digits than 1 + expm1 has, and few chunks matter.
struct Carry {
    float hi, lo;
    __device__ __forceinline__ Carry(float l, int n) {
        const float x = n == 0 ? 0.f : l * static_cast<float>(n);
        if (x > -0.5f && x < 0.5f) {
            const float e = expm1f(x);
            hi = 1.f + e;
            lo = e - (hi - 1.f);
        } else {
            hi = expf(x);
            lo = 0.f;
        }
    }
    __device__ __forceinline__ float next(float& rest) const {
        rest += lo;
        const float f = hi + rest;
        rest -= f - hi;
        return f;
    }
};

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

__device__ __forceinline__ int segments(int len, int seg_len) { return len > 0 ? (len - 1) / seg_len + 1 : 0; }

// What a block works on.
struct DecayItem {
    int b, row, len;   // sequence; first token and tokens, of the segment if it is one
    int slot;          // of its state; negative: a whole sequence
    bool any;
};

// The segments of packed sequences longer than seg_len are counted through first, then the other sequences: item `want` of
// them, or (want < 0) the first slot of sequence ~want.  A sequence that begins before an earlier one's end (bounds before it ran
// backwards) counts as empty, so that there are no more segments than all tokens have.  A warp together.
__device__ __forceinline__ DecayItem packed_item(const DecayParams& P, int want) {
    const uint32_t all = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    DecayItem it = {0, 0, 0, -1, false};
    int before = 0;
#pragma unroll 1
    for (int whole = 0; whole < 2; ++whole) {
        int end = 0;   // of all sequences before
#pragma unroll 1
        for (int s0 = 0; s0 < P.n_seq; s0 += 32) {
            int row = 0, len = -1;
            const bool wrong = s0 + lane < P.n_seq && !sequence(P, s0 + lane, row, len);
            const int upto_here = max(end, __reduce_max_sync(all, row + len));
            if (__any_sync(all, wrong || (len > 0 && row < end))) {   // (else every one of these begins where the last ends)
                int reach = row + len;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) reach = max(reach, __shfl_sync(all, reach, max(lane - o, 0)));
                reach = __shfl_sync(all, reach, max(lane - 1, 0));
                if (len > 0 && row < (lane ? max(reach, end) : end)) row = len = 0;
            }
            end = upto_here;
            const bool cut = len > P.seg_len;
            const int mine = whole ? (len >= 0 && !cut) : cut ? segments(len, P.seg_len) : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(all, upto, o);
                if (lane >= o) upto += y;
            }
            const bool here = want < 0 ? s0 + lane == ~want : want < before + upto;
            const uint32_t hit = __ballot_sync(all, here);
            if (hit) {
                const int at = __ffs(hit) - 1;
                it.b = s0 + at;
                it.row = __shfl_sync(all, row, at);
                it.len = __shfl_sync(all, len, at);
                const int first = __shfl_sync(all, before + upto - mine, at);
                it.any = true;
                if (want < 0) {
                    it.slot = first;
                } else if (!whole) {
                    const int seg = want - first;
                    it.slot = want;
                    it.row += seg * P.seg_len;
                    it.len = min(it.len - seg * P.seg_len, P.seg_len);
                }
                return it;
            }
            before += __shfl_sync(all, upto, 31);
        }
    }
    return it;
}

// Item `item` of a pass.  `report`: bounds that are out of range are noted, where every sequence is an item (of packed sequences that
// are cut, the search for an item ends where it is found: the chaining, which goes through all sequences, notes them).
__device__ __forceinline__ DecayItem find_item(const DecayParams& P, int item, bool report) {
    DecayItem it = {item, 0, 0, -1, true};
    if (P.pass == kWhole) {
        if (!sequence(P, item, it.row, it.len) && report) set_status(P.status, kStatusRange);
    } else if (!P.cu) {
        it.b = item / P.nseg;
        it.slot = item;
        const int seg = item % P.nseg;
        sequence(P, it.b, it.row, it.len);
        it.row += seg * P.seg_len;
        it.len = min(it.len - seg * P.seg_len, P.seg_len);
    } else {
        it = packed_item(P, item);
        if (P.pass == kStates && it.slot < 0) it.any = false;
    }
    return it;
}

}  // namespace kdn
