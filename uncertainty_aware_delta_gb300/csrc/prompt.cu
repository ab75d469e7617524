// Causal attention over whole prompts, CUDA-core path: every size and type (the tcgen05
// kernel takes bf16 with heads of 64 and 128).  fp32 operands (bf16 is widened) as two TF32
// parts, products in 3xTF32 on warp-level MMAs (m16n8k8).
//
// A block has 128 query rows, a warp 32 of them, and walks the keys in tiles of 32: scores in
// registers, a running maximum and sum a row, weights used as the next product's left operand
// where they are (the keys of a step are taken in the order 0, 2, 4, 6, 1, 3, 5, 7, in which the
// accumulators' columns are that operand's).  Operands are split once, when they are put into
// shared memory.  What bounds it: two warps a scheduler (255 registers) that load, split and
// multiply in turn, 24 MMAs against 32 4-byte loads a thread for 32 rows, 8 channels and 32 keys (the
// tensor pipe is busy for 47% of the time, issue slots for 35%); a wider warp tile would not fit its registers.
//
// Measured: 4 prompts of 700 to 1024 tokens in fp32 (16/4 heads of 64, causal) 202 us, 35 TFLOP/s (105 of
// TF32 products), with heads of 128 381; bf16 prompts of 128 tokens (16 of them, 16/4 heads of 128) 84 us against the tcgen05
// kernel's 14, one of 77 tokens 33 against 14.  Calls of a few rows tie (heads of 64, 1 x 16 tokens: 10.6
// against 12.1), so the path goes by type and head size alone.
//
// The MMAs cut sums off instead of rounding them, which a long sum would show: they sum the products of
// 32 channels, or of one tile's keys, and those are added up in fp32 (2000 tokens, heads of 128: an error of
// 3.8e-7 of the outputs' norm, 4.5e-7 with products in fp32; with scores summed over all 128 channels, for 2% less
// time, 1.1e-6).

#include <cuda_bf16.h>

#include "attention.h"
#include "common.cuh"
#include "kdn.h"
#include "mma_tf32x3.cuh"

namespace kdn {
namespace {

constexpr int kThreads = 128, kRows = 128, kKeys = 32;
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}
// Puts four numbers in two TF32 parts at `at`; whether a first part is not finite.
__device__ __forceinline__ bool put4(uint32_t* h, uint32_t* l, int at, float4 x) {
    uint4 hi, lo;
    split_tf32(x.x, hi.x, lo.x);
    split_tf32(x.y, hi.y, lo.y);
    split_tf32(x.z, hi.z, lo.z);
    split_tf32(x.w, hi.w, lo.w);
    *reinterpret_cast<uint4*>(h + at) = hi;
    *reinterpret_cast<uint4*>(l + at) = lo;
    // zero times a number that is not finite is NaN: one test for the four
    const float none = fmaf(__uint_as_float(hi.x), 0.f, fmaf(__uint_as_float(hi.y), 0.f,
                            fmaf(__uint_as_float(hi.z), 0.f, __uint_as_float(hi.w) * 0.f)));
    return !(none == 0.f);
}
// The same where one is not.  An infinity has no second part (or, with `drop`, becomes a zero), and what would round up to one
// (the largest numbers of fp32, such as a mask's lowest value) is cut off instead, in both parts, so that their sum is
// no larger.
__device__ void put4_odd(uint32_t* h, uint32_t* l, int at, float4 v, bool drop) {
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t hi, lo;
        split_tf32(x[i], hi, lo);
        if (!finite(__uint_as_float(hi))) {
            hi = finite(x[i]) ? __float_as_uint(x[i]) & 0xffffe000u : drop ? 0u : hi;
            lo = finite(x[i]) ? __float_as_uint(x[i] - __uint_as_float(hi)) & 0xffffe000u : 0u;
        }
        h[at + i] = hi;
        l[at + i] = lo;
    }
}

// Bounds of a sequence's queries and keys.
__device__ __forceinline__ bool in_range(const PromptArgs& a, int q0, int q1, int k0, int k1) {
    return q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k;
}

// c[i][n] += a[i] b[n]: two 16-row tiles by N 8-column tiles, independent of each other.
template <int N>
__device__ __forceinline__ void products(float (&c)[2][N][4], const uint32_t (&a)[2][4], const uint32_t (&b)[N][2]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) mma_m16n8k8_tf32(c[i][n], a[i], b[n][0], b[n][1]);
}

// A masked key has no influence whatever it holds: keys outside the sequence are read as
// zeros, scores are masked by selection, and a value that is not finite is taken out of the
// tile and added to the rows that see it.  A score with an infinity in it is what its products add up to.
template <typename T, int D> __global__ void __launch_bounds__(kThreads) prompt_kernel(const PromptArgs a) {
    constexpr int LD = D + 4;   // rows 4 banks apart: the fragments' loads are free of conflicts
    extern __shared__ __align__(16) uint32_t prompt_smem[];
    uint32_t* qh = prompt_smem;
    uint32_t* ql = qh + kRows * LD;
    uint32_t* kh = ql + kRows * LD;
    uint32_t* kl = kh + kKeys * LD;
    uint32_t* vh = kl + kKeys * LD;
    uint32_t* vl = vh + kKeys * LD;
    __shared__ int found[5];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int h = blockIdx.x % a.H, kvh = h / (a.H / a.H_kv);
    if (warp == 0) {
        // item -> (sequence, row tile), of every 32 sequences the last tiles first: they have the most keys, and the
        // short ones fill the gaps that they leave (sequence by sequence, the last first, 227 us against 200 on 4 prompts of 700 to 1024)
        int item = static_cast<int>(blockIdx.x / a.H);
        bool here = false;
        if (lane == 0) found[0] = -1;
        for (int s0 = 0; s0 < a.n_seq && !here; s0 += 32) {
            const int s = s0 + lane;
            int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
            if (s < a.n_seq) {
                q0 = a.cu_q[s]; q1 = a.cu_q[s + 1]; k0 = a.cu_k[s]; k1 = a.cu_k[s + 1];
                if (!in_range(a, q0, q1, k0, k1)) q0 = q1 = 0;
            }
            const int tiles = (q1 - q0 + kRows - 1) / kRows;
            // items from row tile t of their sequence on
            auto from = [&](int t) { return __reduce_add_sync(kAll, max(tiles - t, 0)); };
            const int all = from(0);
            here = item < all;
            if (!here) {
                item -= all;
                continue;
            }
            int t = 0, above = a.total_q / kRows + 1, before = 0;   // before: items from `above` on
            while (above - t > 1) {
                const int m = (t + above) / 2, n = from(m);
                if (n > item) {
                    t = m;
                } else {
                    above = m;
                    before = n;
                }
            }
            const uint32_t there = __ballot_sync(kAll, tiles > t);
            if (tiles > t && __popc(there & ((1u << lane) - 1)) == item - before) {
                const int row = t * kRows;
                found[0] = q0 + row;
                found[1] = min(kRows, q1 - q0 - row);
                found[2] = k0;
                found[3] = k1 - k0;
                found[4] = (k1 - k0) - (q1 - q0) + row;   // place of the tile's first row among the keys
            }
        }
    } else {   // the search ends where its item is: the blocks' other warps look at all bounds together
        for (long long s = static_cast<long long>(blockIdx.x) * (kThreads - 32) + tid - 32; s < a.n_seq;
             s += static_cast<long long>(gridDim.x) * (kThreads - 32))
            if (!in_range(a, a.cu_q[s], a.cu_q[s + 1], a.cu_k[s], a.cu_k[s + 1])) set_status(a.status, kStatusRange);
    }
    __syncthreads();
    const int q0 = found[0], rows = found[1], k0 = found[2], n_keys = found[3], place = found[4];
    if (q0 < 0) return;
    const T* qp = static_cast<const T*>(a.q.p) + q0 * a.q.row + h * a.q.head;
    auto queries = [&](int i, auto put) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        return put(qh, ql, r * LD + c, r < rows ? load4(qp + r * a.q.row + c) : make_float4(0.f, 0.f, 0.f, 0.f));
    };
    bool odd_q = false;
    for (int i = tid; i < kRows * (D / 4); i += kThreads) odd_q |= queries(i, put4);
    if (odd_q)   // rare, and every thread has its own: the loads above stay together
#pragma unroll 1
        for (int i = tid; i < kRows * (D / 4); i += kThreads)
            queries(i, [](uint32_t* h, uint32_t* l, int at, float4 x) { put4_odd(h, l, at, x, false); });
    float o[2][D / 8][4], m[4], l[4];   // rows 16 i + g, + 8 of the warp's 32
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    const int last = min(place + rows - 1, n_keys - 1);                       // last key any row sees
    const int low = a.window > 0 && place >= a.window ? place - a.window + 1 : 0;   // first (place may be far below 0)
    const float to_log2 = a.scale * 1.4426950408889634f;
    for (int j0 = low / kKeys * kKeys; j0 <= last; j0 += kKeys) {
        const T* kp = static_cast<const T*>(a.k.p) + (static_cast<long long>(k0) + j0) * a.k.row + kvh * a.k.head;
        const T* vp = static_cast<const T*>(a.v.p) + (static_cast<long long>(k0) + j0) * a.v.row + kvh * a.v.head;
        auto keys = [&](const T* p, long long step, int i, auto put) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            return put(r * LD + c, j0 + r < n_keys ? load4(p + r * step + c) : make_float4(0.f, 0.f, 0.f, 0.f));
        };
        bool odd = false;
        for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
            odd |= keys(kp, a.k.row, i, [&](int at, float4 x) { return put4(kh, kl, at, x); });
            odd |= keys(vp, a.v.row, i, [&](int at, float4 x) { return put4(vh, vl, at, x); });
        }
        if (odd)
#pragma unroll 1
            for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
                keys(kp, a.k.row, i, [&](int at, float4 x) { put4_odd(kh, kl, at, x, false); });
                keys(vp, a.v.row, i, [&](int at, float4 x) { put4_odd(vh, vl, at, x, true); });
            }
        odd = __syncthreads_or(odd || odd_q);
        float s[2][kKeys / 8][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
        constexpr int kSum = D < 32 ? D : 32;   // channels summed by the MMAs; added up in fp32
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += kSum) {
            float t[2][kKeys / 8][4] = {};
#pragma unroll 2
            for (int c = c0; c < c0 + kSum; c += 8) {
                uint32_t ah[2][4], al[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = (32 * warp + 16 * i + g) * LD + c + q;
                    ah[i][0] = qh[at]; ah[i][1] = qh[at + 8 * LD]; ah[i][2] = qh[at + 4]; ah[i][3] = qh[at + 8 * LD + 4];
                    al[i][0] = ql[at]; al[i][1] = ql[at + 8 * LD]; al[i][2] = ql[at + 4]; al[i][3] = ql[at + 8 * LD + 4];
                }
                uint32_t bh[kKeys / 8][2], bl[kKeys / 8][2];
#pragma unroll
                for (int n = 0; n < kKeys / 8; ++n) {
                    const int at = (8 * n + g) * LD + c + q;
                    bh[n][0] = kh[at]; bh[n][1] = kh[at + 4];
                    bl[n][0] = kl[at]; bl[n][1] = kl[at + 4];
                }
                // part by part: the three products of one sum stand apart
                products(t, al, bh);
                products(t, ah, bl);
                products(t, ah, bh);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][n][e] += t[i][n][e];
        }
        if (odd) {
            // an infinity times the other operand's second part, zero or of the other sign, is not the product's: such
            // scores are formed anew, from the products that are not finite (bit 8 r + 2 n + k: row r, key 8 n + 2 q + k)
            uint32_t above = 0, below = 0;
#pragma unroll 1
            for (int b = 0; b < 32; ++b) {
                const int row = 32 * warp + 8 * (b / 8) + g, j = b % 8 / 2 * 8 + 2 * q + b % 2;
                if (row >= rows || j0 + j >= n_keys) continue;
                float t = 0.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 4) {
                    const float4 x = load4(qp + row * a.q.row + c), y = load4(kp + j * a.k.row + c);
                    if (!(finite(x.x) && finite(y.x))) t += x.x * y.x;
                    if (!(finite(x.y) && finite(y.y))) t += x.y * y.y;
                    if (!(finite(x.z) && finite(y.z))) t += x.z * y.z;
                    if (!(finite(x.w) && finite(y.w))) t += x.w * y.w;
                }
                above |= static_cast<uint32_t>(!(t <= 0.f)) << b;   // (both where it is NaN)
                below |= static_cast<uint32_t>(!(t >= 0.f)) << b;
            }
#pragma unroll
            for (int b = 0; b < 32; ++b) {
                float& x = s[b / 16][b % 8 / 2][b / 8 % 2 * 2 + b % 2];
                if (above >> b & 1u) x = below >> b & 1u ? NAN : INFINITY;
                else if (below >> b & 1u) x = -INFINITY;
            }
        }
        // rows 2 i and 2 i + 1 of the thread: 16 i + g and 16 i + g + 8
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = r / 2, e = r % 2 * 2, at = place + 32 * warp + 16 * i + 8 * (r % 2) + g;
            float mx = -INFINITY;
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = j0 + 8 * n + 2 * q + k;
                    const bool see = j <= at && j < n_keys && (a.window <= 0 || j > at - a.window);
                    s[i][n][e + k] = see ? s[i][n][e + k] * to_log2 : -INFINITY;
                    mx = fmaxf(mx, s[i][n][e + k]);
                }
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
            const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[r] - base);
            m[r] = mn;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float p = exp2f(s[i][n][e + k] - base);
                    s[i][n][e + k] = p;
                    sum += p;
                }
            l[r] = l[r] * f + sum;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[i][n][e] *= f;
                o[i][n][e + 1] *= f;
            }
        }
        // 32 channels at a time (16 where there are no more): eight sums side by side
        constexpr int kPart = D / 8 < 4 ? D / 8 : 4;
#pragma unroll
        for (int n0 = 0; n0 < D / 8; n0 += kPart) {
            float t[2][kPart][4] = {};
#pragma unroll
            for (int c = 0; c < kKeys / 8; ++c) {
                uint32_t ph[2][4], pl[2][4], bh[kPart][2], bl[kPart][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    split_tf32(s[i][c][0], ph[i][0], pl[i][0]);
                    split_tf32(s[i][c][2], ph[i][1], pl[i][1]);
                    split_tf32(s[i][c][1], ph[i][2], pl[i][2]);
                    split_tf32(s[i][c][3], ph[i][3], pl[i][3]);
                }
#pragma unroll
                for (int n = 0; n < kPart; ++n) {
                    const int at = (8 * c + 2 * q) * LD + 8 * (n0 + n) + g;
                    bh[n][0] = vh[at]; bh[n][1] = vh[at + LD];
                    bl[n][0] = vl[at]; bl[n][1] = vl[at + LD];
                }
                products(t, pl, bh);
                products(t, ph, bl);
                products(t, ph, bh);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < kPart; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][n0 + n][e] += t[i][n][e];
        }
        if (odd) {   // each row adds what it sees of the values taken out (its weights are positive)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = r / 2, e = r % 2 * 2, at = place + 32 * warp + 16 * i + 8 * (r % 2) + g;
                for (int jj = 0; jj < kKeys; ++jj) {
                    const int j = j0 + jj;
                    if (j > at || j >= n_keys || (a.window > 0 && j <= at - a.window)) continue;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float x = IO<T>::load(vp, jj * a.v.row + 8 * n + 2 * q + k);
                            if (!finite(x)) o[i][n][e + k] += x;
                        }
                }
            }
        }
        __syncthreads();
    }
    T* op = static_cast<T*>(a.o) + (static_cast<size_t>(q0) * a.H + h) * D;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = r / 2, e = r % 2 * 2, row = 32 * warp + 16 * i + 8 * (r % 2) + g;
        float sum = l[r];
        sum += __shfl_xor_sync(kAll, sum, 1);
        sum += __shfl_xor_sync(kAll, sum, 2);
        if (row >= rows) continue;
        const float f = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                IO<T>::store(op, static_cast<size_t>(row) * a.H * D + 8 * n + 2 * q + k, o[i][n][e + k] * f);
        if (q == 0)
            a.lse[(static_cast<size_t>(q0) + row) * a.H + h] = sum != 0.f ? (m[r] + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
}

template <typename T, int D> cudaError_t launch(const PromptArgs& a, cudaStream_t s) {
    const size_t smem = sizeof(float) * 2 * (kRows + 2 * kKeys) * (D + 4);
    const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    // no more row tiles than this, whatever the lengths
    const int items = a.total_q / kRows + (a.n_seq < a.total_q ? a.n_seq : a.total_q);
    const long long grid = static_cast<long long>(items) * a.H;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    prompt_kernel<T, D><<<static_cast<int>(grid), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t by_size(const PromptArgs& a, cudaStream_t s) {
    if (a.d == 128) return launch<T, 128>(a, s);
    if (a.d == 64) return launch<T, 64>(a, s);
    if (a.d == 32) return launch<T, 32>(a, s);
    return launch<T, 16>(a, s);
}

}  // namespace

size_t prompt_scratch(int n_seq, int total_q, int H, int H_kv, int d, int io, uint32_t flags) {
    return !(flags & KDN_FLAG_PORTABLE) && prompt_tc_supported(io, d) ? prompt_tc_scratch(n_seq, total_q, H, H_kv, d) : 0;
}

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s) {
    if (!(a.flags & KDN_FLAG_PORTABLE) && prompt_tc_supported(a.io, a.d)) return launch_prompt_tc(a, s);
    return a.io == 1 ? by_size<__nv_bfloat16>(a, s) : by_size<float>(a, s);
}

}  // namespace kdn
