// Linear attention with a decay for each head: the path of warp-level matrix products (fp32 and small heads), the chaining of
// segments, and the step of one token a sequence.  The tcgen05 path is decay_tc.cu.
//
// Chunk form, for tokens 0 .. m - 1 of a chunk, the state S that it begins with and g = exp(log_decay):
//   o_i  = sum_{j <= i} g^(i - j) (q_i k_j) v_j + g^(i + 1) S^T q_i
//   S'   = g^m S + sum_j g^(m - 1 - j) k_j v_j^T
// and from the end (gradients), with S the state that the tokens behind leave, decayed to the chunk's last token:
//   o_i  = sum_{j >= i} g^(j - i) (q_i k_j) v_j + g^(m - 1 - i) S^T q_i
//   S'   = g^m S + sum_j g^(j + 1) k_j v_j^T
// All powers are of whole numbers >= 0, so none overflows for g <= 1, and g = 0 (log_decay = -infinity) is a memory of the
// token alone.  What is masked is left out by a choice, not by a factor of zero, so that a later token's infinity or NaN
// stays out of earlier rows.
//
// Measured: 8 x 4096 tokens, 16 heads, fp32: heads of 128 1306 us (floor 158), of 64 526 (79), of 32 237 (40); bf16, heads
// of 32, 211 (20).  What bounds it: 3xTF32 on warp-level MMAs (2112 of them a chunk of 32 tokens and 64 value channels for
// heads of 128) and the splitting of every fragment in two, which is two thirds of the instructions; bf16 operands are one
// TF32 part, so that of two sides at most one is split (heads of 32: 341 us when both were).  Gradients of 3 x 777 tokens,
// 4 heads of 64 and 128 in fp32: 110 us in segments of 192 tokens (100 in a graph; 148 whole).

#include <cuda_bf16.h>
#include <algorithm>
#include <math.h>

#include "common.cuh"
#include "decay.h"
#include "decay_common.cuh"
#include "kdn.h"
#include "mma_tf32x3.cuh"

namespace kdn {
namespace {

constexpr int kC = 32, kThreads = 256;   // tokens of a chunk; threads of a block
constexpr int kSMs = 152;                // GB300

// Four values as they are in memory, and as fp32 (apart from the load, so that it does not have to be waited for).
template <bool BF> __device__ __forceinline__ float4 load4(const void* p, long long i) {
    if (!BF) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float2 x = *reinterpret_cast<const float2*>(static_cast<const __nv_bfloat16*>(p) + i);
    return make_float4(x.x, x.y, 0.f, 0.f);
}
template <bool BF> __device__ __forceinline__ float4 widen(float4 v) {
    if (!BF) return v;
    const uint32_t x = __float_as_uint(v.x), y = __float_as_uint(v.y);
    return make_float4(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u), __uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
}

// x = hi + lo, both TF32: hi rounded to nearest, the rest cut off (to 2^-22 of x, of either sign), by integer operations
// where the conversion is a slow one.  A NaN stays one in lo, whatever the carry makes of it in hi; an infinity, too, leaves a NaN there.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

// An operand's fragment: two TF32 parts, or (EXACT: it was bf16) the one that it is.
template <int N, bool EXACT> struct Parts {
    uint32_t hi[N], lo[N];
    __device__ __forceinline__ void set(int i, float x) {
        if (EXACT) hi[i] = __float_as_uint(x);
        else split(x, hi[i], lo[i]);
    }
};
// Sums of the products of parts.  (Few tiles: a sum for each product, as the MMAs of one sum wait for one another.)
template <int NT> constexpr int kSums = NT <= 2 ? 3 : 1;
template <int NT, bool EA, bool EB>
__device__ __forceinline__ void multiply(float (&acc)[kSums<NT>][NT][4], int n, const Parts<4, EA>& a, const Parts<2, EB>& b) {
    constexpr int kLast = kSums<NT> - 1;
    if (!EA) mma_m16n8k8_tf32(acc[kLast][n], a.lo, b.hi[0], b.hi[1]);
    if (!EB) mma_m16n8k8_tf32(acc[kLast / 2][n], a.hi, b.lo[0], b.lo[1]);
    mma_m16n8k8_tf32(acc[0][n], a.hi, b.hi[0], b.hi[1]);
}
template <int NT> __device__ __forceinline__ void add_sums(float (&out)[NT][4], const float (&acc)[kSums<NT>][NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[n][e] += kSums<NT> == 1 ? acc[0][n][e] : acc[0][n][e] + (acc[1 % kSums<NT>][n][e] + acc[kSums<NT> - 1][n][e]);
}

// A warp's 16 x 8 NT tile of A B (fragments: mma_tf32x3.cuh), the MMAs' sums taken over 32 of K and then in fp32 (their
// accumulation is cut off, not rounded).  A(r, k) = A[r lda + k], or A[k lda + r] w[k] where TRANS; B(k, c) = B[k ldb + c].
template <int NT, int K, bool TRANS, bool EB>
__device__ __forceinline__ void warp_product(float (&out)[NT][4], const float* A, int lda, const float* w, const float* B, int ldb) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    constexpr int kSpan = K < 32 ? K : 32;
#pragma unroll 1
    for (int k0 = 0; k0 < K; k0 += kSpan) {
        float acc[kSums<NT>][NT][4] = {};
#pragma unroll
        for (int k = k0; k < k0 + kSpan; k += 8) {
            Parts<4, false> a;
            if (TRANS) {
                const float w0 = w[k + q], w1 = w[k + q + 4];
                a.set(0, A[(k + q) * lda + g] * w0);
                a.set(1, A[(k + q) * lda + g + 8] * w0);
                a.set(2, A[(k + q + 4) * lda + g] * w1);
                a.set(3, A[(k + q + 4) * lda + g + 8] * w1);
            } else {
                a.set(0, A[g * lda + k + q]);
                a.set(1, A[(g + 8) * lda + k + q]);
                a.set(2, A[g * lda + k + q + 4]);
                a.set(3, A[(g + 8) * lda + k + q + 4]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                Parts<2, EB> b;
                b.set(0, B[(k + q) * ldb + 8 * n + g]);
                b.set(1, B[(k + q + 4) * ldb + 8 * n + g]);
                multiply<NT>(acc, n, a, b);
            }
        }
        add_sums<NT>(out, acc);
    }
}

// Two products of the same 16 rows of Q: with 8 rows of K (a tile of the weights) and with 8 NT columns of the state.
template <int NT, int K, bool BF>
__device__ __forceinline__ void query_products(float (&w)[1][4], float (&o)[NT][4], const float* Q, const float* Kt, int ld, const float* S, int lds) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    constexpr int kSpan = K < 32 ? K : 32;
#pragma unroll 1
    for (int k0 = 0; k0 < K; k0 += kSpan) {
        float aw[3][1][4] = {}, ao[kSums<NT>][NT][4] = {};
#pragma unroll
        for (int k = k0; k < k0 + kSpan; k += 8) {
            Parts<4, BF> a;
            a.set(0, Q[g * ld + k + q]);
            a.set(1, Q[(g + 8) * ld + k + q]);
            a.set(2, Q[g * ld + k + q + 4]);
            a.set(3, Q[(g + 8) * ld + k + q + 4]);
            Parts<2, BF> b;
            b.set(0, Kt[g * ld + k + q]);
            b.set(1, Kt[g * ld + k + q + 4]);
            multiply<1>(aw, 0, a, b);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                Parts<2, false> s;
                s.set(0, S[(k + q) * lds + 8 * n + g]);
                s.set(1, S[(k + q + 4) * lds + 8 * n + g]);
                multiply<NT>(ao, n, a, s);
            }
        }
        add_sums<1>(w, aw);
        add_sums<NT>(o, ao);
    }
}

// One block: a head of a sequence (or of a segment of it) and DVS of its value channels; the state in the registers of its
// warps as their products' fragments, and in shared memory as the next chunk's operand.
template <int DK, int DVS, bool BF> __global__ void __launch_bounds__(kThreads, 2) decay_kernel(const __grid_constant__ DecayParams P) {
    // (rows apart by 4 or 8 banks: the fragments' loads meet no bank twice, but those of K^T two)
    constexpr int LQ = DK + 4, LV = DVS + 8, LP = kC + 4;
    extern __shared__ __align__(16) float sm[];
    float *const sq = sm, *const sk = sq + kC * LQ, *const sv = sk + kC * LQ, *const ss = sv + kC * LV, *const sp = ss + DK * LV;
    __shared__ float pw[kC + 1], wt[kC], rowf[kC];
    __shared__ int bad_at[DVS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const DecayJob& J = P.job[blockIdx.z];
    const int slices = J.dv / DVS, slice = blockIdx.x % slices, item = blockIdx.x / slices / P.H, h = blockIdx.x / slices % P.H,
              v0 = slice * DVS;
    const DecayItem it = find_item(P, item, tid < 32 && h == 0);
    if (P.clear && tid == 0 && blockIdx.x + blockIdx.z == 0) *P.status = 0;   // (nothing else can be found then)
    if (!it.any) return;
    const bool outputs = P.pass != kStates;
    const int row0 = it.row, len = it.len;
    const size_t bh = static_cast<size_t>(it.b) * P.H + h;
    const float l = P.log_decay[h];
    if (tid <= kC) pw[tid] = power(l, tid);

    // warps' tiles of the state: 16 rows and NS tiles of 8 columns
    constexpr int RT = DK / 16, WPR = 8 / RT, NS = DVS / 8 / WPR > 0 ? DVS / 8 / WPR : 1;
    const int s_row = (warp / WPR) * 16, s_col = (warp % WPR) * NS * 8;
    const bool s_mine = s_col < DVS;
    const size_t elems = static_cast<size_t>(J.dk) * J.dv;
    const float* in = nullptr;
    float* end = nullptr;
    int i_k = J.s_k, i_v = J.s_v, o_k = J.s_k, o_v = J.s_v;
    if (it.slot < 0) {
        in = J.S0 ? J.S0 + bh * elems : nullptr;
        end = J.S_T ? J.S_T + bh * elems : nullptr;
    } else {
        float* st = P.states[blockIdx.z] + (static_cast<size_t>(it.slot) * P.H + h) * elems;
        i_k = o_k = J.dv;
        i_v = o_v = 1;
        if (P.pass == kStates) end = st;
        else in = st;
    }
    float S[NS][4];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = s_row + g + 8 * (e >> 1), j = v0 + s_col + 8 * n + 2 * q + (e & 1);
            S[n][e] = in && s_mine ? in[static_cast<size_t>(i) * i_k + static_cast<size_t>(j) * i_v] : 0.f;
        }
    __syncthreads();

    constexpr int NQ = (kC * DK / 4 + kThreads - 1) / kThreads, NV = (kC * DVS / 4 + kThreads - 1) / kThreads;
    float4 fq[NQ], fk[NQ], fv[NV];
    const int chunks = (len + kC - 1) / kC;
    // chunk n of the walk: its first token and how many there are
    auto place = [&](int n, int& t0) {
        t0 = (J.reverse ? chunks - 1 - n : n) * kC;
        return min(kC, len - t0);
    };
    auto fetch = [&](int n) {
        int t0;
        const int m = place(n, t0);
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int e = x * kThreads + tid, t = e / (DK / 4), c = e % (DK / 4) * 4;
            const bool there = t < m;
            const long long r = static_cast<long long>(row0) + t0 + t;
            fq[x] = there && outputs ? load4<BF>(J.q.p, r * J.q.row + h * J.q.head + c) : zero;
            fk[x] = there ? load4<BF>(J.k.p, r * J.k.row + h * J.k.head + c) : zero;
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int e = x * kThreads + tid, t = e / (DVS / 4), c = e % (DVS / 4) * 4;
            const long long r = static_cast<long long>(row0) + t0 + t;
            fv[x] = t < m ? load4<BF>(J.v.p, r * J.v.row + h * J.v.head + v0 + c) : zero;
        }
    };
    if (chunks > 0) fetch(0);
    const Carry c_full(l, kC), c_last(l, len - (chunks - 1) * kC);
    float rest = 0.f;
#pragma unroll 1
    for (int n = 0; n < chunks; ++n) {
        int t0;
        const int m = place(n, t0);
        // the state and the chunk's tokens into shared memory
        if (s_mine && outputs)
#pragma unroll
            for (int x = 0; x < NS; ++x) {
                float* d = ss + (s_row + g) * LV + s_col + 8 * x + 2 * q;
                d[0] = S[x][0]; d[1] = S[x][1];
                d[8 * LV] = S[x][2]; d[8 * LV + 1] = S[x][3];
            }
        int bad = 0;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int e = x * kThreads + tid, t = e / (DK / 4), c = e % (DK / 4) * 4;
            if (t < kC) {
                *reinterpret_cast<float4*>(sq + t * LQ + c) = widen<BF>(fq[x]);
                *reinterpret_cast<float4*>(sk + t * LQ + c) = widen<BF>(fk[x]);
            }
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int e = x * kThreads + tid, t = e / (DVS / 4), c = e % (DVS / 4) * 4;
            const float4 y = widen<BF>(fv[x]);
            if (t < kC) *reinterpret_cast<float4*>(sv + t * LV + c) = y;
            bad |= !(fabsf(y.x) + fabsf(y.y) + fabsf(y.z) + fabsf(y.w) < INFINITY);
        }
        if (tid < kC) {
            const int left = max(m - 1 - tid, 0);
            wt[tid] = pw[J.reverse ? tid + 1 : left];
            rowf[tid] = pw[J.reverse ? left : tid + 1];
        }
        bad = __syncthreads_or(bad);
        if (n + 1 < chunks) fetch(n + 1);
        if (bad) {
            // A channel's values that are not finite are taken out of the products (a weight of zero would not stop them)
            // and put into what the first of them reaches: the walk's later rows of the channel, and its state.
            if (tid < DVS) {
                int first = kC;   // in the order of the walk
#pragma unroll 1
                for (int i = m - 1; i >= 0; --i) {
                    float& x = sv[(J.reverse ? m - 1 - i : i) * LV + tid];
                    if (!(fabsf(x) < INFINITY)) {
                        x = 0.f;
                        first = i;
                    }
                }
                bad_at[tid] = first;
            }
            __syncthreads();
        }

        if (outputs) {
            // weights: 2 x 4 tiles, one a warp; the same rows of the outputs in as many parts
            constexpr int NO = DVS / 32 > 0 ? DVS / 32 : 1;
            const int r0 = (warp >> 2) * 16, c0 = (warp & 3) * 8, oc = (warp & 3) * NO * 8;
            float a[1][4] = {}, o[NO][4] = {};
            // (with 16 value channels half of the warps have no outputs: they work on a tile that is not used)
            query_products<NO, DK, BF>(a, o, sq + r0 * LQ, sk + c0 * LQ, LQ, ss + (oc < DVS ? oc : 0), LV);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = r0 + g + 8 * (e >> 1), j = c0 + 2 * q + (e & 1), gap = J.reverse ? j - i : i - j;
                sp[i * LP + j] = gap >= 0 ? a[0][e] * pw[max(gap, 0)] : 0.f;
            }
            __syncthreads();
            if (oc < DVS) {
                float y[NO][4] = {};
                warp_product<NO, kC, false, BF>(y, sp + r0 * LP, LP, nullptr, sv + oc, LV);
                if (bad)
#pragma unroll
                    for (int x = 0; x < NO; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = r0 + g + 8 * (e >> 1);
                            if (bad_at[oc + 8 * x + 2 * q + (e & 1)] <= (J.reverse ? m - 1 - i : i)) y[x][e] = NAN;
                        }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int i = r0 + g + 4 * e;
                    if (i >= m) continue;
                    const float f = rowf[i];
#pragma unroll
                    for (int x = 0; x < NO; ++x) {
                        const long long at = ((static_cast<long long>(row0) + t0 + i) * P.H + h) * J.dv + v0 + oc + 8 * x + 2 * q;
                        const float u = fmaf(f, o[x][e], y[x][e]), w = fmaf(f, o[x][e + 1], y[x][e + 1]);
                        if (!BF) *reinterpret_cast<float2*>(static_cast<float*>(J.o) + at) = make_float2(u, w);
                        else *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(J.o) + at) = __floats2bfloat162_rn(u, w);
                    }
                }
            }
        }
        if (s_mine && (end || n + 1 < chunks)) {
            float u[NS][4] = {};
            warp_product<NS, kC, true, BF>(u, sk + s_row, LQ, wt, sv + s_col, LV);
            const float c = (m == kC ? c_full : c_last).next(rest);
#pragma unroll
            for (int x = 0; x < NS; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[x][e] = fmaf(c, S[x][e], u[x][e]);
                    if (bad && bad_at[s_col + 8 * x + 2 * q + (e & 1)] < kC) S[x][e] = NAN;
                }
        }
        __syncthreads();
    }
    if (end && s_mine)
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = s_row + g + 8 * (e >> 1), j = v0 + s_col + 8 * n + 2 * q + (e & 1);
                end[static_cast<size_t>(i) * o_k + static_cast<size_t>(j) * o_v] = S[n][e];
            }
}

// Segments' own states -> the states that they begin with, and the last one: a few elements a thread.  Bounds that are out of range
// are noted here, by the first block of a sequence.
constexpr int kChainElems = 4;
__global__ void __launch_bounds__(kThreads) decay_chain_kernel(const __grid_constant__ DecayParams P) {
    const DecayJob& J = P.job[blockIdx.z];
    const int elems = J.dk * J.dv, b = blockIdx.y / P.H, h = blockIdx.y % P.H;
    int row0, len, first = b * P.nseg;
    if (!sequence(P, b, row0, len) && threadIdx.x == 0 && blockIdx.x + h + blockIdx.z == 0) set_status(P.status, kStatusRange);
    if (P.cu) {
        if (len <= P.seg_len) return;
        const DecayItem it = packed_item(P, ~b);
        if (it.len == 0) return;   // (it begins before another one's end)
        first = it.slot;
    }
    const float l = P.log_decay[h];
    const int n = segments(len, P.seg_len);
    const Carry full(l, P.seg_len), last(l, len - (n - 1) * P.seg_len);
    const size_t step = static_cast<size_t>(P.H) * elems;
#pragma unroll 1
    for (int y = 0; y < kChainElems; ++y) {
        const int e = (blockIdx.x * kChainElems + y) * kThreads + threadIdx.x;
        if (e >= elems) break;
        const size_t at = static_cast<size_t>(blockIdx.y) * elems + static_cast<size_t>(e / J.dv) * J.s_k + static_cast<size_t>(e % J.dv) * J.s_v;
        float* st = P.states[blockIdx.z] + (static_cast<size_t>(first) * P.H + h) * elems + e;
        float S = J.S0 ? J.S0[at] : 0.f, rest = 0.f;
        // (kBatch segments' loads at a time: one by one, nine segments took 30 us)
        constexpr int kBatch = 8;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            float own[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i0 + i < n) own[i] = st[(J.reverse ? n - 1 - i0 - i : i0 + i) * step];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i0 + i >= n) break;
                const int seg = J.reverse ? n - 1 - i0 - i : i0 + i;
                st[seg * step] = S;
                S = fmaf((seg == n - 1 ? last : full).next(rest), S, own[i]);
            }
        }
        if (J.S_T) J.S_T[at] = S;
    }
}

template <int DK, int DVS, bool BF> cudaError_t start(const DecayParams& P, int n_jobs, cudaStream_t s) {
    constexpr int bytes = 4 * (2 * kC * (DK + 4) + (kC + DK) * (DVS + 8) + kC * (kC + 4));
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(decay_kernel<DK, DVS, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    decay_kernel<DK, DVS, BF><<<dim3(P.items * P.H * (P.job[0].dv / DVS), 1, n_jobs), kThreads, bytes, s>>>(P);
    return cudaGetLastError();
}

template <int DK, int DVS> cudaError_t start_io(const DecayParams& P, int n_jobs, cudaStream_t s) {
    return P.io == KDN_BF16 ? start<DK, DVS, true>(P, n_jobs, s) : start<DK, DVS, false>(P, n_jobs, s);
}

template <int DK> cudaError_t start_dv(const DecayParams& P, int n_jobs, cudaStream_t s) {
    const int dv = P.job[0].dv;
    if (dv == 16) return start_io<DK, 16>(P, n_jobs, s);
    // 64 value channels a block, or 32 where that gives at most two blocks an SM: a chunk is then worked on in less time (fp32
    // gradients of 3 x 777, 4 heads of 128: 112 us for 117).  Where there are more blocks, each one's weights would be made twice.
    const long long blocks = static_cast<long long>(P.items) * P.H * n_jobs * (dv / 32);
    if (dv == 32 || blocks <= 2 * kSMs) return start_io<DK, 32>(P, n_jobs, s);
    return start_io<DK, 64>(P, n_jobs, s);
}

// Jobs of the same head sizes in one launch.
cudaError_t start_path(const DecayParams& P, int n_jobs, bool tc, cudaStream_t s) {
    if (tc) return launch_decay_tc(P, n_jobs, s);
    switch (P.job[0].dk) {
        case 16: return start_dv<16>(P, n_jobs, s);
        case 32: return start_dv<32>(P, n_jobs, s);
        case 64: return start_dv<64>(P, n_jobs, s);
        default: return start_dv<128>(P, n_jobs, s);
    }
}
cudaError_t start_pass(const DecayParams& P, int n_jobs, bool tc, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    for (int i = 0, n; i < n_jobs && e == cudaSuccess; i += n) {
        DecayParams one = P;
        for (n = 0; i + n < n_jobs && P.job[i + n].dk == P.job[i].dk && P.job[i + n].dv == P.job[i].dv; ++n) {
            one.job[n] = P.job[i + n];
            one.states[n] = P.states[i + n];
        }
        e = start_path(one, n, tc, s);
    }
    return e;
}

bool use_tc(int io, int dk, int dv, uint32_t flags) { return !(flags & KDN_FLAG_PORTABLE) && decay_tc_supported(io, dk, dv); }
// Heads of 64 in dense sequences of one chunk of this path: a block of the tcgen05 path, one an SM, has taken some 5 us before its first
// chunk is through.  256 sequences of 1 to 32 tokens, 16 heads: forward 99 to 105 us for 145, gradients 210 to 237 for 405; of 64
// tokens 152 for 145.  (Heads of 128: 307 to 323 for 194 to 199.  Packed sequences may have a long one among them.)
bool short_ones(const DecayArgs& a) {
    return !a.cu && a.job[0].dk == 64 && a.job[0].dv == 64 && a.n_tok <= static_cast<long long>(kC) * a.n_seq;
}

// Tokens of a dense sequence's segments, or none (0) where it is faster whole.  The segments' states take some six tenths of the time
// of their outputs, chaining them 0.3 us a segment, and the launches 9 to 13.  Measured with 420 calls (1 to 5 sequences of 250 to
// 8000 tokens, 2 to 16 heads of 32, 64 and 128, both directions, each whole and with up to nine lengths of segments): this rule's choice
// takes 1 to 2% more than the best on average, 27% at most; cutting wherever at most half as many blocks would be at work, into
// segments of at least 512 tokens (128 on this path), 6 to 12%, and 85 at most.  8 heads of 64: bf16, 1000 tokens 25 us for 29 whole, 500
// tokens 20 for 18; fp32, 500 tokens 21 for 37, 250 tokens 19 for 20.
int dense_segment(long long sequences, int T, int H, int dk, int dv, bool tc, int jobs) {
    // the gradients' jobs are two (of dv keys and dk values) and one in a launch where dk and dv differ
    const bool two = jobs == 3 && dk != dv;
    const int count[2] = {two ? 2 : jobs, 1}, keys[2] = {two ? dv : dk, dk}, values[2] = {two ? dk : dv, dv};
    const long long n = (T + 63) / 64, heads = sequences * H;
    // segments that run at a time (two blocks of 64 channels an SM on this path), but no more than chaining them is worth
    long long blocks = 0;
    for (int i = 0; i <= two; ++i) blocks = std::max(blocks, heads * count[i] * (tc ? 1 : std::max(1, values[i] / 64)));
    const long long fill = (tc ? kSMs : 2 * kSMs) / blocks;
    if (fill < 2) return 0;
    const long long least = std::max(std::max(1ll, static_cast<long long>(sqrt(n / 7.))), (n + fill - 1) / fill);
    if (least >= n) return 0;
    if (tc) return n > 1.7 * least + 0.25 * n / least + 9 ? static_cast<int>(64 * least) : 0;   // in chunks of a whole walk, 1.2 us
    // a walk's chunks in segments of `len` times 64 tokens
    const auto time = [&](long long len) {
        const long long nseg = (n + len - 1) / len;
        double sum = 0;
        for (int i = 0; i <= two; ++i) {
            // blocks of 32 channels, or of 64 (start_dv), and the time of their chunks to that with a block of 32 an SM
            const long long b = heads * count[i] * std::max(1, values[i] / 32) * nseg;
            const double load = b <= kSMs                             ? 1.
                                : b <= 2 * kSMs || values[i] <= 32    ? 1.7 * ((b + 2 * kSMs - 1) / (2 * kSMs))
                                : b / 2 <= kSMs                       ? 2.
                                                                      : 2.8 * std::max(1., b / 2 / (2. * kSMs));
            sum += 2 * len * (0.8 + 0.022 * keys[i]) * load;
        }
        return nseg == 1 ? sum : 13 + 0.3 * nseg + 1.6 * sum;
    };
    long long len = least;
    for (const long long x : {least + 1, 2 * least})
        if (x < n && time(x) < time(len)) len = x;
    return time(len) < 0.97 * time(n) ? static_cast<int>(64 * len) : 0;
}

// The same for packed sequences, whose lengths the host does not know.  The longest has at least their mean, so where dense ones of
// the mean would be cut, they are.  Else, of six or more, one may be far longer than the others and be worked on alone in the end:
// segments a quarter longer than the mean leave sequences of about one length whole, which costs them the launches (some 6 us).
// 2000 tokens and 7 times 20, 4 heads of 64, fp32: 53 us for 139 whole; 8000 and 9 times 100, 8 heads of 64, bf16: 59 for 159;
// 16 times 300, 4 heads of 128, fp32: 79 for 70 (145 when cut).  Where all sequences' heads fill the GPU they are not cut: 24 of 2 to
// 4095 tokens, 16 heads of 64, take 93, of which the longest alone is 90; in segments of an SM's share of all tokens they took 119 (27
// more for the states, 11 for the chaining, the outputs still 75, as every block has some 5 us before its first chunk is through).
long long packed_segment(int n_seq, int n_tok, int H, int dk, int dv, bool tc, int jobs) {
    const int len = dense_segment(n_seq, n_tok / n_seq, H, dk, dv, tc, jobs);
    if (len > 0 || n_seq < 6) return len;
    const int most = std::max(dk, dv);
    const long long n = (n_tok + 63) / 64, per = static_cast<long long>(H) * (jobs == 3 && dk != dv ? 2 : jobs) * (tc ? 1 : std::max(1, most / 64));
    const long long fill = (tc ? kSMs : 2 * kSMs) / per - n_seq;
    const double alone = tc ? 9 + 1.2 * n : 2 * n * (0.8 + 0.022 * most);   // one of all tokens, us
    if (fill < 2 || alone < (tc ? 50 : 100)) return 0;
    const long long least = std::max(static_cast<long long>(sqrt(n / 7.)), (n + fill - 1) / fill);
    return 64 * std::max(least, (n_tok / n_seq * 5ll / 4 + 63) / 64);
}

// Sequences are cut into segments where that is faster.  A segment has a whole number of chunks of both paths.
DecayPlan plan_of(int n_seq, int n_tok, int H, int dk, int dv, int io, uint32_t flags, bool packed, int n_jobs) {
    DecayPlan p = {false, 0, 1, n_seq, 0};
    if ((flags & KDN_FLAG_NO_SPLIT) || n_seq <= 0 || n_tok <= 0 || H <= 0) return p;
    const bool tc = use_tc(io, dk, dv, flags);
    const long long len = packed ? packed_segment(n_seq, n_tok, H, dk, dv, tc, n_jobs) : dense_segment(n_seq, n_tok / n_seq, H, dk, dv, tc, n_jobs);
    if (len == 0 || len >= n_tok) return p;
    p.split = true;
    p.seg_len = static_cast<int>(len);
    p.nseg = static_cast<int>((n_tok / n_seq + len - 1) / len);
    // (packed: a sequence has at most its tokens / len + 1 segments, and only one longer than len more than one)
    p.items = packed ? static_cast<int>(n_tok / len) + n_seq : n_seq * p.nseg;
    p.slots = packed ? static_cast<int>(n_tok / len + std::min<long long>(n_tok / len, n_seq)) : p.items;
    return p;
}

// ---------------------------------------------------------------- one token a sequence
// S = g S + k v^T, o = S^T q: a head a block, its state read once into registers, written once, and summed over the rows.
// Bound by the state's bytes: 256 sequences of 16 heads, 128 x 128, 88 us, 6.2 TB/s, 91% of the copy rate (two blocks an SM
// have 128 KB on their way).
constexpr int kRegs = 16;   // float4 of the state a thread, for 128 x 128
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
decay_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ log_decay,
                  float* __restrict__ S, T* __restrict__ o, int H, int DK, int DV) {
    __shared__ float s_q[128], s_k[128], part[4 * kThreads];
    const int tid = threadIdx.x, n4 = DV / 4, groups = kThreads / n4, c4 = tid % n4, rg = tid / n4;
    const size_t bh = blockIdx.x;
    float4* st = reinterpret_cast<float4*>(S + bh * DK * DV);
    float4 r[kRegs];
#pragma unroll
    for (int m = 0; m < kRegs; ++m) {
        const int i = rg + m * groups;
        if (i < DK) r[m] = st[static_cast<size_t>(i) * n4 + c4];
    }
    if (tid < DK) {
        s_q[tid] = IO<T>::load(q, bh * DK + tid);
        s_k[tid] = IO<T>::load(k, bh * DK + tid);
    }
    // (in two parts: one number's rounding would be the same in every step, and a state of 16384 steps off by 1.1e-3 at -1e-4)
    const Carry a(log_decay[bh % H], 1);
    float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = IO<T>::load(v, bh * DV + c4 * 4 + c);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kRegs; ++m) {
        const int i = rg + m * groups;
        if (i < DK) {
            const float ki = s_k[i], qi = s_q[i];
            float4 z = r[m];
            z.x = fmaf(a.hi, z.x, fmaf(a.lo, z.x, ki * x[0]));
            z.y = fmaf(a.hi, z.y, fmaf(a.lo, z.y, ki * x[1]));
            z.z = fmaf(a.hi, z.z, fmaf(a.lo, z.z, ki * x[2]));
            z.w = fmaf(a.hi, z.w, fmaf(a.lo, z.w, ki * x[3]));
            st[static_cast<size_t>(i) * n4 + c4] = z;
            y[0] = fmaf(qi, z.x, y[0]);
            y[1] = fmaf(qi, z.y, y[1]);
            y[2] = fmaf(qi, z.z, y[2]);
            y[3] = fmaf(qi, z.w, y[3]);
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) part[rg * DV + c4 * 4 + c] = y[c];
    __syncthreads();
    if (tid < DV) {
        float sum = 0.f;
        for (int i = 0; i < min(groups, DK); ++i) sum += part[i * DV + tid];
        IO<T>::store(o, bh * DV + tid, sum);
    }
}

}  // namespace

size_t decay_scratch(int n_seq, int n_tok, int H, int dk, int dv, int io, uint32_t flags, bool packed, int n_jobs) {
    const DecayPlan p = plan_of(n_seq, n_tok, H, dk, dv, io, flags, packed, n_jobs);
    return static_cast<size_t>(n_jobs) * p.slots * H * dk * dv * sizeof(float);
}

cudaError_t launch_decay(const DecayArgs& a, cudaStream_t s) {
    const int dk = a.job[a.n_jobs - 1].dk, dv = a.job[a.n_jobs - 1].dv;   // (the call's: those of the first gradients' jobs change places)
    const bool tc = use_tc(a.io, dk, dv, a.flags) && a.n_tok > 0 && !short_ones(a);
    const DecayPlan plan = plan_of(a.n_seq, a.n_tok, a.H, dk, dv, a.io, a.flags, a.cu != nullptr, a.n_jobs);
    DecayParams P = {};
    for (int i = 0; i < a.n_jobs; ++i) {
        P.job[i] = a.job[i];
        P.states[i] = a.scratch + static_cast<size_t>(i) * plan.slots * a.H * dk * dv;
    }
    P.log_decay = a.log_decay; P.cu = a.cu; P.status = a.status;
    P.n_seq = a.n_seq; P.n_tok = a.n_tok; P.H = a.H; P.io = a.io;
    P.nseg = plan.nseg; P.seg_len = plan.seg_len; P.slots = plan.slots;
    P.probe = (a.flags & KDN_FLAG_TIMEOUT_PROBE) ? 1 : 0;
    // the status word: where a kernel may find something, by a call of its own (else the kernels clear it)
    P.clear = !a.cu && !tc;
    cudaError_t e = cudaSuccess;
    if (!P.clear && (e = cudaMemsetAsync(a.status, 0, sizeof(uint32_t), s)) != cudaSuccess) return e;
    if (plan.split) {
        P.pass = kStates;
        P.items = plan.slots;
        if ((e = start_pass(P, a.n_jobs, tc, s)) != cudaSuccess) return e;
        decay_chain_kernel<<<dim3((dk * dv + kChainElems * kThreads - 1) / (kChainElems * kThreads), a.n_seq * a.H, a.n_jobs), kThreads, 0, s>>>(P);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    P.pass = plan.split ? kOutputs : kWhole;
    P.items = plan.items;
    return start_pass(P, a.n_jobs, tc, s);
}

cudaError_t launch_decay_step(const DecayStepArgs& a, cudaStream_t s) {
    if (a.io == KDN_BF16)
        decay_step_kernel<__nv_bfloat16><<<a.B * a.H, kThreads, 0, s>>>(
            static_cast<const __nv_bfloat16*>(a.q), static_cast<const __nv_bfloat16*>(a.k), static_cast<const __nv_bfloat16*>(a.v),
            a.log_decay, a.S, static_cast<__nv_bfloat16*>(a.o), a.H, a.dk, a.dv);
    else
        decay_step_kernel<float><<<a.B * a.H, kThreads, 0, s>>>(
            static_cast<const float*>(a.q), static_cast<const float*>(a.k), static_cast<const float*>(a.v), a.log_decay, a.S,
            static_cast<float*>(a.o), a.H, a.dk, a.dv);
    return cudaGetLastError();
}

}  // namespace kdn
