// Norm of every token's groups of d channels (the heads of a memory's outputs), with an activation, and its gradients.
//
//   xh = (x - mean) rstd,  n = xh w + b,  y = act(n)  or, with a gate,  y = n act(gate)
//   dn = dy act'(n)  or  dy act(gate),  dgate = dy n act'(gate),  dw = sum over tokens of dn xh,  db = that of dn,
//   dx = rstd (dn w - mean(dn w) - xh mean(dn w xh))
//
// A group's channels lie in neighbouring lanes, eight a lane, so its sums are a few shuffles and x is read once.  A thread
// keeps its channels from token to token: weights stay in registers, and the gradients of weights are sums in registers,
// written once a block and joined by a second kernel in a fixed order.
//
// Measured on 32768 tokens of 16 groups of 128, bf16, SiLU of a gate: 75 us, 5.4 TB/s, 79% of the copy rate (one row of a
// thread at a time 108, two 90, four 74); gradients 123 us, 5.5 TB/s (175 with a row at a time and full exponentials; blocks of
// four an SM 171, of three 154, of two, each with two rows' loads ahead, 121).  fp32: 129 and 201 us in graphs, 92 and 98% of the
// rate.  Bound by the bytes, and in bf16 by the instructions that come with them: issue slots are busy for 61% of the time, and
// 64% in the gradients.

#include <cuda_bf16.h>
#include <algorithm>
#include <math.h>

#include "common.cuh"
#include "decay.h"
#include "kdn.h"
#include "packed.cuh"

namespace kdn {
namespace {

constexpr int kMost = 256, kV = 8;    // threads of a block; channels of a lane
constexpr int kSMs = 152;             // GB300
// rows of a thread whose loads are under way: forward (together), backward (while one is worked on)
template <typename T> constexpr int kAt = sizeof(T) == 2 ? 4 : 2;
template <typename T> constexpr int kNext = sizeof(T) == 2 ? 2 : 1;
constexpr int kForwardBlocks = 3, kBackwardBlocks = 2;   // an SM
constexpr uint32_t kAll = 0xffffffffu;

struct NormParams {
    NormArgs a;
    int lanes, groups, rows;          // lanes of a group; groups and rows that a block has at a time
    int parts;                        // backward: rows of partial sums
};

constexpr int kPairs = kV / 2;
template <typename T> struct Vec;     // eight channels, as they are in memory
template <> struct Vec<__nv_bfloat16> {
    uint4 x;
    __device__ __forceinline__ void load(const void* p, long long i) {
        x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    }
    __device__ __forceinline__ void get(float2 (&y)[kPairs]) const {
        y[0] = unpack2(x.x); y[1] = unpack2(x.y); y[2] = unpack2(x.z); y[3] = unpack2(x.w);
    }
    __device__ __forceinline__ static void store(void* p, long long i, const float2 (&y)[kPairs]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(y[j].x, y[j].y);
            w[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Vec<float> {
    float4 x, z;
    __device__ __forceinline__ void load(const void* p, long long i) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        x = s[0];
        z = s[1];
    }
    __device__ __forceinline__ void get(float2 (&y)[kPairs]) const {
        y[0] = make_float2(x.x, x.y); y[1] = make_float2(x.z, x.w);
        y[2] = make_float2(z.x, z.y); y[3] = make_float2(z.z, z.w);
    }
    __device__ __forceinline__ static void store(void* p, long long i, const float2 (&y)[kPairs]) {
        float4* s = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        s[0] = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
        s[1] = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
    }
};

__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-x)).  The fast exponential is off by |x| 2^-23 of its value, which is nothing beside a rounding to bf16.
template <typename T> __device__ __forceinline__ float2 sigmoid(float2 x) {
    float2 e;
    if (sizeof(T) == 2) {
        e = mul2(x, both(-1.4426950408889634f));
        asm("ex2.approx.f32 %0, %0;" : "+f"(e.x));
        asm("ex2.approx.f32 %0, %0;" : "+f"(e.y));
    } else {
        e = make_float2(expf(-x.x), expf(-x.y));
    }
    e = add2(e, both(1.f));
    return make_float2(reciprocal(e.x), reciprocal(e.y));
}

// The activation of x, and its slope.
template <typename T, int ACT> __device__ __forceinline__ float2 act(float2 x, float2& slope) {
    if (ACT == KDN_ACT_NONE) {
        slope = both(1.f);
        return x;
    }
    const float2 h = sigmoid<T>(x), rest = fma2(h, both(-1.f), both(1.f));
    if (ACT == KDN_ACT_SIGMOID) {
        slope = mul2(h, rest);
        return h;
    }
    slope = mul2(h, fma2(x, rest, both(1.f)));
    return mul2(x, h);
}

// Sum over the lanes of a group (LANES: how many, 0: `lanes`).
template <int LANES> __device__ __forceinline__ float group_sum(float x, int lanes) {
    if (LANES) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    } else {
        for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    }
    return x;
}

// What a thread works on.
struct Place {
    int g, c, row, step;   // group, first channel in it, first row, rows to its next one
    bool mine;             // whether there is such a channel of such a group
};
__device__ __forceinline__ Place place_of(const NormParams& P) {
    Place p;
    const int at = threadIdx.x / P.lanes, lane = threadIdx.x % P.lanes;
    p.g = blockIdx.y * P.groups + at % P.groups;
    p.c = lane * kV;
    const int sub = at / P.groups;
    p.row = blockIdx.x * P.rows + sub;
    p.step = gridDim.x * P.rows;
    p.mine = sub < P.rows && p.g < P.a.groups && p.c < P.a.d;
    return p;
}

// A thread's channels of a weight or bias [groups, d].
__device__ __forceinline__ void parameters(const float* x, const Place& p, int d, float other, float2 (&y)[kPairs]) {
    const float* at = x + p.g * d + p.c;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) y[i] = x && p.mine ? make_float2(at[2 * i], at[2 * i + 1]) : both(other);
}
// Deviations from a group's mean, in place; returns 1 / sigma.
template <int LANES> __device__ __forceinline__ float normalise(float2 (&x)[kPairs], bool mine, float inv, float eps, int lanes) {
    float2 sum = add2(add2(x[0], x[1]), add2(x[2], x[3]));
    const float mean = group_sum<LANES>(sum.x + sum.y, lanes) * inv;
    float2 sq = both(0.f);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        x[i] = add2(x[i], both(-mean));
        sq = fma2(x[i], x[i], sq);
    }
    return rsqrtf(group_sum<LANES>(mine ? sq.x + sq.y : 0.f, lanes) * inv + eps);
}

// Whether the squares of deviations have kept to fp32's range, by what came out for 1 / sigma: not 0 (they were infinite), nor so large
// that they, with eps, were small and have lost digits.  As an unsigned number less one, 0 is the largest (and NaN is out of range, too).
// The kernels keep the worst of a thread's rows, one instruction a row (32768 tokens of 16 groups of 128, bf16, gate, in graphs: 72.9 us
// for 72.1 without, gradients 119.4 for 119.0; with a branch in the loop the forward took 74 to 76).
constexpr uint32_t kMostRstd = (127 + 50) << 23;   // 2^50
__device__ __forceinline__ bool in_range(float rstd) { return __float_as_uint(rstd) - 1 < kMostRstd; }
__device__ __forceinline__ uint32_t largest(float rstd, uint32_t x) { return __viaddmax_u32(__float_as_uint(rstd), 0xffffffffu, x); }

// Rows that were out of range once more, a warp together: their deviations are taken by a power of two before they are squared.  `part_w`,
// `part_b`: the thread's sums for the gradients of weight and bias, which these rows' norms are not in yet.
template <typename T, int ACT, bool GATE, bool BACK> __device__ __forceinline__ void rows_again(const NormParams& P, float* part_w, float* part_b) {
    const NormArgs& A = P.a;
    const Place p = place_of(P);
    float2 w[kPairs], b[kPairs], dw[kPairs] = {}, db[kPairs] = {};
    parameters(A.w, p, A.d, 1.f, w);
    parameters(A.b, p, A.d, 0.f, b);
    const float inv = 1.f / A.d;
#pragma unroll 1
    for (int row = p.row; __any_sync(kAll, row < A.rows); row += p.step) {
        const bool mine = p.mine && row < A.rows;
        Vec<T> v = {}, u = {}, t = {};
        if (mine) {
            v.load(A.x.p, row * A.x.row + p.g * A.x.head + p.c);
            if (BACK) u.load(A.dy.p, row * A.dy.row + p.g * A.dy.head + p.c);
            if (GATE) t.load(A.gate.p, row * A.gate.row + p.g * A.gate.head + p.c);
        }
        float2 x[kPairs], y[kPairs], z[kPairs];
        v.get(x);
        const bool now = !in_range(normalise<0>(x, mine, inv, A.eps, P.lanes)) && mine;
        float most = 0.f;
        for (int i = 0; i < kPairs; ++i) most = fmaxf(most, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
        most = mine ? most : 0.f;
        for (int o = P.lanes >> 1; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
        // 2^-e for a largest deviation of 2^e (from 2^-100 to 2^126)
        const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23), 27), 253);
        const float scale = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        float2 sq = both(0.f);
        for (int i = 0; i < kPairs; ++i) {
            x[i] = mul2(x[i], both(scale));
            sq = fma2(x[i], x[i], sq);
        }
        const float r = rsqrtf(fmaf(group_sum<0>(mine ? sq.x + sq.y : 0.f, P.lanes), inv, A.eps * scale * scale)), rstd = r * scale;
        u.get(y);
        if (GATE) t.get(z);
        float2 t1 = both(0.f), t2 = t1, slope;
        for (int i = 0; i < kPairs; ++i) {
            x[i] = mul2(x[i], both(r));
            const float2 n = fma2(x[i], w[i], b[i]);
            if (!BACK) {
                x[i] = GATE ? mul2(n, act<T, ACT>(z[i], slope)) : act<T, ACT>(n, slope);
                continue;
            }
            const float2 f = act<T, ACT>(GATE ? z[i] : n, slope), dn = mul2(y[i], GATE ? f : slope);
            if (GATE) z[i] = mul2(mul2(y[i], n), slope);
            if (now) dw[i] = fma2(dn, x[i], dw[i]);
            if (now && !GATE) db[i] = add2(db[i], dn);
            y[i] = mul2(dn, w[i]);
            t1 = add2(t1, y[i]);
            t2 = fma2(y[i], x[i], t2);
        }
        const long long at = (static_cast<long long>(row) * A.groups + p.g) * A.d + p.c;
        if (!BACK) {
            if (now) Vec<T>::store(A.y, at, x);
            continue;
        }
        const float s1 = group_sum<0>(mine ? t1.x + t1.y : 0.f, P.lanes) * inv, s2 = group_sum<0>(mine ? t2.x + t2.y : 0.f, P.lanes) * inv;
        if (!now) continue;
        for (int i = 0; i < kPairs; ++i) y[i] = mul2(both(rstd), fma2(x[i], both(-s2), add2(y[i], both(-s1))));
        Vec<T>::store(A.dx, at, y);
        if (GATE) Vec<T>::store(A.dgate, at, z);
    }
    auto add = [&](float* part, const float2 (&more)[kPairs]) {
        if (!part || !p.mine) return;
        float2 sum[kPairs];
        Vec<float> had;
        had.load(part, 0);
        had.get(sum);
        for (int i = 0; i < kPairs; ++i) sum[i] = add2(sum[i], more[i]);
        Vec<float>::store(part, 0, sum);
    };
    if (BACK) {
        add(part_w, dw);
        add(part_b, db);
    }
}

template <typename T, int ACT, bool GATE, int LANES> __global__ void __launch_bounds__(kMost) group_norm_kernel(const __grid_constant__ NormParams P) {
    const NormArgs& A = P.a;
    const Place p = place_of(P);
    float2 w[kPairs], b[kPairs];
    parameters(A.w, p, A.d, 1.f, w);
    parameters(A.b, p, A.d, 0.f, b);
    const float inv = 1.f / A.d;
    uint32_t worst = 0;
    // kAt rows at a time, their loads ahead of all else (all lanes of a warp go on together: the sums are shuffles)
    for (int row = p.row; __any_sync(kAll, row < A.rows); row += kAt<T> * p.step) {
        Vec<T> v[kAt<T>], gate[kAt<T>];
#pragma unroll
        for (int e = 0; e < kAt<T>; ++e) {
            const int r = row + e * p.step;
            if (p.mine && r < A.rows) {
                v[e].load(A.x.p, r * A.x.row + p.g * A.x.head + p.c);
                if (GATE) gate[e].load(A.gate.p, r * A.gate.row + p.g * A.gate.head + p.c);
            } else {
                v[e] = Vec<T>{};
            }
        }
#pragma unroll
        for (int e = 0; e < kAt<T>; ++e) {
            const int r = row + e * p.step;
            const bool mine = p.mine && r < A.rows;
            float2 x[kPairs];
            v[e].get(x);
            const float rstd = normalise<LANES>(x, mine, inv, A.eps, P.lanes);
            if (mine) {
                worst = largest(rstd, worst);
                float2 z[kPairs], slope;
                if (GATE) gate[e].get(z);
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const float2 n = fma2(mul2(x[i], both(rstd)), w[i], b[i]);
                    x[i] = GATE ? mul2(n, act<T, ACT>(z[i], slope)) : act<T, ACT>(n, slope);
                }
                Vec<T>::store(A.y, (static_cast<long long>(r) * A.groups + p.g) * A.d + p.c, x);
            }
        }
    }
    if (__any_sync(kAll, worst >= kMostRstd)) rows_again<T, ACT, GATE, false>(P, nullptr, nullptr);
}

template <typename T, int ACT, bool GATE, int LANES> __global__ void __launch_bounds__(kMost, kBackwardBlocks) group_norm_backward_kernel(const __grid_constant__ NormParams P) {
    const NormArgs& A = P.a;
    const Place p = place_of(P);
    if (blockIdx.x + blockIdx.y + threadIdx.x == 0) *A.status = 0;
    float2 w[kPairs], b[kPairs], dw[kPairs] = {}, db[kPairs] = {};
    parameters(A.w, p, A.d, 1.f, w);
    parameters(A.b, p, A.d, 0.f, b);
    const float inv = 1.f / A.d;
    // the next kNext rows' loads are under way while a row is worked on
    Vec<T> v[kNext<T>] = {}, u[kNext<T>] = {}, t[kNext<T>] = {};
    auto fetch = [&](int row, int e) {
        if (p.mine && row < A.rows) {
            v[e].load(A.x.p, row * A.x.row + p.g * A.x.head + p.c);
            u[e].load(A.dy.p, row * A.dy.row + p.g * A.dy.head + p.c);
            if (GATE) t[e].load(A.gate.p, row * A.gate.row + p.g * A.gate.head + p.c);
        }
    };
#pragma unroll
    for (int e = 0; e < kNext<T>; ++e) fetch(p.row + e * p.step, e);
    uint32_t worst = 0;
    for (int row0 = p.row; __any_sync(kAll, row0 < A.rows); row0 += kNext<T> * p.step)
#pragma unroll
    for (int e = 0; e < kNext<T>; ++e) {
        const int row = row0 + e * p.step;
        const bool mine = p.mine && row < A.rows;
        float2 x[kPairs], y[kPairs], z[kPairs];
        v[e].get(x);
        u[e].get(y);
        if (GATE) t[e].get(z);
        fetch(row + kNext<T> * p.step, e);
        const float rstd = normalise<LANES>(x, mine, inv, A.eps, P.lanes);
        const bool now = in_range(rstd) && mine;   // (else what its norm adds to the weights' gradients comes later)
        float2 t1 = both(0.f), t2 = t1;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const float2 xh = mul2(x[i], both(rstd)), n = fma2(xh, w[i], b[i]);
            float2 slope, dn;
            if (GATE) {
                const float2 f = act<T, ACT>(z[i], slope);
                z[i] = mul2(mul2(y[i], n), slope);
                dn = mul2(y[i], f);
            } else {
                act<T, ACT>(n, slope);
                dn = mul2(y[i], slope);
            }
            if (now) dw[i] = fma2(dn, xh, dw[i]);
            if (GATE ? mine : now) db[i] = add2(db[i], dn);   // (with a gate dn does not depend on the norm)
            x[i] = xh;
            y[i] = mul2(dn, w[i]);
            t1 = add2(t1, y[i]);
            t2 = fma2(y[i], xh, t2);
        }
        const float s1 = group_sum<LANES>(mine ? t1.x + t1.y : 0.f, P.lanes) * inv, s2 = group_sum<LANES>(mine ? t2.x + t2.y : 0.f, P.lanes) * inv;
        if (!mine) continue;
        worst = largest(rstd, worst);
        const long long at = (static_cast<long long>(row) * A.groups + p.g) * A.d + p.c;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) y[i] = mul2(both(rstd), fma2(x[i], both(-s2), add2(y[i], both(-s1))));
        Vec<T>::store(A.dx, at, y);
        if (GATE) Vec<T>::store(A.dgate, at, z);
    }
    float *const part = A.scratch + static_cast<size_t>(p.row) * A.groups * A.d + p.g * A.d + p.c, *const other = part + static_cast<size_t>(P.parts) * A.groups * A.d;
    if (p.mine) {
        if (A.dw) Vec<float>::store(part, 0, dw);
        if (A.db) Vec<float>::store(other, 0, db);
    }
    if (__any_sync(kAll, worst >= kMostRstd)) rows_again<T, ACT, GATE, true>(P, A.dw ? part : nullptr, A.db ? other : nullptr);
}

// Sums of the parts, a channel a lane: eight warps take every eighth part, and one adds them up.
__global__ void __launch_bounds__(kMost) group_norm_join_kernel(const __grid_constant__ NormParams P) {
    __shared__ float sums[8][33];
    const int n = P.a.groups * P.a.d, lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? P.a.db : P.a.dw;
    if (!out) return;
    const float* part = P.a.scratch + static_cast<size_t>(blockIdx.y) * P.parts * n;
    float sum = 0.f;
    if (c < n)
#pragma unroll 8
        for (int i = warp; i < P.parts; i += 8) sum += part[static_cast<size_t>(i) * n + c];
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp || c >= n) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += sums[i][lane];
    out[c] = sum;
}

// How the channels lie in a block's threads.
struct Shape {
    int lanes, groups, rows, blocks_y, threads;
};
Shape shape_of(int groups, int d) {
    Shape s;
    for (s.lanes = 1; s.lanes * kV < d; s.lanes *= 2) {}
    const int most = kMost / s.lanes;
    s.blocks_y = (groups + most - 1) / most;
    s.groups = (groups + s.blocks_y - 1) / s.blocks_y;
    s.rows = most / s.groups;
    s.threads = (s.rows * s.groups * s.lanes + 31) / 32 * 32;
    return s;
}
// Blocks for `each` rows of a thread at least (what more of them would save, the sum of their parts costs), but for 64 of them.
int blocks_x(const Shape& s, int rows, int per_sm, int each) {
    const long long want = (static_cast<long long>(rows) + s.rows - 1) / s.rows, room = std::max(1, per_sm * kSMs / s.blocks_y);
    return static_cast<int>(std::min(std::min(want, room), std::max(64ll, want / each)));
}
constexpr int kBackwardRows = 8;      // of a thread

template <typename T, int ACT, int LANES> void forward_lanes(const NormParams& P, dim3 grid, int threads, cudaStream_t s) {
    if (P.a.gate.p) group_norm_kernel<T, ACT, true, LANES><<<grid, threads, 0, s>>>(P);
    else group_norm_kernel<T, ACT, false, LANES><<<grid, threads, 0, s>>>(P);
}
template <typename T, int ACT> cudaError_t forward(const NormParams& P, dim3 grid, int threads, cudaStream_t s) {
    // heads of 64 and of 128 (the number of lanes known: 8 and 4 fewer instructions a sum), others
    if (P.lanes == 8) forward_lanes<T, ACT, 8>(P, grid, threads, s);
    else if (P.lanes == 16) forward_lanes<T, ACT, 16>(P, grid, threads, s);
    else forward_lanes<T, ACT, 0>(P, grid, threads, s);
    return cudaGetLastError();
}
template <typename T, int ACT, int LANES> void backward_lanes(const NormParams& P, dim3 grid, int threads, cudaStream_t s) {
    if (P.a.gate.p) group_norm_backward_kernel<T, ACT, true, LANES><<<grid, threads, 0, s>>>(P);
    else group_norm_backward_kernel<T, ACT, false, LANES><<<grid, threads, 0, s>>>(P);
}
template <typename T, int ACT> cudaError_t backward(const NormParams& P, dim3 grid, int threads, cudaStream_t s) {
    // heads of 64 and of 128 (the number of lanes known: 8 and 4 fewer instructions a sum), others
    if (P.lanes == 8) backward_lanes<T, ACT, 8>(P, grid, threads, s);
    else if (P.lanes == 16) backward_lanes<T, ACT, 16>(P, grid, threads, s);
    else backward_lanes<T, ACT, 0>(P, grid, threads, s);
    return cudaGetLastError();
}

NormParams params_of(const NormArgs& a, const Shape& s) {
    NormParams P = {};
    P.a = a;
    P.lanes = s.lanes; P.groups = s.groups; P.rows = s.rows;
    return P;
}

}  // namespace

size_t norm_scratch(int rows, int groups, int d) {
    if (rows <= 0 || groups <= 0) return 0;
    const Shape s = shape_of(groups, d);
    return 2 * sizeof(float) * static_cast<size_t>(blocks_x(s, rows, kBackwardBlocks, kBackwardRows)) * s.rows * groups * d;
}

cudaError_t launch_group_norm(const NormArgs& a, cudaStream_t s) {
    const Shape sh = shape_of(a.groups, a.d);
    const NormParams P = params_of(a, sh);
    const dim3 grid(blocks_x(sh, a.rows, kForwardBlocks, 1), sh.blocks_y);
    const auto run = [&](auto type) {
        using T = decltype(type);
        if (a.act == KDN_ACT_NONE) return forward<T, KDN_ACT_NONE>(P, grid, sh.threads, s);
        if (a.act == KDN_ACT_SILU) return forward<T, KDN_ACT_SILU>(P, grid, sh.threads, s);
        return forward<T, KDN_ACT_SIGMOID>(P, grid, sh.threads, s);
    };
    return a.io == KDN_BF16 ? run(__nv_bfloat16()) : run(float());
}

cudaError_t launch_group_norm_backward(const NormArgs& a, cudaStream_t s) {
    const Shape sh = shape_of(a.groups, a.d);
    NormParams P = params_of(a, sh);
    const dim3 grid(blocks_x(sh, a.rows, kBackwardBlocks, kBackwardRows), sh.blocks_y);
    P.parts = grid.x * sh.rows;
    const auto run = [&](auto type) {
        using T = decltype(type);
        if (a.act == KDN_ACT_NONE) return backward<T, KDN_ACT_NONE>(P, grid, sh.threads, s);
        if (a.act == KDN_ACT_SILU) return backward<T, KDN_ACT_SILU>(P, grid, sh.threads, s);
        return backward<T, KDN_ACT_SIGMOID>(P, grid, sh.threads, s);
    };
    const cudaError_t e = a.io == KDN_BF16 ? run(__nv_bfloat16()) : run(float());
    if (e != cudaSuccess || (!a.dw && !a.db)) return e;
    group_norm_join_kernel<<<dim3((a.groups * a.d + 31) / 32, 2), kMost, 0, s>>>(P);
    return cudaGetLastError();
}

}  // namespace kdn
