// Causal attention over whole prompts, CUDA-core path: fp32 operands (bf16 is widened),
// products in 3xTF32 on warp-level tensor-core MMAs.  Every size and type; the tcgen05
// kernel takes bf16 with heads of 64 and 128.

#include <cuda_bf16.h>

#include "attention.h"
#include "common.cuh"
#include "kdn.h"
#include "mma_tf32x3.cuh"

namespace kdn {
namespace {

constexpr int kThreads = 256, kRows = 64, kKeys = 64, kPad = 4;

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// One block per (64 query rows of a sequence, head); key tiles of 64 with the running
// maximum and sum of the softmax.  A masked key has no influence whatever it holds: keys
// outside the sequence are read as zeros, scores are masked by selection, and a value that
// is not finite is taken out of the tile and added to the rows that see it.
template <typename T, int D> __global__ void __launch_bounds__(kThreads) prompt_kernel(const PromptArgs a, int n_items) {
    constexpr int LD = D + kPad, LS = kKeys + kPad;
    extern __shared__ float prompt_smem[];
    float* Q = prompt_smem;
    float* K = Q + kRows * LD;
    float* V = K + kKeys * LD;
    float* O = V + kKeys * LD;
    float* S = O + kRows * LD;
    float* row_m = S + kRows * LS;
    float* row_l = row_m + kRows;
    float* row_f = row_l + kRows;
    __shared__ int found[5], odd_value;
    const int tid = threadIdx.x, h = blockIdx.y, kvh = h / (a.H / a.H_kv);
    if (tid == 0) {
        // item -> (sequence, row tile): sequences in order
        int item = blockIdx.x, s = 0;
        found[0] = -1;
        for (; s < a.n_seq; ++s) {
            const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
            const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k;
            if (!ok) {
                set_status(a.status, kStatusRange);
                continue;
            }
            const int tiles = (q1 - q0 + kRows - 1) / kRows;
            if (item < tiles) {
                found[0] = q0 + item * kRows;
                found[1] = min(kRows, q1 - q0 - item * kRows);
                found[2] = k0;
                found[3] = k1 - k0;
                found[4] = (k1 - k0) - (q1 - q0) + item * kRows;   // place of the tile's first row among the keys
                break;
            }
            item -= tiles;
        }
    }
    __syncthreads();
    const int q0 = found[0], rows = found[1], k0 = found[2], n_keys = found[3], place = found[4];
    if (q0 < 0) return;
    const T* q = static_cast<const T*>(a.q.p) + q0 * a.q.row + h * a.q.head;
    for (int i = tid; i < kRows * D; i += kThreads) {
        const int r = i / D, c = i % D;
        Q[r * LD + c] = r < rows ? IO<T>::load(q, r * a.q.row + c) : 0.f;
        O[r * LD + c] = 0.f;
    }
    for (int i = tid; i < kRows; i += kThreads) {
        row_m[i] = -INFINITY;
        row_l[i] = 0.f;
    }
    const int last = min(place + rows - 1, n_keys - 1);                       // last key any row sees
    const int low = a.window > 0 ? max(place - a.window + 1, 0) : 0;         // first
    const float to_log2 = a.scale * 1.4426950408889634f;
    for (int j0 = low / kKeys * kKeys; j0 <= last; j0 += kKeys) {
        if (tid == 0) odd_value = 0;
        __syncthreads();
        const T* k = static_cast<const T*>(a.k.p) + (static_cast<long long>(k0) + j0) * a.k.row + kvh * a.k.head;
        const T* v = static_cast<const T*>(a.v.p) + (static_cast<long long>(k0) + j0) * a.v.row + kvh * a.v.head;
        for (int i = tid; i < kKeys * D; i += kThreads) {
            const int r = i / D, c = i % D;
            const bool in = j0 + r < n_keys;
            K[r * LD + c] = in ? IO<T>::load(k, r * a.k.row + c) : 0.f;
            const float x = in ? IO<T>::load(v, r * a.v.row + c) : 0.f;
            V[r * LD + c] = finite(x) ? x : 0.f;
            if (!finite(x)) odd_value = 1;
        }
        __syncthreads();
        smem_gemm<4>(kRows, kKeys, D, Q, LD, 1, K, 1, LD, S, LS, 1.f, false);
        __syncthreads();
        {
            const int r = tid >> 2, c0 = (tid & 3) * (kKeys / 4), at = place + r;
            float x[kKeys / 4], mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < kKeys / 4; ++i) {
                const int j = j0 + c0 + i;
                const bool see = r < rows && j <= at && j < n_keys && (a.window <= 0 || j > at - a.window);
                x[i] = see ? S[r * LS + c0 + i] * to_log2 : -INFINITY;
                mx = fmaxf(mx, x[i]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float old = row_m[r], mn = fmaxf(old, mx), base = mn == -INFINITY ? 0.f : mn;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kKeys / 4; ++i) {
                const float p = exp2f(x[i] - base);
                S[r * LS + c0 + i] = p;
                sum += p;
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            __syncwarp();
            if ((tid & 3) == 0) {
                const float f = exp2f(old - base);
                row_f[r] = f;
                row_m[r] = mn;
                row_l[r] = row_l[r] * f + sum;
            }
        }
        __syncthreads();
        for (int i = tid; i < kRows * D; i += kThreads) O[i / D * LD + i % D] *= row_f[i / D];
        __syncthreads();
        smem_gemm<(D >= 32 ? 4 : 2)>(kRows, D, kKeys, S, LS, 1, V, LD, 1, O, LD, 1.f, true);
        __syncthreads();
        if (odd_value) {
            for (int i = tid; i < kRows * D; i += kThreads) {
                const int r = i / D, c = i % D, at = place + r;
                float acc = 0.f;
                for (int jj = 0; jj < kKeys; ++jj) {
                    const int j = j0 + jj;
                    if (r >= rows || j > at || j >= n_keys || (a.window > 0 && j <= at - a.window)) continue;
                    const float x = IO<T>::load(v, jj * a.v.row + c);
                    if (!finite(x)) acc += S[r * LS + jj] * x;
                }
                O[r * LD + c] += acc;
            }
            __syncthreads();
        }
    }
    __syncthreads();
    T* o = static_cast<T*>(a.o) + (static_cast<size_t>(q0) * a.H + h) * D;
    for (int i = tid; i < rows * D; i += kThreads) {
        const int r = i / D, c = i % D;
        const float l = row_l[r];
        IO<T>::store(o, static_cast<size_t>(r) * a.H * D + c, l != 0.f ? O[r * LD + c] / l : 0.f);
        if (c == 0)
            a.lse[(static_cast<size_t>(q0) + r) * a.H + h] =
                l != 0.f ? (row_m[r] + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <typename T, int D> cudaError_t launch(const PromptArgs& a, cudaStream_t s) {
    const size_t smem = sizeof(float) * (4 * kRows * (D + kPad) + kRows * (kKeys + kPad) + 3 * kRows);
    const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    // no more row tiles than this, whatever the lengths
    const long long items = a.total_q / kRows + static_cast<long long>(a.n_seq < a.total_q ? a.n_seq : a.total_q);
    const dim3 grid(static_cast<unsigned>(items), a.H);
    prompt_kernel<T, D><<<grid, kThreads, smem, s>>>(a, static_cast<int>(items));
    return cudaGetLastError();
}

template <typename T> cudaError_t by_size(const PromptArgs& a, cudaStream_t s) {
    if (a.d == 128) return launch<T, 128>(a, s);
    if (a.d == 64) return launch<T, 64>(a, s);
    if (a.d == 32) return launch<T, 32>(a, s);
    return launch<T, 16>(a, s);
}

}  // namespace

size_t prompt_scratch(int, int, int, int, int, int, uint32_t) { return 0; }

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s) {
    if (!(a.flags & KDN_FLAG_PORTABLE) && prompt_tc_supported(a.io, a.d)) return launch_prompt_tc(a, s);
    return a.io == 1 ? by_size<__nv_bfloat16>(a, s) : by_size<float>(a, s);
}

}  // namespace kdn
