// Attention of one query token per sequence over the paged 4-bit cache.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "common.cuh"

namespace kdn {
namespace {

constexpr int kThreads = 128;

// One block per (sequence, head); a tile of 128 tokens at a time, a thread per token for
// the scores and a thread per channel for the weighted sum, with the running maximum and
// sum of the softmax.
template <typename T, int D> __global__ void __launch_bounds__(kThreads) cache_attention_kernel(const CacheAttentionArgs a) {
    constexpr int G = D / 32;
    __shared__ float q[D], p[kThreads], red[kThreads / 32];
    const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, kvh = h / (a.H / a.H_kv);
    const long long room = min(static_cast<long long>(a.max_len), static_cast<long long>(a.table_width) * a.page);
    const int n = static_cast<int>(min(static_cast<long long>(max(a.seq_len[r], 0)), room));
    if (tid == 0 && n != a.seq_len[r]) set_status(a.status, kStatusRange);
    const int first = a.window > 0 ? max(n - a.window, 0) : 0;
    if (tid < D)
        q[tid] = IO<T>::load(static_cast<const T*>(a.q.p), r * a.q.row + h * a.q.head + tid) * a.scale * 1.4426950408889634f;
    __syncthreads();
    float m = -INFINITY, l = 0.f, o = 0.f;
    auto block = [&](int t) -> const uint8_t* {   // null for a page outside the cache
        const int id = a.block_table[static_cast<size_t>(r) * a.table_width + t / a.page];
        if (id < 0 || id >= a.n_pages) return nullptr;
        return a.cache + ((static_cast<size_t>(id) * a.H_kv + kvh) * (a.page / kBlockTokens) + t % a.page / kBlockTokens) *
                             cache_block_bytes(D);
    };
    for (int t0 = first; t0 < n; t0 += kThreads) {
        const int t = t0 + tid;
        const uint8_t* b = t < n ? block(t) : nullptr;
        if (t < n && !b) set_status(a.status, kStatusRange);
        float x = -INFINITY;
        if (b) {
            const int tt = t % kBlockTokens;
            x = 0.f;
            for (int g = 0; g < G; ++g) {
                float acc = 0.f;
                for (int c = 0; c < 4; ++c) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(b + tt * (D / 2) + (c * G + g) * 4);
                    for (int e = 0; e < 8; ++e)
                        acc = fmaf(static_cast<float>((w >> (4 * e)) & 15u) - 8.f, q[32 * g + 8 * c + e], acc);
                }
                x = fmaf(acc, __half2float(*reinterpret_cast<const __half*>(b + 8 * D + (tt * G + g) * 2)), x);
            }
        }
        float mx = x;
        for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        const float mn = fmaxf(fmaxf(m, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
        const float base = mn == -INFINITY ? 0.f : mn, w = exp2f(x - base), f = exp2f(m - base);
        m = mn;
        p[tid] = w;
        __syncthreads();
        o *= f;
        l *= f;
        for (int i = 0; i < kThreads && t0 + i < n; ++i) {
            l += p[i];
            if (tid < D && p[i] != 0.f) {
                const uint8_t* bb = block(t0 + i);
                const int tt = (t0 + i) % kBlockTokens, half = tt >> 3, pair = (tt >> 1) & 3, par = tt & 1;
                const int g8 = tid & 7, nib = (tid >> 3) & 3, g = tid >> 5;
                const uint32_t u = *reinterpret_cast<const uint16_t*>(bb + 9 * D + half * 4 * D + g8 * 16 * G + pair * 4 * G +
                                                                      g * 4 + par * 2);
                const float s = __half2float(
                    *reinterpret_cast<const __half*>(bb + 17 * D + half * (D / 2) + pair * 4 * G + g * 4 + par * 2));
                o = fmaf(p[i], (static_cast<float>((u >> (4 * nib)) & 15u) - 8.f) * s, o);
            }
        }
        __syncthreads();
    }
    const size_t row = static_cast<size_t>(r) * a.H + h;
    if (tid < D) IO<T>::store(static_cast<T*>(a.o), row * D + tid, l != 0.f ? o / l : 0.f);
    if (tid == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T> cudaError_t launch(const CacheAttentionArgs& a, cudaStream_t s) {
    const dim3 grid(a.H, a.n_seq);
    if (a.d == 128) cache_attention_kernel<T, 128><<<grid, kThreads, 0, s>>>(a);
    else if (a.d == 64) cache_attention_kernel<T, 64><<<grid, kThreads, 0, s>>>(a);
    else cache_attention_kernel<T, 32><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t cache_attention_scratch(int, int, int, int, int, int) { return 0; }

cudaError_t launch_cache_attention(const CacheAttentionArgs& a, cudaStream_t s) {
    return a.io == 1 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace kdn
