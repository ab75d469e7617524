// The paged 4-bit key/value cache: block tables and slot maps from request lengths
// (kdn_cache_plan), and tokens quantised into it and read back (kdn_cache_write,
// kdn_cache_read).  The cache's layout and the arithmetic are stated in include/kdn.h.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "common.cuh"

namespace kdn {
namespace {

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512;

__device__ __forceinline__ long long warp_scan(long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

struct Request {
    int ctx, add, held, need;
    bool ok;   // lengths in range
};

__device__ __forceinline__ Request request(const PlanArgs& a, int r) {
    Request q;
    q.ctx = a.context_len[r];
    q.add = a.new_len[r];
    const long long total = static_cast<long long>(q.ctx) + q.add;
    q.ok = q.ctx >= 0 && q.add >= 0 && total <= static_cast<long long>(a.table_width) * a.page;
    q.add = max(q.add, 0);
    q.held = q.ok ? (q.ctx + a.page - 1) / a.page : 0;
    q.need = q.ok ? static_cast<int>((total + a.page - 1) / a.page) - q.held : 0;
    return q;
}

// Every block scans all requests (tokens and pages wanted before each) into shared
// memory and then writes its share of the tokens' slots, the new table entries and the
// per-request results: one launch, and no block waits for another.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanArgs a) {
    extern __shared__ int plan_smem[];
    int* cu = plan_smem;                      // [n_req + 1] tokens before request r
    int* wanted = plan_smem + a.n_req + 1;    // [n_req + 1] pages wanted before request r
    __shared__ long long part[2][kPlanThreads / 32];
    __shared__ int bad_any;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int free_n = min(max(a.free_count[0], 0), a.n_free);
    if (tid == 0) {
        bad_any = a.free_count[0] != free_n;
        cu[0] = 0;
        wanted[0] = 0;
    }
    __syncthreads();
    long long base_t = 0, base_p = 0;
    for (int r0 = 0; r0 < a.n_req; r0 += kPlanThreads) {
        const int r = r0 + tid;
        long long t = 0, p = 0;
        if (r < a.n_req) {
            const Request q = request(a, r);
            t = q.add;
            p = q.need;
            if (!q.ok) bad_any = 1;
        }
        t = warp_scan(t);
        p = warp_scan(p);
        if (lane == 31) {
            part[0][warp] = t;
            part[1][warp] = p;
        }
        __syncthreads();
        long long bt = base_t, bp = base_p;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const long long xt = part[0][w], xp = part[1][w];
            if (w < warp) {
                bt += xt;
                bp += xp;
            }
            base_t += xt;
            base_p += xp;
        }
        if (r < a.n_req) {   // (sums past 32 bits are past every capacity and free list)
            cu[r + 1] = static_cast<int>(min(bt + t, 0x7fffffffll));
            wanted[r + 1] = static_cast<int>(min(bp + p, 0x7fffffffll));
        }
        __syncthreads();
    }
    const int total = cu[a.n_req], stride = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
    if (blockIdx.x == 0 && tid == 0) {
        // pages taken: the largest prefix of wanted pages that the free list covers
        int lo = 0, hi = a.n_req;
        while (lo < hi) {
            const int m = (lo + hi + 1) / 2;
            if (wanted[m] <= free_n) lo = m;
            else hi = m - 1;
        }
        a.free_left[0] = free_n - wanted[lo];
        *a.status = (bad_any || total > a.capacity) ? kStatusRange : 0u;
    }
    // (the need itself decides, not the difference of two prefixes, which may be saturated)
    auto is_granted = [&](const Request& q, int r) { return q.ok && (q.need == 0 || wanted[r + 1] <= free_n); };
    for (int r = first; r <= a.n_req; r += stride) {
        a.cu_new[r] = cu[r];
        if (r == a.n_req) break;
        const Request q = request(a, r);
        const bool g = is_granted(q, r);
        a.granted[r] = g;
        a.seq_len[r] = g ? q.ctx + q.add : q.ctx;
    }
    auto find = [&](const int* pre, int i) {   // the r with pre[r] <= i < pre[r + 1]
        int lo = 0, hi = a.n_req - 1;
        while (lo < hi) {
            const int m = (lo + hi) / 2;
            if (pre[m + 1] > i) hi = m;
            else lo = m + 1;
        }
        return lo;
    };
    const int n_new = min(wanted[a.n_req], free_n);   // entries past the last grant are skipped below
    for (int i = first; i < n_new; i += stride) {
        const int r = find(wanted, i);
        if (wanted[r + 1] > free_n) continue;
        const int held = (a.context_len[r] + a.page - 1) / a.page;
        a.block_table[static_cast<size_t>(r) * a.table_width + held + i - wanted[r]] = a.free_pages[free_n - 1 - i];
    }
    for (int i = first; i < a.capacity; i += stride) {
        int64_t slot = -1;
        int pos = 0;
        if (i < total) {
            const int r = find(cu, i);
            const Request q = request(a, r);
            pos = q.ctx + (i - cu[r]);
            if (is_granted(q, r)) {
                const int p = pos / a.page;
                const int id = p < q.held ? a.block_table[static_cast<size_t>(r) * a.table_width + p]
                                          : a.free_pages[free_n - 1 - (wanted[r] + p - q.held)];
                slot = static_cast<int64_t>(id) * a.page + (pos - p * a.page);
            }
        }
        a.slot_map[i] = slot;
        a.position[i] = pos;
    }
}

// ------------------------------------------------------------------ write and read

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;

template <typename T> __device__ __forceinline__ void load4(const T* p, float (&x)[4]);
template <> __device__ __forceinline__ void load4<float>(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <> __device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}

// Codes (offset 8) and scale of a 32-value group held by 8 neighbouring lanes, 4 values
// each.  The largest magnitude is taken on the bit patterns, which order NaN above
// infinity above every number, so one test afterwards finds a value that is not finite.
__device__ __forceinline__ uint32_t quantise4(const float (&x)[4], __half& scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    scale = m >= 0x7f800000u ? __ushort_as_half(0x7fff)
                             : __float2half_rn(fminf(__fdiv_rn(__uint_as_float(m), 7.0f), 65504.0f));
    const float s = __half2float(scale);
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float q = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.0f), 7.0f) : 0.0f;
        code |= static_cast<uint32_t>(static_cast<int>(q) + 8) << (4 * i);
    }
    return code;
}

// Places of a lane's pieces within a token's block: 4 values of channel dd (a multiple of 4).
struct Place {
    int k_code, k_scale, v_code, v_scale;
};
template <int D> __device__ __forceinline__ Place place(int t, int dd) {
    constexpr int G = D / 32;
    const int m = dd >> 5, c = (dd >> 3) & 3, odd = (dd >> 2) & 1;
    const int half = t >> 3, pair = (t >> 1) & 3, par = t & 1;
    Place p;
    p.k_code = t * (D / 2) + (c * G + m) * 4 + odd * 2;
    p.k_scale = 8 * D + (t * G + m) * 2;
    // the 16-bit unit of channels 32 m + 8 n + (4 odd + c), n = 0..3
    p.v_code = 9 * D + half * 4 * D + (4 * odd + c) * 16 * G + pair * 4 * G + m * 4 + par * 2;
    p.v_scale = 17 * D + half * (D / 2) + pair * 4 * G + m * 4 + par * 2;
    return p;
}

// Whether the warp's 16 slots are one aligned block of the cache, in order.
__device__ __forceinline__ bool whole_block(int64_t slot, int n, int64_t n_slots) {
    const int lane = threadIdx.x & 31;
    const int64_t s0 = __shfl_sync(0xffffffffu, slot, 0);
    const bool fits = lane >= kBlockTokens || slot == s0 + lane;
    return __all_sync(0xffffffffu, fits) && n == kBlockTokens && s0 >= 0 && s0 % kBlockTokens == 0 && s0 < n_slots;
}

template <int D> __device__ __forceinline__ size_t block_offset(const CacheArgs& a, int64_t slot, int h) {
    const int64_t page = slot / a.page;
    const int blk = static_cast<int>(slot - page * a.page) / kBlockTokens;
    return ((static_cast<size_t>(page) * a.H_kv + h) * (a.page / kBlockTokens) + blk) * cache_block_bytes(D);
}

// A warp takes TOK consecutive tokens of one key head, 128 / D of them at a time, each
// lane 4 channels.
template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kRowThreads) cache_write_kernel(const CacheArgs a) {
    constexpr int kBytes = cache_block_bytes(D), kStep = 128 / D;
    __shared__ __align__(16) uint8_t stage[TOK == kBlockTokens ? kRowWarps * kBytes : 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long unit = static_cast<long long>(blockIdx.x) * kRowWarps + warp;
    const int h = static_cast<int>(unit % a.H_kv);
    const long long t0 = unit / a.H_kv * TOK;
    if (t0 >= a.n_tok) return;
    const int n = static_cast<int>(min(static_cast<long long>(TOK), a.n_tok - t0));
    const int64_t n_slots = static_cast<int64_t>(a.n_pages) * a.page;
    const int64_t mine = lane < n ? a.slots[t0 + lane] : -1;
    const bool whole = TOK == kBlockTokens && whole_block(mine, n, n_slots);
    uint8_t* buf = stage + (TOK == kBlockTokens ? warp * kBytes : 0);
    const T* k = static_cast<const T*>(a.k.p) + t0 * a.k.row + h * a.k.head;
    const T* v = static_cast<const T*>(a.v.p) + t0 * a.v.row + h * a.v.head;
    const int dd = (4 * lane) % D;
#pragma unroll 4
    for (int i = 0; i < (TOK + kStep - 1) / kStep; ++i) {
        const int t = i * kStep + 4 * lane / D;
        const int64_t slot = __shfl_sync(0xffffffffu, mine, t & 31);
        const bool live = t < n && slot >= 0 && slot < n_slots;
        float xk[4] = {0.f, 0.f, 0.f, 0.f}, xv[4] = {0.f, 0.f, 0.f, 0.f};
        if (live) {
            load4(k + t * a.k.row + dd, xk);
            load4(v + t * a.v.row + dd, xv);
        }
        __half sk, sv;
        const uint32_t ck = quantise4(xk, sk), cv = quantise4(xv, sv);
        // lanes n = 0..3 of a group half hold nibble n of the half's four 16-bit units:
        // lane n collects unit n
        const int nib = (dd >> 3) & 3;
        uint32_t lo = (cv & 15u) | (((cv >> 4) & 15u) << 16), hi = ((cv >> 8) & 15u) | ((cv >> 12) << 16);
        lo <<= 4 * nib;
        hi <<= 4 * nib;
#pragma unroll
        for (int o = 2; o <= 4; o <<= 1) {
            lo |= __shfl_xor_sync(0xffffffffu, lo, o);
            hi |= __shfl_xor_sync(0xffffffffu, hi, o);
        }
        const uint32_t both = nib < 2 ? lo : hi;
        const uint16_t unit16 = static_cast<uint16_t>((nib & 1) ? both >> 16 : both);
        if (live) {
            uint8_t* blk = whole ? buf : a.cache + block_offset<D>(a, slot, h);
            const Place p = place<D>(static_cast<int>(slot % kBlockTokens), dd);
            *reinterpret_cast<uint16_t*>(blk + p.k_code) = static_cast<uint16_t>(ck);
            *reinterpret_cast<uint16_t*>(blk + p.v_code) = unit16;
            if ((dd & 31) == 0) {
                *reinterpret_cast<__half*>(blk + p.k_scale) = sk;
                *reinterpret_cast<__half*>(blk + p.v_scale) = sv;
            }
        }
    }
    if (whole) {
        __syncwarp();
        uint4* dst = reinterpret_cast<uint4*>(a.cache + block_offset<D>(a, __shfl_sync(0xffffffffu, mine, 0), h));
        for (int i = lane; i < kBytes / 16; i += 32) dst[i] = reinterpret_cast<const uint4*>(buf)[i];
    }
}

template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(const CacheArgs a) {
    constexpr int kBytes = cache_block_bytes(D), kStep = 128 / D;
    __shared__ __align__(16) uint8_t stage[TOK == kBlockTokens ? kRowWarps * kBytes : 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long unit = static_cast<long long>(blockIdx.x) * kRowWarps + warp;
    const int h = static_cast<int>(unit % a.H_kv);
    const long long t0 = unit / a.H_kv * TOK;
    if (t0 >= a.n_tok) return;
    const int n = static_cast<int>(min(static_cast<long long>(TOK), a.n_tok - t0));
    const int64_t n_slots = static_cast<int64_t>(a.n_pages) * a.page;
    const int64_t mine = lane < n ? a.slots[t0 + lane] : -1;
    const bool whole = TOK == kBlockTokens && whole_block(mine, n, n_slots);
    uint8_t* buf = stage + (TOK == kBlockTokens ? warp * kBytes : 0);
    if (whole) {
        const uint4* src =
            reinterpret_cast<const uint4*>(a.cache + block_offset<D>(a, __shfl_sync(0xffffffffu, mine, 0), h));
        for (int i = lane; i < kBytes / 16; i += 32) reinterpret_cast<uint4*>(buf)[i] = src[i];
        __syncwarp();
    }
    T* k = static_cast<T*>(a.k_out) + (t0 * a.H_kv + h) * D;
    T* v = static_cast<T*>(a.v_out) + (t0 * a.H_kv + h) * D;
    const int dd = (4 * lane) % D;
#pragma unroll 4
    for (int i = 0; i < (TOK + kStep - 1) / kStep; ++i) {
        const int t = i * kStep + 4 * lane / D;
        const int64_t slot = __shfl_sync(0xffffffffu, mine, t & 31);
        const bool live = t < n && slot >= 0 && slot < n_slots;
        uint32_t ck = 0x8888u, unit16 = 0x8888u;
        float sk = 0.0f, sv = 0.0f;
        if (live) {
            const uint8_t* blk = whole ? buf : a.cache + block_offset<D>(a, slot, h);
            const Place p = place<D>(static_cast<int>(slot % kBlockTokens), dd);
            ck = *reinterpret_cast<const uint16_t*>(blk + p.k_code);
            unit16 = *reinterpret_cast<const uint16_t*>(blk + p.v_code);
            sk = __half2float(*reinterpret_cast<const __half*>(blk + p.k_scale));
            sv = __half2float(*reinterpret_cast<const __half*>(blk + p.v_scale));
        }
        const int nib = (dd >> 3) & 3;
        float xk[4], xv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // value j: nibble `nib` of the unit that lane j of the half holds
            const uint32_t u = __shfl_sync(0xffffffffu, unit16, (lane & ~6) | (j << 1));
            xk[j] = (static_cast<float>((ck >> (4 * j)) & 15u) - 8.0f) * sk;
            xv[j] = (static_cast<float>((u >> (4 * nib)) & 15u) - 8.0f) * sv;
        }
        if (t < n) {
            store4(k + static_cast<size_t>(t) * a.H_kv * D + dd, xk);
            store4(v + static_cast<size_t>(t) * a.H_kv * D + dd, xv);
        }
    }
}

// Sixteen tokens a warp, so that whole blocks move in 16-byte pieces, unless that
// leaves SMs without a block of threads: then one step of 128 / D tokens a warp.
template <typename T, int D, bool WRITE> cudaError_t launch_rows(const CacheArgs& a, cudaStream_t s) {
    const long long big = (static_cast<long long>(a.n_tok) + kBlockTokens - 1) / kBlockTokens * a.H_kv;
    const bool few = big < 152ll * kRowWarps;
    constexpr int kStep = 128 / D;
    const long long units = few ? (static_cast<long long>(a.n_tok) + kStep - 1) / kStep * a.H_kv : big;
    const long long grid = (units + kRowWarps - 1) / kRowWarps;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    const int g = static_cast<int>(grid);
    if (WRITE) {
        if (few) cache_write_kernel<T, D, kStep><<<g, kRowThreads, 0, s>>>(a);
        else cache_write_kernel<T, D, kBlockTokens><<<g, kRowThreads, 0, s>>>(a);
    } else {
        if (few) cache_read_kernel<T, D, kStep><<<g, kRowThreads, 0, s>>>(a);
        else cache_read_kernel<T, D, kBlockTokens><<<g, kRowThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <bool WRITE> cudaError_t dispatch_rows(const CacheArgs& a, cudaStream_t s) {
    if (a.io == 1) {
        if (a.d == 128) return launch_rows<__nv_bfloat16, 128, WRITE>(a, s);
        if (a.d == 64) return launch_rows<__nv_bfloat16, 64, WRITE>(a, s);
        return launch_rows<__nv_bfloat16, 32, WRITE>(a, s);
    }
    if (a.d == 128) return launch_rows<float, 128, WRITE>(a, s);
    if (a.d == 64) return launch_rows<float, 64, WRITE>(a, s);
    return launch_rows<float, 32, WRITE>(a, s);
}

}  // namespace

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t s) {
    const size_t smem = sizeof(int) * 2 * (static_cast<size_t>(a.n_req) + 1);
    const cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const long long items = a.capacity > a.n_req ? a.capacity : a.n_req + 1;
    const long long want = (items + kPlanThreads - 1) / kPlanThreads;
    cache_plan_kernel<<<static_cast<int>(want < 152 ? want : 152), kPlanThreads, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_write(const CacheArgs& a, cudaStream_t s) { return dispatch_rows<true>(a, s); }
cudaError_t launch_cache_read(const CacheArgs& a, cudaStream_t s) { return dispatch_rows<false>(a, s); }

}  // namespace kdn
