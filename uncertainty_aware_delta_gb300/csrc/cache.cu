// The paged 4-bit key/value cache: block tables and slot maps from request lengths
// (kdn_cache_plan), and tokens quantised into it and read back (kdn_cache_write,
// kdn_cache_read).  The cache's layout and the arithmetic are stated in include/kdn.h.
//
// Plan: two prefix sums over the requests (new tokens, new pages).  A few KB move, so what bounds it is the
// launch and one block's chain of scans: 7.5 us for 256 requests of one token, 16.3 us for 1000 prompts
// of 540,000 tokens (6.5 MB of slots and positions), where every token also takes a search, its request's lengths
// again and three divisions.
// Write: per group of 32 values the scale max |x| / 7 and the codes rint(x / s); read: (code - 8) s.  Bytes bound
// them: 2 d values in, 1.125 d bytes out of a token and head, and back.  65536 tokens of 4 heads of 128 in bf16, both
// ways 345 MB: 89 us, 3.9 TB/s (54 and 37; in fp32 63 and 64).  What is left to the copy rate: some 15 instructions a
// value written, which keep 71% of the issue slots busy (64% where they are read), and in the rest of the time loads
// are waited for.

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

// Pages that n tokens take (n plus a page may pass 2^31 where page is no power of two).
__device__ __forceinline__ int pages_of(int n, int page) {
    return static_cast<int>((static_cast<uint32_t>(n) + static_cast<uint32_t>(page) - 1u) / static_cast<uint32_t>(page));
}

__device__ __forceinline__ Request request(const PlanArgs& a, int r) {
    Request q;
    q.ctx = a.context_len[r];
    q.add = a.new_len[r];
    const long long total = static_cast<long long>(q.ctx) + q.add;
    q.ok = q.ctx >= 0 && q.add >= 0 && total <= static_cast<long long>(a.table_width) * a.page;
    q.add = max(q.add, 0);
    q.held = q.ok ? pages_of(q.ctx, a.page) : 0;
    q.need = q.ok ? pages_of(static_cast<int>(total), a.page) - q.held : 0;
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
        const int held = pages_of(a.context_len[r], a.page);
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

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32, kWriteUnroll = 2;

// 8 neighbouring values as they are stored; as fp32; and the largest bit pattern without sign among
// them, as fp32 bits (patterns order NaN above infinity above every number).
template <typename T> struct Eight;
template <> struct Eight<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const uint4*>(p)[0];
        b = reinterpret_cast<const uint4*>(p)[1];
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]);
    }
    __device__ __forceinline__ uint32_t largest() const {
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, v[i] & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    }
};
template <> struct Eight<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
        const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
    }
    __device__ __forceinline__ uint32_t largest() const {   // two halves at a time
        uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        return max(m << 16, m & 0xffff0000u);
    }
};
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes (offset 8) and scale of a 32-value group held by 4 neighbouring lanes, 8 values each.
// x / s, rounded once, without a division a value, by Markstein's correction (a quotient's residual
// in one fused operation): the product with the approximate reciprocal
// is off by at most 2^-22 of it, and its remainder x - q s (one fused operation) times the reciprocal
// takes that to 2^-44, while x / s, with 24 and 11 bits, is never nearer than 2^-36 to the middle of
// two fp32 numbers without being there.
template <typename T> __device__ __forceinline__ uint32_t quantise8(const Eight<T>& v, __half& scale) {
    const float m = __uint_as_float(v.largest());
    // m / 7, rounded once: the quotient by the rounded reciprocal, corrected by its remainder
    constexpr float kSeventh = 1.0f / 7.0f;
    const float q0 = m * kSeventh, q = fmaf(fmaf(-q0, 7.0f, m), kSeventh, q0);
    scale = m < INFINITY ? __float2half_rn(fminf(q, 65504.0f)) : __ushort_as_half(0x7fff);
    const float s = __half2float(scale);
    if (!(s > 0.0f)) return 0x88888888u;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    constexpr float kRound = 12582912.0f;   // 1.5 2^23: adding and subtracting it rounds to a whole number
    float x[8], t[8];
    v.widen(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = x[i] * inv, z = fmaf(fmaf(-y, s, x[i]), inv, y);
        t[i] = __fsub_rn(__fadd_rn(fminf(fmaxf(z, -7.0f), 7.0f), kRound), kRound);
    }
    // four codes at a time as one exact fp32 number, whose low bits are read off its sum with 2^23
    float lo = 8423560.0f, hi = 8423560.0f;   // 2^23 + 8 (1 + 16 + 256 + 4096)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo = fmaf(t[i], static_cast<float>(1 << (4 * i)), lo);
        hi = fmaf(t[i + 4], static_cast<float>(1 << (4 * i)), hi);
    }
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

// Places of a lane's pieces within a token's block: 8 values of channel dd (a multiple of 8),
// the n-th eight of their group of 32.
struct Place {
    int k_code, k_scale, v_code, v_scale;   // v_code: of the even one of the lane's two units
};
template <int D> __device__ __forceinline__ Place place(int t, int dd) {
    constexpr int G = D / 32;
    const int m = dd >> 5, n = (dd >> 3) & 3, half = t >> 3, pair = (t >> 1) & 3, par = t & 1;
    Place p;
    p.k_code = t * (D / 2) + (n * G + m) * 4;
    p.k_scale = 8 * D + (t * G + m) * 2;
    // the 16-bit units i of channels 32 m + 8 j + i, j = 0..3; lane n of the group has units 2 n, 2 n + 1
    p.v_code = 9 * D + half * 4 * D + 2 * n * 16 * G + pair * 4 * G + m * 4 + par * 2;
    p.v_scale = 17 * D + half * (D / 2) + pair * 4 * G + m * 4 + par * 2;
    return p;
}

// Lanes n = 0..3 of a group hold the codes of channels 8 n + i (i = 0..7) of it; they get the units
// 2 n (low half) and 2 n + 1 (high half): unit i has the codes of channels 8 j + i in nibbles j.
__device__ __forceinline__ uint32_t units_of(uint32_t code, int n) {
    const uint32_t even = code & 0x0f0f0f0fu, odd = (code >> 4) & 0x0f0f0f0fu;
    uint32_t r[4];   // codes 2 i and 2 i + 1, a half each, in nibble n
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (__byte_perm(even, odd, i | (4 + i) << 8) & 0x000f000fu) << (4 * n);
    const uint32_t a = __shfl_xor_sync(0xffffffffu, n & 2 ? r[0] : r[2], 2);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, n & 2 ? r[1] : r[3], 2);
    const uint32_t k0 = (n & 2 ? r[2] : r[0]) | a, k1 = (n & 2 ? r[3] : r[1]) | b;
    return (n & 1 ? k1 : k0) | __shfl_xor_sync(0xffffffffu, n & 1 ? k0 : k1, 1);
}

// Whether the warp's 16 slots are one aligned block of the cache, in order.
__device__ __forceinline__ bool whole_block(int64_t slot, int n, int64_t n_slots) {
    const int lane = threadIdx.x & 31;
    const int64_t s0 = __shfl_sync(0xffffffffu, slot, 0);
    const bool fits = lane >= kBlockTokens || slot == s0 + lane;
    return __all_sync(0xffffffffu, fits) && n == kBlockTokens && s0 >= 0 && (s0 & (kBlockTokens - 1)) == 0 && s0 < n_slots;
}

template <int D> __device__ __forceinline__ size_t block_offset(const CacheArgs& a, int64_t slot, int h) {
    // a division of 64-bit numbers costs some hundred instructions: only where a slot needs one
    const int64_t page = slot >> 32 ? slot / a.page : static_cast<int64_t>(static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page));
    const int blk = static_cast<int>(slot - page * a.page) / kBlockTokens;
    return ((static_cast<size_t>(page) * a.H_kv + h) * (a.page / kBlockTokens) + blk) * cache_block_bytes(D);
}

// A warp takes TOK consecutive tokens of one key head, 256 / D of them at a time, each
// lane 8 channels.
template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kRowThreads) cache_write_kernel(const CacheArgs a) {
    constexpr int kBytes = cache_block_bytes(D), kStep = 256 / D, G = D / 32;
    __shared__ __align__(16) uint8_t stage[TOK == kBlockTokens ? kRowWarps * kBytes : 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kRowWarps + warp, tile = unit / static_cast<unsigned>(a.H_kv);   // (below 2^31)
    const int h = static_cast<int>(unit - tile * a.H_kv);
    const long long t0 = static_cast<long long>(tile) * TOK;
    if (t0 >= a.n_tok) return;
    const int n_here = static_cast<int>(min(static_cast<long long>(TOK), a.n_tok - t0));
    const int64_t n_slots = static_cast<int64_t>(a.n_pages) * a.page;
    const int64_t mine = lane < n_here ? a.slots[t0 + lane] : -1;
    const bool whole = TOK == kBlockTokens && whole_block(mine, n_here, n_slots);
    uint8_t* buf = stage + (TOK == kBlockTokens ? warp * kBytes : 0);
    const int dd = (8 * lane) % D, n = (dd >> 3) & 3;
    const T* k = static_cast<const T*>(a.k.p) + t0 * a.k.row + h * a.k.head + dd;
    const T* v = static_cast<const T*>(a.v.p) + t0 * a.v.row + h * a.v.head + dd;
#pragma unroll kWriteUnroll
    for (int i = 0; i < (TOK + kStep - 1) / kStep; ++i) {
        const int t = i * kStep + 8 * lane / D;
        const int64_t slot = __shfl_sync(0xffffffffu, mine, t & 31);
        const bool live = whole || (t < n_here && slot >= 0 && slot < n_slots);
        Eight<T> kk = {}, vv = {};
        if (live) {
            kk.load(k + t * a.k.row);
            vv.load(v + t * a.v.row);
        }
        __half sk, sv;
        const uint32_t ck = quantise8(kk, sk), units = units_of(quantise8(vv, sv), n);
        if (whole) {
            // a token's unit and the next's are one word: the even token's lane writes unit 2 n, the odd one's 2 n + 1
            const uint32_t next = __shfl_xor_sync(0xffffffffu, units, D / 8);
            const Place p = place<D>(t, dd);
            *reinterpret_cast<uint32_t*>(buf + p.k_code) = ck;
            *reinterpret_cast<uint32_t*>(buf + p.v_code + (t & 1) * (16 * G - 2)) =
                t & 1 ? (next >> 16) | (units & 0xffff0000u) : (units & 0xffffu) | (next << 16);
            if (n == 0) {
                *reinterpret_cast<__half*>(buf + p.k_scale) = sk;
                *reinterpret_cast<__half*>(buf + p.v_scale) = sv;
            }
        } else if (live) {
            uint8_t* blk = a.cache + block_offset<D>(a, slot, h);
            const Place p = place<D>(static_cast<int>(slot & (kBlockTokens - 1)), dd);
            *reinterpret_cast<uint32_t*>(blk + p.k_code) = ck;
            *reinterpret_cast<uint16_t*>(blk + p.v_code) = static_cast<uint16_t>(units);
            *reinterpret_cast<uint16_t*>(blk + p.v_code + 16 * G) = static_cast<uint16_t>(units >> 16);
            if (n == 0) {
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
    constexpr int kBytes = cache_block_bytes(D), kStep = 256 / D, G = D / 32;
    __shared__ __align__(16) uint8_t stage[TOK == kBlockTokens ? kRowWarps * kBytes : 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kRowWarps + warp, tile = unit / static_cast<unsigned>(a.H_kv);   // (below 2^31)
    const int h = static_cast<int>(unit - tile * a.H_kv);
    const long long t0 = static_cast<long long>(tile) * TOK;
    if (t0 >= a.n_tok) return;
    const int n_here = static_cast<int>(min(static_cast<long long>(TOK), a.n_tok - t0));
    const int64_t n_slots = static_cast<int64_t>(a.n_pages) * a.page;
    const int64_t mine = lane < n_here ? a.slots[t0 + lane] : -1;
    const bool whole = TOK == kBlockTokens && whole_block(mine, n_here, n_slots);
    uint8_t* buf = stage + (TOK == kBlockTokens ? warp * kBytes : 0);
    if (whole) {
        const uint4* src =
            reinterpret_cast<const uint4*>(a.cache + block_offset<D>(a, __shfl_sync(0xffffffffu, mine, 0), h));
        for (int i = lane; i < kBytes / 16; i += 32) reinterpret_cast<uint4*>(buf)[i] = src[i];
        __syncwarp();
    }
    const int dd = (8 * lane) % D, n = (dd >> 3) & 3;
    T* k = static_cast<T*>(a.k_out) + (t0 * a.H_kv + h) * D + dd;
    T* v = static_cast<T*>(a.v_out) + (t0 * a.H_kv + h) * D + dd;
#pragma unroll 4
    for (int i = 0; i < (TOK + kStep - 1) / kStep; ++i) {
        const int t = i * kStep + 8 * lane / D;
        const int64_t slot = __shfl_sync(0xffffffffu, mine, t & 31);
        const bool live = whole || (t < n_here && slot >= 0 && slot < n_slots);
        uint32_t ck = 0x88888888u, units = 0x88888888u;
        float sk = 0.0f, sv = 0.0f;
        if (live) {
            const uint8_t* blk = whole ? buf : a.cache + block_offset<D>(a, slot, h);
            const Place p = place<D>(whole ? t : static_cast<int>(slot & (kBlockTokens - 1)), dd);
            ck = *reinterpret_cast<const uint32_t*>(blk + p.k_code);
            units = *reinterpret_cast<const uint16_t*>(blk + p.v_code) |
                    static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(blk + p.v_code + 16 * G)) << 16;
            sk = __half2float(*reinterpret_cast<const __half*>(blk + p.k_scale));
            sv = __half2float(*reinterpret_cast<const __half*>(blk + p.v_scale));
        }
        // 2^23 + code as fp32 bits, less 2^23 + 8
        auto value = [](uint32_t code, float s) { return (__uint_as_float((code & 15u) | 0x4b000000u) - 8388616.0f) * s; };
        float xk[8], xv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xk[j] = value(ck >> (4 * j), sk);
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // units 2 j and 2 j + 1, of lane j of the group; this lane's are nibbles n
            const uint32_t u = __shfl_sync(0xffffffffu, units, (lane & ~3) | j) >> (4 * n);
            xv[2 * j] = value(u, sv);
            xv[2 * j + 1] = value(u >> 16, sv);
        }
        if (t < n_here) {
            store8(k + static_cast<size_t>(t) * a.H_kv * D, xk);
            store8(v + static_cast<size_t>(t) * a.H_kv * D, xv);
        }
    }
}

// One step of 256 / D tokens a warp: many short warps.  For large calls sixteen tokens, so that whole blocks
// move in 16-byte pieces.  Tokens of 4 heads of 128 in page order, write and read in us, steps against sixteens:
// 256: 4.1 and 4.1 against 10.2 and 6.2; 8192: 10.3 and 8.2 against 12.3 and 8.2; 16384: 16.4 and 12.3 against
// 18.4 and 12.3; 65536: 57.9 and 43.0 against 55.3 and 36.9; 131072: 111 and 82 against 100 and 68 (scattered, the
// two are within a tenth from 24576 on).
template <typename T, int D, bool WRITE> cudaError_t launch_rows(const CacheArgs& a, cudaStream_t s) {
    const long long big = (static_cast<long long>(a.n_tok) + kBlockTokens - 1) / kBlockTokens * a.H_kv;
    const bool few = big * kBlockTokens * D <= 1ll << 23;
    constexpr int kStep = 256 / D;
    const long long units = few ? (static_cast<long long>(a.n_tok) + kStep - 1) / kStep * a.H_kv : big;
    const long long grid = (units + kRowWarps - 1) / kRowWarps;
    if (grid > 0x7fffffffll / kRowWarps) return cudaErrorInvalidValue;
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
    auto bytes = [](int n_req) { return static_cast<int>(sizeof(int)) * 2 * (n_req + 1); };
    // the limit is the kernel's, shared by all host threads: always the same one, whatever this call needs
    const int smem = bytes(a.n_req);
    const cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               bytes(kPlanMaxRequests));
    if (e != cudaSuccess) return e;
    const long long items = a.capacity > a.n_req ? a.capacity : a.n_req + 1;
    const long long want = (items + kPlanThreads - 1) / kPlanThreads;
    cache_plan_kernel<<<static_cast<int>(want < 152 ? want : 152), kPlanThreads, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_write(const CacheArgs& a, cudaStream_t s) { return dispatch_rows<true>(a, s); }
cudaError_t launch_cache_read(const CacheArgs& a, cudaStream_t s) { return dispatch_rows<false>(a, s); }

}  // namespace kdn
