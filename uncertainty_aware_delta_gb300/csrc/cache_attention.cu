// Attention of one query token per sequence over the paged 4-bit cache.
//
// The work is a row of units, 256 tokens of one sequence for up to eight query heads of one key
// head, and every block takes an equal share of it: a segment of one or several rows.  A
// block's warps each take every fourth step of 64 tokens with a running maximum and sum and
// are joined in shared memory; a second kernel joins the rows that were cut.
//
// What bounds it: the cache's bytes, 1.125 d a token and key head.  At HBM's rate an SM
// gets 23.5 bytes a cycle, 98 cycles for 16 tokens of d = 128, in which it must unpack
// 4096 codes and multiply them with 8 heads.  So key codes are never converted: a 4-bit code
// u under a mask, read as fp16, is the subnormal number u 2^-24 (u 2^-20 for the second
// nibble), exactly, and warp-level MMAs take subnormal operands at full rate; the factors go
// into the queries, and -8 sum q is where the sums start.  Value codes, whose sums are long
// and may cancel, are widened to u - 8 by one logical operation and one subtraction of
// constants.  Scales multiply the scores per group (fp32), and the softmax weights per
// group (values).
//
// Measured: 64 sequences of 1000 to 32768 tokens (bf16, 32/4 heads of 128) 89 us, 4.1 TB/s of cache.  The bytes do not
// bound it there, nor does a pipe (issue slots 55% busy, ALU 45%, tensor 24%): registers leave three warps a
// scheduler, and each mostly waits for its own last instruction.  256 of 512 to 1536 tokens (fp32, 16/4
// heads of 128) 72 us, 1.97 TB/s: two warps a scheduler, two fp16 parts double the MMAs, and 4 of their 8 columns are
// heads.  One of 4096 tokens (bf16, 16/4) 14.4 us, the latency of a memset and two kernels.  256 sequences through a
// window of 1024 (16/4 heads of 128) 57 us in bf16, 76 in fp32.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "common.cuh"
#include "sm100.cuh"

namespace kdn {
namespace {

using namespace sm100;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStepBlocks = 4, kStepTokens = kStepBlocks * kBlockTokens, kStages = 2, kResident = 3;
constexpr int kUnit = kWarps * kStepTokens;   // a step of every warp
constexpr int kTile = 8;                      // query heads of one key head a block
// Blocks an SM.  fp32's two parts need the registers of two (three spilled: 80 us against 73 on 256
// sequences of up to 1536 tokens, 16/4 heads of 128); bf16 is the faster for a third (101 against 103 on 64 of
// up to 32768, 32/4 heads).
template <typename T> constexpr int resident() { return sizeof(T) == 4 ? 2 : kResident; }
constexpr uint32_t kWaitLimit = 2000000u;     // polls of about a microsecond at most
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kAll = 0xffffffffu;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// d = a b + c (m16n8k16; not volatile, so that independent products are interleaved)
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                    float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    mma(c, a0, a1, a2, a3, b0, b1, c[0], c[1], c[2], c[3]);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) { return bits(__floats2half2_rn(lo, hi)); }

// Codes - 8 of the first (second) nibbles of both halves, as fp16: 1024 + u and 64 + u hold u exactly.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "r"(mask), "r"(magic));
    return y;
}
__device__ __forceinline__ uint32_t low_values(uint32_t w) {
    return bits(__hsub2(half2_of(and_or(w, kLow, 0x64006400u)), half2_of(0x64086408u)));
}
__device__ __forceinline__ uint32_t high_values(uint32_t w) {
    return bits(__hsub2(half2_of(and_or(w, kHigh, 0x54005400u)), half2_of(0x54805480u)));
}

// N 32-bit words of shared memory
template <int N> __device__ __forceinline__ void load_words(uint32_t p, uint32_t (&w)[N]) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(p));
}
// N fp16 numbers
template <int N> __device__ __forceinline__ void load_scales(uint32_t p, float (&s)[N]) {
    if constexpr (N == 1) {
        uint16_t x;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(p));
        s[0] = __half2float(__ushort_as_half(x));
    } else {
        uint32_t w[N / 2];
        load_words<N / 2>(p, w);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = __half22float2(half2_of(w[i]));
            s[2 * i] = f.x;
            s[2 * i + 1] = f.y;
        }
    }
}

// What a sequence's row sees: tokens lo .. n - 1, taken from the 16-token block that holds
// lo on, in units of kUnit tokens.
struct Span {
    int n, lo, first, units;
};
__device__ __forceinline__ Span span_of(const CacheAttentionArgs& a, int r) {
    Span s;
    const long long room = min(static_cast<long long>(a.max_len), static_cast<long long>(a.table_width) * a.page);
    s.n = static_cast<int>(min(static_cast<long long>(max(a.seq_len[r], 0)), room));
    s.lo = a.window > 0 ? max(s.n - a.window, 0) : 0;
    s.first = s.lo / kBlockTokens * kBlockTokens;
    s.units = (s.n - s.first + kUnit - 1) / kUnit;
    return s;
}

// The work in a row: sequence after sequence, its tiles of heads one after another, each
// `cost` + `units` long, as a row's start and end take about as long as `cost` of its units.  Block b of
// the grid takes places b share .. (b + 1) share - 1, so every block has the same work whatever the
// lengths; a share is no less than 1 / kMaxParts of a row, so that no row is in more parts than the
// join can take.  Small shares leave the cost out: a block more counts for more there.
// (64 rows of 1000 to 32768 tokens, 32/4 heads of 128, at a cost of 0, 1, 2, 3, 4 and 6 units: 101, 94, 90, 91, 91
// and 95 us; 256 of 512 to 1536 in fp32, 16/4 heads: 73, 72, 72, 74, 75 and 76.)
constexpr int kMaxParts = 128, kRowCost = 2, kCostedShare = 8;
__device__ __forceinline__ void work_of(const CacheAttentionArgs& a, int tiles, long long& total, long long& share, int& cost) {
    __shared__ long long part_sum[kWarps];
    __shared__ int part_max[kWarps], part_rows[kWarps];
    long long sum = 0;
    int top = 0, rows = 0;
    for (int i = threadIdx.x; i < a.n_seq; i += kThreads) {
        const int u = span_of(a, i).units;
        sum += u;
        top = max(top, u);
        rows += u > 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(kAll, sum, o);
        top = max(top, __shfl_xor_sync(kAll, top, o));
        rows += __shfl_xor_sync(kAll, rows, o);
    }
    if (threadIdx.x % 32 == 0) {
        part_sum[threadIdx.x / 32] = sum;
        part_max[threadIdx.x / 32] = top;
        part_rows[threadIdx.x / 32] = rows;
    }
    __syncthreads();
    sum = 0;
    top = rows = 0;
    for (int w = 0; w < kWarps; ++w) {
        sum += part_sum[w];
        top = max(top, part_max[w]);
        rows += part_rows[w];
    }
    cost = sum * tiles >= static_cast<long long>(kCostedShare) * gridDim.x ? kRowCost : 0;
    total = (sum + static_cast<long long>(rows) * cost) * tiles;
    // (a row of top units that starts inside a share spans at most kMaxParts of this length)
    share = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>((top + kMaxParts - 2) / (kMaxParts - 1)));
}

// Places of one tile of a sequence's heads.
__device__ __forceinline__ int places_of(const Span& s, int cost) { return s.units ? cost + s.units : 0; }

// The sequence that holds place `at` of the work, and the places before it; n_seq past the end.
__device__ __forceinline__ void find_sequence(const CacheAttentionArgs& a, long long at, int tiles, int cost, int& r, long long& before) {
    __shared__ long long part[kWarps], found_before;
    __shared__ int found;
    const int per = (a.n_seq + kThreads - 1) / kThreads, r0 = min(static_cast<int>(threadIdx.x) * per, a.n_seq),
              r1 = min(r0 + per, a.n_seq);
    long long mine = 0;
    for (int i = r0; i < r1; ++i) mine += static_cast<long long>(places_of(span_of(a, i), cost)) * tiles;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kAll, upto, o);
        if (threadIdx.x % 32 >= o) upto += y;
    }
    if (threadIdx.x % 32 == 31) part[threadIdx.x / 32] = upto;
    if (threadIdx.x == 0) found = a.n_seq;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(threadIdx.x) / 32; ++w) upto += part[w];
    if (at < upto && at >= upto - mine) {
        long long x = upto - mine;
        for (int i = r0; i < r1; ++i) {
            const long long u = static_cast<long long>(places_of(span_of(a, i), cost)) * tiles;
            if (at < x + u) {
                found = i;
                found_before = x;
                break;
            }
            x += u;
        }
    }
    __syncthreads();
    r = found;
    before = found_before;
}

// A segment's result where it is not a whole row's: sums [kTile][D], then the maxima and the
// denominators.  A block has at most two, one of a row that began in an earlier block (its
// first record) and one of a row that goes on in the next (its second).  Before the records,
// a header for every block: the row that begins in it and goes on, and its number of parts (0: none).
template <int D> struct Record {
    static constexpr int kFloats = kTile * D + 2 * kTile;
};
struct Header {
    int seq, tile, parts, unused;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, resident<T>()) cache_attention_kernel(const CacheAttentionArgs a) {
    constexpr int G = D / 32, kBytes = cache_block_bytes(D), kStageBytes = kStepBlocks * kBytes;
    constexpr uint32_t kAllBlocks = (1u << kStepBlocks) - 1;
    // fp32 queries and weights go as two fp16 parts (22 bits), bf16 ones as one (exact, and 11 bits)
    constexpr bool TWO = sizeof(T) == 4;
    extern __shared__ __align__(128) uint8_t cache_smem[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ float join_m[kWarps][kTile], join_l[kWarps][kTile];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, c = lane & 3;
    const int rep = a.H / a.H_kv, ht = (rep + kTile - 1) / kTile, tiles = a.H_kv * ht;
    asm volatile("griddepcontrol.launch_dependents;");
    if (lane < kStages) mbar_init(smem_addr(&bars[warp][lane]), 1);
    mbar_fence_init();
    for (int i = blockIdx.x; i < a.n_seq; i += gridDim.x) {
        const Span sp = span_of(a, i);
        if (tid == 0 && sp.n != a.seq_len[i]) set_status(a.status, kStatusRange);
        if (sp.units) continue;   // nothing to see
        for (int j = tid; j < a.H * D; j += kThreads) IO<T>::store(static_cast<T*>(a.o), static_cast<size_t>(i) * a.H * D + j, 0.f);
        for (int j = tid; j < a.H; j += kThreads) a.lse[static_cast<size_t>(i) * a.H + j] = -INFINITY;
    }
    long long place, end, row_place, total, share;   // this block's share of the work; places before sequence r
    Header* headers = static_cast<Header*>(a.scratch);
    float* records = reinterpret_cast<float*>(headers + gridDim.x);
    int r, cost;
    {
        work_of(a, tiles, total, share, cost);
        place = share * blockIdx.x;
        end = min(place + share, total);
        if (tid == 0 && a.scratch) headers[blockIdx.x] = Header{0, 0, 0, 0};
        if (place >= end) return;
        find_sequence(a, place, tiles, cost, r, row_place);
    }
    const uint32_t ring = smem_addr(cache_smem) + warp * kStages * kStageBytes;
    const int per_page = a.page / kBlockTokens, ahead = kUnit / a.page, ahead_off = kUnit - ahead * a.page;
    int used = 0;   // stages filled so far
    Span sp = span_of(a, r);

    while (place < end) {
    const int at = static_cast<int>(place - row_place), tile = at / (cost + sp.units), at0 = at - tile * (cost + sp.units);
    const int n_places = static_cast<int>(min(static_cast<long long>(cost + sp.units - at0), end - place));
    // the cost stands before the row's first unit; a row of which a block has no more than that begins in the next
    const int u0 = max(at0 - cost, 0), n_units = at0 + n_places - cost - u0;
    if (n_units <= 0) break;
    const int kvh = tile / ht, h0 = kvh * rep + tile % ht * kTile, heads = min(kTile, rep - tile % ht * kTile);
    const int t_begin = sp.first + u0 * kUnit, t_end = min(sp.n, t_begin + n_units * kUnit);
    const int32_t* table = a.block_table + static_cast<size_t>(r) * a.table_width;

    // the first lanes fetch the step's blocks, walking along the table kUnit tokens at a time; a block
    // of a page outside the cache is not fetched, and its tokens count as not visible
    int walk_t = t_begin + warp * kStepTokens + lane * kBlockTokens, walk_page = walk_t / a.page,
        walk_off = walk_t - walk_page * a.page;
    int walk_id = -1;
    auto look_up = [&]() { walk_id = lane < kStepBlocks && walk_t < t_end ? table[walk_page] : -1; };
    uint32_t present = 0;   // kStepBlocks bits a stage
    auto issue = [&](int step) {
        const int st = step % kStages;
        const bool ok = walk_id >= 0 && walk_id < a.n_pages;
        if (lane < kStepBlocks && walk_t < t_end && !ok) set_status(a.status, kStatusRange);
        const uint32_t have = __ballot_sync(kAll, ok);
        present = (present & ~(kAllBlocks << (kStepBlocks * st))) | have << (kStepBlocks * st);
        const uint32_t bar = smem_addr(&bars[warp][st]);
        if (lane == 0) mbar_expect_tx(bar, __popc(have) * kBytes);
        __syncwarp();
        if (ok)
            bulk_load(ring + st * kStageBytes + lane * kBytes,
                      a.cache + ((static_cast<size_t>(walk_id) * a.H_kv + kvh) * per_page + walk_off / kBlockTokens) * kBytes,
                      kBytes, bar);
        walk_t += kUnit;
        walk_page += ahead;
        walk_off += ahead_off;
        if (walk_off >= a.page) {
            walk_off -= a.page;
            ++walk_page;
        }
        look_up();   // the next step's, a step before it is needed
    };
    look_up();
    // steps of this warp, counted on from those of the segments before
    const int first_step = used, last_step = used + (t_end - t_begin - warp * kStepTokens + kUnit - 1) / kUnit;
    int issued = used;
    __syncwarp();
    for (; issued < used + kStages && issued < last_step; ++issued) issue(issued);

    // queries: lane (g8, c) holds channels 32 g + 8 c .. + 7 of head g8, scaled by a power of two
    // that brings the head's largest to 2^13..2^14, in the order of the key codes' nibbles
    uint32_t bq[TWO ? 2 : 1][G][4];
    float f0, f1;   // score (in powers of two) of one unit of the products, heads 2 c and 2 c + 1
    {
        float x[G][8], top = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[g][i] = 0.f;
            if (g8 < heads) {
                const T* q = static_cast<const T*>(a.q.p) + r * a.q.row + (h0 + g8) * a.q.head + 32 * g + 8 * c;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[g][i] = IO<T>::load(q, i);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[g][i]));
        }
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
        // exponent field of the largest, kept where both factors below are normal numbers
        const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 24), 253);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);   // 2^(127 - e)
        const float f = fminf(fmaxf(a.scale * kLog2e * (TWO ? 1.f / 8192.f : 2048.f) *   // 2^-13, and 2^24 for the codes
                                            __uint_as_float(static_cast<uint32_t>(e) << 23), 1e-37f), 3e38f);   // neither 0 nor infinite: it multiplies -infinity and 0
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float k = (i & 1) && !TWO ? 512.f : 8192.f;   // the second nibble counts 16 times
                const float lo = x[g][i] * down * k, hi = x[g][i + 4] * down * k;
                const uint32_t w = pack(lo, hi);
                bq[0][g][i] = w;
                if constexpr (TWO) {
                    const float2 y = __half22float2(half2_of(w));
                    bq[1][g][i] = pack(lo - y.x, hi - y.y);
                }
            }
        f0 = __shfl_sync(kAll, f, 8 * c);
        f1 = __shfl_sync(kAll, f, 8 * c + 4);
    }
    float minus8[G][2];   // -8 sum q of a group, heads 2 c and 2 c + 1 (fp32: the codes are widened instead)
    if constexpr (!TWO) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma(t, 0x00080008u, 0x00080008u, 0x00800080u, 0x00800080u, bq[0][g][0], bq[0][g][1]);
            mma(t, 0x00080008u, 0x00080008u, 0x00800080u, 0x00800080u, bq[0][g][2], bq[0][g][3]);
            minus8[g][0] = -t[0];
            minus8[g][1] = -t[1];
        }
    }

    // Running state, heads 2 c and 2 c + 1.  With m the largest score so far and E the exponent of the
    // largest value scale, weights are formed as 2^(x - m + 10 - En), En = E cut to [-5, 0], and reach
    // the MMAs multiplied by scale 2^-Ep, Ep = max(E, 0): at most 2^15 and 2^11 (2^15 both when m lags
    // behind by up to 2^4, see slack), so fp16 holds them, and what its subnormal range loses of a weight is below 2^-34 of the largest (for scales
    // from 2^-5 on; below, by as much more as the scales are smaller).  m0, m1: m - 10 + En; the sums o
    // carry 2^-Ep besides.
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int E = -5;
    float scale_end = 0.0625f;   // 2^(E + 1)
    float o[2 * G][4];
#pragma unroll
    for (int i = 0; i < 2 * G; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

    int done = first_step;
    bool gave_up = false;
    for (; done < last_step; ++done) {
        const int st = done % kStages;
        if (!mbar_wait(smem_addr(&bars[warp][st]), (done / kStages) & 1, kWaitLimit)) {
            set_status(a.status, kStatusTimeout);
            gave_up = true;
            break;
        }
        const uint32_t stage = ring + st * kStageBytes;
        const int t0 = t_begin + ((done - first_step) * kWarps + warp) * kStepTokens;
        const uint32_t have = (present >> (kStepBlocks * st)) & kAllBlocks;
        const bool whole = t0 >= sp.lo && t0 + kStepTokens <= t_end && have == kAllBlocks;
        float x[kStepBlocks][4];
#pragma unroll
        for (int b = 0; b < kStepBlocks; ++b) {
            const uint32_t blk = stage + b * kBytes;
            uint32_t w0[G], w1[G];
            float s0[G], s1[G];
            load_words<G>(blk + g8 * (D / 2) + c * (4 * G), w0);
            load_words<G>(blk + (g8 + 8) * (D / 2) + c * (4 * G), w1);
            load_scales<G>(blk + 8 * D + g8 * (2 * G), s0);
            load_scales<G>(blk + 8 * D + (g8 + 8) * (2 * G), s1);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float t[4];
                const uint32_t v0 = w0[g] >> 8, v1 = w1[g] >> 8;
                if constexpr (TWO) {
                    uint32_t n[2][4] = {{low_values(w0[g]), low_values(w1[g]), high_values(w0[g]), high_values(w1[g])},
                                        {low_values(v0), low_values(v1), high_values(v0), high_values(v1)}};
                    mma(t, n[0][0], n[0][1], n[0][2], n[0][3], bq[1][g][0], bq[1][g][1], 0.f, 0.f, 0.f, 0.f);
                    mma(t, n[1][0], n[1][1], n[1][2], n[1][3], bq[1][g][2], bq[1][g][3]);
                    mma(t, n[0][0], n[0][1], n[0][2], n[0][3], bq[0][g][0], bq[0][g][1]);
                    mma(t, n[1][0], n[1][1], n[1][2], n[1][3], bq[0][g][2], bq[0][g][3]);
                } else {
                    mma(t, w0[g] & kLow, w1[g] & kLow, w0[g] & kHigh, w1[g] & kHigh, bq[0][g][0], bq[0][g][1], minus8[g][0],
                        minus8[g][1], minus8[g][0], minus8[g][1]);
                    mma(t, v0 & kLow, v1 & kLow, v0 & kHigh, v1 & kHigh, bq[0][g][2], bq[0][g][3]);
                }
                x[b][0] = g ? fmaf(s0[g], t[0], x[b][0]) : s0[g] * t[0];
                x[b][1] = g ? fmaf(s0[g], t[1], x[b][1]) : s0[g] * t[1];
                x[b][2] = g ? fmaf(s1[g], t[2], x[b][2]) : s1[g] * t[2];
                x[b][3] = g ? fmaf(s1[g], t[3], x[b][3]) : s1[g] * t[3];
            }
            if (!whole) {
                const int t = t0 + b * kBlockTokens + g8;
                const bool in = (have >> b) & 1u;
                if (!(in && t >= sp.lo && t < t_end)) x[b][0] = x[b][1] = -INFINITY;
                if (!(in && t + 8 >= sp.lo && t + 8 < t_end)) x[b][2] = x[b][3] = -INFINITY;
            }
        }
        // value scales of tokens 2 c, 2 c + 1 and 2 c + 8, 2 c + 9; zero where not visible
        uint32_t sv[kStepBlocks][2][G];
        __half2 smax = __float2half2_rn(0.f);
#pragma unroll
        for (int b = 0; b < kStepBlocks; ++b)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                load_words<G>(stage + b * kBytes + 17 * D + hf * (D / 2) + c * (4 * G), sv[b][hf]);
                if (!whole) {
                    const int t = t0 + b * kBlockTokens + 8 * hf + 2 * c;
                    const bool in = (have >> b) & 1u;
                    const uint32_t keep = (in && t >= sp.lo && t < t_end ? 0xffffu : 0u) |
                                          (in && t + 1 >= sp.lo && t + 1 < t_end ? 0xffff0000u : 0u);
#pragma unroll
                    for (int g = 0; g < G; ++g) sv[b][hf][g] &= keep;
                }
#pragma unroll
                for (int g = 0; g < G; ++g) smax = __hmax2(smax, half2_of(sv[b][hf][g]));
            }
        float stop = fmaxf(__low2float(smax), __high2float(smax));
        float n0 = fmaxf(x[0][0], x[0][2]), n1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
        for (int b = 1; b < kStepBlocks; ++b) {
            n0 = fmaxf(n0, fmaxf(x[b][0], x[b][2]));
            n1 = fmaxf(n1, fmaxf(x[b][1], x[b][3]));
        }
        n0 *= f0;
        n1 *= f1;
        const float shift = static_cast<float>(min(E, 0) - 10);
        // m is raised when a score passes it by more than the headroom that fp16 leaves: rarely after
        // the first steps
        const float slack = static_cast<float>(min(4, 5 + min(E, 0)));
        if (__any_sync(kAll, n0 + shift > m0 + slack || n1 + shift > m1 + slack || stop >= scale_end)) {
            stop = fmaxf(stop, __shfl_xor_sync(kAll, stop, 1));
            stop = fmaxf(stop, __shfl_xor_sync(kAll, stop, 2));
            const int e_new = max(E, static_cast<int>(__float_as_uint(stop) >> 23) - 127);
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(kAll, n0, s));
                n1 = fmaxf(n1, __shfl_xor_sync(kAll, n1, s));
            }
            // a head that has seen no finite score keeps m = -infinity
            const float up = static_cast<float>(min(e_new, 0) - 10);
            const float u0 = fmaxf(m0 - shift, n0) + up, u1 = fmaxf(m1 - shift, n1) + up;
            const float k0 = m0 == -INFINITY ? 0.f : ex2(m0 - u0), k1 = m1 == -INFINITY ? 0.f : ex2(m1 - u1);
            const float down = ex2(static_cast<float>(max(E, 0) - max(e_new, 0)));
            const float j0 = k0 * down, j1 = k1 * down;
            m0 = u0;
            m1 = u1;
            E = e_new;
            scale_end = ex2(static_cast<float>(E + 1));
            l0 *= k0;
            l1 *= k1;
#pragma unroll
            for (int i = 0; i < 2 * G; ++i) {
                o[i][0] *= j0; o[i][1] *= j1; o[i][2] *= j0; o[i][3] *= j1;
            }
        }
        if (E > 0) {   // large scales: the products stay in fp16's range
            const __half2 down = __float2half2_rn(ex2(static_cast<float>(-E)));
#pragma unroll
            for (int b = 0; b < kStepBlocks; ++b)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    sv[b][0][g] = bits(__hmul2(half2_of(sv[b][0][g]), down));
                    sv[b][1][g] = bits(__hmul2(half2_of(sv[b][1][g]), down));
                }
        }
        const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
        for (int b = 0; b < kStepBlocks; ++b) {
            const uint32_t blk = stage + b * kBytes;
            const float p0 = ex2(fmaf(x[b][0], f0, -b0)), p1 = ex2(fmaf(x[b][1], f1, -b1));
            const float p2 = ex2(fmaf(x[b][2], f0, -b0)), p3 = ex2(fmaf(x[b][3], f1, -b1));
            l0 += p0 + p2;
            l1 += p1 + p3;
            const uint32_t ph0 = pack(p0, p1), ph1 = pack(p2, p3);
            // weights of head g8, tokens 2 c, 2 c + 1 (w0) and 2 c + 8, 2 c + 9 (w1)
            const uint32_t w0 = transpose8x8(ph0), w1 = transpose8x8(ph1);
            uint32_t r0 = 0, r1 = 0;
            if constexpr (TWO) {
                const float2 y0 = __half22float2(half2_of(ph0)), y1 = __half22float2(half2_of(ph1));
                r0 = transpose8x8(pack(p0 - y0.x, p1 - y0.y));
                r1 = transpose8x8(pack(p2 - y1.x, p3 - y1.y));
            }
            uint32_t v0[G], v1[G];
            load_words<G>(blk + 9 * D + lane * (4 * G), v0);
            load_words<G>(blk + 13 * D + lane * (4 * G), v1);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const __half2 s0 = half2_of(sv[b][0][g]), s1 = half2_of(sv[b][1][g]);
                const __half2 q0 = __hmul2(half2_of(w0), s0), q1 = __hmul2(half2_of(w1), s1);
                const uint32_t u0 = v0[g] >> 8, u1 = v1[g] >> 8;
                const uint32_t n0 = low_values(v0[g]), n1 = high_values(v0[g]), n2 = low_values(v1[g]),
                               n3 = high_values(v1[g]), n4 = low_values(u0), n5 = high_values(u0),
                               n6 = low_values(u1), n7 = high_values(u1);
                if constexpr (TWO) {
                    // what the rounded products left out (both residuals are exact); the MMAs' sums, which are
                    // cut off and not rounded, stay short, and are added up in fp32
                    const __half2 z0 = __hfma2(half2_of(r0), s0, __hfma2(half2_of(w0), s0, __hneg2(q0)));
                    const __half2 z1 = __hfma2(half2_of(r1), s1, __hfma2(half2_of(w1), s1, __hneg2(q1)));
                    float t[4], u[4];
                    mma(t, n0, n1, n2, n3, bits(z0), bits(z1), 0.f, 0.f, 0.f, 0.f);
                    mma(u, n4, n5, n6, n7, bits(z0), bits(z1), 0.f, 0.f, 0.f, 0.f);
                    mma(t, n0, n1, n2, n3, bits(q0), bits(q1));
                    mma(u, n4, n5, n6, n7, bits(q0), bits(q1));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[2 * g][j] += t[j];
                        o[2 * g + 1][j] += u[j];
                    }
                } else {
                    mma(o[2 * g], n0, n1, n2, n3, bits(q0), bits(q1));
                    mma(o[2 * g + 1], n4, n5, n6, n7, bits(q0), bits(q1));
                }
            }
        }
        __syncwarp();   // every lane has read the stage
        if (issued < last_step) {
            issue(issued);
            ++issued;
        }
    }
    // a warp that gave up lets its copies land
    for (; done < issued; ++done) mbar_wait(smem_addr(&bars[warp][done % kStages]), (done / kStages) & 1, kWaitLimit);
#pragma unroll
    for (int s = 4; s < 32; s <<= 1) {
        l0 += __shfl_xor_sync(kAll, l0, s);
        l1 += __shfl_xor_sync(kAll, l1, s);
    }
    used = last_step;
    if (__syncthreads_or(gave_up)) return;   // the rings are free

    float* sums = reinterpret_cast<float*>(cache_smem);   // [kWarps][kTile][D]
    {
        float* mine = sums + warp * kTile * D + 2 * c * D + g8;
        const float up = ex2(static_cast<float>(max(E, 0)));
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
            mine[16 * i] = o[i][0] * up;
            mine[16 * i + D] = o[i][1] * up;
            mine[16 * i + 8] = o[i][2] * up;
            mine[16 * i + 8 + D] = o[i][3] * up;
        }
        if (g8 == 0) {
            join_m[warp][2 * c] = m0;
            join_m[warp][2 * c + 1] = m1;
            join_l[warp][2 * c] = l0;
            join_l[warp][2 * c + 1] = l1;
        }
    }
    __syncthreads();
    const bool whole_row = n_units == sp.units;
    float* rec = records + (2 * static_cast<size_t>(blockIdx.x) + (u0 == 0)) * Record<D>::kFloats;
    if (tid == 0 && !whole_row && u0 == 0)
        headers[blockIdx.x] = Header{r, tile, static_cast<int>((place - at0 + cost + sp.units - 1) / share) - static_cast<int>(blockIdx.x) + 1, 0};
    for (int i = tid; i < heads * D; i += kThreads) {
        const int h = i / D, d = i % D;
        float m = join_m[0][h];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, join_m[w][h]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float k = ex2(join_m[w][h] - base);
            l = fmaf(k, join_l[w][h], l);
            s = fmaf(k, sums[(w * kTile + h) * D + d], s);
        }
        if (!whole_row) {
            rec[i] = s;
            if (d == 0) {
                rec[kTile * D + h] = m;
                rec[kTile * D + kTile + h] = l;
            }
        } else {
            const size_t row = static_cast<size_t>(r) * a.H + h0 + h;
            IO<T>::store(static_cast<T*>(a.o), row * D + d, l != 0.f ? s / l : 0.f);
            if (d == 0) a.lse[row] = l != 0.f ? (base + log2f(l)) * kLn2 : -INFINITY;
        }
    }
    place += n_places;
    if (place - row_place >= static_cast<long long>(cost + sp.units) * tiles) {
        row_place = place;
        do {
            if (++r >= a.n_seq) return;
            sp = span_of(a, r);
        } while (sp.units == 0);
    }
    __syncthreads();       // what was written to the rings above is read,
    fence_proxy_async();   // and the next copies into them come after it
    }
}

// Joins the parts of the row that begins in block x of the first kernel and goes on, for one of
// its heads: groups of D threads take every kGroups-th part, the groups are added up in order.
constexpr int kJoinThreads = 512;
template <typename T, int D> __global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const CacheAttentionArgs a, int blocks) {
    constexpr int kGroups = kJoinThreads / D;
    __shared__ float sum[kGroups][D], weight[kMaxParts], top[kMaxParts / 32], den[kMaxParts / 32];
    const int rep = a.H / a.H_kv, ht = (rep + kTile - 1) / kTile, row_h = blockIdx.y, tid = threadIdx.x, d = tid % D, grp = tid / D;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Header head = static_cast<const Header*>(a.scratch)[blockIdx.x];
    const int parts = head.parts, hh = head.tile % ht * kTile + row_h, h = head.tile / ht * rep + hh;
    if (parts == 0 || hh >= rep) return;
    // the second record of that block, and the first ones of the blocks after
    const float* rec = reinterpret_cast<const float*>(static_cast<const Header*>(a.scratch) + blocks) +
                       2 * static_cast<size_t>(blockIdx.x) * Record<D>::kFloats;
    auto at = [&](int p) { return rec + (p ? 2 * p : 1) * Record<D>::kFloats; };
    float m = -INFINITY, l = 0.f;
    if (tid < kMaxParts) {
        if (tid < parts) {
            m = at(tid)[kTile * D + row_h];
            l = at(tid)[kTile * D + kTile + row_h];
        }
        float x = m;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, s));
        if (tid % 32 == 0) top[tid / 32] = x;
    }
    __syncthreads();
    float base = top[0];
#pragma unroll
    for (int i = 1; i < kMaxParts / 32; ++i) base = fmaxf(base, top[i]);
    if (base == -INFINITY) base = 0.f;
    if (tid < kMaxParts) {
        const float k = ex2(m - base);
        weight[tid] = k;
        l = warp_sum(tid < parts ? k * l : 0.f);
        if (tid % 32 == 0) den[tid / 32] = l;
    }
    __syncthreads();
    float s = 0.f;
#pragma unroll 8
    for (int p = grp; p < parts; p += kGroups) s = fmaf(weight[p], at(p)[row_h * D + d], s);
    sum[grp][d] = s;
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) s += sum[g][d];
    l = den[0];
#pragma unroll
    for (int i = 1; i < kMaxParts / 32; ++i) l += den[i];
    const size_t row = static_cast<size_t>(head.seq) * a.H + h;
    IO<T>::store(static_cast<T*>(a.o), row * D + d, l != 0.f ? s / l : 0.f);
    if (d == 0) a.lse[row] = l != 0.f ? (base + log2f(l)) * kLn2 : -INFINITY;
}

// As many blocks as are resident at once, or a unit each; whether a row can be cut.
struct Grid {
    int blocks;
    bool cut;
};
constexpr int kSMs = 152;   // GB300's
Grid grid_of(int n_seq, int H, int H_kv, int max_len, int window, int most_blocks) {
    if (H <= 0 || H_kv <= 0) return {0, false};
    const long long tiles = static_cast<long long>(H_kv) * ((H / H_kv + kTile - 1) / kTile);
    const long long seen = window > 0 && window < max_len ? static_cast<long long>(window) + kBlockTokens - 1 : max_len;
    const long long units = (seen + kUnit - 1) / kUnit, all = (units > 1 ? units : 1) * n_seq * tiles;
    return {static_cast<int>(all < most_blocks ? all : most_blocks), units > 1};
}

template <typename T, int D> cudaError_t launch(const CacheAttentionArgs& a, cudaStream_t s) {
    const Grid g = grid_of(a.n_seq, a.H, a.H_kv, a.max_len, a.window, kSMs * resident<T>());
    constexpr int ring = kWarps * kStages * kStepBlocks * cache_block_bytes(D), joined = kWarps * kTile * D * 4;
    constexpr int smem = ring > joined ? ring : joined;
    cudaError_t e = cudaFuncSetAttribute(cache_attention_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    CacheAttentionArgs b = a;
    if (!g.cut) b.scratch = nullptr;   // no row can be cut
    cache_attention_kernel<T, D><<<g.blocks, kThreads, smem, s>>>(b);
    if ((e = cudaGetLastError()) != cudaSuccess || !g.cut) return e;
    // started while the first kernel runs; it waits for it before it reads
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int rep = a.H / a.H_kv;
    cfg.gridDim = dim3(g.blocks, rep < kTile ? rep : kTile);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_join_kernel<T, D>, a, g.blocks);
}

template <typename T> cudaError_t by_size(const CacheAttentionArgs& a, cudaStream_t s) {
    if (a.d == 128) return launch<T, 128>(a, s);
    if (a.d == 64) return launch<T, 64>(a, s);
    return launch<T, 32>(a, s);
}

}  // namespace

size_t cache_attention_scratch(int n_seq, int H, int H_kv, int d, int max_len, int window) {
    const Grid g = grid_of(n_seq, H, H_kv, max_len, window, kSMs * kResident);
    return g.cut ? static_cast<size_t>(g.blocks) * (sizeof(Header) + 2 * sizeof(float) * (kTile * d + 2 * kTile)) : 0;
}

cudaError_t launch_cache_attention(const CacheAttentionArgs& a, cudaStream_t s) {
    return a.io == 1 ? by_size<__nv_bfloat16>(a, s) : by_size<float>(a, s);
}

}  // namespace kdn
