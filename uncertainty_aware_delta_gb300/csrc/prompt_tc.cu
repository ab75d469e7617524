// Causal attention over packed prompts on tcgen05 tensor cores: bf16, heads of 64 or 128.
//
// One block takes two units of 128 query rows that read the same keys: two heads of one key
// head where there are an even number of them, else two neighbouring row tiles of one head.
// Per key tile of 128 and unit: S = Q K^T into TMEM, the softmax by one warpgroup with a row
// a thread, P = exp(S - m) as bf16 back into S's TMEM columns, O += P V with P read from
// TMEM.  While one unit's warpgroup works on its scores, the tensor cores run the other
// unit's P V and next Q K^T.  What bounds it: the products (4 x 128 x 128 x d multiply-adds a pair of
// tiles, 2048 cycles for d = 128) on long prompts, the softmax (2 x 128 x 128 exponentials and
// as many maxima, sums and roundings) where d = 64, and on short rows what lies between items: the
// masked last tile, an item's outputs, code that has left the instruction cache.
//
// Measured: 8 prompts of 4096 tokens (16/4 heads of 128, causal) 391 to 409 us, 1344 to 1406 TFLOP/s, 70 to 73% of the
// cuBLAS rate, and a pair of tiles in 2900 cycles; 24 prompts of up to 4095 through a window of
// 1024 (16 heads of 64) 102 us, 495 TFLOP/s; 16 x up to 256 tokens over prefixes of up to 3840 (16/2 heads of
// 128) 57 us, 390 TFLOP/s (42 of it this kernel, in which an SM is active for 62 to 92% of the time); one of 77 tokens 14.4 us.
//
// The running maximum is raised only when a row's score passes it by 2^8: fp32 sums and
// accumulators and bf16 weights have the range, and O (in TMEM) is then hardly ever rescaled.
// Weights are rounded to bf16 for the product (the type of V in the MMA); their sum is taken
// before rounding, in fp32.

#include <cuda.h>
#include <cuda_bf16.h>
#include <algorithm>
#include <mutex>

#include "attention.h"
#include "common.cuh"
#include "kdn.h"
#include "sm100.cuh"

namespace kdn {
namespace {

using namespace sm100;

constexpr int kTileRows = 128, kTileKeys = 128;
constexpr int kThreads = 512;                 // loader, two product warps, finder and guard; 2 softmax and 1 output warpgroups
// registers: launched with 128 a thread; 96 + 2 x 168 + 80 = 4 x 128, and 96 + 2 x 152 + 112 where outputs may be parts
constexpr int kAuxRegs = 96;
template <bool SPLIT> constexpr int kSoftmaxRegs = SPLIT ? 152 : 168;
template <bool SPLIT> constexpr int kOutputRegs = SPLIT ? 112 : 80;
constexpr int kItems = 3, kChunks = 128;     // items known ahead; chunks of sequences
constexpr uint32_t kWaitLimit = 1u << 20, kProbeLimit = 4096;   // polls of about a microsecond at most
constexpr int kSMs = 152;                     // GB300
constexpr float kLazy = 8.0f;                 // powers of two a score may pass the running maximum by
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xffffffffu;

struct PromptParams {
    CUtensorMap tq, tk, tv;
    const __nv_bfloat16* v;
    long long v_row, v_head;
    const int32_t *cu_q, *cu_k;
    __nv_bfloat16* o;
    float* lse;
    uint32_t *status, *counter;   // counter: items taken
    int n_seq, total_q, total_k, H, H_kv, window, groups, items, chunk, chunks, probe, wide;
    struct SplitPlan* plan;
    struct SplitHead* heads;
    float* rows;         // [n_rows][d]
    float2* sums;        // [n_rows]: maximum and sum
    int n_rows, dense, row_step, unit_step;   // dense: rows by part, row and head, else by record
    float scale_log2;
};

template <int D> struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kHalves * 16384;      // 128 rows of d bf16 in 128-byte-swizzled halves
    static constexpr int kSlots = D == 128 ? 4 : 8;         // K and V tiles in turn
    static constexpr int kSums = 2 * 2 * 128 * 8;           // the rows' maxima and sums, of two items
    static constexpr int kSmem = 2 * kTileBytes + kSlots * kTileBytes + kSums + 1024;
};

// TMEM columns: scores (then weights) of the units, their outputs
constexpr uint32_t kTmS = 0, kTmO = 256, kTmCols = 512;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// One look at a barrier, without the suspension of mbar_try_wait (which costs some 300 cycles
// even where the phase is complete).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The MMA warp runs as a whole, so that descriptors stay in uniform registers, and one lane's
// predicate issues.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead));
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead));
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %1, 0;"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar), "r"(lead)
        : "memory");
}
// Ones in bits 0 .. n.
__device__ __forceinline__ uint32_t bits_to(int n) { return n < 0 ? 0u : n >= 31 ? 0xffffffffu : (2u << n) - 1u; }
// two fp32 operations an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
// After tmem_wait_ld(): ties the loaded registers to that point of the program.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// What a block works on: a row tile of one sequence and a group of heads.
// Few items, some of them long: the keys of a long one are split over several, whose sums a second kernel joins.
// Measured (us, split against whole, 16/2 heads of 128 unless stated): one token over 32768 46 / 384, 128 over 32768
// 53 / 385, 4 x 64 over 16384 (8/1 heads of 64) 51 / 176, 8192 alone (2/1 heads) 71 / 105, 16384 alone (2/1) 172 / 199,
// 16 x 256 over up to 3840 57 / 66, 8192 alone (4/1 heads of 64) 89 / 93, 8 x 64 over 4096 (16/4) 63 / 61: the
// longest item has to be longer than an SM's share of all by some 16 tiles.
// A part's outputs stand in rows of d, with the rows' maxima and sums beside them: a record of 2 x 128 rows for every
// part, or, where that is less, kMaxParts rows for every row that there is.
constexpr int kMaxParts = 16, kMinPart = 6, kWorthParts = 16;   // of a row; key tiles of a part; see above
constexpr int kSplitItems = 3 * kSMs;         // more items than this fill the SMs
struct SplitPlan {
    int items, unused[15];    // items that are split, the first so many by their length
    int base[kMaxParts];      // record of the first one's part p (where there are records)
    int unused_too[32];
};
struct SplitHead {
    int q0, rows, group, parts, unused[4];   // first query, queries
};
constexpr int kRecord = 2 * kTileRows;

struct Item {
    int q0, n_q, k0, n_k;    // the sequence's rows
    int row;                 // first row of the item in its sequence; negative: no more items
    int group;
    int from, to, slot;      // where rows may be split: key tiles that the item has, the first row of its part (negative: not a part)
};
struct Unit {
    int head, row, rows;     // rows: valid ones
    int place;               // place of its first row among the keys
    int lo, hi;              // key tiles; hi < lo: none
    int all_from, all_to;    // of these, tiles all_from < b < all_to are seen whole by every valid row
    __device__ __forceinline__ bool any() const { return hi >= lo; }
    __device__ __forceinline__ bool masked(int b) const { return b >= all_to || b <= all_from; }
};
template <bool PAIR, bool SPLIT> __device__ __forceinline__ Unit unit_of(const Item& it, int s, int window) {
    Unit u;
    u.head = PAIR ? 2 * it.group + s : it.group;
    u.row = it.row + (PAIR ? 0 : s * kTileRows);
    u.rows = min(kTileRows, it.n_q - u.row);
    u.place = it.n_k - it.n_q + u.row;
    // (place may be far below 0)
    const int last = u.place + u.rows - 1, first = window > 0 && u.place >= window ? u.place - window + 1 : 0;
    u.lo = first / kTileKeys;
    u.hi = u.rows > 0 && last >= 0 ? last / kTileKeys : u.lo - 1;
    if (SPLIT) {
        u.lo = max(u.lo, it.from);
        u.hi = min(u.hi, it.to);
    }
    u.all_to = max(u.place + 1, 0) / kTileKeys;
    u.all_from = window > 0 && last >= window ? (last - window) / kTileKeys : -1;
    return u;
}
// Key tiles of an item: all, and those the guard looks at (all that some unit masks).
struct Tiles {
    int lo, hi, cut_from, cut_to;
    __device__ __forceinline__ bool cut(int b) const { return b >= cut_to || b <= cut_from; }
};
__device__ __forceinline__ Tiles tiles_of(const Unit& u0, const Unit& u1) {
    const bool a0 = u0.any(), a1 = u1.any();
    Tiles t;
    t.lo = min(a0 ? u0.lo : 0x7ffffff0, a1 ? u1.lo : 0x7ffffff0);
    t.hi = max(a0 ? u0.hi : -1, a1 ? u1.hi : -1);
    t.cut_to = min(a0 ? u0.all_to : 0x7fffffff, a1 ? u1.all_to : 0x7fffffff);
    t.cut_from = max(a0 ? u0.all_from : -1, a1 ? u1.all_from : -1);
    return t;
}

// Values that are not finite in the tiles that the guard looked at, added to a row that sees
// them (channels i .. i + 31; its weights are positive, so they come out as they are).
template <bool PAIR, bool SPLIT>
__device__ __forceinline__ void give_back(const PromptParams& P, const Item& it, int last, int head, int i, uint32_t (&x)[32]) {
    const Tiles t = tiles_of(unit_of<PAIR, SPLIT>(it, 0, P.window), unit_of<PAIR, SPLIT>(it, 1, P.window));
    const int first = P.window > 0 ? last - P.window + 1 : 0, kvh = head / (P.H / P.H_kv);
#pragma unroll 1
    for (int b = t.lo; b <= t.hi; ++b) {
        if (!t.cut(b)) continue;
#pragma unroll 1
        for (int k = max(b * kTileKeys, first); k <= min(b * kTileKeys + kTileKeys - 1, last); ++k) {
            const __nv_bfloat16* v = P.v + (static_cast<long long>(it.k0) + k) * P.v_row + kvh * P.v_head + i;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float y = __bfloat162float(v[j]);
                if ((__float_as_uint(y) & 0x7f800000u) == 0x7f800000u) x[j] = __float_as_uint(__uint_as_float(x[j]) + y);
            }
        }
    }
}

// 16 words to a row's own place, whole sectors at a time where the output is aligned to them.  (Through shared
// memory, with whole lines an instruction, 24 prompts through a window took 107.6 us against 106.2, one of 77 tokens
// 16.4 against 14.4: the code is shorter, and a new item's first products wait for the last's outputs to be read.)
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint32_t (&y)[16], bool wide) {
    if (wide) {
#pragma unroll
        for (int j = 0; j < 16; j += 8)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + 2 * j), "r"(y[j]), "r"(y[j + 1]),
                         "r"(y[j + 2]), "r"(y[j + 3]), "r"(y[j + 4]), "r"(y[j + 5]), "r"(y[j + 6]), "r"(y[j + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int j = 0; j < 16; j += 4) *reinterpret_cast<uint4*>(p + 2 * j) = make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]);
    }
}

// Blocks stay (one an SM) and take items from a counter.  Warp 0 loads, warps 1 and 2 issue
// the units' products, warp 3 finds the items and guards, warps 4 .. 11 are the units' softmax, 12 .. 15
// write the outputs of both.  Everything is counted on from item to item, so the next item's first products run
// while the last one's outputs are written.
template <int D, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) prompt_tc_kernel(const __grid_constant__ PromptParams P) {
    using L = Layout<D>;
    constexpr int kItemRows = PAIR ? kTileRows : 2 * kTileRows;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * L::kSlots + 28 + 2 * kItems];
    __shared__ Item items[kItems];
    __shared__ int chunk_tiles[kChunks], dirty[kItems];
    __shared__ volatile int aborted;
    __shared__ uint32_t tmem_slot;
    const uint32_t sb = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t sq = sb, skv = sb + 2 * L::kTileBytes, sums = skv + L::kSlots * L::kTileBytes;
    const uint32_t bar_full = smem_addr(bars), bar_empty = bar_full + 8 * L::kSlots, bar_q = bar_empty + 8 * L::kSlots,
                   bar_q_free = bar_q + 16, bar_s = bar_q_free + 16, bar_p = bar_s + 16, bar_o = bar_p + 16,
                   bar_o_free = bar_o + 16, bar_v = bar_o_free + 16, bar_cut = bar_v + 32, bar_item = bar_cut + 32,
                   bar_item_free = bar_item + 8 * kItems, bar_turn = bar_item_free + 8 * kItems, bar_l = bar_turn + 16, bar_drain = bar_l + 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (SPLIT) asm volatile("griddepcontrol.launch_dependents;");

    if (tid == 0) {
        aborted = 0;
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 2);   // both units' products
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_q + 8 * i, 1);
            mbar_init(bar_q_free + 8 * i, 1);
            mbar_init(bar_s + 8 * i, 1);
            mbar_init(bar_p + 8 * i, 4);
            mbar_init(bar_turn + 8 * i, 1);
            mbar_init(bar_l + 16 * i, 4);   // two a unit in turn: of an item of one tile, they may be there before the last
            mbar_init(bar_l + 16 * i + 8, 4);   // item's have been read
            mbar_init(bar_o + 8 * i, 1);
            mbar_init(bar_o_free + 8 * i, 4);
        }
        // four in turn: the loader may be several tiles ahead of the guard, and it of the products
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar_v + 8 * i, 1);
            mbar_init(bar_cut + 8 * i, 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(bar_item + 8 * i, 1);
            mbar_init(bar_item_free + 8 * i, 4 + 12);   // loader, products, guard; softmax and output warps
        }
        mbar_init(bar_drain, 1);   // also the probe's: completed by nothing before the end
        mbar_init(bar_drain + 8, 1);
        mbar_fence_init();
    }
    // row tiles of every chunk of sequences (32, or more where there are many)
    auto tiles_of_sequence = [&](int s, Item& it) {
        const int q0 = P.cu_q[s], q1 = P.cu_q[s + 1], k0 = P.cu_k[s], k1 = P.cu_k[s + 1];
        if (q0 < 0 || q1 < q0 || q1 > P.total_q || k0 < 0 || k1 < k0 || k1 > P.total_k) {
            if (blockIdx.x == 0) set_status(P.status, kStatusRange);
            return 0;
        }
        it.q0 = q0; it.n_q = q1 - q0; it.k0 = k0; it.n_k = k1 - k0;
        return (q1 - q0 + kItemRows - 1) / kItemRows;
    };
    for (int i = warp; i < P.chunks; i += kThreads / 32) {
        int n = 0;
        Item it;
#pragma unroll 1
        for (int j = lane; j < P.chunk; j += 32)
            if (i * P.chunk + j < P.n_seq) n += tiles_of_sequence(i * P.chunk + j, it);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
        if (lane == 0) chunk_tiles[i] = n;
    }
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(smem_addr(&tmem_slot), kTmCols);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_test(bar, parity)) return true;
#pragma unroll 1
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if (aborted) return false;
        }
        aborted = 1;
        set_status(P.status, kStatusTimeout);
        return false;
    };
    // the item in place n of a role's walk; false when the walk is over
    auto take = [&](int n, Item& it, bool& ok) {
        ok = wait(bar_item + 8 * (n % kItems), (n / kItems) & 1);
        if (!ok) return false;
        it = items[n % kItems];
        return it.row >= 0;
    };
    auto release = [&](int n) { mbar_arrive(bar_item_free + 8 * (n % kItems)); };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
        if (warp == 0 && lane == 0) {
            // ---- loader: Q, then K and V tiles in turn
            const int rep = P.H / P.H_kv;
            int n = 0, nq = 0, nq_sent[2] = {0, 0};
            uint32_t nc = 0;
            bool ok = true;
            Item it;
            for (int w = 0; take(w, it, ok); ++w) {
                release(w);
                const Unit u0 = unit_of<PAIR, SPLIT>(it, 0, P.window), u1 = unit_of<PAIR, SPLIT>(it, 1, P.window);
                const Tiles t = tiles_of(u0, u1);
                if (t.hi < t.lo) continue;
                const int kvh = u0.head / rep;
#pragma unroll 1
                for (int b = t.lo; ok && b <= t.hi; ++b)
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        const int slot = n % L::kSlots;
                        if (n >= L::kSlots && !(ok = wait(bar_empty + 8 * slot, (n / L::kSlots - 1) & 1))) break;
                        mbar_expect_tx(bar_full + 8 * slot, L::kTileBytes);
                        for (int f = 0; f < L::kHalves; ++f)
                            tma_load_3d(skv + slot * L::kTileBytes + f * 16384, i ? &P.tv : &P.tk, 64 * f, kvh,
                                        it.k0 + b * kTileKeys, bar_full + 8 * slot);
                        ++n;
                        // the first keys are asked for before the queries: these wait for the last products of the
                        // item before, each unit's for its own
                        if (i == 0 && b == t.lo) {
                            for (int s = 0; s < 2; ++s) {
                                const Unit& u = s ? u1 : u0;
                                if (nq > 0 && !(ok = wait(bar_q_free + 8 * s, (nq - 1) & 1))) break;
                                mbar_expect_tx(bar_q + 8 * s, u.any() ? L::kTileBytes : 0);
                                nq_sent[s] = nq + 1;
                                if (u.any())
                                    for (int f = 0; f < L::kHalves; ++f)
                                        tma_load_3d(sq + s * L::kTileBytes + f * 16384, &P.tq, 64 * f, u.head, it.q0 + u.row,
                                                    bar_q + 8 * s);
                            }
                            if (!ok) break;
                            ++nq;
                        }
                        if (i && t.cut(b)) mbar_arrive(bar_cut + 8 * (nc++ & 3));
                        if (P.probe && n == 1 && !mbar_wait(bar_drain, 0, kProbeLimit)) {
                            aborted = 1;
                            set_status(P.status, kStatusTimeout);
                        }
                        if (aborted) {
                            ok = false;
                            break;
                        }
                    }
                if (!ok) break;
            }
            if (aborted) {   // copies already issued land before the block's shared memory goes away
                for (int s = 0; s < 2; ++s)
                    if (nq_sent[s] > 0) mbar_wait(bar_q + 8 * s, (nq_sent[s] - 1) & 1, kWaitLimit);
                for (int j = max(n - L::kSlots, 0); j < n; ++j)
                    mbar_wait(bar_full + 8 * (j % L::kSlots), (j / L::kSlots) & 1, kWaitLimit);
            }
        } else if (warp == 1 || warp == 2) {
            // ---- products of a unit: P V of a key tile, then Q K^T of the next (of this item or the one after it).
            // A warp a unit, issuing in turn: all that a warp waits for, it waits for during the other's turn, and
            // one unit's softmax runs beside the other's products (issued as they come, the two units' products
            // share the tensor cores and both end late, and both softmaxes then run at once).
            constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0, 0), id_o = idesc_bf16(128, D, 0, 1, 0);
            const uint32_t lead = elect_one();
            auto one = [](int x) { return __shfl_sync(kAll, x, 0); };
            const int s = one(warp - 1);
            const uint32_t ts = one(tmem) + kTmS + 128 * s, to = one(tmem) + kTmO + 128 * s, fb = one(bar_full), eb = one(bar_empty),
                           bs = one(bar_s) + 8 * s, bp = one(bar_p) + 8 * s, bo = one(bar_o) + 8 * s, bf = one(bar_o_free) + 8 * s;
            auto await = [&](uint32_t bar, uint32_t parity) { return __all_sync(kAll, wait(bar, parity)); };
            const uint64_t qd = sw128_desc(one(sq) + s * L::kTileBytes, 16, 1024), kd = sw128_desc(one(skv), 16, 1024),
                           vd = sw128_desc(one(skv), 16384, 1024);
            auto scores = [&](int slot) {
                const uint64_t b = desc_add(kd, slot * L::kTileBytes);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * 16384 + (k % 4) * 32;
                    mma_ss(lead, ts, desc_add(qd, off), desc_add(b, off), id_s, k > 0);
                }
                commit(lead, bs);
            };
            auto output = [&](int slot, bool add) {
                const uint64_t b = desc_add(vd, slot * L::kTileBytes);
#pragma unroll
                for (int k = 0; k < kTileKeys / 16; ++k) mma_ts(lead, to, ts + 8 * k, desc_add(b, k * 2048), id_o, k > 0 ? 1u : add);
            };
            struct Walk {   // key tile b of an item (tiles lo .. hi), of which the unit has mine_lo .. mine_hi
                int b, lo, hi, mine_lo, mine_hi, cut_from, cut_to;
            };
            int w = 0;
            bool ok = true;
            // the first tile of the next item that has any; false when there is none
            auto next_item = [&](Walk& x) {
                for (;;) {
                    Item it;
                    bool fine;
                    const bool got = take(w, it, fine);
                    if (!__all_sync(kAll, fine)) {
                        ok = false;
                        return false;
                    }
                    if (!one(got)) return false;
                    if (lead) release(w);
                    ++w;
                    const Unit u0 = unit_of<PAIR, SPLIT>(it, 0, P.window), u1 = unit_of<PAIR, SPLIT>(it, 1, P.window);
                    const Unit& u = s ? u1 : u0;
                    const Tiles t = tiles_of(u0, u1);
                    x = Walk{one(t.lo), one(t.lo), one(t.hi), one(u.any() ? u.lo : 0x7ffffff0), one(u.any() ? u.hi : -1),
                             one(t.cut_from), one(t.cut_to)};
                    if (x.hi >= x.lo) return true;
                }
            };
            uint32_t slot = L::kSlots - 1, phase = 1;   // of the tile used last
            auto next = [&]() {
                if (++slot == L::kSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            uint32_t nq = 0, np = 0, no = 1, nv = 0, turn = s ^ 1;
            const uint32_t my_turn = one(bar_turn) + 8 * s, other_turn = one(bar_turn) + 8 * (s ^ 1);
            // K of the walk's tile, the next in the ring, has landed
            auto have_keys = [&](const Walk& x) {
                next();
                if (!await(fb + 8 * slot, phase)) return false;
                if (x.b == x.lo) {
                    if (!await(one(bar_q) + 8 * s, nq)) return false;
                    nq ^= 1;
                }
                return true;
            };
            auto take_turn = [&]() {
                const bool got = await(my_turn, turn);
                turn ^= 1;
                tc_fence_after();
                return got;
            };
            Walk cur = {}, nxt;
            bool have = false;   // cur is a tile (its scores are under way)
            while (ok) {
                nxt = cur;
                const bool fresh = !have || cur.b == cur.hi;
                bool more = true;
                if (fresh) more = next_item(nxt);
                else ++nxt.b;
                if (!ok) break;
                uint32_t vslot = 0;
                bool mine = false;
                if (have) {
                    next();
                    vslot = slot;
                    if (!(ok = await(fb + 8 * vslot, phase))) break;
                    if (cur.b >= cur.cut_to || cur.b <= cur.cut_from) {
                        if (!(ok = await(bar_v + 8 * (nv & 3), (nv >> 2) & 1))) break;
                        ++nv;
                    }
                    mine = cur.b >= cur.mine_lo && cur.b <= cur.mine_hi;
                    if (mine) {
                        if (cur.b == cur.mine_lo) {   // the last item's output has been read
                            if (!(ok = await(bf, no))) break;
                            no ^= 1;
                        }
                    }
                }
                // (a new item's queries, too: they are asked for when this unit's last scores are done)
                if (more && !(ok = have_keys(nxt))) break;
                if (!(ok = take_turn())) break;
                if (have) {
                    if (mine) {
                        if (!(ok = await(bp, np))) break;
                        np ^= 1;
                        tc_fence_after();
                        output(vslot, cur.b > cur.mine_lo);
                        if (cur.b == cur.mine_hi) commit(lead, bo);
                    }
                    commit(lead, eb + 8 * vslot);
                }
                if (!more) {
                    if (lead) mbar_arrive(other_turn);
                    break;
                }
                if (nxt.b >= nxt.mine_lo && nxt.b <= nxt.mine_hi) scores(slot);
                commit(lead, eb + 8 * slot);
                if (nxt.b == nxt.hi) commit(lead, bar_q_free + 8 * s);
                if (lead) mbar_arrive(other_turn);
                cur = nxt;
                have = true;
            }
            if (!ok) {   // products already issued end before TMEM goes away
                commit(lead, bar_drain + 8 * s);
                mbar_wait(bar_drain + 8 * s, 0, kWaitLimit);
            }
        } else if (warp == 3) {
            // ---- finder: the next item, the longest rows first: of up to 32 sequences by their length (24 ragged prompts
            // 102 us against 107.5 sequence by sequence), of more by sequence, its last tiles first; false when there is none
            const int all = P.items * P.groups;
            // up to 32: a sequence a lane, its row tiles first + 1 .. first + tiles row tiles long
            constexpr int kRatio = kItemRows / kTileKeys;
            Item own;
            int tiles = 0, first = 0, part_len = 1, n_part = 0, base = 0, n_parts = 1, seen = 0x7fffffff;
            auto from = [&](int x) {   // row tiles at least x + 1 long
                return __reduce_add_sync(kAll, max(first + tiles - max(x, first), 0));
            };
            const bool ordered = SPLIT || P.n_seq <= 32;
            if (ordered) {
                if (lane < P.n_seq) tiles = tiles_of_sequence(lane, own);
                if (tiles) first = max(own.n_k - own.n_q, 0) / kItemRows;
                const int n = P.groups * from(0);
                if (lane == 0) n_part = n;
            }
            if (SPLIT) {
                if (P.window > 0) seen = (P.window + kItemRows) / kTileKeys + 2;   // key tiles at most
                const int k = min(max(seen / kRatio - first, 0), tiles);
                float work = kRatio * (static_cast<float>(k) * first + 0.5f * k * (k + 1)) + (tiles - k) * static_cast<float>(tiles > k ? seen : 0);
                const int top = __reduce_max_sync(kAll, first + tiles);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(kAll, work, o);
                const int longest = min(top > seen / kRatio ? seen : top * kRatio, seen);
                // a part is no longer than an SM's share of the work
                const int share = static_cast<int>(work * P.groups / kSMs) + 1;
                part_len = max(max(kMinPart, share), (longest + kMaxParts - 1) / kMaxParts);
                n_parts = longest - share > kWorthParts ? (longest + part_len - 1) / part_len : 1;
                int records = 0;
#pragma unroll 1
                for (int q = 0; q < n_parts; ++q) {   // lane q: items with more than q parts
                    const int n = P.groups * from(q * part_len / kRatio);
                    if (lane == q) {
                        n_part = n;
                        base = records;
                    }
                    if (q == 1) records = n;
                    if (q == 1 && lane == 1) base = n;
                    if (q) records += n;
                }
                // (sequences may overlap where bounds are out of order: then there may be more items than room)
                if (__shfl_sync(kAll, n_part, 0) > all || (!P.dense && records > P.n_rows / kRecord)) n_parts = 1;
                const int split = __shfl_sync(kAll, n_part, 1);
                if (blockIdx.x == 0) {
                    if (lane == 0) P.plan->items = n_parts > 1 ? split : 0;
                    if (lane < kMaxParts) P.plan->base[lane] = base;
                }
            }
            // a part of the longest rows first
            auto find_part = [&](int i, Item& it) {
                int q = n_parts - 1;
#pragma unroll 1
                for (; q >= 0; --q) {
                    const int n = __shfl_sync(kAll, n_part, q);
                    if (i < n) break;
                    i -= n;
                }
                if (q < 0) return -1;
                const int want = i / P.groups, record = __shfl_sync(kAll, base, q) + i;
                int lo = 0, hi = __reduce_max_sync(kAll, first + tiles), before = 0;
#pragma unroll 1
                while (hi - lo > 1) {   // from(lo) > want >= from(hi) = before
                    const int m = (lo + hi) / 2, n = from(m);
                    if (n > want) {
                        lo = m;
                    } else {
                        hi = m;
                        before = n;
                    }
                }
                const bool has = lo >= first && lo < first + tiles;
                const uint32_t there = __ballot_sync(kAll, has);
                const bool me = has && __popc(there & ((1u << lane) - 1)) == want - before;
                if (me) {
                    it = own;
                    it.row = (lo - first) * kItemRows;
                    it.group = i % P.groups;
                    it.from = 0;
                    it.to = 0x7fffffff;
                    it.slot = -1;
                    const int parts = SPLIT && n_parts > 1 ? min((min(lo >= seen / kRatio ? seen : (lo + 1) * kRatio, seen) + part_len - 1) / part_len, n_parts) : 1;
                    if (parts > 1) {
                        const Tiles t = tiles_of(unit_of<PAIR, SPLIT>(it, 0, P.window), unit_of<PAIR, SPLIT>(it, 1, P.window));
                        const int len = (max(t.hi - t.lo + 1, 0) + parts - 1) / parts;
                        if (len > 0) {
                            it.from = t.lo + q * len;
                            it.to = it.from + len - 1;
                        }
                        it.slot = P.dense ? (q * P.total_q + it.q0 + it.row) * P.H + (PAIR ? 2 : 1) * it.group : record * kRecord;
                        if (q == 0) {
                            P.heads[i].q0 = it.q0 + it.row;
                            P.heads[i].rows = it.n_q - it.row;
                            P.heads[i].group = it.group;
                            P.heads[i].parts = parts;
                        }
                    }
                }
                return __ffs(__ballot_sync(kAll, me)) - 1;
            };
            auto find = [&](int w) {
                int found = -1;
                Item it;
#pragma unroll 1
                while (found < 0) {
                    int i = 0;
                    if (lane == 0) i = static_cast<int>(atomicAdd(P.counter, 1u));
                    i = __shfl_sync(kAll, i, 0);
                    if (ordered) {
                        found = find_part(i, it);
                        break;
                    }
                    if (i >= all) break;
                    int want = P.items - 1 - i / P.groups;
                    // its chunk of sequences
                    int c = -1;
#pragma unroll 1
                    for (int c0 = 0; c0 < P.chunks; c0 += 32) {
                        const int mine = c0 + lane < P.chunks ? chunk_tiles[c0 + lane] : 0;
                        int upto = mine;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int y = __shfl_up_sync(kAll, upto, o);
                            if (lane >= o) upto += y;
                        }
                        const uint32_t hit = __ballot_sync(kAll, want < upto);
                        if (hit) {
                            const int at = __ffs(hit) - 1;
                            c = c0 + at;
                            want -= __shfl_sync(kAll, upto - mine, at);
                            break;
                        }
                        want -= __shfl_sync(kAll, upto, 31);
                    }
                    if (c < 0) continue;   // fewer tiles than there could be
#pragma unroll 1
                    for (int j0 = 0; j0 < P.chunk; j0 += 32) {
                        const int q = c * P.chunk + j0 + lane;
                        const int mine = j0 + lane < P.chunk && q < P.n_seq ? tiles_of_sequence(q, it) : 0;
                        int upto = mine;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int y = __shfl_up_sync(kAll, upto, o);
                            if (lane >= o) upto += y;
                        }
                        const uint32_t hit = __ballot_sync(kAll, want < upto);
                        if (hit) {
                            found = __ffs(hit) - 1;
                            it.row = (want - (upto - mine)) * kItemRows;
                            it.group = i % P.groups;
                            break;
                        }
                        want -= __shfl_sync(kAll, upto, 31);
                    }
                }
                if (found < 0) it.row = -1;
                if (lane == max(found, 0)) {
                    items[w % kItems] = it;
                    dirty[w % kItems] = 0;
                    mbar_arrive(bar_item + 8 * (w % kItems));
                }
                __syncwarp();
                return found >= 0;
            };
            // ---- and guard: in tiles that some row does not see all of, a value that is not finite is taken out
            // (a weight of zero would not stop it in the product), and keys past the sequence are zeroed; the
            // rows that see such a value get it at the end
            int n = 0;
            uint32_t nv = 0;
            bool ok = true, left = true;
#pragma unroll 1
            for (int w = -1; ok; ++w) {
                if (left) {   // one item ahead
                    if (w + 1 >= kItems)
                        ok = __all_sync(kAll, wait(bar_item_free + 8 * ((w + 1) % kItems), ((w + 1) / kItems - 1) & 1));
                    if (!ok) break;
                    left = find(w + 1);
                }
                if (w < 0) continue;
                const Item it = items[w % kItems];
                if (it.row < 0) break;
                const Unit u0 = unit_of<PAIR, SPLIT>(it, 0, P.window), u1 = unit_of<PAIR, SPLIT>(it, 1, P.window);
                const Tiles t = tiles_of(u0, u1);
#pragma unroll 1
                for (int b = t.lo; b <= t.hi; ++b, n += 2) {
                    if (!t.cut(b)) continue;
                    const int slot = (n + 1) % L::kSlots;
                    // only once its copy is under way does the slot's phase tell whether it has landed
                    ok = __all_sync(kAll, wait(bar_cut + 8 * (nv & 3), (nv >> 2) & 1)) &&
                         __all_sync(kAll, wait(bar_full + 8 * slot, ((n + 1) / L::kSlots) & 1));
                    if (!ok) break;
                    uint8_t* tile = smem_raw + (skv - smem_addr(smem_raw)) + slot * L::kTileBytes;
                    const int keys = it.n_k - b * kTileKeys;
                    uint4* v = reinterpret_cast<uint4*>(tile) + lane;
                    constexpr int kPieces = L::kTileBytes / 16 / 32;   // a lane's
                    if (keys < kTileKeys)
#pragma unroll 1
                        for (int i = 0; i < kPieces; ++i)
                            if ((i * 32 + lane) % 1024 / 8 >= keys) v[i * 32] = make_uint4(0, 0, 0, 0);
                    // where the exponent field is all ones, its sum with one carries into the sign's place
                    auto odd = [](uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                    uint32_t found = 0;
#pragma unroll 1
                    for (int i = 0; i < kPieces; i += 8) {
                        uint4 x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = v[(i + j) * 32];
#pragma unroll
                        for (int j = 0; j < 8; ++j) found |= odd(x[j].x) | odd(x[j].y) | odd(x[j].z) | odd(x[j].w);
                    }
                    if (found) {
                        uint32_t* word = reinterpret_cast<uint32_t*>(v);
#pragma unroll 1
                        for (int i = 0; i < 4 * kPieces; ++i) {
                            uint32_t& x = word[i / 4 * 128 + i % 4];
                            const uint32_t bad = odd(x);
                            x &= ~((bad & 0x8000u ? 0xffffu : 0u) | (bad & 0x80000000u ? 0xffff0000u : 0u));
                        }
                    }
                    if (__any_sync(kAll, found != 0)) dirty[w % kItems] = 1;
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_v + 8 * (nv & 3));
                    ++nv;
                }
                if (ok && lane == 0) release(w);
            }
        }
    } else if (warp < 12) {
        // ---- softmax: warpgroup s has unit s, a row a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<SPLIT>));
        const int s = (warp - 4) / 4, row = tid % 128;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + kTmS + 128 * s + lanes, to = tmem + kTmO + 128 * s + lanes;
        const float c = P.scale_log2;
        uint32_t ns = 0, nl = 0;   // nl: items that the unit was in
        bool ok = true;
        Item it;
        for (int w = 0; __all_sync(kAll, take(w, it, ok)); ++w) {
            const Unit u = unit_of<PAIR, SPLIT>(it, s, P.window);
            float m = -INFINITY, l = 0.f;   // m: running maximum, in powers of two
#pragma unroll 1
            for (int b = u.lo; b <= u.hi; ++b) {
                if (!(ok = __all_sync(kAll, wait(bar_s + 8 * s, ns)))) break;
                ns ^= 1;
                tc_fence_after();
                // Scores of keys 64 h .. 64 h + 63, what the row does not see at -infinity.  The second half is read
                // twice, for the maximum and for the weights: TMEM gives 64 columns in some 60 cycles, and the code
                // stays short (unrolled over 128 keys the kernel's code was several times the instruction
                // cache, and every pass through a rarely run part of it cost thousands of cycles).
                uint32_t x[64];
                auto load = [&](int h) {
                    tmem_ld32(ts + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
                    tmem_ld32(ts + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 64; ++i) asm volatile("" : "+r"(x[i]));
                    if (u.masked(b)) {
                        const int last = u.place + row - b * kTileKeys - 64 * h, first = P.window > 0 ? last - P.window + 1 : 0;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t seen = bits_to(last - 32 * i) & ~bits_to(first - 32 * i - 1);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!(seen >> j & 1u)) x[32 * i + j] = 0xff800000u;
                        }
                    }
                };
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll 1
                for (int h = 1; h >= 0; --h) {
                    load(h);
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        t0 = fmaxf(t0, fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
                        t1 = fmaxf(t1, fmaxf(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])));
                    }
                }
                const float top = fmaxf(t0, t1) * c;
                const bool raise = top > m + kLazy;
                if (__any_sync(kAll, raise)) {
                    const float f = raise ? ex2(m - top) : 1.f;   // (0 from -infinity)
                    if (raise) m = top;
                    l *= f;
                    if (b > u.lo) {
                        // the scores are complete, so the product before them is: O may be changed
#pragma unroll 1
                        for (int i = 0; i < D; i += 32) {
                            uint32_t x[32];
                            tmem_ld32(to + i, x);
                            tmem_wait_ld();
                            loaded(x);
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                            tmem_st32(to + i, x);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : -m;
                const float2 cc = make_float2(c, c), bb = make_float2(base, base);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (h) load(1);
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float2 y = fma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, bb);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        if (i & 1) sum1 = add2(sum1, y);
                        else sum0 = add2(sum0, y);
                        p[i] = pack_bf16(y.x, y.y);
                    }
                    tmem_st32(ts + 32 * h, p);
                }
                sum0 = add2(sum0, sum1);
                l += sum0.x + sum0.y;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p + 8 * s);
            }
            if (!ok) break;
            if (u.any()) {
                asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(sums + (((nl & 1) * 2 + s) * 128 + row) * 8), "f"(m), "f"(l)
                             : "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_l + 16 * s + 8 * (nl & 1));
                ++nl;
            }
            if (lane == 0) release(w);
        }
    } else {
        // ---- outputs of both units, a row a thread, while the softmax goes on with the next item
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutputRegs<SPLIT>));
        const int row = tid % 128;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t no[2] = {0, 0};
        bool ok = true;
        Item it;
#pragma unroll 1
        for (int w = 0; __all_sync(kAll, take(w, it, ok)); ++w) {
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
                const Unit u = unit_of<PAIR, SPLIT>(it, s, P.window);
                const uint32_t to = tmem + kTmO + 128 * s + lanes;
                float m = 0.f, l = 0.f;
                if (u.any()) {
                    const uint32_t n = s ? no[1]++ : no[0]++;
                    if (!(ok = __all_sync(kAll, wait(bar_l + 16 * s + 8 * (n & 1), n >> 1 & 1)) &&
                               __all_sync(kAll, wait(bar_o + 8 * s, n & 1))))
                        break;
                    tc_fence_after();
                    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(m), "=f"(l) : "r"(sums + (((n & 1) * 2 + s) * 128 + row) * 8) : "memory");
                }
                const bool part = SPLIT && it.slot >= 0;
                const float f = part ? 1.f : l != 0.f ? 1.f / l : 0.f;
                const bool mine = row < u.rows;
                // (set, if at all, before the products that bar_o told of)
                const bool add = u.any() && *const_cast<volatile int*>(&dirty[w % kItems]);
                __nv_bfloat16* const out = P.o + (static_cast<long long>(it.q0 + u.row + row) * P.H + u.head) * D;
#pragma unroll 1
                for (int i = 0; i < D && u.rows > 0; i += 32) {
                    uint32_t x[32];
                    if (u.any()) {
                        tmem_ld32(to + i, x);
                        tmem_wait_ld();
                        loaded(x);
                    }
                    if (i == D - 32) {   // the next item may have O
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0 && u.any()) mbar_arrive(bar_o_free + 8 * s);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = u.any() ? __float_as_uint(__uint_as_float(x[j]) * f) : 0u;
                    if (add && mine) give_back<PAIR, SPLIT>(P, it, u.place + row, u.head, i, x);
                    if (part) {
                        float* p = P.rows + static_cast<size_t>(it.slot + s * P.unit_step + row * P.row_step) * D + i;
                        if (mine && u.any())
#pragma unroll
                            for (int j = 0; j < 32; j += 8)
                                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + j), "r"(x[j]), "r"(x[j + 1]),
                                             "r"(x[j + 2]), "r"(x[j + 3]), "r"(x[j + 4]), "r"(x[j + 5]), "r"(x[j + 6]), "r"(x[j + 7])
                                             : "memory");
                    } else if (mine) {
                        uint32_t y[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) y[j] = pack_bf16(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                        store16(out + i, y, P.wide);
                    }
                    __syncwarp();
                }
                if (part) {
                    if (mine) P.sums[it.slot + s * P.unit_step + row * P.row_step] = make_float2(m, l);
                } else if (mine)
                    P.lse[static_cast<long long>(it.q0 + u.row + row) * P.H + u.head] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) release(w);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmCols);
    }
}

// Joins the records of the split items, a row a warp.  After a timeout, whose results are invalid, plan and heads
// may hold anything: they are checked before they are followed.
constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 32, kJoinSteps = 2 * kTileRows / kJoinRows;
template <int D, bool PAIR> __global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const __grid_constant__ PromptParams P) {
    constexpr int C = D / 32;   // channels a lane
    const int lane = threadIdx.x % 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (*P.status == kStatusTimeout) return;
    const long long steps = static_cast<long long>(min(max(P.plan->items, 0), P.items * P.groups)) * kJoinSteps;
#pragma unroll 1
    for (long long step = blockIdx.x; step < steps; step += gridDim.x) {
        const int item = static_cast<int>(step / kJoinSteps), at = static_cast<int>(step % kJoinSteps) * kJoinRows + threadIdx.x / 32,
                  s = at / kTileRows;
        const SplitHead head = P.heads[item];
        const int h = PAIR ? 2 * head.group + s : head.group, row = PAIR ? at % kTileRows : at;   // the item's row
        if (row >= head.rows || head.q0 < 0 || head.q0 >= P.total_q - row || h < 0 || h >= P.H) continue;
        float2 ml = make_float2(-INFINITY, 0.f);
        const float* y = nullptr;
        if (lane < min(head.parts, kMaxParts)) {
            const long long id = (P.dense ? (static_cast<long long>(lane) * P.total_q + head.q0) * P.H + (PAIR ? 2 : 1) * head.group
                                          : (static_cast<long long>(P.plan->base[lane]) + item) * kRecord) +
                                 s * P.unit_step + at % kTileRows * P.row_step;
            if (id >= 0 && id < P.n_rows) {
                y = P.rows + id * D;
                ml = P.sums[id];
            }
        }
        float m = ml.y != 0.f ? ml.x : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        const float base = m == -INFINITY ? 0.f : m, k = ml.y != 0.f ? ex2(ml.x - base) : 0.f;
        float l = ml.y != 0.f ? k * ml.y : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
        uint32_t some = __ballot_sync(kAll, ml.y != 0.f);   // (the others' outputs may not be there)
        float x[C];
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = 0.f;
#pragma unroll 1
        while (some) {   // four at a time, in order
            float v[4][C], kp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = some ? __ffs(some) - 1 : -1;
                kp[i] = __shfl_sync(kAll, k, max(p, 0));
                const float* z = reinterpret_cast<const float*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(y), max(p, 0)));
                some &= some - 1;
#pragma unroll
                for (int c = 0; c < C; ++c) v[i][c] = p >= 0 ? z[C * lane + c] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < C; ++c)   // a value that is not finite counts whatever the weight has become
                    x[c] += fabsf(v[i][c]) < INFINITY ? kp[i] * v[i][c] : v[i][c];
        }
        const float f = l != 0.f ? 1.f / l : 0.f;
        const long long out = (static_cast<long long>(head.q0) + row) * P.H + h;
        uint32_t w[C / 2];
#pragma unroll
        for (int c = 0; c < C / 2; ++c) w[c] = pack_bf16(x[2 * c] * f, x[2 * c + 1] * f);
        if constexpr (C == 4) *reinterpret_cast<uint2*>(P.o + out * D + C * lane) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(P.o + out * D + C * lane) = w[0];
        if (lane == 0) P.lse[out] = l != 0.f ? (base + log2f(l)) * kLn2 : -INFINITY;
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// [rows, heads, d] bf16, tiles of 128 rows and 64 channels of one head.
bool encode(CUtensorMap* m, const Strided& x, int rows, int heads, int d) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(x.head) * 2, static_cast<cuuint64_t>(x.row) * 2};
    const cuuint32_t box[3] = {64, 1, kTileKeys}, step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.p), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows for parts, of at most kSplitItems items.
int part_rows(int total_q, int H, long long items) {
    return static_cast<int>(std::min((items + kSMs) * kRecord, static_cast<long long>(kMaxParts) * total_q * H));
}

bool can_split(int n_seq, long long items) { return n_seq <= 32 && items <= kSplitItems; }

// Whether an item is longer than an SM's share of all by more than parts cost, as far as the host can tell: with the
// prefixes spread evenly, or, by far, with one sequence having them all.  (Where the kernel then finds rows that are
// not worth it, being ready for it has cost some 4 us: 16 x 256 over 740 each, 43 against 39.)
bool worth_splitting(const PromptArgs& a, long long items) {
    const double prefix = a.total_k > a.total_q ? static_cast<double>(a.total_k) - a.total_q : 0.0,
                 rows = static_cast<double>(a.total_q) / a.n_seq, seen = a.window > 0 ? a.window : 2147483648.0;
    const double even = std::min(prefix / a.n_seq + rows, seen), most = std::min(prefix + rows, seen),
                 share = items * std::min(prefix / a.n_seq + rows / 2, seen) / kSMs;
    return even - share > kWorthParts * kTileKeys || most - share > 3.0 * kWorthParts * kTileKeys;
}

template <int D, bool PAIR, bool SPLIT> cudaError_t start(const PromptParams& P, int blocks, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<D, PAIR, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Layout<D>::kSmem);
    if (e != cudaSuccess) return e;
    prompt_tc_kernel<D, PAIR, SPLIT><<<blocks, kThreads, Layout<D>::kSmem, s>>>(P);
    return cudaGetLastError();
}

template <int D, bool PAIR> cudaError_t launch(const PromptArgs& a, cudaStream_t s) {
    PromptParams P;
    // without keys nothing is loaded; the maps then describe the queries
    const Strided &k = a.total_k ? a.k : a.q, &v = a.total_k ? a.v : a.q;
    const int nk = a.total_k ? a.total_k : a.total_q, hk = a.total_k ? a.H_kv : a.H;
    if (!encode(&P.tq, a.q, a.total_q, a.H, D) || !encode(&P.tk, k, nk, hk, D) || !encode(&P.tv, v, nk, hk, D))
        return cudaErrorInvalidValue;
    P.v = static_cast<const __nv_bfloat16*>(a.v.p);
    P.v_row = a.v.row; P.v_head = a.v.head;
    P.cu_q = a.cu_q; P.cu_k = a.cu_k;
    P.o = static_cast<__nv_bfloat16*>(a.o); P.lse = a.lse; P.status = a.status;
    P.n_seq = a.n_seq; P.total_q = a.total_q; P.total_k = a.total_k; P.H = a.H; P.H_kv = a.H_kv; P.window = a.window;
    P.wide = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 ? 1 : 0;
    P.probe = (a.flags & KDN_FLAG_TIMEOUT_PROBE) ? 1 : 0;
    P.scale_log2 = a.scale * kLog2e;
    constexpr int rows = PAIR ? kTileRows : 2 * kTileRows;
    P.groups = PAIR ? a.H / 2 : a.H;
    // no more tiles than this, whatever the lengths
    P.items = a.total_q / rows + (a.n_seq < a.total_q ? a.n_seq : a.total_q);
    const long long grid = static_cast<long long>(P.items) * P.groups;
    if (grid > 0x7fff0000ll) return cudaErrorInvalidValue;   // (the counter goes on past the last item, once a block)
    P.counter = a.status + 1;
    P.chunk = 32 * ((a.n_seq + 32 * kChunks - 1) / (32 * kChunks));
    P.chunks = (a.n_seq + P.chunk - 1) / P.chunk;
    const bool split = can_split(a.n_seq, grid) && worth_splitting(a, grid);
    if (split) {
        // (records are written in pieces of 32 bytes)
        P.plan = reinterpret_cast<SplitPlan*>((reinterpret_cast<uintptr_t>(a.scratch) + 31) / 32 * 32);
        P.heads = reinterpret_cast<SplitHead*>(P.plan + 1);
        P.rows = reinterpret_cast<float*>(P.heads + grid);
        P.n_rows = part_rows(a.total_q, a.H, grid);
        P.sums = reinterpret_cast<float2*>(P.rows + static_cast<size_t>(P.n_rows) * D);
        P.dense = P.n_rows < (grid + kSMs) * kRecord ? 1 : 0;
        P.row_step = P.dense ? a.H : 1;
        P.unit_step = P.dense && PAIR ? 1 : kTileRows * P.row_step;
        cudaError_t e = start<D, PAIR, true>(P, kSMs, s);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(4 * kSMs);
        cfg.blockDim = dim3(kJoinThreads);
        cfg.stream = s;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, prompt_join_kernel<D, PAIR>, P);
    }
    return start<D, PAIR, false>(P, static_cast<int>(grid < kSMs ? grid : kSMs), s);
}

}  // namespace

bool prompt_tc_supported(int io, int d) { return io == 1 && (d == 64 || d == 128); }

size_t prompt_tc_scratch(int n_seq, int total_q, int H, int H_kv, int d) {
    if (n_seq <= 0 || total_q <= 0 || H <= 0 || H_kv <= 0) return 0;
    const bool pair = (H / H_kv) % 2 == 0;
    const long long tiles = total_q / (pair ? kTileRows : 2 * kTileRows) + (n_seq < total_q ? n_seq : total_q),
                    items = tiles * (pair ? H / 2 : H);
    if (!can_split(n_seq, items)) return 0;
    return 32 + sizeof(SplitPlan) + items * sizeof(SplitHead) + part_rows(total_q, H, items) * sizeof(float) * (d + 2);
}

cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t s) {
    const bool pair = (a.H / a.H_kv) % 2 == 0;
    if (a.d == 128) return pair ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return pair ? launch<64, true>(a, s) : launch<64, false>(a, s);
}

}  // namespace kdn
