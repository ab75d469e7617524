// Linear attention with a decay for each head on tcgen05 tensor cores: bf16, dk and dv 64 or 128.
//
// One block walks a head of a sequence (or of a segment of it) in chunks of 64 tokens (the chunk form: decay.cu).  All
// products have the value channels in their rows (TMEM lanes), so that the state lies in the registers of one warpgroup, a
// value channel a thread, and goes back into the products through TMEM:
//   W  = Q K^T              (64 rows of 128: an MMA of 64 takes as long)
//   P  = W g^(i-j)          bf16, shared memory
//   U^T = V'^T K            V'_j = g^(m-1-j) v_j in bf16 parts, written to TMEM by a warpgroup that reads V transposed
//   S   = g^m S + U         fp32, registers;  bf16 S^T to TMEM
//   O^T = V^T P^T + (S^T Q^T) g^(i+1)
// V' has three parts (24 bits), and two (16) where dense sequences that were cut are walked for their outputs alone: one part
// would add as much to the error of o as its own rounding does.  (Whole walks of the gradients of q and k have three, too, though
// no state comes out of them: with the parts chosen at run time heads of 64 took 98 us for 88.)
// S^T and P go in as bf16, one part each: the roundings of the terms that they are multiplied into are independent, and with them
// the error of o is 0.0023 of its norm where its own rounding to bf16 gives 0.0017.  Two parts of each would be twice the products
// of the outputs, and S^T's second one has no place in TMEM beside three parts of V' (480 of 512 columns are taken).
//
// U depends on no state, so a chunk's products run while the last chunk's state is still on its way: the walk's only serial
// step is S = g^m S + U, a fused multiply-add an element.
//
// Measured: 8 sequences of 4096 tokens, 16 heads of 128, 107 us, 5.1 TB/s of what it has to move, 76% of the copy rate
// on 128 of the 152 SMs (the first form, with the roles' loops unrolled and values read one by one, 250); its gradients 303 us
// (three walks, 384 blocks: two and a half turns of the SMs); 65536 tokens alone 292 to 299 (states 98, chaining 5, outputs 175); 24 of 2
// to 4095, heads of 64, 93 (the longest one's 64 chunks).  A chunk takes 1.5 us for heads of 128 and 1.35 for heads of 64, where
// its bytes would take 1.24 and its products 0.7.  What bounds it is the chain of the roles: V' (some 260 instructions a warp and
// chunk, five cycles each, as an SM's quarter has five warps, all of other roles), the state, the outputs, and what a barrier takes
// between them.  Bytes do not: with all copies from the same two chunks (L2) it took 112.5 us against 113.  Less work
// anywhere helps a little (left out of copies of this file: the weights' arithmetic 7 us, W's products 8, a part and a half
// of V' 11, the stores 3); longer code costs more than it saves, as the roles' loops hardly fit the instruction caches
// (V' unrolled, and computed ahead of its turn: 116 us for 106).  Also slower: looking at barriers without suspension (128 for
// 118), tiles asked for into L2 ahead (119 to 141 for 118), copies asked for by the warps that issue products (see the loader).  No
// faster for heads of 64: TMEM for V' of two chunks (89.3 us for 88.2), or for outputs of two (88.8).

#include <cuda.h>
#include <cuda_bf16.h>
#include <mutex>

#include "common.cuh"
#include "decay.h"
#include "decay_common.cuh"
#include "kdn.h"
#include "packed.cuh"
#include "sm100.cuh"

namespace kdn {
namespace {

using namespace sm100;

constexpr int kC = 64;                        // tokens of a chunk
// two weight warps and two product warps; the state; V' of a chunk's first and second 32 tokens; outputs: a warpgroup each.  (A
// warp more would leave 80 registers a thread at launch: a quarter of the SM's registers is for six warps then.)
constexpr int kThreads = 640;
constexpr int kStateRegs = 184, kValueRegs = 64, kOutputRegs = 72;   // the first warpgroup has 96 as launched: 96 + 184 + 2 x 64 + 72 = 5 x 96
constexpr uint32_t kWaitLimit = 1u << 20, kProbeLimit = 4096;   // polls of about a microsecond at most
constexpr uint32_t kAll = 0xffffffffu;
constexpr uint32_t kHalf = 8192;              // 64 tokens of 64 channels
constexpr uint32_t kFRow = 36 * 4;            // 32 powers; rows apart by 4 banks
constexpr int kMarks = 4;                     // chunks whose marks of values that are not finite are kept

struct TcParams {
    CUtensorMap q[kMaxDecayJobs], k[kMaxDecayJobs], v[kMaxDecayJobs], o[kMaxDecayJobs];
    DecayParams d;
};

template <int DK, int DV, bool OUT> struct Layout {
    static constexpr int kStages = OUT ? (DK + DV == 128 ? 6 : 3) : 6, kKHalves = DK / 64, kVHalves = DV / 64;
    // a stage: halves of K, of Q, of V.  (Products read 128 rows of Q and 128 value channels: what lies behind a half, or behind
    // 64 channels, is multiplied too, and its rows are not used.)
    static constexpr uint32_t kQ = kKHalves * kHalf, kV = (OUT ? 2 : 1) * kQ, kStage = kV + kVHalves * kHalf;
    static constexpr uint32_t kP = kStages * kStage, kO = kP + 2 * kHalf;   // weights of two chunks; outputs: 4 KB a warp, twice
    static constexpr uint32_t kF = kO + 2 * 4 * 4096;   // the weights' powers, 2 x 32 rows
    static constexpr uint32_t kSmem = (OUT ? kF + 2 * 32 * kFRow : kP + kHalf) + 1024;
};

// TMEM columns: W; O within the chunk and from the state; U; parts of V'; S^T.  Where the state alone is wanted there is room
// for U and V' of two chunks.
template <bool OUT> struct Tm {
    static constexpr int kBufs = OUT ? 1 : 2;
    static constexpr uint32_t kW = 0, kI = 64, kX = 128, kU = 192, kV = OUT ? 320 : 0, kS = 416;
};
constexpr uint32_t kTmCols = 512;

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(c0), "r"(c1),
                 "r"(c2), "r"(src)
                 : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// The warp that issues products runs as a whole, so that descriptors stay in uniform registers; one lane's predicate issues.
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
template <int N> __device__ __forceinline__ void loaded(uint32_t (&r)[N]) {   // after tmem_wait_ld(): ties the registers to that point
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// Fragments of 16 lanes: 32-bit column t % 4 of lanes t / 4 and t / 4 + 8 ...
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, uint32_t r0, uint32_t r1) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x1.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(r0), "r"(r1));
}
// ... and columns 2 (t % 4), + 1 of lane t / 4, then those of lane t / 4 + 8 (and again eight columns on).
__device__ __forceinline__ void tmem_ld_frag4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
// Four 8 x 8 matrices of 16 bits, transposed: a lane's address is a row's (matrix lane / 8, row lane % 8).
__device__ __forceinline__ void ldmatrix_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void stmatrix_t(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a));
    return x;
}

// OUT: outputs, else the state alone.  PARTS: of V'.
template <int DK, int DV, bool OUT, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) decay_tc_kernel(const __grid_constant__ TcParams T) {
    using L = Layout<DK, DV, OUT>;
    using M = Tm<OUT>;
    constexpr int kStages = L::kStages;
    const DecayParams& P = T.d;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[4 * kStages + 13];
    __shared__ float pw[kC + 1];
    __shared__ __align__(16) float vf[2][kC], rf[2][kC];   // factors of the chunk's tokens in V' and in outputs: whole chunk, last one
    __shared__ int marks[kMarks][2][128];                  // per value channel, the first token of the walk (in a half) that is not finite
    __shared__ volatile int aborted;
    __shared__ uint32_t tmem_slot;
    const uint32_t sb = (smem_addr(smem_raw) + 1023u) & ~1023u;
    // a barrier a stage: loaded, free, V' of the first 32 tokens, V' of all (and what is not to be multiplied taken out)
    const uint32_t bar_full = smem_addr(bars), bar_empty = bar_full + 8 * kStages, bar_v1 = bar_empty + 8 * kStages,
                   bar_v2 = bar_v1 + 8 * kStages, bar_u = bar_v2 + 8 * kStages, bar_u_free = bar_u + 16, bar_u1 = bar_u_free + 16,
                   bar_w = bar_u1 + 8, bar_p = bar_w + 8, bar_s = bar_p + 8, bar_s_free = bar_s + 8, bar_o = bar_s_free + 8,
                   bar_o_free = bar_o + 8, bar_drain = bar_o_free + 8, bar_probe = bar_drain + 8;   // bar_u1: the first 32 tokens
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // (the jobs of a head side by side: those of one direction read the same tokens at about the same time)
    const int job = blockIdx.x % P.n_jobs, item = blockIdx.x / P.n_jobs / P.H, h = blockIdx.x / P.n_jobs % P.H;
    const DecayJob& J = P.job[job];
    const bool rev = J.reverse != 0;

    const DecayItem it = find_item(P, item, tid < 32 && h == 0 && job == 0);
    if (!it.any) return;
    const int row0 = it.row, len = it.len;
    constexpr size_t elems = static_cast<size_t>(DK) * DV;
    const size_t bh = static_cast<size_t>(it.b) * P.H + h;
    const float* in = nullptr;
    float* end = nullptr;
    int s_k = J.s_k, s_v = J.s_v;
    if (it.slot < 0) {
        in = J.S0 ? J.S0 + bh * elems : nullptr;
        end = J.S_T ? J.S_T + bh * elems : nullptr;
    } else {
        float* st = P.states[job] + (static_cast<size_t>(it.slot) * P.H + h) * elems;
        s_k = DV;
        s_v = 1;
        if (P.pass == kStates) end = st;
        else in = st;
    }
    if (len == 0) {
        if (end)
            for (int i = tid; i < static_cast<int>(elems); i += kThreads) end[i] = in ? in[i] : 0.f;   // (the same layout)
        return;
    }
    const int chunks = (len + kC - 1) / kC, m_last = len - (chunks - 1) * kC;   // tokens of the chunk that may be short
    const float l = P.log_decay[h];
    // chunk n of the walk: its place among the chunks, and whether it is the short one
    auto place = [&](int n) { return rev ? chunks - 1 - n : n; };
    auto is_last = [&](int n) { return place(n) == chunks - 1; };

    // copies of chunk n of the walk; the first ones by the first thread, the others by one of those that make weights
    const int early = P.probe ? 1 : min(chunks, kStages);
    auto copy = [&](int n) {
        const int slot = n % kStages, t = row0 + place(n) * kC;
        const uint32_t st = sb + slot * L::kStage, full = bar_full + 8 * slot;
        mbar_expect_tx(full, L::kStage);
        tma_load_4d(st, &T.k[job], 0, t, 0, h, full);
        if (OUT) tma_load_4d(st + L::kQ, &T.q[job], 0, t, 0, h, full);
        tma_load_4d(st + L::kV, &T.v[job], 0, t, 0, h, full);
        if (P.probe && n == 0 && !mbar_wait(bar_probe, 0, kProbeLimit)) {
            aborted = 1;
            set_status(P.status, kStatusTimeout);
        }
    };
    if (tid == 0) {
        aborted = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, OUT ? 2 : 1);
            mbar_init(bar_v1 + 8 * i, 4);
            mbar_init(bar_v2 + 8 * i, 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_u + 8 * i, 1);
            mbar_init(bar_u_free + 8 * i, 4);
        }
        mbar_init(bar_u1, 1);
        mbar_init(bar_w, 1);
        mbar_init(bar_p, 2);
        mbar_init(bar_s, 4);
        mbar_init(bar_s_free, 1);
        mbar_init(bar_o, 1);
        mbar_init(bar_o_free, 4);
        mbar_init(bar_drain, OUT ? 2 : 1);
        mbar_init(bar_probe, 1);   // completed by nothing
        mbar_fence_init();
        fence_proxy_async();
        for (int i = 0; i < early && !aborted; ++i) copy(i);   // (before all else: the first of them takes longer than that)
    }
    if (tid <= kC) pw[tid] = power(l, tid);
    if (warp == 8) {
        tmem_alloc(smem_addr(&tmem_slot), kTmCols);
        tc_fence_before();
    }
    __syncthreads();
    if (tid < 2 * kC) {
        const int last = tid / kC, i = tid % kC, m = last ? m_last : kC, left = m - 1 - i;
        vf[last][i] = left < 0 ? 0.f : pw[rev ? i + 1 : left];
        rf[last][i] = left < 0 ? 0.f : pw[rev ? left : i + 1];
    }
    // powers of the weights' two blocks of 32 x 32
    for (int e = tid; OUT && e < 2 * 32 * 32; e += kThreads) {
        const int i = e / 32 % 32, j = e % 32, gap = rev ? j - i : i - j;
        const float f = e < 1024 ? pw[abs(gap)] : pw[32 + gap];
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(sb + L::kF + (e / 32) * kFRow + 4 * j), "f"(f) : "memory");
    }
    tc_fence_after();
    __syncthreads();
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
    auto await = [&](uint32_t bar, uint32_t parity) { return __all_sync(kAll, wait(bar, parity)); };

    if (warp < 4) {
        constexpr uint32_t id_w = idesc_bf16(128, 64, 0, 0, 0), id_u = idesc_bf16(128, DK, 0, 1, 0), id_i = idesc_bf16(128, 64, 1, 0, 0);
        auto one = [](uint32_t x) { return __shfl_sync(kAll, x, 0); };
        const uint32_t base = one(sb), tm = one(tmem);
        if (warp == 2) {
            // ---- products of the state
            const uint32_t lead = elect_one();
            const uint64_t kt = sw128_desc(base, kHalf, 1024);
            uint32_t slot = 0, phase = 0;
            bool ok = true;
#pragma unroll 1
            for (int n = 0; n < chunks; ++n) {
                const uint32_t at = slot * L::kStage, buf = n % M::kBufs, turn = n / M::kBufs;
                if (turn > 0 && !(ok = await(bar_u_free + 8 * buf, (turn - 1) & 1))) break;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    if (!(ok = await((half ? bar_v2 : bar_v1) + 8 * slot, phase))) break;
                    tc_fence_after();
                    // (the small parts first: the sums' last bits are cut off)
#pragma unroll
                    for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma_ts(lead, tm + M::kU + 128 * buf, tm + M::kV + 96 * buf + 32 * p + 16 * half + 8 * k,
                                   desc_add(kt, at + half * 4096 + k * 2048), id_u, half || p < PARTS - 1 || k > 0);
                    if (half) commit(lead, bar_u + 8 * buf);
                    else if (OUT) commit(lead, bar_u1);
                }
                if (!ok) break;
                commit(lead, bar_empty + 8 * slot);
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            // products already issued end before TMEM goes away
            commit(lead, bar_drain);
            mbar_wait(bar_drain, 0, kWaitLimit);
        } else if (warp == 3 && OUT) {
            // ---- products of the outputs
            const uint32_t lead = elect_one();
            const uint64_t kd = sw128_desc(base, 16, 1024), qd = sw128_desc(base + L::kQ, 16, 1024), vt = sw128_desc(base + L::kV, kHalf, 1024), pd = sw128_desc(base + L::kP, 16, 1024);
            auto weights = [&](uint32_t at) {
#pragma unroll 1
                for (int f = 0; f < L::kKHalves; ++f)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t x = at + f * kHalf + k * 32;
                        mma_ss(lead, tm + M::kW, desc_add(qd, x), desc_add(kd, x), id_w, f > 0 || k > 0);
                    }
                commit(lead, bar_w);
            };
            uint32_t slot = 0, phase = 0;
            bool ok = await(bar_full, 0);
            tc_fence_after();
            if (ok) weights(0);
#pragma unroll 1
            for (int n = 0; ok && n < chunks; ++n) {
                const uint32_t here = slot, at = here * L::kStage, par = n & 1, turn = phase;
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1;
                }
                if (!(ok = await(bar_p, par))) break;
                if (n + 1 < chunks) {
                    if (!(ok = await(bar_full + 8 * slot, phase))) break;
                    tc_fence_after();
                    weights(slot * L::kStage);
                }
                if (!(ok = await(bar_s, par))) break;
                if (n > 0 && !(ok = await(bar_o_free, par ^ 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int f = 0; f < L::kKHalves; ++f)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(lead, tm + M::kX, tm + M::kS + 32 * f + 8 * k, desc_add(qd, at + f * kHalf + k * 32), id_w, f > 0 || k > 0);
                commit(lead, bar_s_free);
                if (!(ok = await(bar_v2 + 8 * here, turn))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kC / 16; ++k)
                    mma_ss(lead, tm + M::kI, desc_add(vt, at + k * 2048), desc_add(pd, par * kHalf + k * 32), id_i, k > 0);
                commit(lead, bar_o);
                commit(lead, bar_empty + 8 * here);
            }
            commit(lead, bar_drain);
            mbar_wait(bar_drain, 0, kWaitLimit);
        } else if (warp < 2) {
            // ---- loader, a lane of the warp that has less to do otherwise (asked for by the warp of the state's products or of
            // the outputs, copies held these up by 600 to 1000 cycles a chunk)
            const bool loads = lane == 0 && warp == (rev ? 1 : 0);
            int sent = early;
            auto load = [&]() {   // the next chunk, once its stage is free
                if (!wait(bar_empty + 8 * (sent % kStages), (sent / kStages - 1) & 1)) return;
                copy(sent);
                ++sent;
            };
            if (loads && !OUT)
#pragma unroll 1
                while (sent < chunks && !aborted) load();
            __syncwarp();
            // ---- weights: row i of the chunk a thread.  Of the two blocks of 32 columns one is cut by the
            // diagonal, with the same powers in every chunk, and one is seen whole or not at all.
            const int low = warp, i = lane;   // rows 32 low + i
            const bool whole = rev ? low == 0 : low == 1;
            const uint32_t tw = tmem + M::kW + (static_cast<uint32_t>(warp * 32) << 16), mine = sb + L::kF + i * kFRow;
            const uint32_t cut = rev ? ~((1u << i) - 1u) : (2u << i) - 1u;   // columns of the block that the row sees
            auto to = [&](int n, int c, int j) { return sb + L::kP + (n & 1) * kHalf + sw128_off(32 * low + i, 4 * c + j); };
            auto put = [&](uint32_t a, const uint32_t* x) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = pack_bf16(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
            };
            if (OUT && !whole)
                for (int n = 0; n < 2; ++n)
                    for (int j = 0; j < 4; ++j)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to(n, low ^ 1, j)), "r"(0) : "memory");
#pragma unroll 1
            for (int n = 0; OUT && n < chunks; ++n) {
                if (!await(bar_w, n & 1)) break;
                tc_fence_after();
                // (a short chunk's last columns are masked by the diagonal in a forward walk)
                const int m = rev && is_last(n) ? m_last : kC;
#pragma unroll 1
                for (int e = 0; e < (whole ? 2 : 1); ++e) {   // the block that is cut, then the other
                    const int c = low ^ e;
                    uint32_t x[32];
                    float f[32];
                    tmem_ld32(tw + 32 * c, x);
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(f[j]), "=f"(f[j + 1]), "=f"(f[j + 2]), "=f"(f[j + 3])
                                     : "r"(mine + e * 32 * kFRow + 4 * j));
                    uint32_t seen = e ? kAll : cut;
                    if (m - 32 * c < 32) seen &= m > 32 * c ? (1u << (m - 32 * c)) - 1u : 0u;
                    tmem_wait_ld();
                    loaded(x);
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = seen >> j & 1u ? __float_as_uint(__uint_as_float(x[j]) * f[j]) : 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) put(to(n, c, j), x + 8 * j);
                }
                tc_fence_before();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p);
                // (the stage of the last chunk: done with by the time that this one's weights are used)
                if (loads && n > 0 && sent < chunks && !aborted) load();
                __syncwarp();
            }
            // copies already issued land before the block's shared memory goes away (where there are outputs, a walk that was not
            // given up has waited for all of them here)
            if (loads && (aborted || !OUT))
                for (int i = max(sent - kStages, 0); i < sent; ++i) mbar_wait(bar_full + 8 * (i % kStages), (i / kStages) & 1, kWaitLimit);
        }
    } else if (warp < 8) {
        // ---- state: value channel j a thread, all key channels in its registers
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
        const int j = tid - 128;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16, tu = tmem + M::kU + lanes, ts = tmem + M::kS + lanes;
        const bool mine = j < DV;
        float S[DK];
        if (in && mine) {
            const float* p = in + static_cast<size_t>(j) * s_v;
            if (s_k == 1) {
#pragma unroll
                for (int i = 0; i < DK; i += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(p + i);
                    S[i] = x.x; S[i + 1] = x.y; S[i + 2] = x.z; S[i + 3] = x.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < DK; ++i) S[i] = p[static_cast<size_t>(i) * s_k];
            }
        } else {
#pragma unroll
            for (int i = 0; i < DK; ++i) S[i] = 0.f;
        }
        auto give = [&]() {   // S^T as the next products' operand
#pragma unroll
            for (int c = 0; c < DK; c += 64) {
                uint32_t x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = pack_bf16(S[c + 2 * i], S[c + 2 * i + 1]);
                tmem_st32(ts + c / 2, x);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_s);
        };
        if (OUT) give();
        const Carry f_full(l, kC), f_last(l, m_last);
        float rest = 0.f;
#pragma unroll 1
        for (int n = 0; n < chunks; ++n) {
            const uint32_t buf = n % M::kBufs, here = tu + 128 * buf;
            if (!await(bar_u + 8 * buf, n / M::kBufs & 1)) break;
            tc_fence_after();
            const float f = (is_last(n) ? f_last : f_full).next(rest);
            const float2 ff = make_float2(f, f);
            uint32_t x[2][32];   // the next columns are on their way while these are added
            tmem_ld32(here, x[0]);
#pragma unroll
            for (int c = 0; c < DK; c += 32) {
                tmem_wait_ld();
                loaded(x[c / 32 % 2]);
                if (c + 32 < DK) tmem_ld32(here + c + 32, x[(c / 32 + 1) % 2]);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const uint32_t* u = x[c / 32 % 2] + i;
                    const float2 z = fma2(ff, make_float2(S[c + i], S[c + i + 1]), make_float2(__uint_as_float(u[0]), __uint_as_float(u[1])));
                    S[c + i] = z.x;
                    S[c + i + 1] = z.y;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_u_free + 8 * buf);
            if (OUT && n + 1 < chunks) {
                if (!await(bar_s_free, n & 1)) break;
                tc_fence_after();
                give();
            }
        }
        if (end && mine && !aborted)
#pragma unroll
            for (int i = 0; i < DK; ++i) end[static_cast<size_t>(i) * s_k + static_cast<size_t>(j) * s_v] = S[i];
    } else if (warp < 16) {
        // ---- V': 32 value channels a warp, transposed on the way from shared memory to fragments: a thread has tokens
        // 8 t + 2 (lane % 4), + 1 of channels lane / 4 + 0, 8, 16, 24.  A warpgroup has tokens 0 .. 31, the other the rest.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kValueRegs));
        const int j = tid % 128, half = warp >= 12;   // the channel whose marks the thread keeps
        const uint32_t tv = tmem + M::kV + 16 * half + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t rows = L::kV + (j / 64) * kHalf + half * 4096 + (lane & 7) * 128 + (((j % 64 / 32 * 4 + lane / 8) ^ (lane & 7)) << 4);
        uint32_t slot = 0, phase = 0;
#pragma unroll 1
        for (int n = 0; n < chunks; ++n) {
            const uint32_t buf = n % M::kBufs;
            if (!await(bar_full + 8 * slot, phase)) break;
            // the place of V' has been read
            if (n >= M::kBufs && !await(OUT && !half ? bar_u1 : bar_u + 8 * buf, (n / M::kBufs - 1) & 1)) break;
            tc_fence_after();
            const bool last = is_last(n);
            const int m = (last ? m_last : kC) - 32 * half;   // tokens from the half's first on
            const uint32_t st = sb + slot * L::kStage;
            float2 odd = make_float2(0.f, 0.f);   // NaN where a value is not finite
            // (in a loop, as short as may be: the block's roles together hardly fit the instruction cache)
#pragma unroll 1
            for (int t = 0; t < 4; ++t) {
                uint32_t v[4] = {};
                if (j - lane < DV) ldmatrix_t(st + rows + t * 1024, v);
                const int at = 8 * t + 2 * (lane % 4);
                const float2 f = *reinterpret_cast<const float2*>(&vf[last][32 * half + at]);
                if (m < 32) {   // rows of other sequences
                    const uint32_t there = at + 1 < m ? 0xffffffffu : at < m ? 0xffffu : 0u;
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] &= there;
                }
                uint32_t part[PARTS][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float2 x = unpack2(v[c]);
                    if (OUT) odd = fma2(x, make_float2(0.f, 0.f), odd);
                    x = mul2(x, f);
                    // (parts cut off, not rounded: three have all 24 bits, and cutting off takes one instruction a pair)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        part[p][c] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
                        if (p + 1 < PARTS)
                            x = fma2(make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u), __uint_as_float(__float_as_uint(x.y) & 0xffff0000u)),
                                     make_float2(-1.f, -1.f), x);
                    }
                }
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {   // lanes 0 .. 15, and 16 .. 31
                    tmem_st_frag(tv + 96 * buf + 32 * p + 4 * t, part[p][0], part[p][1]);
                    tmem_st_frag(tv + 96 * buf + 32 * p + 4 * t + (16u << 16), part[p][2], part[p][3]);
                }
            }
            if (OUT) {
                // Values that are not finite are taken out of the product with the weights (a weight of zero would not stop
                // them); the walk's rows from the first of them on get it back.
                int mark = kC;
                if (__any_sync(kAll, odd.x + odd.y != 0.f)) {
                    if (j < DV)
#pragma unroll 1
                        for (int i = 31; i >= 0; --i) {
                            const int t = rev ? 31 - i : i;
                            const uint32_t a = st + L::kV + (j / 64) * kHalf + half * 4096 + t * 128 + (((j % 64 / 8) ^ (t & 7)) << 4) + (j % 8) * 2;
                            if (t < m && (lds16(a) & 0x7f80u) == 0x7f80u) {
                                mark = 32 * half + t;
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(0)) : "memory");
                            }
                        }
                    fence_proxy_async();
                }
                marks[n % kMarks][half][j] = mark;
            }
            if (m < 32) {   // rows of other sequences
                constexpr int kRows = (L::kKHalves + L::kVHalves) * 8;   // pieces of a token
                const int gone = max(m, 0);
                for (int i = j; i < (32 - gone) * kRows; i += 128) {
                    const int t = 32 * half + gone + i / kRows, c = i % kRows / 8;
                    const uint32_t a = st + (c < L::kKHalves ? c * kHalf : L::kV + (c - L::kKHalves) * kHalf) + t * 128 + (i % 8) * 16;
                    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(0) : "memory");
                }
                fence_proxy_async();
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (!half) mbar_arrive(bar_v1 + 8 * slot);
                mbar_arrive(bar_v2 + 8 * slot);
            }
            if (++slot == kStages) {
                slot = 0;
                phase ^= 1;
            }
        }
    } else {
        // ---- outputs: 32 value channels a warp, as fragments like those of V', put in token order and stored
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutputRegs));
        const int j = tid - 512;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16, ti = tmem + M::kI + lanes, tx = tmem + M::kX + lanes;
        if (OUT) {
#pragma unroll 1
            for (int n = 0; n < chunks; ++n) {
                const bool last = is_last(n);
                const int m = last ? m_last : kC;
                const uint32_t out = sb + L::kO + ((n & 1) * 4 + (warp & 3)) * 4096;
                // 16 bytes `c` of token t
                auto piece = [&](int t, int c) { return out + t * 64 + ((c ^ (t >> 1 & 3)) << 4); };
                if (lane == 0) bulk_wait_read1();   // the store of two chunks ago has read its place
                __syncwarp();
                if (!await(bar_o, n & 1)) break;
                tc_fence_after();
                const int mark0 = marks[n % kMarks][0][j], mark1 = marks[n % kMarks][1][j];
                // 16 channels and 32 tokens at a time, the next ones on their way while these are put in order
                auto at = [](int e) { return ((e >> 1) * 16u << 16) + 32 * (e & 1); };
                uint32_t x[2][16], y[2][16];
                tmem_ld_frag4(ti, x[0]);
                tmem_ld_frag4(tx, y[0]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t (&xi)[16] = x[e & 1], (&yi)[16] = y[e & 1];
                    tmem_wait_ld();
                    loaded(xi);
                    loaded(yi);
                    if (e < 3) {
                        tmem_ld_frag4(ti + at(e + 1), x[~e & 1]);
                        tmem_ld_frag4(tx + at(e + 1), y[~e & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_o_free);
                    }
                    uint32_t z[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 f = *reinterpret_cast<const float2*>(&rf[last][32 * (e & 1) + 4 * i + 2 * (lane % 4)]);
#pragma unroll
                        for (int c = i; c < i + 2; ++c) {
                            const float2 o = fma2(f, make_float2(__uint_as_float(yi[2 * c]), __uint_as_float(yi[2 * c + 1])),
                                                  make_float2(__uint_as_float(xi[2 * c]), __uint_as_float(xi[2 * c + 1])));
                            z[c] = pack_bf16(o.x, o.y);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; t += 2)
                        stmatrix_t(piece(32 * (e & 1) + 8 * (t + lane / 16) + lane % 8, (e & 2) + lane / 8 % 2), z[2 * t], z[2 * t + 1], z[2 * t + 2],
                                   z[2 * t + 3]);
                }
                if (__any_sync(kAll, min(mark0, mark1) < kC)) {
                    __syncwarp();
                    const int first = rev ? (mark1 < kC ? mark1 : mark0 < kC ? mark0 : -1) : min(mark0, mark1);   // the walk's first
#pragma unroll 1
                    for (int t = rev ? 0 : first; t < (rev ? first + 1 : m); ++t)
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(piece(t, lane / 8) + lane % 8 * 2), "h"(static_cast<uint16_t>(0x7fc0)) : "memory");
                }
                const int t = row0 + place(n) * kC;
                if (j - lane >= DV) continue;   // (the warps behind the value channels)
                if (m == kC) {
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&T.o[job], out, j, h, t);
                        bulk_commit();
                    }
                } else {   // the rows behind are another sequence's
                    __syncwarp();
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(J.o) + (static_cast<long long>(t) * P.H + h) * DV + (j - lane);
                    for (int i = lane / 4; i < m; i += 8) {
                        uint4 x;
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                     : "r"(piece(i, lane % 4)));
                        *reinterpret_cast<uint4*>(o + static_cast<long long>(i) * P.H * DV + lane % 4 * 8) = x;
                    }
                    __syncwarp();
                    if (lane == 0) bulk_commit();   // (an empty group: the count of groups goes on)
                }
            }
            if (lane == 0) bulk_wait_all();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmCols);
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

// [rows, heads, d] bf16 as (channel of a half, row, half, head): tiles of 64 rows of one head, half after half.
bool encode(CUtensorMap* m, const Strided& x, int rows, int heads, int d) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(d / 64), static_cast<cuuint64_t>(heads)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(x.row) * 2, 128, static_cast<cuuint64_t>(x.head) * 2};
    const cuuint32_t box[4] = {64, kC, static_cast<cuuint32_t>(d / 64), 1}, step[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The same for outputs: tiles of 64 rows and 32 channels.
bool encode_out(CUtensorMap* m, void* p, int rows, int heads, int d) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(heads) * d * 2};
    const cuuint32_t box[3] = {32, 1, kC}, step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool OUT, int PARTS> cudaError_t start(const TcParams& T, int n_jobs, cudaStream_t s) {
    constexpr int bytes = Layout<DK, DV, OUT>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(decay_tc_kernel<DK, DV, OUT, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    decay_tc_kernel<DK, DV, OUT, PARTS><<<T.d.items * T.d.H * n_jobs, kThreads, bytes, s>>>(T);
    return cudaGetLastError();
}

template <int DK, int DV> cudaError_t start_pass(const TcParams& T, int n_jobs, cudaStream_t s) {
    if (T.d.pass == kStates) return start<DK, DV, false, 3>(T, n_jobs, s);
    // (of packed sequences some may be whole, and have a final state to give)
    if (T.d.pass == kOutputs && !T.d.cu) return start<DK, DV, true, 2>(T, n_jobs, s);
    return start<DK, DV, true, 3>(T, n_jobs, s);
}

}  // namespace

bool decay_tc_supported(int io, int dk, int dv) { return io == KDN_BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

cudaError_t launch_decay_tc(const DecayParams& P, int n_jobs, cudaStream_t s) {
    TcParams T;
    T.d = P;
    T.d.n_jobs = n_jobs;
    const int dk = P.job[0].dk, dv = P.job[0].dv;
    for (int i = 0; i < n_jobs; ++i) {
        const DecayJob& j = P.job[i];
        if (!encode(&T.q[i], j.q, P.n_tok, P.H, dk) || !encode(&T.k[i], j.k, P.n_tok, P.H, dk) ||
            !encode(&T.v[i], j.v, P.n_tok, P.H, dv) || !encode_out(&T.o[i], j.o, P.n_tok, P.H, dv))
            return cudaErrorInvalidValue;
    }
    if (dk == 128) return dv == 128 ? start_pass<128, 128>(T, n_jobs, s) : start_pass<128, 64>(T, n_jobs, s);
    return dv == 128 ? start_pass<64, 128>(T, n_jobs, s) : start_pass<64, 64>(T, n_jobs, s);
}

}  // namespace kdn
