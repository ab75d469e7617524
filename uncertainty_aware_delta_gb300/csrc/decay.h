// Internal launchers of a retention layer's operators (host side; not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "attention.h"

namespace kdn {

// One walk of a memory with a fixed decay g a head along the tokens of every sequence:
//   S_t = g S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t.
// The gradients are walks, too, with other tensors in the places of q, k and v: that of q a forward one, those of k and v from
// the end (then the state that a walk begins with is taken as that of its last token: not decayed before it).
struct DecayJob {
    Strided q, k, v;         // [tokens, H, dk or dv]
    void* o;                 // [tokens, H, dv] dense, or null: states alone
    const float* S0;         // [n_seq, H] states, or null (zero): element (i, j) at i s_k + j s_v
    float* S_T;              // the same, or null
    int dk, dv, s_k, s_v, reverse;
};
constexpr int kMaxDecayJobs = 3;

// Segments of sequences that run side by side: one pass gives the states that they end with from zero, a short one chains
// them, and a last one gives the outputs.  Dense sequences all have the same segments.  Of packed ones those longer than
// seg_len are cut (the lengths are known on the device alone), the others run whole in the last pass.
struct DecayPlan {
    bool split;
    int seg_len, nseg;       // nseg: of a dense sequence
    int items, slots;        // blocks a head in the last pass, at most; segments that have a state
};

struct DecayArgs {
    int n_seq, n_tok, H, io;                 // io: 0 fp32, 1 bf16
    uint32_t flags;
    const float* log_decay;                  // [H]
    const int32_t* cu;                       // [n_seq + 1], or null: n_tok / n_seq tokens each
    uint32_t* status;
    float* scratch;                          // decay_scratch() bytes
    int n_jobs;
    DecayJob job[kMaxDecayJobs];
};
size_t decay_scratch(int n_seq, int n_tok, int H, int dk, int dv, int io, uint32_t flags, bool packed, int n_jobs);
cudaError_t launch_decay(const DecayArgs& a, cudaStream_t s);

// What a pass's kernel takes.
struct DecayParams {
    DecayJob job[kMaxDecayJobs];
    float* states[kMaxDecayJobs];            // [slots, H, dk, dv] of the job
    const float* log_decay;
    const int32_t* cu;
    uint32_t* status;
    int n_seq, n_tok, H, io, n_jobs, nseg, seg_len, items, slots, pass, probe, clear;   // pass: kWhole, kStates or kOutputs
};
enum { kWhole = 0, kStates = 1, kOutputs = 2 };

// tcgen05 path: bf16, dk and dv 64 or 128.  decay_tc.cu
bool decay_tc_supported(int io, int dk, int dv);
cudaError_t launch_decay_tc(const DecayParams& P, int n_jobs, cudaStream_t s);

struct DecayStepArgs {
    int B, H, dk, dv, io;
    const void *q, *k, *v;
    const float* log_decay;
    float* S;
    void* o;
};
cudaError_t launch_decay_step(const DecayStepArgs& a, cudaStream_t s);

// Norm of every token's groups of d channels, with an activation.  group_norm.cu
struct NormArgs {
    int rows, groups, d, io, act;            // act: KDN_ACT_*
    float eps;
    Strided x, gate, dy;                     // gate.p null: the activation is of the norm itself
    const float *w, *b;                      // [groups, d], or null
    void *y, *dx, *dgate;                    // dense
    float *dw, *db;                          // [groups, d]
    uint32_t* status;                        // backward: there is nothing to report, 0
    float* scratch;                          // backward: norm_scratch() bytes
};
size_t norm_scratch(int rows, int groups, int d);
cudaError_t launch_group_norm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_group_norm_backward(const NormArgs& a, cudaStream_t s);

}  // namespace kdn
