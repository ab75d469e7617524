// C ABI of a retention layer's operators: argument validation and dispatch.  See include/kdn.h for the contract of every
// entry point.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_checks.h"
#include "decay.h"
#include "kdn.h"

namespace {

bool good_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
size_t size_of(int io) { return io == KDN_BF16 ? 2 : 4; }

constexpr uint32_t kDecayFlags = KDN_FLAG_PORTABLE | KDN_FLAG_NO_SPLIT | KDN_FLAG_TIMEOUT_PROBE;

kdn_status check_sizes(int n_seq, int n_tok, int H, int dk, int dv, int io, uint32_t flags) {
    if (io != KDN_F32 && io != KDN_BF16) return KDN_ERR_DTYPE;
    if (n_seq < 0 || n_tok < 0 || H < 0) return KDN_ERR_SHAPE;
    if (!good_dim(dk) || !good_dim(dv) || (flags & ~kDecayFlags)) return KDN_ERR_UNSUPPORTED;
    // (tokens of 8-byte rows and the like stay far below 2^63 bytes, blocks below 2^31)
    if (n_tok > kMostRows || n_seq > kMostRows || H > 65535) return KDN_ERR_SHAPE;
    if ((double)n_tok * H * 128 > 1.0e12 || (double)n_seq * H > 1.0e8) return KDN_ERR_SHAPE;
    return KDN_OK;
}

// Bytes of scratch, whether the sequences' lengths are on the device or not.
size_t scratch_bytes(int n_seq, int n_tok, int H, int dk, int dv, int io, uint32_t flags, int n_jobs) {
    const size_t a = kdn::decay_scratch(n_seq, n_tok, H, dk, dv, io, flags, false, n_jobs),
                 b = kdn::decay_scratch(n_seq, n_tok, H, dk, dv, io, flags, true, n_jobs);
    return kStatusBytes + align_up(a > b ? a : b);
}

// Tokens of dense sequences are split evenly.
kdn_status check_lengths(int n_seq, int n_tok, const int32_t* cu) {
    if (cu) return KDN_OK;
    return n_seq == 0 ? (n_tok == 0 ? KDN_OK : KDN_ERR_SHAPE) : (n_tok % n_seq ? KDN_ERR_SHAPE : KDN_OK);
}

void fill(kdn::DecayArgs& a, int n_seq, int n_tok, int H, int io, uint32_t flags, const float* log_decay, const int32_t* cu, void* ws) {
    a.n_seq = n_seq; a.n_tok = n_tok; a.H = H; a.io = io; a.flags = flags;
    a.log_decay = log_decay; a.cu = cu;
    a.status = static_cast<uint32_t*>(ws);
    a.scratch = reinterpret_cast<float*>(static_cast<char*>(ws) + kStatusBytes);
}

}  // namespace

extern "C" {

size_t kdn_decay_workspace_size(int n_seq, int n_tok, int H, int dk, int dv, int io_dtype, uint32_t flags) {
    if (check_sizes(n_seq, n_tok, H, dk, dv, io_dtype, flags) != KDN_OK) return 0;
    return scratch_bytes(n_seq, n_tok, H, dk, dv, io_dtype, flags, 1);
}

kdn_status kdn_decay_forward(int n_seq, int n_tok, int H, int dk, int dv, int io_dtype, uint32_t flags,
                             const void* q, int64_t q_row, int64_t q_head, const void* k, int64_t k_row, int64_t k_head,
                             const void* v, int64_t v_row, int64_t v_head, const float* log_decay, const float* S0,
                             const int32_t* cu, void* o, float* S_T, void* workspace, size_t workspace_bytes,
                             kdn_stream_t stream) {
    kdn_status st = check_sizes(n_seq, n_tok, H, dk, dv, io_dtype, flags);
    if (st == KDN_OK) st = check_lengths(n_seq, n_tok, cu);
    if (st != KDN_OK) return st;
    const size_t need = kdn_decay_workspace_size(n_seq, n_tok, H, dk, dv, io_dtype, flags);
    if (!workspace || workspace_bytes < need) return KDN_ERR_WORKSPACE;
    const bool any = n_seq > 0 && H > 0, tokens = any && n_tok > 0;
    if (any && (!log_decay || !S_T)) return KDN_ERR_NULL;
    if (tokens && (!q || !k || !v || !o)) return KDN_ERR_NULL;
    const void* const ptrs[] = {q, k, v, log_decay, S0, cu, o, S_T, workspace};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t esz = size_of(io_dtype), states = (size_t)n_seq * H * dk * dv * 4;
    kdn::DecayArgs a = {};
    fill(a, n_seq, n_tok, H, io_dtype, flags, log_decay, cu, workspace);
    a.n_jobs = 1;
    a.job[0] = {{q, q_row, q_head}, {k, k_row, k_head}, {v, v_row, v_head}, o, S0, S_T, dk, dv, dv, 1, 0};
    kdn::DecayJob& j = a.job[0];
    if (tokens) {
        if ((st = check_strided(&j.q, n_tok, H, dk, esz)) != KDN_OK) return st;
        if ((st = check_strided(&j.k, n_tok, H, dk, esz)) != KDN_OK) return st;
        if ((st = check_strided(&j.v, n_tok, H, dv, esz)) != KDN_OK) return st;
    }
    const Range out[] = {{o, (size_t)n_tok * H * dv * esz}, {S_T, states}, {workspace, need}};
    const Range in[] = {range_of(j.q, n_tok, H, dk, esz), range_of(j.k, n_tok, H, dk, esz), range_of(j.v, n_tok, H, dv, esz),
                        {log_decay, 4 * (size_t)H}, {cu, cu ? 4 * ((size_t)n_seq + 1) : 0},
                        {S0 == S_T ? nullptr : S0, states}};   // (states resumed in place are allowed)
    if ((st = check_alias(out, in)) != KDN_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!any) return done(cudaMemsetAsync(a.status, 0, sizeof(uint32_t), s));
    return done(kdn::launch_decay(a, s));
}

kdn_status kdn_decay_step(int B, int H, int dk, int dv, int io_dtype, const void* q, const void* k, const void* v,
                          const float* log_decay, float* S, void* o, kdn_stream_t stream) {
    const kdn_status st = check_sizes(B, B, H, dk, dv, io_dtype, 0);
    if (st != KDN_OK) return st;
    if (B == 0 || H == 0) return KDN_OK;
    if (!q || !k || !v || !log_decay || !S || !o) return KDN_ERR_NULL;
    const void* const ptrs[] = {q, k, v, log_decay, S, o};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t n = (size_t)B * H, esz = size_of(io_dtype);
    const Range out[] = {{S, n * dk * dv * 4}, {o, n * dv * esz}};
    const Range in[] = {{q, n * dk * esz}, {k, n * dk * esz}, {v, n * dv * esz}, {log_decay, 4 * (size_t)H}};
    const kdn_status al = check_alias(out, in);
    if (al != KDN_OK) return al;
    kdn::DecayStepArgs a = {B, H, dk, dv, io_dtype, q, k, v, log_decay, S, o};
    return done(kdn::launch_decay_step(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kdn_decay_backward_workspace_size(int n_seq, int n_tok, int H, int dk, int dv, int io_dtype, uint32_t flags) {
    if (check_sizes(n_seq, n_tok, H, dk, dv, io_dtype, flags) != KDN_OK) return 0;
    return scratch_bytes(n_seq, n_tok, H, dk, dv, io_dtype, flags, 3);
}

kdn_status kdn_decay_backward(int n_seq, int n_tok, int H, int dk, int dv, int io_dtype, uint32_t flags,
                              const void* q, int64_t q_row, int64_t q_head, const void* k, int64_t k_row, int64_t k_head,
                              const void* v, int64_t v_row, int64_t v_head, const float* log_decay, const float* S0,
                              const int32_t* cu, const void* dO, int64_t dO_row, int64_t dO_head, const float* dS_T,
                              void* grad_q, void* grad_k, void* grad_v, float* grad_S0, void* workspace,
                              size_t workspace_bytes, kdn_stream_t stream) {
    kdn_status st = check_sizes(n_seq, n_tok, H, dk, dv, io_dtype, flags);
    if (st == KDN_OK) st = check_lengths(n_seq, n_tok, cu);
    if (st != KDN_OK) return st;
    const size_t need = kdn_decay_backward_workspace_size(n_seq, n_tok, H, dk, dv, io_dtype, flags);
    if (!workspace || workspace_bytes < need) return KDN_ERR_WORKSPACE;
    const bool any = n_seq > 0 && H > 0, tokens = any && n_tok > 0;
    if (any && (!log_decay || !grad_S0)) return KDN_ERR_NULL;
    if (tokens && (!q || !k || !v || !dO || !grad_q || !grad_k || !grad_v)) return KDN_ERR_NULL;
    const void* const ptrs[] = {q, k, v, log_decay, S0, cu, dO, dS_T, grad_q, grad_k, grad_v, grad_S0, workspace};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t esz = size_of(io_dtype), states = (size_t)n_seq * H * dk * dv * 4;
    kdn::Strided sq = {q, q_row, q_head}, sk = {k, k_row, k_head}, sv = {v, v_row, v_head}, so = {dO, dO_row, dO_head};
    if (tokens) {
        if ((st = check_strided(&sq, n_tok, H, dk, esz)) != KDN_OK) return st;
        if ((st = check_strided(&sk, n_tok, H, dk, esz)) != KDN_OK) return st;
        if ((st = check_strided(&sv, n_tok, H, dv, esz)) != KDN_OK) return st;
        if ((st = check_strided(&so, n_tok, H, dv, esz)) != KDN_OK) return st;
    }
    const size_t rows = (size_t)n_tok * H * esz;
    const Range out[] = {{grad_q, rows * dk}, {grad_k, rows * dk}, {grad_v, rows * dv}, {grad_S0, states}, {workspace, need}};
    const Range in[] = {range_of(sq, n_tok, H, dk, esz), range_of(sk, n_tok, H, dk, esz), range_of(sv, n_tok, H, dv, esz),
                        range_of(so, n_tok, H, dv, esz), {log_decay, 4 * (size_t)H}, {cu, cu ? 4 * ((size_t)n_seq + 1) : 0},
                        {S0, states}, {dS_T, states}};
    if ((st = check_alias(out, in)) != KDN_OK) return st;
    kdn::DecayArgs a = {};
    fill(a, n_seq, n_tok, H, io_dtype, flags, log_decay, cu, workspace);
    // dq_t = S_t dO_t; from the end R_t = g R_{t+1} + q_t dO_t^T (and dS_T): dk_t = R_t v_t, dv_t = R_t^T k_t, dS0 = g R_0.
    // The walks of dq and dk have the states transposed.
    a.n_jobs = 3;
    a.job[0] = {so, sv, sk, grad_q, S0, nullptr, dv, dk, 1, dv, 0};
    a.job[1] = {sv, so, sq, grad_k, dS_T, nullptr, dv, dk, 1, dv, 1};
    a.job[2] = {sk, sq, so, grad_v, dS_T, grad_S0, dk, dv, dv, 1, 1};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!any) return done(cudaMemsetAsync(a.status, 0, sizeof(uint32_t), s));
    return done(kdn::launch_decay(a, s));
}

static kdn_status check_norm(int rows, int groups, int d, int io, int act, float eps) {
    if (io != KDN_F32 && io != KDN_BF16) return KDN_ERR_DTYPE;
    if (rows < 0 || groups < 0 || d < 0) return KDN_ERR_SHAPE;
    if (d < 8 || d > 256 || d % 8 || act < KDN_ACT_NONE || act > KDN_ACT_SIGMOID) return KDN_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f) || !isfinite(eps)) return KDN_ERR_SHAPE;
    if (rows > kMostRows || groups > 65535 || (double)rows * groups * d > 1.0e12) return KDN_ERR_SHAPE;
    return KDN_OK;
}

kdn_status kdn_group_norm(int rows, int groups, int d, int act, float eps, int io_dtype, const void* x, int64_t x_row,
                          int64_t x_head, const float* weight, const float* bias, const void* gate, int64_t gate_row,
                          int64_t gate_head, void* y, kdn_stream_t stream) {
    kdn_status st = check_norm(rows, groups, d, io_dtype, act, eps);
    if (st != KDN_OK) return st;
    if (rows == 0 || groups == 0) return KDN_OK;
    if (!x || !y) return KDN_ERR_NULL;
    const void* const ptrs[] = {x, weight, bias, gate, y};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t esz = size_of(io_dtype), params = 4 * (size_t)groups * d;
    kdn::NormArgs a = {};
    a.rows = rows; a.groups = groups; a.d = d; a.io = io_dtype; a.act = act; a.eps = eps;
    a.x = {x, x_row, x_head}; a.gate = {gate, gate_row, gate_head};
    a.w = weight; a.b = bias; a.y = y;
    if ((st = check_strided(&a.x, rows, groups, d, esz)) != KDN_OK) return st;
    if (gate && (st = check_strided(&a.gate, rows, groups, d, esz)) != KDN_OK) return st;
    const Range out[] = {{y, (size_t)rows * groups * d * esz}};
    const Range in[] = {range_of(a.x, rows, groups, d, esz), gate ? range_of(a.gate, rows, groups, d, esz) : Range{nullptr, 0},
                        {weight, params}, {bias, params}};
    if ((st = check_alias(out, in)) != KDN_OK) return st;
    return done(kdn::launch_group_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kdn_group_norm_backward_workspace_size(int rows, int groups, int d, int io_dtype) {
    if (check_norm(rows, groups, d, io_dtype, KDN_ACT_NONE, 0.0f) != KDN_OK) return 0;
    return kStatusBytes + align_up(kdn::norm_scratch(rows, groups, d));
}

kdn_status kdn_group_norm_backward(int rows, int groups, int d, int act, float eps, int io_dtype, const void* x, int64_t x_row,
                                   int64_t x_head, const float* weight, const float* bias, const void* gate, int64_t gate_row,
                                   int64_t gate_head, const void* dy, int64_t dy_row, int64_t dy_head, void* grad_x,
                                   void* grad_gate, float* grad_weight, float* grad_bias, void* workspace,
                                   size_t workspace_bytes, kdn_stream_t stream) {
    kdn_status st = check_norm(rows, groups, d, io_dtype, act, eps);
    if (st != KDN_OK) return st;
    const size_t need = kdn_group_norm_backward_workspace_size(rows, groups, d, io_dtype);
    if (!workspace || workspace_bytes < need) return KDN_ERR_WORKSPACE;
    if (groups > 0 && ((weight && !grad_weight) || (bias && !grad_bias))) return KDN_ERR_NULL;
    const bool any = rows > 0 && groups > 0;
    if (any && (!x || !dy || !grad_x || (gate && !grad_gate))) return KDN_ERR_NULL;
    const void* const ptrs[] = {x, weight, bias, gate, dy, grad_x, grad_gate, grad_weight, grad_bias, workspace};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t esz = size_of(io_dtype), params = 4 * (size_t)groups * d, whole = (size_t)rows * groups * d * esz;
    kdn::NormArgs a = {};
    a.rows = rows; a.groups = groups; a.d = d; a.io = io_dtype; a.act = act; a.eps = eps;
    a.x = {x, x_row, x_head}; a.gate = {gate, gate_row, gate_head}; a.dy = {dy, dy_row, dy_head};
    a.w = weight; a.b = bias;
    a.dx = grad_x; a.dgate = gate ? grad_gate : nullptr;
    a.dw = weight ? grad_weight : nullptr; a.db = bias ? grad_bias : nullptr;
    a.status = static_cast<uint32_t*>(workspace);
    a.scratch = reinterpret_cast<float*>(static_cast<char*>(workspace) + kStatusBytes);
    if (any) {
        if ((st = check_strided(&a.x, rows, groups, d, esz)) != KDN_OK) return st;
        if ((st = check_strided(&a.dy, rows, groups, d, esz)) != KDN_OK) return st;
        if (gate && (st = check_strided(&a.gate, rows, groups, d, esz)) != KDN_OK) return st;
    }
    const Range out[] = {{grad_x, whole}, {a.dgate, whole}, {a.dw, params}, {a.db, params}, {workspace, need}};
    const Range in[] = {range_of(a.x, rows, groups, d, esz), range_of(a.dy, rows, groups, d, esz),
                        gate ? range_of(a.gate, rows, groups, d, esz) : Range{nullptr, 0}, {weight, params}, {bias, params}};
    if ((st = check_alias(out, in)) != KDN_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!any) {   // sums of nothing
        if (cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) != cudaSuccess) return KDN_ERR_CUDA;
        if (params && a.dw && cudaMemsetAsync(a.dw, 0, params, s) != cudaSuccess) return KDN_ERR_CUDA;
        if (params && a.db && cudaMemsetAsync(a.db, 0, params, s) != cudaSuccess) return KDN_ERR_CUDA;
        return KDN_OK;
    }
    return done(kdn::launch_group_norm_backward(a, s));
}

}  // extern "C"
