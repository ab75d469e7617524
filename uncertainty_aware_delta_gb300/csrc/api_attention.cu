// C ABI of the attention operators and the 4-bit cache: argument validation and
// dispatch.  See include/kdn.h for the contract of every entry point.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "abi_checks.h"
#include "attention.h"
#include "kdn.h"

namespace {

constexpr int kMostTokens = 0x7ffffc00;   // of a cached sequence

bool cache_dim(int d) { return d == 32 || d == 64 || d == 128; }
bool prompt_dim(int d) { return d == 16 || cache_dim(d); }
bool cache_page(int page) { return page >= kdn::kBlockTokens && page <= 1024 && page % kdn::kBlockTokens == 0; }

size_t cache_size(int n_pages, int page, int H_kv, int d) {
    return (size_t)n_pages * H_kv * (page / kdn::kBlockTokens) * kdn::cache_block_bytes(d);
}

bool good_scale(float scale) { return isfinite(scale) && scale >= 0.0f; }

}  // namespace

extern "C" {

kdn_status kdn_cache_plan(int n_req, int page, int table_width, int n_free, int capacity, const int32_t* context_len,
                          const int32_t* new_len, int32_t* block_table, const int32_t* free_pages,
                          const int32_t* free_count, int64_t* slot_map, int32_t* position, int32_t* cu_new,
                          int32_t* seq_len, int32_t* granted, int32_t* free_left, void* workspace,
                          size_t workspace_bytes, kdn_stream_t stream) {
    if (n_req < 0 || table_width < 0 || n_free < 0 || capacity < 0) return KDN_ERR_SHAPE;
    if (!cache_page(page) || n_req > kdn::kPlanMaxRequests) return KDN_ERR_UNSUPPORTED;
    if (n_free > kMostRows || capacity > kMostRows) return KDN_ERR_SHAPE;
    if ((long long)table_width * page > 0x7fffffffll) return KDN_ERR_SHAPE;
    if (!workspace || workspace_bytes < kStatusBytes) return KDN_ERR_WORKSPACE;
    if (!free_count || !free_left || !cu_new) return KDN_ERR_NULL;
    if (n_req > 0 && (!context_len || !new_len || !seq_len || !granted)) return KDN_ERR_NULL;
    if (n_req > 0 && table_width > 0 && !block_table) return KDN_ERR_NULL;
    if (n_free > 0 && !free_pages) return KDN_ERR_NULL;
    if (capacity > 0 && (!slot_map || !position)) return KDN_ERR_NULL;
    const void* const ptrs[] = {context_len, new_len, block_table, free_pages, free_count, slot_map,
                                position, cu_new, seq_len, granted, free_left, workspace};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t n = (size_t)n_req;
    const Range out[] = {{block_table, 4 * n * table_width}, {slot_map, 8 * (size_t)capacity},
                         {position, 4 * (size_t)capacity}, {cu_new, 4 * (n + 1)}, {seq_len, 4 * n},
                         {granted, 4 * n}, {free_left, 4}, {workspace, kStatusBytes}};
    const Range in[] = {{context_len, 4 * n}, {new_len, 4 * n}, {free_pages, 4 * (size_t)n_free}, {free_count, 4}};
    const kdn_status st = check_alias(out, in);
    if (st != KDN_OK) return st;
    kdn::PlanArgs a;
    a.n_req = n_req; a.page = page; a.table_width = table_width; a.n_free = n_free; a.capacity = capacity;
    a.context_len = context_len; a.new_len = new_len; a.block_table = block_table; a.free_pages = free_pages;
    a.free_count = free_count; a.slot_map = slot_map; a.position = position; a.cu_new = cu_new; a.seq_len = seq_len;
    a.granted = granted; a.free_left = free_left; a.status = static_cast<uint32_t*>(workspace);
    return done(kdn::launch_cache_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kdn_cache_size(int n_pages, int page, int H_kv, int d) {
    if (n_pages < 0 || H_kv < 0 || !cache_page(page) || !cache_dim(d)) return 0;
    return cache_size(n_pages, page, H_kv, d);
}

static kdn_status cache_rows(bool write, kdn::CacheArgs& a, cudaStream_t s) {
    if (a.io != KDN_F32 && a.io != KDN_BF16) return KDN_ERR_DTYPE;
    if (a.n_tok < 0 || a.n_pages < 0 || a.H_kv < 0) return KDN_ERR_SHAPE;
    if (!cache_dim(a.d) || !cache_page(a.page)) return KDN_ERR_UNSUPPORTED;
    if (a.n_tok == 0 || a.H_kv == 0) return KDN_OK;
    const void* kp = write ? a.k.p : a.k_out;
    const void* vp = write ? a.v.p : a.v_out;
    if (!kp || !vp || !a.slots || (!a.cache && a.n_pages > 0)) return KDN_ERR_NULL;
    const void* const ptrs[] = {kp, vp, a.slots, a.cache};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t esz = a.io == KDN_BF16 ? 2 : 4;
    if (write) {
        kdn_status st = check_strided(&a.k, a.n_tok, a.H_kv, a.d, esz);
        if (st == KDN_OK) st = check_strided(&a.v, a.n_tok, a.H_kv, a.d, esz);
        if (st != KDN_OK) return st;
    }
    const Range cache = {a.cache, cache_size(a.n_pages, a.page, a.H_kv, a.d)}, slots = {a.slots, 8 * (size_t)a.n_tok};
    kdn_status st;
    if (write) {
        const Range out[] = {cache};
        const Range in[] = {range_of(a.k, a.n_tok, a.H_kv, a.d, esz), range_of(a.v, a.n_tok, a.H_kv, a.d, esz), slots};
        st = check_alias(out, in);
    } else {
        const size_t bytes = (size_t)a.n_tok * a.H_kv * a.d * esz;
        const Range out[] = {{a.k_out, bytes}, {a.v_out, bytes}};
        const Range in[] = {cache, slots};
        st = check_alias(out, in);
    }
    if (st != KDN_OK) return st;
    return done(write ? kdn::launch_cache_write(a, s) : kdn::launch_cache_read(a, s));
}

kdn_status kdn_cache_write(int n_tok, int n_pages, int page, int H_kv, int d, int io_dtype, const void* k,
                           int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                           const int64_t* slot_map, void* cache, kdn_stream_t stream) {
    kdn::CacheArgs a = {};
    a.n_tok = n_tok; a.n_pages = n_pages; a.page = page; a.H_kv = H_kv; a.d = d; a.io = io_dtype;
    a.k = {k, k_row, k_head}; a.v = {v, v_row, v_head};
    a.slots = slot_map; a.cache = static_cast<uint8_t*>(cache);
    return cache_rows(true, a, reinterpret_cast<cudaStream_t>(stream));
}

kdn_status kdn_cache_read(int n_tok, int n_pages, int page, int H_kv, int d, int io_dtype, const void* cache,
                          const int64_t* slot_map, void* k, void* v, kdn_stream_t stream) {
    kdn::CacheArgs a = {};
    a.n_tok = n_tok; a.n_pages = n_pages; a.page = page; a.H_kv = H_kv; a.d = d; a.io = io_dtype;
    a.k_out = k; a.v_out = v; a.slots = slot_map;
    a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
    return cache_rows(false, a, reinterpret_cast<cudaStream_t>(stream));
}

static kdn_status check_cache_attention(int n_seq, int H, int H_kv, int d, int page, int n_pages, int table_width,
                                        int max_len, int window) {
    if (n_seq < 0 || H < 0 || H_kv < 0 || n_pages < 0 || table_width < 0 || max_len < 0 || window < 0)
        return KDN_ERR_SHAPE;
    if (H > 0 && (H_kv == 0 || H % H_kv)) return KDN_ERR_SHAPE;
    if (!cache_dim(d) || !cache_page(page)) return KDN_ERR_UNSUPPORTED;
    if ((double)n_seq * H * d > 1.0e12 || n_seq > 65535 || H > 65535) return KDN_ERR_SHAPE;
    return KDN_OK;
}

size_t kdn_cache_attention_workspace_size(int n_seq, int H, int H_kv, int d, int max_len, int window) {
    if (check_cache_attention(n_seq, H, H_kv, d, kdn::kBlockTokens, 0, 0, max_len, window) != KDN_OK) return 0;
    return kStatusBytes + align_up(kdn::cache_attention_scratch(n_seq, H, H_kv, d, max_len, window));
}

kdn_status kdn_cache_attention(int n_seq, int H, int H_kv, int d, int page, int n_pages, int table_width, int max_len,
                               int window, float scale, int io_dtype, const void* q, int64_t q_row, int64_t q_head,
                               const void* cache, const int32_t* block_table, const int32_t* seq_len, void* o,
                               float* lse, void* workspace, size_t workspace_bytes, kdn_stream_t stream) {
    if (io_dtype != KDN_F32 && io_dtype != KDN_BF16) return KDN_ERR_DTYPE;
    kdn_status st = check_cache_attention(n_seq, H, H_kv, d, page, n_pages, table_width, max_len, window);
    if (st != KDN_OK) return st;
    if (!good_scale(scale)) return KDN_ERR_SHAPE;
    const size_t need = kdn_cache_attention_workspace_size(n_seq, H, H_kv, d, max_len, window);
    if (!workspace || workspace_bytes < need) return KDN_ERR_WORKSPACE;
    const bool any = n_seq > 0 && H > 0;
    if (any && (!q || !seq_len || !o || !lse)) return KDN_ERR_NULL;
    if (any && ((table_width > 0 && !block_table) || (n_pages > 0 && !cache))) return KDN_ERR_NULL;
    const void* const ptrs[] = {q, cache, block_table, seq_len, o, lse, workspace};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t esz = io_dtype == KDN_BF16 ? 2 : 4, rows = (size_t)n_seq * H;
    kdn::CacheAttentionArgs a = {};
    a.q = {q, q_row, q_head};
    if (any && (st = check_strided(&a.q, n_seq, H, d, esz)) != KDN_OK) return st;
    const Range out[] = {{o, rows * d * esz}, {lse, rows * 4}, {workspace, need}};
    const Range in[] = {range_of(a.q, n_seq, H, d, esz), {cache, cache_size(n_pages, page, H_kv, d)},
                        {block_table, 4 * (size_t)n_seq * table_width}, {seq_len, 4 * (size_t)n_seq}};
    if ((st = check_alias(out, in)) != KDN_OK) return st;
    a.n_seq = n_seq; a.H = H; a.H_kv = H_kv; a.d = d; a.page = page; a.n_pages = n_pages;
    a.table_width = table_width;
    // the kernel's places run up to a thousand past the last token
    a.max_len = max_len < kMostTokens ? max_len : kMostTokens;
    a.window = window; a.io = io_dtype;
    a.scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)d);
    a.cache = static_cast<const uint8_t*>(cache); a.block_table = block_table; a.seq_len = seq_len;
    a.o = o; a.lse = lse;
    a.status = static_cast<uint32_t*>(workspace);
    a.scratch = static_cast<char*>(workspace) + kStatusBytes;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(a.status, 0, sizeof(uint32_t), s) != cudaSuccess) return KDN_ERR_CUDA;
    if (!any) return KDN_OK;
    return done(kdn::launch_cache_attention(a, s));
}

static kdn_status check_prompt(int n_seq, int total_q, int total_k, int H, int H_kv, int d, int window, int io) {
    if (io != KDN_F32 && io != KDN_BF16) return KDN_ERR_DTYPE;
    if (n_seq < 0 || total_q < 0 || total_k < 0 || H < 0 || H_kv < 0 || window < 0) return KDN_ERR_SHAPE;
    if (H > 0 && (H_kv == 0 || H % H_kv)) return KDN_ERR_SHAPE;
    if (!prompt_dim(d)) return KDN_ERR_UNSUPPORTED;
    if (n_seq > kMostRows || total_q > kMostRows || total_k > kMostRows) return KDN_ERR_SHAPE;
    if (H > 65535 || (double)total_q * H * d > 1.0e12 || (double)total_k * H_kv * d > 1.0e12) return KDN_ERR_SHAPE;
    return KDN_OK;
}

size_t kdn_prompt_attention_workspace_size(int n_seq, int total_q, int H, int H_kv, int d, int io_dtype,
                                           uint32_t flags) {
    if (check_prompt(n_seq, total_q, 0, H, H_kv, d, 0, io_dtype) != KDN_OK) return 0;
    return kStatusBytes + align_up(kdn::prompt_scratch(n_seq, total_q, H, H_kv, d, io_dtype, flags));
}

kdn_status kdn_prompt_attention(int n_seq, int total_q, int total_k, int H, int H_kv, int d, int window, float scale,
                                int io_dtype, uint32_t flags, const void* q, int64_t q_row, int64_t q_head,
                                const void* k, int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                int64_t v_head, const int32_t* cu_q, const int32_t* cu_k, void* o, float* lse,
                                void* workspace, size_t workspace_bytes, kdn_stream_t stream) {
    kdn_status st = check_prompt(n_seq, total_q, total_k, H, H_kv, d, window, io_dtype);
    if (st != KDN_OK) return st;
    if (!good_scale(scale)) return KDN_ERR_SHAPE;
    if (flags & ~(KDN_FLAG_PORTABLE | KDN_FLAG_TIMEOUT_PROBE)) return KDN_ERR_UNSUPPORTED;
    const size_t need = kdn_prompt_attention_workspace_size(n_seq, total_q, H, H_kv, d, io_dtype, flags);
    if (!workspace || workspace_bytes < need) return KDN_ERR_WORKSPACE;
    const bool any = n_seq > 0 && total_q > 0 && H > 0;
    if (any && (!q || !cu_q || !o || !lse)) return KDN_ERR_NULL;
    if (any && total_k > 0 && (!k || !v)) return KDN_ERR_NULL;
    if (!cu_k) {   // self-attention over the same tokens
        if (total_k != total_q) return KDN_ERR_SHAPE;
        cu_k = cu_q;
    }
    const void* const ptrs[] = {q, k, v, cu_q, cu_k, o, lse, workspace};
    if (!all_aligned(ptrs)) return KDN_ERR_ALIGN;
    const size_t esz = io_dtype == KDN_BF16 ? 2 : 4, rows = (size_t)total_q * H;
    kdn::PromptArgs a = {};
    a.q = {q, q_row, q_head}; a.k = {k, k_row, k_head}; a.v = {v, v_row, v_head};
    if (any) {
        if ((st = check_strided(&a.q, total_q, H, d, esz)) != KDN_OK) return st;
        if ((st = check_strided(&a.k, total_k, H_kv, d, esz)) != KDN_OK) return st;
        if ((st = check_strided(&a.v, total_k, H_kv, d, esz)) != KDN_OK) return st;
    }
    const Range out[] = {{o, rows * d * esz}, {lse, rows * 4}, {workspace, need}};
    const Range in[] = {range_of(a.q, total_q, H, d, esz), range_of(a.k, total_k, H_kv, d, esz),
                        range_of(a.v, total_k, H_kv, d, esz), {cu_q, 4 * ((size_t)n_seq + 1)},
                        {cu_k, 4 * ((size_t)n_seq + 1)}};
    if ((st = check_alias(out, in)) != KDN_OK) return st;
    a.n_seq = n_seq; a.total_q = total_q; a.total_k = total_k; a.H = H; a.H_kv = H_kv; a.d = d;
    // a window of all keys or more masks nothing: the kernels' sums with it stay in 32 bits
    a.window = window < total_k ? window : 0;
    a.io = io_dtype; a.flags = flags;
    a.scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)d);
    a.cu_q = cu_q; a.cu_k = cu_k; a.o = o; a.lse = lse;
    a.status = static_cast<uint32_t*>(workspace);
    a.scratch = static_cast<char*>(workspace) + kStatusBytes;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the status word and the kernel's item counter beside it
    if (cudaMemsetAsync(a.status, 0, 2 * sizeof(uint32_t), s) != cudaSuccess) return KDN_ERR_CUDA;
    if (!any) return KDN_OK;
    return done(kdn::launch_prompt_attention(a, s));
}

}  // extern "C"
