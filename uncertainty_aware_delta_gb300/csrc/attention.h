// Internal launchers of the attention operators (host side; not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kdn {

// Bytes of one 16-token block of one key head of the 4-bit cache (layout: include/kdn.h).
__host__ __device__ constexpr int cache_block_bytes(int d) { return 18 * d; }
constexpr int kBlockTokens = 16;

// A [rows, heads, d] operand with the last axis dense; strides in elements.
struct Strided {
    const void* p;
    long long row, head;
};

struct PlanArgs {
    int n_req, page, table_width, n_free, capacity;
    const int32_t *context_len, *new_len;
    int32_t* block_table;
    const int32_t *free_pages, *free_count;
    int64_t* slot_map;
    int32_t *position, *cu_new, *seq_len, *granted, *free_left;
    uint32_t* status;
};
constexpr int kPlanMaxRequests = 16384;   // two prefix arrays in shared memory
cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t s);

struct CacheArgs {
    int n_tok, n_pages, page, H_kv, d, io;   // io: 0 fp32, 1 bf16
    Strided k, v;                            // write: inputs
    void *k_out, *v_out;                     // read: outputs, dense
    const int64_t* slots;
    uint8_t* cache;
};
cudaError_t launch_cache_write(const CacheArgs& a, cudaStream_t s);
cudaError_t launch_cache_read(const CacheArgs& a, cudaStream_t s);

struct CacheAttentionArgs {
    int n_seq, H, H_kv, d, page, n_pages, table_width, max_len, window, io;
    float scale;
    Strided q;
    const uint8_t* cache;
    const int32_t *block_table, *seq_len;
    void* o;
    float* lse;
    uint32_t* status;
    void* scratch;
};
size_t cache_attention_scratch(int n_seq, int H, int H_kv, int d, int max_len, int window);
cudaError_t launch_cache_attention(const CacheAttentionArgs& a, cudaStream_t s);

struct PromptArgs {
    int n_seq, total_q, total_k, H, H_kv, d, window, io;
    float scale;
    uint32_t flags;
    Strided q, k, v;
    const int32_t *cu_q, *cu_k;
    void* o;
    float* lse;
    uint32_t* status;
    void* scratch;
};
size_t prompt_scratch(int n_seq, int total_q, int H, int H_kv, int d, int io, uint32_t flags);
cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s);
bool prompt_tc_supported(int io, int d);   // prompt_tc.cu
size_t prompt_tc_scratch(int n_seq, int total_q, int H, int H_kv, int d);
cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t s);

}  // namespace kdn
