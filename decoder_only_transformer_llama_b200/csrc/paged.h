// Host-side descriptions shared by the paged-cache operators and their entry
// points (api_paged.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/llama_b200.h"

namespace llb {

constexpr int kPagedMaxRequests = 1024;   // requests one call may hold (one thread of the plan kernel each)

// Bytes at the start of a paged-attention workspace that hold arrival counters,
// zero between launches; both kernels keep to them, so one workspace serves both.
constexpr size_t kPagedCounters = 12288;

struct PlanArgs {
    const int32_t* ctx_lens;
    const int32_t* new_lens;
    int B, page_size, max_pages, n_pages, T;
    int32_t* block_tables;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t* seq_lens;
    int32_t* cu_new;
    int64_t* slots;
    int32_t* positions;
    int32_t* free_left;
    int32_t* status;
};

struct AppendArgs {
    const void* q;
    const void* k;
    const void* v;
    long long q_stride, k_stride, v_stride;   // elements between token rows
    int T, nh, nkv, hd;
    const float* q_norm;                      // [hd] or null
    const float* k_norm;
    float eps;
    const float2* rope;                       // [rope_len][hd / 2] (cos, sin)
    int rope_len;
    const int32_t* positions;
    const int64_t* slots;
    void* q_out;
    void* k_pages;
    void* v_pages;
    long long n_slots;                        // n_pages * page_size
    int page_shift;
    int32_t* status;
};

struct PagedAttnArgs {
    const void* q;
    const void* k_pages;
    const void* v_pages;
    int T, nh, nkv, hd, B;
    const int32_t* cu_new;
    const int32_t* seq_lens;
    const int32_t* block_tables;
    int max_pages, n_pages, page_shift, max_new;
    float scale;
    void* out;
    void* workspace;
    int32_t* status;
};

int launch_paged_plan(const PlanArgs& a, cudaStream_t st);
int launch_paged_append(const AppendArgs& a, int in_dtype, int dtype, cudaStream_t st);
size_t paged_attention_ws(int nh, int nkv, int hd, int dtype, int max_new);
// Chunks on tcgen05 (16-bit caches, head_dim 64 or 128, scale > 0).
size_t paged_attention_tile_ws(int hd);
int launch_paged_attention_tile(const PagedAttnArgs& a, int dtype, cudaStream_t st);
// The next launch of that kernel, by any thread, stalls stage `stage` of CTA 0 (llama_debug_stall); -1: none.
void arm_paged_stall(int stage, long long wait_ns);
int launch_paged_attention(const PagedAttnArgs& a, int dtype, cudaStream_t st);
int launch_sample_rows(const float* logits, int B, int V, const float* temperature, const int32_t* top_k,
                       const float* top_p, const float* min_p, const float* uniforms, int32_t* out, cudaStream_t st);

}  // namespace llb
