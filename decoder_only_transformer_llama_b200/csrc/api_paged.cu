// C entry points of the paged-cache operators and the per-row sampler:
// argument checks on the host, then one launch.
#include "common.cuh"
#include "paged.h"
#include "../../include/llama_b200_ops.h"

namespace llb {

int launch_rope_table(float2* rope, int S, int hd, float theta, cudaStream_t st);

namespace {
bool is_dtype(int d) { return d == LLAMA_F32 || d == LLAMA_BF16 || d == LLAMA_F16; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

constexpr int kMaxSampleRows = 1 << 28;       // the grid holds up to 4 CTAs a row

// log2(page_size), or -1 for a size that is not supported.
int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

int bad(const char* what) {
    set_error("%s", what);
    return LLAMA_ERR_INVALID_ARG;
}

// Checks that paged_append and paged_attention share; *shift = log2(page_size).
int cache_args(int T, int nh, int nkv, int hd, int dtype, int n_pages, int page_size, int* shift) {
    if (T < 0) return bad("T must be >= 0");
    if (!is_dtype(dtype)) return bad("dtype must be LLAMA_F32, LLAMA_BF16 or LLAMA_F16");
    if (nh <= 0 || nkv <= 0 || nh % nkv) return bad("n_heads must be a positive multiple of n_kv_heads");
    const int rep = nh / nkv;
    if (rep != 1 && rep != 2 && rep != 4 && rep != 8) return bad("n_heads / n_kv_heads must be 1, 2, 4 or 8");
    if (hd != 32 && hd != 64 && hd != 128) { set_error("head_dim %d unsupported (32, 64, 128)", hd); return LLAMA_ERR_INVALID_ARG; }
    if (nh > 1024) return bad("n_heads must be at most 1024");
    if (n_pages <= 0) return bad("n_pages must be positive");
    if (static_cast<long long>(n_pages) * nkv > 0x7fffffffLL) return bad("n_pages * n_kv_heads must be below 2^31");
    *shift = page_shift_of(page_size);
    if (*shift < 0) { set_error("page_size %d must be 16, 32, 64, 128 or 256", page_size); return LLAMA_ERR_INVALID_ARG; }
    return LLAMA_OK;
}
}  // namespace
}  // namespace llb

using namespace llb;

extern "C" {

int llama_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size, int32_t* block_tables,
                     int max_pages, int32_t* free_pages, int n_pages, const int32_t* free_count, int T,
                     int32_t* seq_lens, int32_t* cu_new, int64_t* slots, int32_t* positions, int32_t* free_left,
                     int32_t* status, void* stream) {
    if (!ctx_lens || !new_lens || !block_tables || !free_pages || !free_count || !seq_lens || !cu_new || !free_left)
        return bad("a length, table, page-list or offset pointer is NULL");
    if (B <= 0 || max_pages <= 0 || n_pages <= 0 || T < 0) return bad("B, max_pages and n_pages must be positive, T >= 0");
    if (T > 0 && (!slots || !positions)) return bad("slots or positions is NULL");
    if (B > kPagedMaxRequests) { set_error("B=%d > %d requests", B, kPagedMaxRequests); return LLAMA_ERR_CAPACITY; }
    if (page_shift_of(page_size) < 0) { set_error("page_size %d must be 16, 32, 64, 128 or 256", page_size); return LLAMA_ERR_INVALID_ARG; }
    const PlanArgs a = {ctx_lens, new_lens, B, page_size, max_pages, n_pages, T, block_tables, free_pages, free_count,
                        seq_lens, cu_new, slots, positions, free_left, status};
    return launch_paged_plan(a, static_cast<cudaStream_t>(stream));
}

int llama_rope_table(float* rope, int len, int head_dim, float theta, void* stream) {
    if (!rope) return bad("rope is NULL");
    if (len <= 0 || head_dim <= 0 || head_dim % 2 || !(theta > 0.f)) return bad("len and theta must be positive, head_dim positive and even");
    if (static_cast<long long>(len) * (head_dim / 2) > 0x7fffff00LL) return bad("rope table too large");
    if ((reinterpret_cast<uintptr_t>(rope) & 7) != 0) return bad("rope must be 8-byte aligned");
    return launch_rope_table(reinterpret_cast<float2*>(rope), len, head_dim, theta, static_cast<cudaStream_t>(stream));
}

int llama_paged_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int in_dtype, int T, int n_heads, int n_kv_heads, int head_dim,
                       const float* q_norm, const float* k_norm, float eps, const float* rope, int rope_len,
                       const int32_t* positions, const int64_t* slots, void* q_out, void* k_pages, void* v_pages,
                       int n_pages, int page_size, int dtype, int32_t* status, void* stream) {
    int shift = 0;
    const int rc = cache_args(T, n_heads, n_kv_heads, head_dim, dtype, n_pages, page_size, &shift);
    if (rc != LLAMA_OK) return rc;
    if (in_dtype != dtype && in_dtype != LLAMA_F32) return bad("in_dtype must be LLAMA_F32 or the cache's dtype");
    if (!k_pages || !v_pages || !rope || rope_len <= 0) return bad("k_pages, v_pages or rope is NULL, or rope_len is not positive");
    if (!(eps >= 0.f)) return bad("eps must be >= 0");
    if (T == 0) return LLAMA_OK;
    if (!q || !k || !v || !positions || !slots || !q_out) return bad("q, k, v, positions, slots or q_out is NULL");
    const int e = in_dtype == LLAMA_F32 ? 4 : 2;
    if (q_stride < static_cast<int64_t>(n_heads) * head_dim || k_stride < static_cast<int64_t>(n_kv_heads) * head_dim ||
        v_stride < static_cast<int64_t>(n_kv_heads) * head_dim)
        return bad("a row stride is smaller than its row");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || (q_stride * e) % 16 || (k_stride * e) % 16 ||
        (v_stride * e) % 16 || !aligned16(q_out) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(rope) ||
        !aligned16(q_norm) || !aligned16(k_norm))
        return bad("q, k, v (bases and rows), q_out, the pages, rope and the norm weights must be 16-byte aligned");
    const AppendArgs a = {q, k, v, q_stride, k_stride, v_stride, T, n_heads, n_kv_heads, head_dim, q_norm, k_norm, eps,
                          reinterpret_cast<const float2*>(rope), rope_len, positions, slots, q_out, k_pages, v_pages,
                          static_cast<long long>(n_pages) << shift, shift, status};
    return launch_paged_append(a, in_dtype, dtype, static_cast<cudaStream_t>(stream));
}

size_t llama_paged_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int dtype, int max_new) {
    int shift = 0;
    if (cache_args(0, n_heads, n_kv_heads, head_dim, dtype, 1, 16, &shift) != LLAMA_OK) return 0;
    if (max_new < 1) { bad("max_new must be positive"); return 0; }
    return paged_attention_ws(n_heads, n_kv_heads, head_dim, dtype, max_new);
}

int llama_paged_attention(const void* q, const void* k_pages, const void* v_pages, int dtype, int T, int n_heads,
                          int n_kv_heads, int head_dim, int B, const int32_t* cu_new, const int32_t* seq_lens,
                          const int32_t* block_tables, int max_pages, int n_pages, int page_size, int max_new,
                          float scale, void* out, void* workspace, size_t workspace_bytes, int32_t* status,
                          void* stream) {
    int shift = 0;
    const int rc = cache_args(T, n_heads, n_kv_heads, head_dim, dtype, n_pages, page_size, &shift);
    if (rc != LLAMA_OK) return rc;
    if (!k_pages || !v_pages || !cu_new || !seq_lens || !block_tables) return bad("a page, offset, length or table pointer is NULL");
    if (B <= 0 || max_pages <= 0 || max_new < 1) return bad("B, max_pages and max_new must be positive");
    if (B > kPagedMaxRequests) { set_error("B=%d > %d requests", B, kPagedMaxRequests); return LLAMA_ERR_CAPACITY; }
    if ((static_cast<long long>(max_pages) << shift) > 0x40000000LL) return bad("max_pages * page_size must be at most 2^30");
    if (!(scale == scale) || scale - scale != 0.f) return bad("scale must be finite");
    if (T == 0) return LLAMA_OK;
    if (!q || !out) return bad("q or out is NULL");
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_pages) || !aligned16(v_pages)) return bad("q, out and the pages must be 16-byte aligned");
    const size_t need = paged_attention_ws(n_heads, n_kv_heads, head_dim, dtype, max_new);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need) {
        set_error("paged attention needs a 256-byte aligned workspace of %zu bytes", need);
        return LLAMA_ERR_INVALID_ARG;
    }
    const PagedAttnArgs a = {q, k_pages, v_pages, T, n_heads, n_kv_heads, head_dim, B, cu_new, seq_lens, block_tables,
                             max_pages, n_pages, shift, max_new, scale, out, workspace, status};
    return launch_paged_attention(a, dtype, static_cast<cudaStream_t>(stream));
}

int llama_sample_rows(const float* logits, int B, int V, const float* temperature, const int32_t* top_k,
                      const float* top_p, const float* min_p, const float* uniforms, int32_t* out, void* stream) {
    if (B < 0 || B > kMaxSampleRows || V <= 0 || V > 262144) return bad("B must be 0 .. 2^28 and V 1 .. 262144");
    if (B == 0) return LLAMA_OK;
    if (!logits || !temperature || !uniforms || !out) return bad("logits, temperature, uniforms or out is NULL");
    return launch_sample_rows(logits, B, V, temperature, top_k, top_p, min_p, uniforms, out,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
