// Causal attention of each request's new tokens over its pages (Admin Guide
// §8.4, Attention steps 5-7 and the mask NOTE; repeat_kv from the source tour):
//   o = softmax_j(q . K[j] * scale) V[j],  keys j = 0 .. position of the token.
//
// One warp per (token, head): a lane holds HD / 32 dims; online softmax.
#include "common.cuh"
#include "paged.h"

namespace llb {

template <typename T, int HD>
__global__ void __launch_bounds__(128) paged_attn_kernel(PagedAttnArgs a) {
    constexpr int E = HD / 32;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += 128)
            if (a.cu_new[b] < 0 || a.cu_new[b + 1] < a.cu_new[b] || a.cu_new[b + 1] > a.T)
                report_status(a.status, LLAMA_ERR_INVALID_ARG);
    const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(a.T) * a.nh) return;
    const int t = static_cast<int>(item / a.nh), h = static_cast<int>(item % a.nh);
    int lo = 0, hi = a.B - 1;                       // the request that holds row t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu_new[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int q0 = a.cu_new[lo], q1 = a.cu_new[lo + 1];
    if (t < q0 || t >= q1 || q1 > a.T) return;      // behind the last request: left as it was
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    long long seq = a.seq_lens[lo];
    if (seq < 0 || seq > cap) {
        if (lane == 0) report_status(a.status, LLAMA_ERR_CAPACITY);
        seq = seq < 0 ? 0 : cap;
    }
    const long long keys = min(seq, seq - (q1 - q0) + (t - q0) + 1);
    const int g = h / (a.nh / a.nkv);
    const T* qp = static_cast<const T*>(a.q) + item * HD + lane * E;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) { q[e] = to_f32<T>(qp[e]) * a.scale; o[e] = 0.f; }
    for (long long j = 0; j < keys; ++j) {
        const int page = a.block_tables[static_cast<long long>(lo) * a.max_pages + (j >> a.page_shift)];
        float s = 0.f, v[E];
        if (page < 0 || page >= a.n_pages) {
            if (lane == 0) report_status(a.status, LLAMA_ERR_INVALID_ARG);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = 0.f;
        } else {
            const long long at = ((((static_cast<long long>(page) * a.nkv + g) << a.page_shift) +
                                   (j & ((1 << a.page_shift) - 1))) * HD) + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s = fmaf(q[e], to_f32<T>(static_cast<const T*>(a.k_pages)[at + e]), s);
                v[e] = to_f32<T>(static_cast<const T*>(a.v_pages)[at + e]);
            }
            s = warp_sum(s);
        }
        const float mn = fmaxf(m, s);
        const float c = expf(m - mn), p = expf(s - mn);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, v[e], o[e] * c);
        m = mn;
    }
    T* op = static_cast<T*>(a.out) + item * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) op[e] = from_f32<T>(keys > 0 ? o[e] / l : 0.f);
}

template <typename T>
static int attn_hd(const PagedAttnArgs& a, cudaStream_t st) {
    const long long blocks = (static_cast<long long>(a.T) * a.nh + 3) / 4;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (a.hd == 32) paged_attn_kernel<T, 32><<<grid, 128, 0, st>>>(a);
    else if (a.hd == 64) paged_attn_kernel<T, 64><<<grid, 128, 0, st>>>(a);
    else paged_attn_kernel<T, 128><<<grid, 128, 0, st>>>(a);
    LLB_CHECK_LAUNCH("paged_attn_kernel");
    return LLAMA_OK;
}

size_t paged_attention_ws(int, int, int, int, int) { return 256; }

int launch_paged_attention(const PagedAttnArgs& a, int dtype, cudaStream_t st) {
    if (dtype == LLAMA_BF16) return attn_hd<bf16>(a, st);
    if (dtype == LLAMA_F16) return attn_hd<f16>(a, st);
    return attn_hd<float>(a, st);
}

}  // namespace llb
