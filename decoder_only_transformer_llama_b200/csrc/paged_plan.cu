// Block tables, slot maps, positions and offsets of one serving step, from
// the requests' lengths (the cache indexed by position, Admin Guide §8.4 and
// §6.2, cut into pages).
//
// One CTA: thread b holds request b; three block scans give every request its
// first token row, its place among the released pages and its place among the
// pages taken.  Latency bound: a step moves a few hundred kilobytes at most.
#include "common.cuh"
#include "paged.h"

namespace llb {

namespace {
constexpr int kThreads = 1024;

// Exclusive scan of v over the CTA's threads; *total = the sum.
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    long long before = 0, sum = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        sum += s_warp[w];
    }
    *total = sum;
    return before + incl - v;
}
}  // namespace

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(PlanArgs a) {
    __shared__ long long s_warp[kThreads / 32];
    __shared__ int s_cu[kThreads + 1];
    __shared__ int s_ctx[kThreads];
    const int b = threadIdx.x;
    const bool in = b < a.B;
    const long long ctx = in ? a.ctx_lens[b] : 0;
    const int nl = in ? a.new_lens[b] : 0;
    const long long count = a.free_count[0];
    const bool ended = nl < 0;
    const long long n = ended ? 0 : nl;
    const long long ps = a.page_size;
    const long long have = (ctx + ps - 1) / ps;
    const long long want = ended ? 0 : (ctx + n + ps - 1) / ps - have;
    long long n_tok, n_back, n_take;
    const long long tok_at = block_scan(n, s_warp, &n_tok);
    const long long back_at = block_scan(ended ? have : 0, s_warp, &n_back);
    const long long take_at = block_scan(want, s_warp, &n_take);
    int err = 0;
    if (ctx < 0 || count < 0 || count + n_back > a.n_pages) err = LLAMA_ERR_INVALID_ARG;
    else if (have + want > a.max_pages || n_tok > a.T || n_take > count + n_back) err = LLAMA_ERR_CAPACITY;
    if (err) report_status(a.status, err);
    if (__syncthreads_or(err)) {
        // nothing is granted and nothing changes: no tokens in this step
        if (in) a.seq_lens[b] = static_cast<int32_t>(ctx);
        for (int i = b; i <= a.B; i += kThreads) a.cu_new[i] = 0;
        for (int t = b; t < a.T; t += kThreads) { a.slots[t] = -1; a.positions[t] = -1; }
        if (b == 0) a.free_left[0] = static_cast<int32_t>(count);
        return;
    }
    int32_t* row = a.block_tables + static_cast<long long>(b) * a.max_pages;
    if (in && ended)
        for (long long i = 0; i < have; ++i) a.free_pages[count + back_at + i] = row[i];
    __syncthreads();
    if (in) {
        for (long long i = 0; i < want; ++i) row[have + i] = a.free_pages[count + n_back - 1 - (take_at + i)];
        a.seq_lens[b] = ended ? 0 : static_cast<int32_t>(ctx + n);
        a.cu_new[b] = static_cast<int32_t>(tok_at);
        s_cu[b] = static_cast<int>(tok_at);
        s_ctx[b] = static_cast<int>(ctx);
    }
    if (b == 0) {
        a.cu_new[a.B] = static_cast<int32_t>(n_tok);
        s_cu[a.B] = static_cast<int>(n_tok);
        a.free_left[0] = static_cast<int32_t>(count + n_back - n_take);
    }
    __syncthreads();
    for (int t = b; t < a.T; t += kThreads) {
        long long slot = -1;
        int pos = -1;
        if (t < s_cu[a.B]) {
            int lo = 0, hi = a.B - 1;               // last request with s_cu <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
            }
            pos = s_ctx[lo] + t - s_cu[lo];
            const int page = a.block_tables[static_cast<long long>(lo) * a.max_pages + pos / a.page_size];
            if (page >= 0) slot = static_cast<long long>(page) * a.page_size + pos % a.page_size;
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
}

int launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
    paged_plan_kernel<<<1, kThreads, 0, st>>>(a);
    LLB_CHECK_LAUNCH("paged_plan_kernel");
    return LLAMA_OK;
}

}  // namespace llb
