// Block tables, slot maps, positions and offsets of one serving step, from
// the requests' lengths (the cache indexed by position, Admin Guide §8.4 and
// §6.2, cut into pages).
//
// Every request's first token row, its place among the released pages and its
// place among the pages taken are prefix sums over the requests.  Page i that
// the step takes is known without any exchange: it is entry count + released -
// 1 - i of the stack, which lies in free_pages below count and in the table of
// the ended request that returns it above.  So each CTA scans the lengths by
// itself and writes its share of slots, pages and offsets from the inputs
// alone; a cluster barrier between the last read of an input and the first
// write lets seq_lens and free_left be the inputs they follow.  Latency bound (a
// step moves a few hundred kilobytes at most): 3.5 us for 32 decodes, 7.9 us for
// 256 requests with 11000 new tokens; one CTA with a thread per request that
// moved its pages one after the other took 23.6 us for the former.
#include "common.cuh"
#include "paged.h"

namespace llb {

namespace {
constexpr int kThreads = 512;
constexpr int kPer = kPagedMaxRequests / kThreads;   // requests per thread
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr long long kMaxTokens = 1LL << 30;          // of one request, as in paged attention

// The last of n ascending entries that is <= v (a[0] <= v).
__device__ __forceinline__ int last_le(const int* a, int n, int v) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
}
}  // namespace

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(PlanArgs a, int shift) {
    __shared__ int s_tok[kPagedMaxRequests + 1], s_take[kPagedMaxRequests + 1], s_back[kPagedMaxRequests + 1];
    __shared__ int s_ctx[kPagedMaxRequests];
    __shared__ long long s_sum[3][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, step = gridDim.x * kThreads, first = cta * kThreads + tid;
    const long long ps1 = (1 << shift) - 1;
    const long long count = a.free_count[0];
    long long ctx[kPer], n[kPer], v[3] = {0, 0, 0};   // tokens, released pages, taken pages
    bool ended[kPer];
    int err = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int b = tid * kPer + e;
        ctx[e] = b < a.B ? a.ctx_lens[b] : 0;
        const int nl = b < a.B ? a.new_lens[b] : 0;
        ended[e] = nl < 0;
        n[e] = ended[e] ? 0 : nl;
    }
    long long have[kPer], want[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        have[e] = (ctx[e] + ps1) >> shift;
        want[e] = ended[e] ? 0 : ((ctx[e] + n[e] + ps1) >> shift) - have[e];
        v[0] += n[e];
        v[1] += ended[e] ? have[e] : 0;
        v[2] += want[e];
        if (ctx[e] < 0) err = LLAMA_ERR_INVALID_ARG;
        else if (!err && (have[e] + want[e] > a.max_pages || ctx[e] + n[e] > kMaxTokens)) err = LLAMA_ERR_CAPACITY;
    }
    long long incl[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const long long y = __shfl_up_sync(0xffffffffu, incl[x], o);
            if (lane >= o) incl[x] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int x = 0; x < 3; ++x) s_sum[x][warp] = incl[x];
    __syncthreads();
    long long total[3], at[3];
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        long long w = lane < kWarps ? s_sum[x][lane] : 0;
        long long before = lane < warp ? w : 0;
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            w += __shfl_xor_sync(0xffffffffu, w, o);
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        total[x] = __shfl_sync(0xffffffffu, w, 0);
        at[x] = __shfl_sync(0xffffffffu, before, 0) + incl[x] - v[x];
    }
    if (count < 0 || count + total[1] > a.n_pages) err = LLAMA_ERR_INVALID_ARG;
    else if (!err && (total[0] > a.T || total[2] > count + total[1])) err = LLAMA_ERR_CAPACITY;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int b = tid * kPer + e;
        if (b <= a.B && b < kPagedMaxRequests) {
            s_tok[b] = static_cast<int>(at[0]);
            s_back[b] = static_cast<int>(at[1]);
            s_take[b] = static_cast<int>(at[2]);
            s_ctx[b] = static_cast<int>(ctx[e]);
        }
        at[0] += n[e];
        at[1] += ended[e] ? have[e] : 0;
        at[2] += want[e];
    }
    // everyone has read the lengths and the count (the sums, and in a cluster its other CTAs)
    const bool invalid = __syncthreads_or(err == LLAMA_ERR_INVALID_ARG);
    const bool fails = __syncthreads_or(err);
    if (gridDim.x > 1) cluster_sync();
    if (fails) {
        // nothing is granted and nothing changes: no tokens in this step
        if (first == 0) report_status(a.status, invalid ? LLAMA_ERR_INVALID_ARG : LLAMA_ERR_CAPACITY);
        for (int b = first; b <= a.B; b += step) {
            if (b < a.B) a.seq_lens[b] = s_ctx[b];
            a.cu_new[b] = 0;
        }
        for (int t = first; t < a.T; t += step) { a.slots[t] = -1; a.positions[t] = -1; }
        if (first == 0) a.free_left[0] = static_cast<int32_t>(count);
        return;
    }
    const int n_tok = static_cast<int>(total[0]), n_back = static_cast<int>(total[1]), n_take = static_cast<int>(total[2]);
    auto released = [&](int i) {                      // page i of the released ones
        const int b = last_le(s_back, a.B, i);
        return a.block_tables[static_cast<long long>(b) * a.max_pages + (i - s_back[b])];
    };
    auto taken = [&](int i) {                         // page i of the taken ones
        const long long at_stack = count + n_back - 1 - i;
        return at_stack < count ? a.free_pages[at_stack] : released(static_cast<int>(at_stack - count));
    };
    for (int t = first; t < a.T; t += step) {
        long long slot = -1;
        int pos = -1;
        if (t < n_tok) {
            const int b = last_le(s_tok, a.B, t);
            pos = s_ctx[b] + t - s_tok[b];
            const int pg = pos >> shift, held = static_cast<int>((s_ctx[b] + ps1) >> shift);
            const int page = pg < held ? a.block_tables[static_cast<long long>(b) * a.max_pages + pg]
                                       : taken(s_take[b] + pg - held);
            if (page >= 0) slot = (static_cast<long long>(page) << shift) + (pos & ps1);
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    for (int i = first; i < n_take; i += step) {
        const int b = last_le(s_take, a.B, i);
        const int held = static_cast<int>((s_ctx[b] + ps1) >> shift);
        a.block_tables[static_cast<long long>(b) * a.max_pages + held + i - s_take[b]] = taken(i);
    }
    for (int i = first; i < n_back; i += step) a.free_pages[count + i] = released(i);
    if (cta == 0) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int b = tid * kPer + e;
            if (b < a.B) {
                a.seq_lens[b] = ended[e] ? 0 : static_cast<int32_t>(ctx[e] + n[e]);
                a.cu_new[b] = s_tok[b];
            }
        }
        if (tid == 0) {
            a.cu_new[a.B] = n_tok;
            a.free_left[0] = static_cast<int32_t>(count + n_back - n_take);
        }
    }
}

int launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
    int shift = 4;
    while ((1 << shift) < a.page_size) ++shift;
    // CTAs for up to four token rows a thread, as one cluster
    int ctas = 1;
    while (ctas < kMaxCtas && ctas * kThreads * 4 < a.T) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_plan_kernel, a, shift);
    count_launch();
    if (e != cudaSuccess) return cuda_fail(e, "paged_plan_kernel");
    return LLAMA_OK;
}

}  // namespace llb
