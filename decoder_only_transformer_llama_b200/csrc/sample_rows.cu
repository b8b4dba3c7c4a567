// Next-token draws with parameters of their own for each row: temperature,
// top-k, top-p and min-p (Admin Guide §6.3 and §8.5; the nucleus rule of the
// source tour, sample_top_p).
//
// With tokens in sampling order (logit descending, ties by id ascending),
// e_i = exp((l_i - l_max) / T), each filter keeps a prefix of the order:
//   top-k  the first k tokens, of mass Zk
//   top-p  the tokens whose mass before them is <= top_p * Zk, of mass Zp
//   min-p  the tokens with e_i >= min_p, of mass Zm
// so the kept tokens are the shortest of the three prefixes, their mass is
// Z = min(Zk, Zp, Zm), and the draw is the first token whose cumulative mass
// exceeds u * Z: it lies in the kept prefix by itself, and no filter needs
// the identity of its last token.  Masses are fp64 exponentials held as
// 64-bit fixed point (2^-46 resolution): every prefix sum is an exact integer
// in any order.
//
// One CTA per row; the prefix masses and the draw are found by a
// most-significant-digit radix select over the 64-bit (logit, id) key, with
// histograms of mass and count.
#include "common.cuh"
#include "paged.h"

namespace llb {

namespace {
constexpr int kThreads = 1024;
constexpr double kFix = 70368744177664.0;     // 2^46: V * 2^46 < 2^64 for V <= 262144

typedef unsigned long long u64;

// Order key: larger for a larger logit, among equal logits for the lower id.
// NaN orders with -inf: it is never drawn.  -0 and 0 are one value.
__device__ __forceinline__ u64 row_key(float l, int id) {
    if (!(l == l)) l = -INFINITY;
    if (l == 0.f) l = 0.f;
    uint32_t u = __float_as_uint(l);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (static_cast<u64>(u) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(id));
}

struct RowShared {
    u64 mass[256];
    unsigned int cnt[256];
    float red_f[32];
    u64 red_u[32];
    u64 prefix, before;
    unsigned int before_cnt;
};

struct RowParams {
    float lmax;
    double inv_t;
};

// e_i as a double; an infinite maximum leaves only its equals.
__device__ __forceinline__ double row_exp(const RowParams& p, float l) {
    if (!(l == l) || l == -INFINITY) return 0.0;
    if (l == p.lmax) return 1.0;
    if (p.lmax == INFINITY) return 0.0;
    return exp((static_cast<double>(l) - static_cast<double>(p.lmax)) * p.inv_t);
}
__device__ __forceinline__ u64 row_mass(const RowParams& p, float l) {
    return static_cast<u64>(row_exp(p, l) * kFix + 0.5);
}

// In sampling order, the first key whose inclusive mass exceeds `target`
// (by_count: whose inclusive count exceeds it), or the last key; *before =
// the mass of the keys ahead of it.
__device__ u64 row_select(RowShared& sh, const float* row, int V, const RowParams& p, bool by_count, u64 target,
                          u64* before_out) {
    u64 prefix = 0, mask = 0, before = 0;
    u64 before_cnt = 0;
    for (int shift = 56; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += kThreads) { sh.mass[i] = 0; sh.cnt[i] = 0; }
        __syncthreads();
        for (int i = threadIdx.x; i < V; i += kThreads) {
            const float l = row[i];
            const u64 key = row_key(l, i);
            if ((key & mask) != prefix) continue;
            const int bin = static_cast<int>((key >> shift) & 255u);
            atomicAdd(&sh.mass[bin], row_mass(p, l));
            atomicAdd(&sh.cnt[bin], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 cm = before, cc = before_cnt, bm = before, bc = before_cnt;
            int chosen = -1;
            for (int bin = 255; bin >= 0; --bin) {
                if (!sh.cnt[bin]) continue;
                chosen = bin;
                bm = cm;
                bc = cc;
                cm += sh.mass[bin];
                cc += sh.cnt[bin];
                if ((by_count ? cc : cm) > target) break;
            }
            sh.prefix = prefix | (static_cast<u64>(chosen) << shift);
            sh.before = bm;
            sh.before_cnt = static_cast<unsigned int>(bc);
        }
        __syncthreads();
        prefix = sh.prefix;
        before = sh.before;
        before_cnt = sh.before_cnt;
        mask |= 255ull << shift;
    }
    *before_out = before;
    return prefix;
}
}  // namespace

__global__ void __launch_bounds__(kThreads)
sample_rows_kernel(const float* __restrict__ logits, int V, const float* __restrict__ temperature,
                   const int32_t* __restrict__ top_k, const float* __restrict__ top_p,
                   const float* __restrict__ min_p, const float* __restrict__ uniforms, int32_t* __restrict__ out) {
    __shared__ RowShared sh;
    const int b = blockIdx.x;
    const float* row = logits + static_cast<long long>(b) * V;
    const float T = temperature[b];
    const int k = top_k ? top_k[b] : 0;
    const float tp = top_p ? top_p[b] : 1.f;
    const float mp = min_p ? min_p[b] : 0.f;
    if (!(T >= 0.f) || T == INFINITY || !(tp >= 0.f) || !(mp >= 0.f) || mp > 1.f) {
        if (threadIdx.x == 0) out[b] = -1;
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    u64 best = 0;
    for (int i = threadIdx.x; i < V; i += kThreads) {
        const u64 key = row_key(row[i], i);
        best = key > best ? key : best;
    }
    best = warp_max_u64(best);
    if (lane == 0) sh.red_u[warp] = best;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) best = sh.red_u[w] > best ? sh.red_u[w] : best;
    const int first = static_cast<int>(~static_cast<uint32_t>(best & 0xffffffffu));
    RowParams p;
    p.lmax = row[first];
    if (!(p.lmax == p.lmax)) p.lmax = -INFINITY;
    if (T == 0.f || p.lmax == -INFINITY) {
        if (threadIdx.x == 0) out[b] = first;
        return;
    }
    p.inv_t = 1.0 / static_cast<double>(T);
    __syncthreads();
    // all tokens, and those of min-p
    u64 s = 0, zm = 0;
    for (int i = threadIdx.x; i < V; i += kThreads) {
        const double e = row_exp(p, row[i]);
        const u64 m = static_cast<u64>(e * kFix + 0.5);
        s += m;
        if (e >= static_cast<double>(mp)) zm += m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        zm += __shfl_xor_sync(0xffffffffu, zm, o);
    }
    __shared__ u64 s_m[32];
    if (lane == 0) { sh.red_u[warp] = s; s_m[warp] = zm; }
    __syncthreads();
    s = 0;
    zm = 0;
    for (int w = 0; w < kThreads / 32; ++w) { s += sh.red_u[w]; zm += s_m[w]; }
    u64 z = s, before;
    if (k > 0 && k < V) {
        const u64 key = row_select(sh, row, V, p, true, static_cast<u64>(k - 1), &before);
        z = before + row_mass(p, row[~static_cast<uint32_t>(key & 0xffffffffu)]);
    }
    if (tp < 1.f) {
        const u64 target = static_cast<u64>(static_cast<double>(tp) * static_cast<double>(z));
        const u64 key = row_select(sh, row, V, p, false, target, &before);
        const u64 zp = before + row_mass(p, row[~static_cast<uint32_t>(key & 0xffffffffu)]);
        z = zp < z ? zp : z;
    }
    z = zm < z ? zm : z;
    // u below 1, so the target stays below the kept mass
    const double u = fmin(fmax(static_cast<double>(uniforms[b]), 0.0), 1.0 - 1.0 / 16777216.0);
    const u64 key = row_select(sh, row, V, p, false, static_cast<u64>(u * static_cast<double>(z)), &before);
    if (threadIdx.x == 0) out[b] = static_cast<int32_t>(~static_cast<uint32_t>(key & 0xffffffffu));
}

int launch_sample_rows(const float* logits, int B, int V, const float* temperature, const int32_t* top_k,
                       const float* top_p, const float* min_p, const float* uniforms, int32_t* out, cudaStream_t st) {
    sample_rows_kernel<<<B, kThreads, 0, st>>>(logits, V, temperature, top_k, top_p, min_p, uniforms, out);
    LLB_CHECK_LAUNCH("sample_rows_kernel");
    return LLAMA_OK;
}

}  // namespace llb
