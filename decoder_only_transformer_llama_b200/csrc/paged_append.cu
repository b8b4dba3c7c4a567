// Per-head RMSNorm of queries and keys, rotation by position, and the write
// of K and V into their cache slots, in one pass over a step's projections
// (Admin Guide §8.4: RMSNorm, apply_rotary_emb, Attention step 4).
//
//   y = x / sqrt(mean(x^2) + eps) * w          per head; without weights y = x
//   (y[2j], y[2j+1]) -> (y[2j] c - y[2j+1] s, y[2j] s + y[2j+1] c),  (c, s) = rope[position][j]
//
// in fp32, rounded once to the cache's type.  Bound by HBM: every value is
// read once and written once.  A lane holds two vectors of 16 bytes of a head,
// half a head apart (each coalesced, and the work per head shared by twice the
// values); the HD * sizeof(input) / 32 lanes of a head sum its squares by
// shuffles.  A thread asks for its kHeads heads' values and the slot together,
// so that a CTA waits for memory once and then once more for the rotation, which
// serves all of its heads.  What a thread does besides its heads costs about as
// much as one of them: three heads a thread where a token has enough, one where
// a CTA takes a token in one go or the step is short (16384 tokens of 48 heads,
// 16-bit, with norms: 81 us with three, 5.05 TB/s; 122 with one and 105 with two in
// CTAs of 256, which leave a quarter of the places empty; 64 tokens of 80 heads:
// 2.5 us with one, 2.9 with three).
#include <type_traits>

#include "common.cuh"
#include "paged.h"

namespace llb {

namespace {
constexpr int kThreads = 128;

template <typename TI, int N>
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[N]) {
    const TI* h = reinterpret_cast<const TI*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32<TI>(h[i]);
}
// 16 bytes that are read once.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}

template <typename TO, int N>
__device__ __forceinline__ void store_vec(TO* p, const float (&v)[N]) {
    if constexpr (sizeof(TO) == 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else if constexpr (N == 8) {
        uint4 u;
        u.x = pack2<TO>(v[0], v[1]); u.y = pack2<TO>(v[2], v[3]);
        u.z = pack2<TO>(v[4], v[5]); u.w = pack2<TO>(v[6], v[7]);
        *reinterpret_cast<uint4*>(p) = u;
    } else {
        uint2 u;
        u.x = pack2<TO>(v[0], v[1]); u.y = pack2<TO>(v[2], v[3]);
        *reinterpret_cast<uint2*>(p) = u;
    }
}
}  // namespace

template <typename TI, typename TO, int HD, int kHeads>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(AppendArgs a) {
    constexpr int N = 16 / static_cast<int>(sizeof(TI));   // values per vector
    constexpr int LPH = HD / (2 * N);                      // lanes per head
    constexpr int GROUPS = kThreads / LPH;
    const int t = blockIdx.x;
    const int sub = threadIdx.x % LPH;
    const int heads = a.nh + 2 * a.nkv;
    const int h0 = blockIdx.y * (GROUPS * kHeads) + threadIdx.x / LPH;
    const long long slot = a.slots[t];
    const int pos = a.positions[t];
    const TI* rows[3] = {static_cast<const TI*>(a.q) + t * a.q_stride,
                         static_cast<const TI*>(a.k) + t * a.k_stride - a.nh * HD,
                         static_cast<const TI*>(a.v) + t * a.v_stride - (a.nh + a.nkv) * HD};
    uint4 raw[kHeads][2];
#pragma unroll
    for (int e = 0; e < kHeads; ++e) {
        const int h = h0 + e * GROUPS;
        raw[e][0] = raw[e][1] = make_uint4(0u, 0u, 0u, 0u);
        if (h >= heads) continue;
        const TI* src = (h < a.nh ? rows[0] : h < a.nh + a.nkv ? rows[1] : rows[2]) + h * HD + sub * N;
        raw[e][0] = load_once(src);
        raw[e][1] = load_once(src + HD / 2);
    }
    if (slot < 0) return;                                  // padding: nothing is written
    if (slot >= a.n_slots || pos < 0 || pos >= a.rope_len) {
        if (threadIdx.x == 0) report_status(a.status, LLAMA_ERR_CAPACITY);
        return;
    }
    // Both vectors' rotations at once where they take few registers (fp32 input),
    // else one after the other (16-bit: 64 registers instead of 87, 86 -> 81 us for
    // 16384 tokens of 48 heads).
    constexpr bool kBoth = sizeof(TI) == 4;
    float4 turn[kBoth ? 2 : 1][N / 4];
    const float4* turns = reinterpret_cast<const float4*>(a.rope + static_cast<long long>(pos) * (HD / 2) + sub * (N / 2));
#pragma unroll
    for (int v = 0; v < (kBoth ? 2 : 1); ++v)
#pragma unroll
        for (int i = 0; i < N / 4; ++i) turn[v][i] = __ldg(turns + v * (HD / 8) + i);
    // a position's rows of one page's heads lie 2^page_shift rows apart
    const long long cell = (((slot >> a.page_shift) * a.nkv) << a.page_shift) + (slot & ((1LL << a.page_shift) - 1));
    float inv[kHeads];                                     // 1 / rms of each head
    if (a.q_norm || a.k_norm) {                            // the same for every thread: the shuffles stay warp-wide
#pragma unroll
        for (int e = 0; e < kHeads; ++e) {
            float x[2][N], s0 = 0.f, s1 = 0.f;
            unpack<TI, N>(raw[e][0], x[0]);
            unpack<TI, N>(raw[e][1], x[1]);
#pragma unroll
            for (int i = 0; i < N; ++i) { s0 = fmaf(x[0][i], x[0][i], s0); s1 = fmaf(x[1][i], x[1][i], s1); }
            s0 += s1;
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
            inv[e] = rsqrtf(s0 * (1.f / HD) + a.eps);
        }
    }
    // vector v of head e, rotated by f
    auto finish = [&](int e, int v, const float4 (&f)[N / 4]) {
        const int h = h0 + e * GROUPS;
        const bool is_q = h < a.nh, is_k = !is_q && h < a.nh + a.nkv;
        if (h >= heads) return;
        TO* dst;
        if (is_q) {
            dst = static_cast<TO*>(a.q_out) + (static_cast<long long>(t) * a.nh + h) * HD;
        } else {
            const int g = is_k ? h - a.nh : h - a.nh - a.nkv;
            dst = static_cast<TO*>(is_k ? a.k_pages : a.v_pages) + (cell + (static_cast<long long>(g) << a.page_shift)) * HD;
        }
        dst += sub * N + v * (HD / 2);
        float x[N];
        unpack<TI, N>(raw[e][v], x);
        if (is_q || is_k) {
            const float* w = is_q ? a.q_norm : a.k_norm;
            if (w) {
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const float4 g = __ldg(reinterpret_cast<const float4*>(w + v * (HD / 2) + sub * N + i));
                    x[i] *= inv[e] * g.x; x[i + 1] *= inv[e] * g.y; x[i + 2] *= inv[e] * g.z; x[i + 3] *= inv[e] * g.w;
                }
            }
            float y[N];
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {              // two pairs: (cos, sin), (cos, sin)
                const float* p = x + 4 * i;
                y[4 * i] = p[0] * f[i].x - p[1] * f[i].y;
                y[4 * i + 1] = p[0] * f[i].y + p[1] * f[i].x;
                y[4 * i + 2] = p[2] * f[i].z - p[3] * f[i].w;
                y[4 * i + 3] = p[2] * f[i].w + p[3] * f[i].z;
            }
            store_vec<TO, N>(dst, y);
        } else if constexpr (std::is_same<TI, TO>::value) {
            *reinterpret_cast<uint4*>(dst) = raw[e][v];                        // the value's own bits
        } else {
            store_vec<TO, N>(dst, x);
        }
    };
    if constexpr (kBoth) {
#pragma unroll
        for (int e = 0; e < kHeads; ++e) { finish(e, 0, turn[0]); finish(e, 1, turn[1]); }
    } else {
#pragma unroll
        for (int e = 0; e < kHeads; ++e) finish(e, 0, turn[0]);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) turn[0][i] = __ldg(turns + HD / 8 + i);
#pragma unroll
        for (int e = 0; e < kHeads; ++e) finish(e, 1, turn[0]);
    }
}

template <typename TI, typename TO, int HD>
static int append_go(const AppendArgs& a, cudaStream_t st) {
    constexpr int groups = kThreads / (HD * static_cast<int>(sizeof(TI)) / 32);   // heads a CTA works on at a time
    const int heads = a.nh + 2 * a.nkv;
    const int one = (heads + groups - 1) / groups;
    if (one == 1 || static_cast<long long>(a.T) * one <= 1024)
        paged_append_kernel<TI, TO, HD, 1><<<dim3(a.T, one), kThreads, 0, st>>>(a);
    else
        paged_append_kernel<TI, TO, HD, 3><<<dim3(a.T, (one + 2) / 3), kThreads, 0, st>>>(a);
    LLB_CHECK_LAUNCH("paged_append_kernel");
    return LLAMA_OK;
}

template <typename TI, typename TO>
static int append_hd(const AppendArgs& a, cudaStream_t st) {
    switch (a.hd) {
        case 32: return append_go<TI, TO, 32>(a, st);
        case 64: return append_go<TI, TO, 64>(a, st);
        default: return append_go<TI, TO, 128>(a, st);
    }
}

int launch_paged_append(const AppendArgs& a, int in_dtype, int dtype, cudaStream_t st) {
    if (in_dtype == LLAMA_BF16) return append_hd<bf16, bf16>(a, st);
    if (in_dtype == LLAMA_F16) return append_hd<f16, f16>(a, st);
    if (dtype == LLAMA_BF16) return append_hd<float, bf16>(a, st);
    if (dtype == LLAMA_F16) return append_hd<float, f16>(a, st);
    return append_hd<float, float>(a, st);
}

}  // namespace llb
