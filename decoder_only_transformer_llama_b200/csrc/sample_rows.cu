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
// 64-bit fixed point (2^-46 resolution, 2^-45 for 2^18 tokens): every prefix sum
// is an exact integer below 2^64 in any order, and tokens below half a unit
// weigh nothing.
//
// Measured: 1 x 32000 logits 11 us (six exchanges over the cluster, latency), 64 x 128000
// with parameters of every kind 63 us (rows with top-k 34, with min-p 40, with top-p 75; of
// the histogram pass of the latter, 14 us, the additions to shared memory take 8, whose
// lanes meet in banks, and the exponentials 4), against 1.28 ms and 5.2 ms of one CTA per row
// with a radix select over whole-row passes.
//
// A row is spread over a cluster of R = 8, 4 or 2 CTAs.  A histogram over 1024 equal steps
// of l_max - l (bins are ordered like the tokens), summed over the cluster
// through distributed shared memory, turns each of the three searches (k-th
// token, nucleus edge, draw) into the choice of a bin; the tokens up to that
// bin, or in it, are gathered into a list of at most 256, which every CTA sorts
// and resolves alike.  A row with a small top_k needs counts only: its list
// holds every token that may be drawn, and only their exponentials are taken.
// Other rows add masses to the histogram.  A bin with more tokens than a list
// holds is cut into 1024 steps by a second histogram; a step with more (ties)
// by histograms over the order key, 10 bits of it at a time.
#include "common.cuh"
#include "paged.h"
#include "per_device.cuh"
#include "sample_mass.cuh"

namespace llb {

namespace {
typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kCap = 256;                     // tokens one list holds
constexpr int kKept = 8192;                   // logits of a slice that stay in shared memory
constexpr int kSlice = 65536;                 // most logits of a slice: the sums of 16 mass bits stay below 2^32
constexpr double kOne = 4503599627370496.0;   // 2^52: adding it rounds a double to an integer, in its low 52 bits
constexpr u64 kKeep = 1ull << 63;             // beside a mass: min-p keeps the token
constexpr float kReach = 32.625f;             // 47 ln 2 = 32.58: masses beyond round to 0

struct Prefix {
    u64 mass[kBins + 1];                      // before each bin
    unsigned int cnt[kBins + 1];
};
struct __align__(16) RowShared {
    unsigned int h[4][kBins];                 // this CTA's histogram: counts, mass bits 0-15, 16-31, 32-46
    Prefix p0, p1;                            // cluster totals: of the whole row, of a bin being cut
    u64 seg_key[2][kCap], seg_mass[2][kCap];  // tokens this CTA gathered, read by the cluster
    u64 key[kCap], mass[kCap];                // the cluster's list as gathered
    u64 s_key[kCap], s_pre[kCap + 1];         // and in sampling order: keys, mass before each (and behind the last)
    u64 x_zm, x_k0, x_k1;                     // this CTA's part of a maximum or sum, read by the cluster
    float x_max, x_min;
    int x_id;
    bool s_keep[kCap];                        // min-p keeps it
    int seg_n[2];
    u64 red_a[kWarps], red_b[kWarps];
    float red_f[kWarps], red_g[kWarps];
    double table[32][32];                     // 2^(mass_bits - j / 32), a column for each lane
    int bin, hit;
};

// Order key: larger for a larger logit, among equal logits for the lower id.
// NaN orders with -inf: it is never drawn.  -0 and 0 are one value.
__device__ __forceinline__ u64 row_key(float l, int id) {
    if (!(l == l)) l = -INFINITY;
    if (l == 0.f) l = 0.f;
    uint32_t u = __float_as_uint(l);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (static_cast<u64>(u) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(id));
}
__device__ __forceinline__ int key_id(u64 k) { return static_cast<int>(~static_cast<uint32_t>(k & 0xffffffffu)); }

__device__ __forceinline__ u64 ld_peer64(const void* p, uint32_t rank) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ unsigned int ld_peer32(const void* p, uint32_t rank) {
    unsigned int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void st_peer64(const void* p, uint32_t rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(cluster_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void st_peer32(const void* p, uint32_t rank, unsigned int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(cluster_addr(p, rank)), "r"(v) : "memory");
}

// One row's scales.  e = 2^(-y / 32), y = (l_max - l) * c32 with c32 = 32 log2(e) / T.
struct Scale {
    float lmax, lcut;    // tokens below lcut weigh nothing
    double dmax, c32;    // l_max
    float cbin;          // bins per unit of l_max - l
};

constexpr double kMagic = 6755399441055744.0;    // 1.5 * 2^52: adding it rounds to an integer, in the low word

// Tokens that may weigh something (never NaN or -inf).
__device__ __forceinline__ bool within(const Scale& s, float l) { return l >= s.lcut; }

// A token's mass, e * 2^mass_bits rounded to an integer, plus 2^52; for tokens within
// reach only (others give anything).  y = n + r, |r| <= 1/2, is cut into n =
// 32 q + j, and 2^(-y/32) = 2^-q * 2^(-j/32) * exp(-r ln2 / 32) with the exponential's
// Taylor terms up to the fifth power (|r ln2 / 32| < 0.011: the rest is below 2.3e-15,
// a third of the masses' resolution).  Table-driven exponentials after Tang (1989).
// Every lane has a copy of the table in its own banks: lanes that look up different
// entries of one copy wait for one another, 5 passes instead of 2.
__device__ __forceinline__ double row_mass(const double* table, const Scale& s, float l) {
    constexpr double c = 0.69314718055994530942 / 32.0;
    const double d = s.dmax - static_cast<double>(l);
    const double t = fma(d, s.c32, kMagic);
    const int n = __double2loint(t);
    const double r = fma(d, s.c32, kMagic - t);
    double p = fma(r, -c * c * c * c * c / 120.0, c * c * c * c / 24.0);
    p = fma(p, r, -c * c * c / 6.0);
    p = fma(p, r, c * c / 2.0);
    p = fma(p, r, -c);
    p = fma(p, r, 1.0);
    const double v = table[(n & 31) * 32];
    const double scale = __hiloint2double(__double2hiint(v) - ((n & ~31) << 15), __double2loint(v));   // * 2^-q
    return fma(p, scale, kOne);
}
__device__ __forceinline__ u64 mass_of(double m) { return static_cast<u64>(__double_as_longlong(m)) & 0xfffffffffffffull; }
// A token's bin, the distance in steps rounded to an integer: as a float, 2^23 + bin
// (ordered like the tokens; two additions and no conversion), and as a number.
constexpr float kBinBase = 8388608.f;
__device__ __forceinline__ float row_place(const Scale& s, float l) {
    return fminf(fmaf(s.lmax - l, s.cbin, kBinBase), kBinBase + (kBins - 1));
}
__device__ __forceinline__ int row_bin(const Scale& s, float l) {
    return __float_as_int(row_place(s, l)) - __float_as_int(kBinBase);
}
// The step within the bin at `place`, of 1024.
__device__ __forceinline__ int row_step(const Scale& s, float l, float place) {
    const float part = fmaf(s.lmax - l, s.cbin, kBinBase - place);          // -1/2 .. 1/2
    return max(0, min(static_cast<int>((part + 0.5f) * kBins), kBins - 1));
}

// Adds a token of mass m (row_mass) to this CTA's histogram (shared address h), to its
// counts if asked to: nothing if not `in`, without branches.
__device__ __forceinline__ void hist_add(uint32_t h, int bin, double m, bool in, bool counted) {
    const uint32_t lo = __double2loint(m), hi = __double2hiint(m) & 0xfffff, at = h + 4 * bin;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t@p red.shared.add.u32 [%0 + %5], %1;\n\t"
                 "@p red.shared.add.u32 [%0 + %6], %2;\n\t@p red.shared.add.u32 [%0 + %7], %3;\n\t}"
                 :: "r"(at), "r"(lo & 0xffffu), "r"(lo >> 16), "r"(hi), "r"(static_cast<uint32_t>(in)),
                    "n"(4 * kBins), "n"(8 * kBins), "n"(12 * kBins) : "memory");
    if (counted && in && (lo | hi)) asm volatile("red.shared.add.u32 [%0], 1;" :: "r"(at) : "memory");
}
__device__ __forceinline__ void hist_clear(RowShared& sh) {
    for (int i = threadIdx.x; i < 4 * kBins; i += kThreads) sh.h[i / kBins][i % kBins] = 0u;
}

// The most tokens that may lie in a bin of mass m (each weighs 1 at least), from the
// smallest mass within it: 2^(bits - (bin + 1/2) step), less its rounding.
__device__ __forceinline__ unsigned int most_tokens(u64 m, int bin, float step, int bits) {
    const float least = exp2f(static_cast<float>(bits) - (static_cast<float>(bin) + 0.5f) * step) * 0.999f - 1.f;
    return static_cast<unsigned int>(fminf(__ull2float_ru(m) / fmaxf(least, 1.f) * 1.0001f, 262144.f));
}

// The cluster's totals of the histograms, as sums before each bin, into `p` of every CTA.
// step > 0: no counts were taken, the bound of most_tokens takes their place.
template <int R, bool MASS>
__device__ __forceinline__ void hist_reduce(RowShared& sh, Prefix& p, uint32_t rank, float step = 0.f, int bits = 0) {
    cluster_sync();
    {
        // CTA r adds up its share of the bins: R / 2 threads a bin, two CTAs each
        const int bin = static_cast<int>(rank) * (kBins / R) + threadIdx.x / (R / 2), q = threadIdx.x % (R / 2);
        u64 m = 0;
        unsigned int c = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t from = 2 * q + x;
            c += ld_peer32(&sh.h[0][bin], from);
            if (MASS)
                m += ld_peer32(&sh.h[1][bin], from) + (static_cast<u64>(ld_peer32(&sh.h[2][bin], from)) << 16) +
                     (static_cast<u64>(ld_peer32(&sh.h[3][bin], from)) << 32);
        }
#pragma unroll
        for (int o = 1; o < R / 2; o <<= 1) {
            m += __shfl_xor_sync(0xffffffffu, m, o);
            c += __shfl_xor_sync(0xffffffffu, c, o);
        }
        if (MASS && step > 0.f) c = most_tokens(m, bin, step, bits);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (MASS) st_peer64(&p.mass[bin + 1], 2 * q + x, m);
            st_peer32(&p.cnt[bin + 1], 2 * q + x, c);
        }
    }
    cluster_sync();
    // prefix sums: two bins a thread
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = 2 * threadIdx.x;
    const u64 m0 = MASS ? p.mass[b + 1] : 0ull, m1 = MASS ? p.mass[b + 2] : 0ull;
    const unsigned int c0 = p.cnt[b + 1], c1 = p.cnt[b + 2];
    u64 m = m0 + m1;
    unsigned int c = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 ym = __shfl_up_sync(0xffffffffu, m, o);
        const unsigned int yc = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) { m += ym; c += yc; }
    }
    if (lane == 31) { sh.red_a[warp] = m; sh.red_b[warp] = c; }
    __syncthreads();
    u64 bm = m - m0 - m1;
    unsigned int bc = c - c0 - c1;
    for (int w = 0; w < warp; ++w) { bm += sh.red_a[w]; bc += static_cast<unsigned int>(sh.red_b[w]); }
    p.mass[b + 1] = bm + m0;
    p.cnt[b + 1] = bc + c0;
    p.mass[b + 2] = bm + m0 + m1;
    p.cnt[b + 2] = bc + c0 + c1;
    if (threadIdx.x == 0) { p.mass[0] = 0; p.cnt[0] = 0; }
    __syncthreads();
}

// The bin that holds the first token whose inclusive mass (by_count: count)
// exceeds `target`, counted from `p`'s first bin; the caller knows there is one.
__device__ __forceinline__ int choose_bin(RowShared& sh, const Prefix& p, bool by_count, u64 target) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
        const u64 lo = by_count ? p.cnt[b] : p.mass[b], hi = by_count ? p.cnt[b + 1] : p.mass[b + 1];
        if (lo <= target && target < hi) sh.bin = b;
    }
    __syncthreads();
    const int bin = sh.bin;
    __syncthreads();
    return bin;
}
}  // namespace

// KEPT: the CTA's slice of the row stays in shared memory (up to 8192 logits);
// otherwise each pass reads it again (from L2).
template <int R, bool KEPT>
__global__ void __launch_bounds__(kThreads, 2)
sample_rows_kernel(const float* __restrict__ logits, int V, const float* __restrict__ temperature,
                   const int32_t* __restrict__ top_k, const float* __restrict__ top_p,
                   const float* __restrict__ min_p, const float* __restrict__ uniforms, int32_t* __restrict__ out) {
    extern __shared__ __align__(16) uint8_t smem[];
    RowShared& sh = *reinterpret_cast<RowShared*>(smem);
    const uint32_t rank = cluster_rank();
    const int b = blockIdx.x / R;
    const float T = temperature[b];
    const int k = top_k ? top_k[b] : 0;
    const float tp = top_p ? top_p[b] : 1.f;
    const float mp = min_p ? min_p[b] : 0.f;
    // (1e30f lies above 1e30)
    if (!(T >= 0.f) || T >= 1e30f || !(tp >= 0.f) || !(mp >= 0.f) || mp > 1.f) {
        if (rank == 0 && threadIdx.x == 0) out[b] = -1;
        return;                                // the whole cluster, before any exchange
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int S = (V + R - 1) / R, lo = static_cast<int>(rank) * S;
    const int n = max(0, min(S, V - lo));
    const float* row = logits + static_cast<long long>(b) * V + lo;
    // The slice as 16-byte vectors of aligned addresses; its first and last may
    // reach outside the slice, where values read as -inf and are skipped.
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 2) & 3);
    const int nv = n > 0 ? (n + mis + 3) >> 2 : 0;
    float4* kept = reinterpret_cast<float4*>(smem + sizeof(RowShared));
    const float4* vectors = reinterpret_cast<const float4*>(row - mis);
    auto fetch = [&](int i) {
        if (i > 0 && i < nv - 1) return __ldg(vectors + i);
        const int j = 4 * i - mis;
        float4 v;
        v.x = j >= 0 ? __ldg(row + j) : -INFINITY;
        v.y = j + 1 >= 0 && j + 1 < n ? __ldg(row + j + 1) : -INFINITY;
        v.z = j + 2 >= 0 && j + 2 < n ? __ldg(row + j + 2) : -INFINITY;
        v.w = j + 3 < n ? __ldg(row + j + 3) : -INFINITY;
        return v;
    };
    bool infinite = false;
    // f(four logits, first id) for every vector of the slice (-inf outside it); the next
    // one is asked for while f works on this one.  f's code is there once: four vectors
    // asked for and worked on together, by four copies of it, took 66 us for 62.
    auto each4 = [&](auto f) __attribute__((always_inline)) {
        float4 next;
        if (threadIdx.x < nv) next = KEPT ? kept[threadIdx.x] : fetch(threadIdx.x);
        for (int i = threadIdx.x; i < nv; i += kThreads) {
            float l[4] = {next.x, next.y, next.z, next.w};
            if (i + kThreads < nv) next = KEPT ? kept[i + kThreads] : fetch(i + kThreads);
            if (infinite) {                    // only the equals of an infinite maximum weigh anything
#pragma unroll
                for (int y = 0; y < 4; ++y) l[y] = l[y] == INFINITY ? 0.f : -INFINITY;
            }
            f(l, lo + 4 * i - mis);
        }
    };
    // f(logit, id) for the tokens that `in` accepts
    auto each_of = [&](auto in, auto f) __attribute__((always_inline)) {
        each4([&](const float (&l)[4], int id) {
            bool t[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) t[y] = in(l[y], id + y);
            if (t[0] || t[1] || t[2] || t[3]) {
#pragma unroll 1
                for (int y = 0; y < 4; ++y)
                    if (in(l[y], id + y)) f(l[y], id + y);
            }
        });
    };
    // ---- the largest logit of the row and its smallest finite one
    constexpr int kAhead = KEPT ? 2 : 4;       // vectors a thread has in flight
    float4 v[kAhead];
    auto ask = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int i = i0 + x * kThreads;
            v[x] = i < nv ? fetch(i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
    };
    ask(threadIdx.x);
    {
        const double e = exp2(mass_bits(V) - static_cast<double>(lane) / 32.0);
#pragma unroll
        for (int j = warp; j < 32; j += kWarps) sh.table[j][lane] = __shfl_sync(0xffffffffu, e, j);
    }
    const double* const table = &sh.table[0][lane];
    const uint32_t hist = smem_u32(&sh.h[0][0]);
    hist_clear(sh);
    if (threadIdx.x == 0) { sh.hit = 0; sh.bin = 0; }
    float lmax = -INFINITY, least = INFINITY;
    for (int i0 = threadIdx.x; i0 < nv;) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (KEPT && i0 + x * kThreads < nv) kept[i0 + x * kThreads] = v[x];   // read back by this thread only
            const float l[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                lmax = fmaxf(lmax, l[y]);                      // NaN never wins
                if (l[y] > -INFINITY) least = fminf(least, l[y]);
            }
        }
        i0 += kAhead * kThreads;
        ask(i0);
    }
    lmax = warp_max(lmax);
    least = -warp_max(-least);
    if (lane == 0) { sh.red_f[warp] = lmax; sh.red_g[warp] = least; }
    __syncthreads();
    if (warp == 0) {
        lmax = warp_max(lane < kWarps ? sh.red_f[lane] : -INFINITY);
        least = -warp_max(lane < kWarps ? -sh.red_g[lane] : -INFINITY);
        if (lane == 0) { sh.x_max = lmax; sh.x_min = least; }
    }
    cluster_sync();
    lmax = warp_max(lane < R ? __uint_as_float(ld_peer32(&sh.x_max, lane)) : -INFINITY);
    least = -warp_max(lane < R ? -__uint_as_float(ld_peer32(&sh.x_min, lane)) : -INFINITY);
    infinite = lmax == INFINITY;
    if (infinite) lmax = least = 0.f;
    if (T == 0.f || lmax == -INFINITY) {
        // greedy: the lowest id at the maximum (a row without a finite logit: token 0)
        int id0 = 0x7fffffff;
        if (lmax > -INFINITY)
            each_of([&](float l, int) { return l == lmax; }, [&](float, int id) { id0 = min(id0, id); });
        id0 = __reduce_min_sync(0xffffffffu, id0);
        if (lane == 0) sh.red_b[warp] = static_cast<u64>(id0);
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWarps; ++w) id0 = min(id0, static_cast<int>(sh.red_b[w]));
            sh.x_id = id0;
        }
        cluster_sync();
        if (rank == 0 && warp == 0) {
            id0 = lane < R ? static_cast<int>(ld_peer32(&sh.x_id, lane)) : 0x7fffffff;
            id0 = __reduce_min_sync(0xffffffffu, id0);
            if (lane == 0) out[b] = id0 == 0x7fffffff ? 0 : id0;
        }
        cluster_sync();                        // no CTA leaves while its shared memory may be read
        return;
    }
    Scale sc;
    sc.lmax = lmax;
    sc.c32 = 32.0 * 1.4426950408889634074 / static_cast<double>(T);
    // tokens further from the maximum than kReach * T weigh nothing; without top-k and top-p,
    // neither do those that min-p drops (a little further, for its own exact test)
    float reach = kReach * T;
    if (k <= 0 && tp >= 1.f && mp > 0.f) reach = fminf(reach, (-logf(mp) * 1.0001f + 1e-4f) * T);
    sc.lcut = fmaxf(least, lmax - reach);
    sc.dmax = static_cast<double>(lmax);
    reach = lmax - sc.lcut;
    sc.cbin = reach > 0.f ? static_cast<float>(kBins - 1) / reach : 0.f;
    if (!(sc.cbin < INFINITY)) sc.cbin = 3e38f;
    const double mp52 = static_cast<double>(mp) * static_cast<double>(1ull << mass_bits(V)) + kOne;   // masses from here on are kept by min-p

    // ---- lists
    int turn = 0;                              // buffer of the next gather
    int list_n = 0;
    // Gathers the tokens that `in` accepts (at most kCap over the cluster) and
    // sorts them; `before` is the mass ahead of the list.
    auto gather = [&](u64 before, auto in) __attribute__((always_inline)) {
        if (threadIdx.x == 0) sh.seg_n[turn] = 0;
        __syncthreads();
        each_of([&](float l, int id) { return in(l, id) && within(sc, l); }, [&](float l, int id) {
            const double w = row_mass(table, sc, l);
            const u64 m = mass_of(w);
            if (m == 0) return;
            const int at = atomicAdd(&sh.seg_n[turn], 1);
            if (at >= kCap) return;            // never: the callers count or bound what they accept,
                                               // and the lists are cut at kCap here and below
            sh.seg_key[turn][at] = row_key(l, id);
            sh.seg_mass[turn][at] = m | (w >= mp52 ? kKeep : 0ull);
        });
        cluster_sync();
        // warp r copies CTA r's tokens
        int at = lane < R ? min(static_cast<int>(ld_peer32(&sh.seg_n[turn], lane)), kCap) : 0;
        const int mine = __shfl_sync(0xffffffffu, at, warp & (R - 1));
#pragma unroll
        for (int o = 1; o < R; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += y;
        }
        list_n = min(__shfl_sync(0xffffffffu, at, R - 1), kCap);
        at = __shfl_sync(0xffffffffu, at, warp & (R - 1)) - mine;
        if (warp < R)
            for (int i = lane; i < min(mine, kCap - at); i += 32) {
                const u64 key = ld_peer64(&sh.seg_key[turn][i], warp), m = ld_peer64(&sh.seg_mass[turn][i], warp);
                sh.key[at + i] = key;
                sh.mass[at + i] = m;
            }
        turn ^= 1;
        __syncthreads();
        // rank and mass before of entry threadIdx.x / 2, half of the list in each of two threads
        {
            const int i = threadIdx.x >> 1, half = (list_n + 1) >> 1;
            const int j0 = (threadIdx.x & 1) * half, j1 = min(list_n, j0 + half);
            const u64 key = i < list_n ? sh.key[i] : ~0ull;
            u64 bm = 0;
            int rk = 0;
            if (i < list_n) {
#pragma unroll 4
                for (int j = j0; j < j1; ++j) {
                    const bool ahead = sh.key[j] > key;
                    bm += ahead ? sh.mass[j] & ~kKeep : 0ull;
                    rk += ahead;
                }
            }
            bm += __shfl_xor_sync(0xffffffffu, bm, 1);
            rk += __shfl_xor_sync(0xffffffffu, rk, 1);
            if (i < list_n && (threadIdx.x & 1) == 0) {
                const u64 m = sh.mass[i];
                sh.s_key[rk] = key;
                sh.s_pre[rk] = before + bm;
                sh.s_keep[rk] = (m & kKeep) != 0;
                if (rk == list_n - 1) sh.s_pre[list_n] = before + bm + (m & ~kKeep);
            }
        }
        __syncthreads();
    };
    // Index in the list of the first token whose inclusive mass exceeds `target`.
    auto hit_of = [&](u64 target) __attribute__((always_inline)) {
        for (int i = threadIdx.x; i < list_n; i += kThreads)
            if (sh.s_pre[i] <= target && target < sh.s_pre[i + 1]) sh.hit = i;
        __syncthreads();
        const int i = sh.hit;
        __syncthreads();
        return i;
    };
    // u below 1, so that the target stays below the kept mass
    const double u = fmin(fmax(static_cast<double>(uniforms[b]), 0.0), 1.0 - 1.0 / 16777216.0);
    auto finish = [&](int i) {
        if (rank == 0 && threadIdx.x == 0) out[b] = key_id(sh.s_key[i]);
        cluster_sync();                        // no CTA leaves while its shared memory may be read
    };

    // ---- a small top_k: counts, one list with every token that may be drawn
    if (k > 0 && k <= kCap) {
        each4([&](const float (&l)[4], int) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (within(sc, l[y])) atomicAdd(&sh.h[0][row_bin(sc, l[y])], 1u);
        });
        hist_reduce<R, false>(sh, sh.p0, rank);
        const unsigned int all = sh.p0.cnt[kBins];
        const int bin = choose_bin(sh, sh.p0, true, min(static_cast<unsigned int>(k), all) - 1);
        if (sh.p0.cnt[bin + 1] <= kCap) {
            const float last = kBinBase + bin;
            gather(0, [&](float l, int) { return row_place(sc, l) <= last; });
            u64 z = sh.s_pre[min(k, list_n)];
            if (tp < 1.f) {
                const u64 zp = sh.s_pre[hit_of(static_cast<u64>(static_cast<double>(tp) * static_cast<double>(z))) + 1];
                z = zp < z ? zp : z;
            }
            if (mp > 0.f) {
                for (int i = threadIdx.x; i < list_n; i += kThreads)
                    if (sh.s_keep[i] && (i + 1 == list_n || !sh.s_keep[i + 1])) sh.hit = i;
                __syncthreads();
                const u64 zm = sh.s_pre[sh.hit + 1];
                z = zm < z ? zm : z;
                __syncthreads();
            }
            finish(hit_of(static_cast<u64>(u * static_cast<double>(z))));
            return;
        }
        hist_clear(sh);                        // its last readers passed the sums' second barrier
        __syncthreads();
    }

    // ---- histogram of masses; the row's mass and min-p's.  Bound by shared-memory
    // passes and integer instructions alike: counts are taken for top-k only
    const bool counted = k > 0;
    u64 zm = 0;
    each4([&](const float (&l)[4], int) {
        if (!within(sc, fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])))) return;   // all four weigh nothing
        double m[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) m[y] = row_mass(table, sc, l[y]);
        if (mp > 0.f) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (within(sc, l[y]) && m[y] >= mp52) zm += mass_of(m[y]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
            hist_add(hist, row_bin(sc, l[y]), m[y], within(sc, l[y]), counted);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) zm += __shfl_xor_sync(0xffffffffu, zm, o);
    if (lane == 0) sh.red_b[warp] = zm;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) zm += sh.red_b[w];
        sh.x_zm = zm;
    }
    // a bin's width in powers of two
    const float step = sc.cbin > 0.f ? static_cast<float>(sc.c32 / 32.0 / static_cast<double>(sc.cbin)) : 0.f;
    hist_reduce<R, true>(sh, sh.p0, rank, counted ? 0.f : fmaxf(step, 1e-30f), mass_bits(V));
    {
        u64 m = lane < R ? ld_peer64(&sh.x_zm, lane) : 0ull;
#pragma unroll
        for (int o = R / 2; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        zm = __shfl_sync(0xffffffffu, m, 0);
    }
    int have_lo = 1, have_hi = 0;              // bins that the list holds whole
    unsigned int list_cnt = 0;                 // tokens before the list
    // Index in the list of the first token whose inclusive mass (by_count: count)
    // exceeds `target`; there is one.
    auto find = [&](bool by_count, u64 target) __attribute__((always_inline)) {
        const int bin = choose_bin(sh, sh.p0, by_count, target);
        if (bin < have_lo || bin > have_hi) {
            const unsigned int upto = sh.p0.cnt[bin + 1], inside0 = upto - sh.p0.cnt[bin];
            if (inside0 <= kCap) {
                have_lo = upto <= kCap ? 0 : bin;
                have_hi = bin;
                list_cnt = sh.p0.cnt[have_lo];
                const float from = kBinBase + have_lo, to = kBinBase + bin;
                gather(sh.p0.mass[have_lo], [&](float l, int) { const float x = row_place(sc, l); return x >= from && x <= to; });
            } else {
                have_lo = 1;                   // a list of part of a bin serves no other search
                have_hi = 0;
                // cut the bin into 1024 steps of the distance
                __syncthreads();
                hist_clear(sh);
                __syncthreads();
                auto add = [&](int at, float l) { hist_add(hist, at, row_mass(table, sc, l), true, true); };
                const float place = kBinBase + bin;
                each_of([&](float l, int) { return row_place(sc, l) == place && within(sc, l); },
                        [&](float l, int) { add(row_step(sc, l, place), l); });
                hist_reduce<R, true>(sh, sh.p1, rank);
                u64 before = sh.p0.mass[bin];
                list_cnt = sh.p0.cnt[bin];
                const int step = choose_bin(sh, sh.p1, by_count, target - (by_count ? list_cnt : before));
                before += sh.p1.mass[step];
                list_cnt += sh.p1.cnt[step];
                unsigned int inside = sh.p1.cnt[step + 1] - sh.p1.cnt[step];
                auto in_step = [&](float l, int) {
                    return row_place(sc, l) == place && within(sc, l) && row_step(sc, l, place) == step;
                };
                if (inside <= kCap) {
                    gather(before, in_step);
                    return by_count ? static_cast<int>(target - list_cnt) : hit_of(target);
                }
                // near ties: cut the step by its order keys [k0, k1]
                u64 k1 = 0, k0 = ~0ull;
                each_of(in_step, [&](float l, int id) {
                    if (mass_of(row_mass(table, sc, l)) == 0) return;
                    const u64 key = row_key(l, id);
                    k1 = key > k1 ? key : k1;
                    k0 = key < k0 ? key : k0;
                });
                k1 = warp_max_u64(k1);
                k0 = ~warp_max_u64(~k0);
                if (lane == 0) { sh.red_a[warp] = k1; sh.red_b[warp] = k0; }
                __syncthreads();
                if (threadIdx.x == 0) {
                    for (int w = 1; w < kWarps; ++w) {
                        k1 = sh.red_a[w] > k1 ? sh.red_a[w] : k1;
                        k0 = sh.red_b[w] < k0 ? sh.red_b[w] : k0;
                    }
                    sh.x_k1 = k1;
                    sh.x_k0 = k0;
                }
                cluster_sync();
                k1 = warp_max_u64(lane < R ? ld_peer64(&sh.x_k1, lane) : 0ull);
                k0 = ~warp_max_u64(lane < R ? ~ld_peer64(&sh.x_k0, lane) : 0ull);
                while (inside > kCap) {
                    const int bits = 64 - __clzll(static_cast<long long>(k1 - k0));
                    const int shift = bits > 10 ? bits - 10 : 0;
                    __syncthreads();
                    hist_clear(sh);
                    __syncthreads();
                    each_of([&](float l, int id) { const u64 key = row_key(l, id); return key >= k0 && key <= k1; },
                            [&](float l, int id) { add(static_cast<int>((k1 - row_key(l, id)) >> shift), l); });
                    hist_reduce<R, true>(sh, sh.p1, rank);
                    const int cut = choose_bin(sh, sh.p1, by_count, target - (by_count ? list_cnt : before));
                    before += sh.p1.mass[cut];
                    list_cnt += sh.p1.cnt[cut];
                    inside = sh.p1.cnt[cut + 1] - sh.p1.cnt[cut];
                    const u64 top = k1 - (static_cast<u64>(cut) << shift);
                    const u64 low = top - ((1ull << shift) - 1);
                    k0 = low > k0 && low <= top ? low : k0;
                    k1 = top;
                }
                gather(before, [&](float l, int id) { const u64 key = row_key(l, id); return key >= k0 && key <= k1; });
            }
        }
        return by_count ? static_cast<int>(target - list_cnt) : hit_of(target);
    };
    const u64 s = sh.p0.mass[kBins];
    u64 z = s;
    if (k > 0 && static_cast<unsigned int>(k) < sh.p0.cnt[kBins]) z = sh.s_pre[find(true, static_cast<u64>(k - 1)) + 1];
    if (tp < 1.f) {
        const u64 target = static_cast<u64>(static_cast<double>(tp) * static_cast<double>(z));
        if (target < s) {
            const u64 zp = sh.s_pre[find(false, target) + 1];
            z = zp < z ? zp : z;
        }
    }
    if (mp > 0.f && zm < z) z = zm;
    __syncthreads();
    finish(find(false, static_cast<u64>(u * static_cast<double>(z))));
}

template <int R, bool KEPT>
static int rows_go(const float* logits, int B, int V, const float* temperature, const int32_t* top_k,
                   const float* top_p, const float* min_p, const float* uniforms, int32_t* out, cudaStream_t st) {
    constexpr int most = static_cast<int>(sizeof(RowShared)) + (KEPT ? (kKept + 4) * 4 : 0);
    static PerDevice<int> per_device;          // the attribute's value
    int room = 0;
    cudaError_t e = per_device.get(&room, [&](int, int* out) {
        *out = most;
        return cudaFuncSetAttribute(sample_rows_kernel<R, KEPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(sample_rows_kernel)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(B * R);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(RowShared) + (KEPT ? ((V + R - 1) / R + 4) * sizeof(float) : 0);
    cfg.dynamicSmemBytes = (cfg.dynamicSmemBytes + 15) & ~size_t(15);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = R;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sample_rows_kernel<R, KEPT>, logits, V, temperature, top_k, top_p, min_p,
                                       uniforms, out);
    count_launch();
    if (e != cudaSuccess) return cuda_fail(e, "sample_rows_kernel");
    return LLAMA_OK;
}

template <int R>
static int rows_keep(const float* logits, int B, int V, const float* temperature, const int32_t* top_k,
                     const float* top_p, const float* min_p, const float* uniforms, int32_t* out, cudaStream_t st) {
    if (V <= R * kKept) return rows_go<R, true>(logits, B, V, temperature, top_k, top_p, min_p, uniforms, out, st);
    return rows_go<R, false>(logits, B, V, temperature, top_k, top_p, min_p, uniforms, out, st);
}

int launch_sample_rows(const float* logits, int B, int V, const float* temperature, const int32_t* top_k,
                       const float* top_p, const float* min_p, const float* uniforms, int32_t* out, cudaStream_t st) {
    // the widest clusters whose rows all fit on the GPU at once (two CTAs an SM): 64 rows of
    // 128000 with top-k 33 us on clusters of 4, 45 on 8; 32 rows 24 us on 8
    if (B <= 32) return rows_keep<8>(logits, B, V, temperature, top_k, top_p, min_p, uniforms, out, st);
    if (B <= 64 || V > 2 * kSlice) return rows_keep<4>(logits, B, V, temperature, top_k, top_p, min_p, uniforms, out, st);
    return rows_keep<2>(logits, B, V, temperature, top_k, top_p, min_p, uniforms, out, st);
}

}  // namespace llb
