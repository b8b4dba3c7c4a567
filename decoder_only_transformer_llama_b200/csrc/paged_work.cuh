// The work list of one paged-attention call, cut into equal runs.
//
// Request b with n new tokens over a context of ctx cached ones holds, for
// each of its nkv KV heads, ceil(n / R) tiles of R = 2^lr tokens (with their
// n_heads / n_kv_heads query heads each); tile i attends keys 0 .. ctx +
// min((i + 1) R, n) - 1, i.e. units_of(i) units of K = 2^lk keys.  Units are
// numbered by (request, head, tile, unit); CTA c of P takes the run [c W / P,
// (c + 1) W / P), whatever the mix of lengths, and splits a tile between CTAs
// where its run starts or ends inside it.  Where a split costs more than a tile's
// few units, run_bound moves such a boundary to the nearer end of the tile.
#pragma once

#include "common.cuh"

namespace llb {

struct TileShape {
    int lr, lk;   // log2 of the tokens per tile and of the keys per unit
};

// Units of tiles 0 .. m-1, each with all its R tokens: the sum over i = 1 .. m
// of ceil((ctx + i R) / K).
__host__ __device__ __forceinline__ long long tiles_units(TileShape s, long long ctx, long long m) {
    if (s.lr >= s.lk) {
        const long long c = (ctx + (1LL << s.lk) - 1) >> s.lk;
        return m * c + (m * (m + 1) / 2 << (s.lr - s.lk));
    }
    // K = 2^d R: ceil((ctx + i R) / K) = ceil((c + i) / 2^d) with c = ceil(ctx / R),
    // and the sum of ceil(j / 2^d) over j = 1 .. x, x = 2^d q + r, is
    // 2^d q (q + 1) / 2 + r (q + 1)
    const int d = s.lk - s.lr;
    const long long c = (ctx + (1LL << s.lr) - 1) >> s.lr;
    const long long x1 = c + m, q1 = x1 >> d, r1 = x1 & ((1LL << d) - 1);
    const long long q0 = c >> d, r0 = c & ((1LL << d) - 1);
    return (q1 * (q1 + 1) / 2 << d) + r1 * (q1 + 1) - (q0 * (q0 + 1) / 2 << d) - r0 * (q0 + 1);
}
__host__ __device__ __forceinline__ int tiles_of(TileShape s, int n) { return (n + (1 << s.lr) - 1) >> s.lr; }
// Units of tile i of a request with n >= 1 new tokens.
__host__ __device__ __forceinline__ int units_of(TileShape s, int ctx, int n, int i) {
    const long long end = (static_cast<long long>(i) + 1) << s.lr;
    return static_cast<int>((ctx + (end < n ? end : n) + (1LL << s.lk) - 1) >> s.lk);
}
// Units of one KV head of a request (0 without new tokens).
__host__ __device__ __forceinline__ long long request_units(TileShape s, int ctx, int n) {
    if (n <= 0) return 0;
    const int t = tiles_of(s, n);
    return tiles_units(s, ctx, t - 1) + units_of(s, ctx, n, t - 1);
}
// The tile that holds unit u of a request's head.
__host__ __device__ __forceinline__ int tile_at(TileShape s, int ctx, int n, long long u) {
    int lo = 0, hi = tiles_of(s, n) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tiles_units(s, ctx, mid) <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// (32-bit divisions where the products fit: a 64-bit one takes about 100 instructions)
__host__ __device__ __forceinline__ long long run_start(long long c, long long W, long long P) {
    const long long x = c * W;
    if (x <= 0xffffffffLL) return static_cast<uint32_t>(x) / static_cast<uint32_t>(P);
    return x / P;
}
// The run that holds unit u.
__host__ __device__ __forceinline__ int run_of(long long u, long long W, long long P) {
    const long long x = (u + 1) * P - 1;
    if (x <= 0xffffffffLL && W <= 0xffffffffLL) return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(W));
    return static_cast<int>(x / W);
}

// One request as the kernels hold it in shared memory.
struct WorkReq {
    int q0, n, seq;   // first packed row, new tokens (0: nothing to do), tokens in the cache
};

// A place in the work list, the same in every thread that holds one.
struct WorkCur {
    int b, g, tile, j, nu;   // request, KV head, tile, unit of it and the tile's units
};

__host__ __device__ __forceinline__ int ctx_of(const WorkReq& r) { return r.seq > r.n ? r.seq - r.n : 0; }

__host__ __device__ __forceinline__ WorkCur work_at(TileShape s, const WorkReq* req, const long long* cum, int B, int nkv,
                                           long long u) {
    int lo = 0, hi = B - 1;          // the last request with cum <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const WorkReq r = req[lo];
    const long long per = request_units(s, ctx_of(r), r.n);
    const long long rem = u - cum[lo];
    WorkCur c;
    c.b = lo;
    c.g = rem <= 0xffffffffLL && per <= 0xffffffffLL ? static_cast<uint32_t>(rem) / static_cast<uint32_t>(per)
                                                     : static_cast<int>(rem / per);
    const long long v = rem - c.g * per;
    c.tile = tile_at(s, ctx_of(r), r.n, v);
    c.j = static_cast<int>(v - tiles_units(s, ctx_of(r), c.tile));
    c.nu = units_of(s, ctx_of(r), r.n, c.tile);
    return c;
}

// The first unit of the tile after c's (b == B behind the last one).
__host__ __device__ __forceinline__ void next_tile(TileShape s, const WorkReq* req, int B, int nkv, WorkCur& c) {
    c.j = 0;
    if (++c.tile >= tiles_of(s, req[c.b].n)) {
        c.tile = 0;
        if (++c.g >= nkv) {
            c.g = 0;
            do { ++c.b; } while (c.b < B && req[c.b].n <= 0);
            if (c.b >= B) return;
        }
    }
    const WorkReq r = req[c.b];
    c.nu = units_of(s, ctx_of(r), r.n, c.tile);
}

// The run boundary at unit u (0 .. W), moved to the nearer end of its tile if
// that has at most `most` units, with the place it lies at (undefined at W).
__host__ __device__ __forceinline__ long long run_bound(TileShape s, const WorkReq* req, const long long* cum, int B,
                                                        int nkv, long long u, int most, WorkCur& at) {
    if (u >= cum[B]) return cum[B];
    at = work_at(s, req, cum, B, nkv, u);
    if (at.j == 0 || at.nu > most) return u;
    if (2 * at.j < at.nu) {
        u -= at.j;
        at.j = 0;
    } else {
        u += at.nu - at.j;
        next_tile(s, req, B, nkv, at);
    }
    return u;
}

#ifdef __CUDACC__
// Fills req[0 .. B) and cum[0 .. B] (units before each request) from the
// call's offsets and lengths, with the checks of the entry point; CTA 0
// reports.  All NT threads of the CTA; scratch: 2 NT / 32 values.  *tiles = the
// tiles of all requests and heads.
template <int NT>
__device__ __forceinline__ void build_work(const int32_t* cu, const int32_t* seq_lens, int B, int T, long long cap,
                                           int nkv, TileShape shape, WorkReq* req, long long* cum, long long* scratch,
                                           long long* tiles, int* status) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (B + NT - 1) / NT;
    const int b0 = threadIdx.x * per;
    long long mine = 0, my_tiles = 0;
    for (int b = b0; b < b0 + per && b < B; ++b) {
        const int q0 = cu[b], q1 = cu[b + 1];
        int seq = seq_lens[b], n = q1 - q0;
        if (q0 < 0 || q1 < q0 || q1 > T) {
            n = 0;
            if (blockIdx.x == 0) report_status(status, LLAMA_ERR_INVALID_ARG);
        }
        if (seq < 0 || seq > cap) {
            if (blockIdx.x == 0 && n > 0) report_status(status, LLAMA_ERR_CAPACITY);
            seq = seq < 0 ? 0 : static_cast<int>(cap);
        }
        req[b] = {q0, n, seq};
        mine += request_units(shape, seq > n ? seq - n : 0, n) * nkv;
        my_tiles += static_cast<long long>(tiles_of(shape, n)) * nkv;
        cum[b + 1] = mine;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) my_tiles += __shfl_xor_sync(0xffffffffu, my_tiles, o);
    if (lane == 31) { scratch[warp] = incl; scratch[NT / 32 + warp] = my_tiles; }
    __syncthreads();
    long long before = incl - mine;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    for (int b = b0; b < b0 + per && b < B; ++b) cum[b + 1] += before;
    if (threadIdx.x == 0) {
        cum[0] = 0;
        long long t = 0;
        for (int w = 0; w < NT / 32; ++w) t += scratch[NT / 32 + w];
        *tiles = t;
    }
    __syncthreads();
}

#endif

}  // namespace llb
