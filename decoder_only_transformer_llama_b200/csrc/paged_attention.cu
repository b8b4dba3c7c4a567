// Causal attention of each request's new tokens over its pages (Admin Guide
// §8.4, Attention steps 5-7 and the mask NOTE; repeat_kv from the source tour):
//   o = softmax_j(q . K[j] * scale) V[j],  keys j = 0 .. position of the token,
// in one pass over the keys with the running maximum m and sum l of the
// softmax (o, l rescaled by 2^(m - m') when m moves, scores in the log2 domain).
//
// A tile is 16 query rows that share one KV head (16 * n_kv_heads / n_heads
// tokens with their query heads), a unit 32 KB of K and V.  Short steps are
// bound by reading the cache: the units of all tiles form one list, and every
// CTA takes an equal run of it (paged_work.cuh), so each reads the same bytes
// whatever the mix of lengths.  Units arrive by 16-byte asynchronous copies
// with zero fill (each row's page is looked up one unit ahead; rows behind the
// request's last key and pages outside the pool read as zeros) in a ring of
// three.
//
// Measured: 32 tokens over 1000-2000 keys (32 heads of 128, bf16, pages of 16) 133 us,
// 5.8 TB/s; one token over 53000 keys (64/8 heads, fp16) 46 us, 6.0 TB/s in its loop,
// 6 us before it and 6 behind it; 190 keys 7.7 us.  32 KB units three deep with two
// CTAs per SM keep 128 KB in flight on each; TMA boxes would need a map per page
// size and could not zero the rows behind the last key.
//
// 16-bit caches: warp w takes keys 16 w .. 16 w + 15 of a unit for all 16 rows,
// S = Q K^T and O += P V as mma.sync m16n8k16 fragments (a tile of 16 rows is
// far below tcgen05's 128; longer chunks take the kernel of
// paged_attention_tile.cu); the warps' states are merged at the end of a tile.
// fp32 caches: CUDA-core products (no TF32), a thread holding a 2 x 2 block of
// scores and 16 HD / 128 outputs.
//
// A tile split between CTAs: each publishes its unnormalised (o, m, l) and
// counts itself; the last to arrive merges, in CTA order (the same bits from run
// to run; nobody waits), and clears the counter.
#include <type_traits>

#include "common.cuh"
#include "paged.h"
#include "paged_work.cuh"
#include "per_device.cuh"

namespace llb {

namespace {
constexpr int kThreads = 128;
constexpr int kRows = 16;
constexpr int kStages = 3;
constexpr int kMaxCtas = 512;
// Units per CTA below which fewer CTAs run: a split costs a publish and a merge.
constexpr int kMinUnits = 4;

template <typename T> constexpr int kUnitKeys = sizeof(T) == 2 ? 64 : 32;

// Workspace: counters, (m, l) and o of two partial tiles per CTA.
constexpr int kFan = 8;                     // partial results merged at a time
constexpr int kLevels = 3;                  // kFan^3 contributors: every CTA
static_assert(kFan * kFan * kFan >= kMaxCtas && 2 * kLevels * kMaxCtas * sizeof(int) <= kPagedCounters, "merge tree");
constexpr size_t kOffMl = kPagedCounters;
constexpr size_t kOffO = kOffMl + 2ull * kMaxCtas * kRows * sizeof(float2);
constexpr size_t ws_bytes(int hd) { return kOffO + 2ull * kMaxCtas * kRows * hd * sizeof(float); }

// Byte offset of 16-byte chunk `c` of row `row` in a unit's K or V block:
// chunks are permuted within a row so that 8 rows read at one chunk index
// (ldmatrix, or the fp32 score loop's rows two apart) fall into different banks.
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t unit_off(int row, int c) {
    if constexpr (ROW_BYTES == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    else return row * ROW_BYTES + ((c ^ (row & 7)) << 4);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// With zeros in place of the source's bytes unless `ok`.
__device__ __forceinline__ void cp16_if(uint32_t dst, const void* src, bool ok) {
    const int n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, bf16>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A value whose exponent bits are all ones: infinity or NaN.
template <typename T> __device__ __forceinline__ bool not_finite16(uint32_t h) {
    constexpr uint32_t e = std::is_same<T, bf16>::value ? 0x7f80u : 0x7c00u;
    return (h & e) == e;
}
}  // namespace

// Merges the partial results of n <= kFan contributors of a tile, x = first, first
// + stride, ... (contributor x's in slot 2 x, the tile's first one cf's in slot
// 2 cf + 1), in their order.  A thread holds four columns of a row and asks for
// everything it needs at once.  With `out` the rows are finished: row r of the
// tile lies at out + (r >> lrep) * token + (r & (2^lrep - 1)) * HD and sees lim0 +
// (r >> lrep) keys; without it the merged partial result takes the place of the
// first one: a row's threads lie in one warp, which all goes through the loop
// together and has read the first one's (m, l) before one lane overwrites it.
template <typename T, int HD>
__device__ __forceinline__ void merge_tile(float2* part_ml, float* part_o, int cf, int first, int n, int stride, int rows,
                                           T* out, int lrep, long long token, int lim0) {
    auto slot_of = [&](int k) {
        const int x = first + k * stride;
        return static_cast<long long>(2 * x + (x == cf ? 1 : 0)) * kRows;
    };
    static_assert(HD / 4 <= 32 && kThreads % 32 == 0, "a row's threads lie in one warp");
    const int all = rows * (HD / 4);
#pragma unroll 2
    for (int idx = threadIdx.x; (idx & ~31) < all; idx += kThreads) {
        const bool in = idx < all;                // the same number of turns for a whole warp
        const int r = idx / (HD / 4), d = (idx % (HD / 4)) * 4;
        float2 ml[kFan];
        float4 v[kFan];
#pragma unroll
        for (int k = 0; k < kFan; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < n && in) {
                ml[k] = __ldcg(part_ml + slot_of(k) + r);
                v[k] = __ldcg(reinterpret_cast<const float4*>(part_o + (slot_of(k) + r) * HD + d));
            }
        }
        float M = -INFINITY, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kFan; ++k) M = fmaxf(M, ml[k].x);
        const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int k = 0; k < kFan; ++k) {
            if (k >= n) break;
            const float f = ex2(ml[k].x - Ms);
            L += ml[k].y * f;
            o.x = fmaf(v[k].x, f, o.x); o.y = fmaf(v[k].y, f, o.y);
            o.z = fmaf(v[k].z, f, o.z); o.w = fmaf(v[k].w, f, o.w);
        }
        if (!out) {
            __syncwarp();                         // every lane has read the first one's (m, l)
            if (in) *reinterpret_cast<float4*>(part_o + (slot_of(0) + r) * HD + d) = o;
            if (in && d == 0) part_ml[slot_of(0) + r] = make_float2(M, L);
            continue;
        }
        if (!in) continue;
        T* dst = out + (r >> lrep) * token + (r & ((1 << lrep) - 1)) * HD + d;
        const float4 y = lim0 + (r >> lrep) > 0 ? make_float4(o.x / L, o.y / L, o.z / L, o.w / L)
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (sizeof(T) == 2) {
            uint2 w;
            w.x = pack2<T>(y.x, y.y);
            w.y = pack2<T>(y.z, y.w);
            *reinterpret_cast<uint2*>(dst) = w;
        } else {
            *reinterpret_cast<float4*>(dst) = y;
        }
    }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 2) paged_attn_kernel(PagedAttnArgs a, TileShape shape) {
    constexpr bool H16 = sizeof(T) == 2;
    constexpr int KU = kUnitKeys<T>;
    constexpr int ROW = HD * static_cast<int>(sizeof(T));
    constexpr int BLK = KU * ROW;                 // K or V of a unit
    constexpr int CPR = ROW / 16;                 // 16-byte chunks per row
    constexpr int RPP = kThreads / CPR;           // rows one pass of the CTA copies
    constexpr int NPG = KU / 16;                  // most pages of a unit
    // P is rounded to the cache's type for the second product (relative to P at most
    // half a step, of the size of the output's own rounding; l sums it unrounded).
    // fp16 loses relative precision below 2^-14: all weights carry a factor 2^8 there.
    constexpr float kLift = std::is_same<T, f16>::value ? 8.f : 0.f;
    extern __shared__ __align__(128) uint8_t smem[];
    // ring | scratch (16-bit: o of 4 warps x 4 rows; fp32: q, scores) | work list
    constexpr int SCR = H16 ? 4 * 4 * HD * 4 : kRows * HD * 4 + kRows * KU * 4;
    uint8_t* scr = smem + kStages * 2 * BLK;
    long long* cum = reinterpret_cast<long long*>(scr + SCR);
    WorkReq* req = reinterpret_cast<WorkReq*>(cum + a.B + 1);
    __shared__ long long s_scan[2 * kThreads / 32], s_tiles;
    __shared__ float s_m[4][kRows], s_l[4][kRows], s_corr[kRows];
    __shared__ int s_bad, s_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    build_work<kThreads>(a.cu_new, a.seq_lens, a.B, a.T, cap, a.nkv, shape, req, cum, s_scan, &s_tiles, a.status);
    const long long W = cum[a.B];
    // a CTA for every kMinUnits units or every tile, whichever is more
    const long long parts = max((W + kMinUnits - 1) / kMinUnits, min(s_tiles, W));
    const int P = static_cast<int>(parts < gridDim.x ? parts : gridDim.x), c = blockIdx.x;
    if (c >= P) return;
    const long long u0 = run_start(c, W, P), u1 = run_start(c + 1, W, P);
    const int len = static_cast<int>(u1 - u0);
    WorkCur ic = work_at(shape, req, cum, a.B, a.nkv, u0);   // the next unit to copy
    const int rep = a.nh / a.nkv, lrep = 4 - shape.lr;      // 16 rows = 2^lr tokens * rep heads
    const int R = 1 << shape.lr;

    int* counters = static_cast<int*>(a.workspace);
    float2* part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(a.workspace) + kOffMl);
    float* part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kOffO);
    const T* kp = static_cast<const T*>(a.k_pages);
    const T* vp = static_cast<const T*>(a.v_pages);

    // ---- copies: the cursor of the next unit to issue, its tile's last key and its pages
    int pg[NPG], ikend = 0;
    const int32_t* itable = nullptr;
    auto issue_tile = [&]() {
        if (ic.b >= a.B) return;
        const WorkReq r = req[ic.b];
        ikend = min(r.seq, r.seq - r.n + min((ic.tile + 1) << shape.lr, r.n));
        itable = a.block_tables + static_cast<long long>(ic.b) * a.max_pages;
    };
    issue_tile();
    WorkCur cc = ic;                              // the unit at hand
    auto load_pages = [&]() {
#pragma unroll
        for (int i = 0; i < NPG; ++i) {
            const int at = (ic.j * KU + i * 16) >> a.page_shift;
            pg[i] = ic.b < a.B && at < a.max_pages ? __ldg(itable + at) : -1;
        }
    };
    const int ch = tid % CPR, r0 = tid / CPR;     // this thread's 16-byte chunk and first row
    const long long page_elems = static_cast<long long>(HD) << a.page_shift;
    auto issue = [&](int i) {                     // the i-th unit of the run
        const uint32_t base = smem_u32(smem + (i % kStages) * 2 * BLK);
        const int left = ikend - ic.j * KU;       // keys of the unit that exist
        bool inside = true;
        long long off[NPG];                       // elements to this thread's chunk in each 16 rows
#pragma unroll
        for (int x = 0; x < NPG; ++x) {
            inside = inside && static_cast<unsigned>(pg[x]) < static_cast<unsigned>(a.n_pages);
            off[x] = (static_cast<long long>(pg[x]) * a.nkv + ic.g) * page_elems +
                     ((ic.j * KU + x * 16) & ((1 << a.page_shift) - 1)) * HD + ch * (16 / static_cast<int>(sizeof(T)));
        }
        auto group = [&](int p) {                 // offset of the 16 rows that pass p's row lies in
            if constexpr (RPP <= 16) return off[p * RPP / 16];
            else return (r0 & 16) ? off[2 * p + 1] : off[2 * p];
        };
        if (inside && left >= KU) {
#pragma unroll
            for (int p = 0; p < KU / RPP; ++p) {
                const long long o = group(p) + ((p * RPP + r0) & 15) * HD;
                const uint32_t dst = base + unit_off<ROW>(p * RPP + r0, ch);
                cp16(dst, kp + o);
                cp16(dst + BLK, vp + o);
            }
        } else {
            // the request's last unit, or a page outside the pool: rows that do not exist read as zeros
#pragma unroll
            for (int p = 0; p < KU / RPP; ++p) {
                const int row = p * RPP + r0;
                int page = pg[0];
#pragma unroll
                for (int x = 1; x < NPG; ++x) page = (row >> 4) == x ? pg[x] : page;
                const bool known = static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
                const bool ok = row < left && known;
                if (row < left && !known && ch == 0) report_status(a.status, LLAMA_ERR_INVALID_ARG);
                const long long o = ok ? group(p) + (row & 15) * HD : 0;
                const uint32_t dst = base + unit_off<ROW>(row, ch);
                cp16_if(dst, kp + o, ok);
                cp16_if(dst + BLK, vp + o, ok);
            }
        }
        if (++ic.j >= ic.nu) { next_tile(shape, req, a.B, a.nkv, ic); issue_tile(); }
    };
    load_pages();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < len) { issue(i); load_pages(); }
        cp_commit();
    }

    // ---- the tile at hand
    WorkReq rq = {0, 0, 0};
    int t0 = 0, lim0 = 0, kend = 0, rows = 0;     // first token, keys its first and last row see, rows in use
    const float sl2 = a.scale * 1.4426950408889634f;
    // keys that row r of the tile sees (<= 0: none); rows behind the request's last token see none
    auto limit = [&](int r) {
        const int t = t0 + (r >> lrep);
        return t < rq.n ? min(rq.seq, rq.seq - rq.n + t + 1) : 0;
    };
    // 16-bit: lane (g = lane / 4, tq = lane % 4) holds rows g and g + 8
    const int g8 = lane >> 2, tq = lane & 3;
    uint32_t qa[H16 ? HD / 16 : 1][4];
    float m2[2], l2[2], oacc[H16 ? HD / 8 : 1][4];
    int lim2[2];
    // fp32: q in shared memory; this warp's rows 4 warp .. +3 for the softmax,
    // this thread's outputs: rows fr .. fr + FR - 1, columns fc .. fc + 3
    constexpr int CG = HD / 4, RG = kThreads / CG, FR = kRows / RG;
    const int fc = (tid % CG) * 4, fr = (tid / CG) * FR;
    float mf[4], lf[4], of[H16 ? 1 : FR][4];
    float* s_q = reinterpret_cast<float*>(scr);
    float* s_p = s_q + kRows * HD;
    auto start_tile = [&]() {
        rq = req[cc.b];
        t0 = cc.tile << shape.lr;
        lim0 = limit(0);
        kend = min(rq.seq, rq.seq - rq.n + min(t0 + R, rq.n));
        rows = min(kRows, (rq.n - t0) << lrep);
        if (tid == 0) s_bad = 0;
        const T* qb = static_cast<const T*>(a.q);
        auto qrow = [&](int r) {
            return qb + (static_cast<long long>(rq.q0 + t0 + (r >> lrep)) * a.nh + cc.g * rep + (r & (rep - 1))) * HD;
        };
        if constexpr (H16) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = g8 + 8 * x;
                const bool in = t0 + (r >> lrep) < rq.n;
                const T* p = in ? qrow(r) : qb;
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks) {
                    qa[ks][x] = in ? *reinterpret_cast<const uint32_t*>(p + 16 * ks + 2 * tq) : 0u;
                    qa[ks][2 + x] = in ? *reinterpret_cast<const uint32_t*>(p + 16 * ks + 2 * tq + 8) : 0u;
                }
                m2[x] = -INFINITY;
                l2[x] = 0.f;
                lim2[x] = limit(r);
            }
#pragma unroll
            for (int nd = 0; nd < HD / 8; ++nd)
#pragma unroll
                for (int e = 0; e < 4; ++e) oacc[nd][e] = 0.f;
        } else {
            for (int i = tid; i < kRows * (HD / 4); i += kThreads) {
                const int r = i / (HD / 4), ch = i % (HD / 4);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (t0 + (r >> lrep) < rq.n) v = *reinterpret_cast<const float4*>(qrow(r) + ch * 4);
                *reinterpret_cast<float4*>(s_q + r * HD + ((ch ^ ((r >> 1) & 7)) << 2)) = v;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) { mf[i] = -INFINITY; lf[i] = 0.f; }
#pragma unroll
            for (int i = 0; i < FR; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) of[i][e] = 0.f;
        }
    };
    start_tile();
    int seg_j0 = cc.j;                            // first unit of this CTA's part of the tile

    for (int i = 0; i < len; ++i) {
        cp_wait<kStages - 2>();
        __syncthreads();                          // unit i landed; everyone is past unit i - 1
        if (i + kStages - 1 < len) { issue(i + kStages - 1); load_pages(); }
        cp_commit();
        uint8_t* sK = smem + (i % kStages) * 2 * BLK;
        uint8_t* sV = sK + BLK;
        const int key0 = cc.j * KU;
        const bool masked = key0 + KU > lim0;     // some row does not see some key
        if (H16 && masked && kend > lim0) {
            // A key that some rows see and others do not: a weight of 0 times
            // an infinity or NaN of its V would reach the rows that do not see
            // it.  Such values become 0 here and are added at the tile's end.
            const int from = max(0, lim0 - key0);
            for (int x = from * CPR + tid; x < KU * CPR; x += kThreads) {
                uint32_t* p = reinterpret_cast<uint32_t*>(sV + x * 16);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t v = p[w];
                    const bool lo = not_finite16<T>(v & 0xffffu), hi = not_finite16<T>(v >> 16);
                    if (lo || hi) {
                        p[w] = v & ((lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u));
                        s_bad = 1;
                    }
                }
            }
            __syncthreads();
        }
        if constexpr (H16) {
            const uint32_t kb = smem_u32(sK), vb = smem_u32(sV);
            const int mi = lane >> 3, rr = lane & 7;
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) {
                uint32_t b[4];                    // keys 0-7: dims 0-7, 8-15; keys 8-15: dims 0-7, 8-15
                ldsm4(kb + unit_off<ROW>(16 * warp + ((mi >> 1) << 3) + rr, 2 * ks + (mi & 1)), b);
                mma16<T>(sc[0], qa[ks], b[0], b[1]);
                mma16<T>(sc[1], qa[ks], b[2], b[3]);
            }
            uint32_t pa[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int x = 0; x < 2; ++x) {         // rows g8 and g8 + 8
                if (x == 1 && rows <= 8) break;
                float s[4] = {sc[0][2 * x] * sl2, sc[0][2 * x + 1] * sl2, sc[1][2 * x] * sl2, sc[1][2 * x + 1] * sl2};
                if (masked) {
                    const int k0 = key0 + 16 * warp + 2 * tq;
                    if (k0 >= lim2[x]) s[0] = -INFINITY;
                    if (k0 + 1 >= lim2[x]) s[1] = -INFINITY;
                    if (k0 + 8 >= lim2[x]) s[2] = -INFINITY;
                    if (k0 + 9 >= lim2[x]) s[3] = -INFINITY;
                }
                float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m2[x], mx);
                const float ms = mn == -INFINITY ? 0.f : mn;     // no key so far: every weight is 0
                const float corr = ex2(m2[x] - ms);
                float p[4], rs = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) { p[e] = ex2(s[e] - (ms - kLift)); rs += p[e]; }
                l2[x] = l2[x] * corr + rs;        // this lane's keys; summed over the quad at the end
                m2[x] = mn;
                pa[x] = pack2<T>(p[0], p[1]);
                pa[2 + x] = pack2<T>(p[2], p[3]);
                if (__any_sync(0xffffffffu, corr != 1.f)) {      // some row's maximum moved
#pragma unroll
                    for (int nd = 0; nd < HD / 8; ++nd) { oacc[nd][2 * x] *= corr; oacc[nd][2 * x + 1] *= corr; }
                }
            }
#pragma unroll
            for (int np = 0; np < HD / 16; ++np) {
                uint32_t b[4];                    // dims 16 np ..: keys 0-7, 8-15; dims + 8: keys 0-7, 8-15
                ldsm4_t(vb + unit_off<ROW>(16 * warp + ((mi & 1) << 3) + rr, 2 * np + (mi >> 1)), b);
                mma16<T>(oacc[2 * np], pa, b[0], b[1]);
                mma16<T>(oacc[2 * np + 1], pa, b[2], b[3]);
            }
        } else {
            // scores: rows 2 (tid % 8) + {0, 1}, keys 2 (tid / 8) + {0, 1}
            const int sr = (tid & 7) * 2, sk = (tid >> 3) * 2;
            float s[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 4
            for (int ch = 0; ch < HD / 4; ++ch) {
                float4 q4[2], k4[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    q4[x] = *reinterpret_cast<const float4*>(s_q + (sr + x) * HD + ((ch ^ ((sr >> 1) & 7)) << 2));
                    k4[x] = *reinterpret_cast<const float4*>(sK + unit_off<ROW>(sk + x, ch));
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        s[x][y] = fmaf(q4[x].x, k4[y].x, fmaf(q4[x].y, k4[y].y, fmaf(q4[x].z, k4[y].z, fmaf(q4[x].w, k4[y].w, s[x][y]))));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                *reinterpret_cast<float2*>(s_p + (sr + x) * KU + sk) = make_float2(s[x][0] * sl2, s[x][1] * sl2);
            __syncthreads();
            // softmax: rows 4 warp .. + 3, lane = key
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int r = 4 * warp + x;
                const float v = key0 + lane < limit(r) ? s_p[r * KU + lane] : -INFINITY;
                const float mn = fmaxf(mf[x], warp_max(v));
                const float ms = mn == -INFINITY ? 0.f : mn;
                const float p = ex2(v - ms), corr = ex2(mf[x] - ms);
                lf[x] = lf[x] * corr + warp_sum(p);
                mf[x] = mn;
                s_p[r * KU + lane] = p;
                if (lane == 0) s_corr[r] = corr;
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < FR; ++x) {
                const float cr = s_corr[fr + x];
#pragma unroll
                for (int e = 0; e < 4; ++e) of[x][e] *= cr;
            }
            int lims[FR];
#pragma unroll
            for (int x = 0; x < FR; ++x) lims[x] = limit(fr + x) - key0;
#pragma unroll 4
            for (int k = 0; k < KU; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(sV + unit_off<ROW>(k, fc >> 2));
#pragma unroll
                for (int x = 0; x < FR; ++x) {
                    if (masked && k >= lims[x]) continue;        // not 0 times whatever the slot holds
                    const float p = s_p[(fr + x) * KU + k];
                    of[x][0] = fmaf(p, v.x, of[x][0]);
                    of[x][1] = fmaf(p, v.y, of[x][1]);
                    of[x][2] = fmaf(p, v.z, of[x][2]);
                    of[x][3] = fmaf(p, v.w, of[x][3]);
                }
            }
        }
        if (cc.j + 1 < cc.nu && i + 1 < len) { ++cc.j; continue; }

        // ---- end of the tile, or of this CTA's part of it
        const bool whole = seg_j0 == 0 && cc.j + 1 == cc.nu;
        const long long tile_u0 = u0 + i - cc.j;                 // the tile's first unit in the list
        const int cf = whole ? c : run_of(tile_u0, W, P), cl = whole ? c : run_of(tile_u0 + cc.nu - 1, W, P);
        const int slot = 2 * c + (c == cf ? 1 : 0);
        auto out_at = [&](int r) {
            return static_cast<T*>(a.out) +
                   (static_cast<long long>(rq.q0 + t0 + (r >> lrep)) * a.nh + cc.g * rep + (r & (rep - 1))) * HD;
        };
        if constexpr (H16) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l2[x] += __shfl_xor_sync(0xffffffffu, l2[x], 1);
                l2[x] += __shfl_xor_sync(0xffffffffu, l2[x], 2);
                if (tq == 0) { s_m[warp][g8 + 8 * x] = m2[x]; s_l[warp][g8 + 8 * x] = l2[x]; }
            }
            __syncthreads();
            if (tid < kRows) {                    // each row's maximum, sum and the warps' weights
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w][tid]);
                const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float f = ex2(s_m[w][tid] - Ms);
                    L += s_l[w][tid] * f;
                    s_m[w][tid] = f;
                }
                s_l[0][tid] = L;
                if (!whole && tid < rows) part_ml[slot * kRows + tid] = make_float2(M, L);
            }
            float* s_o = reinterpret_cast<float*>(scr);          // [4 warps][4 rows][HD]
            constexpr int CG4 = HD / 4;                          // four columns a thread
            for (int r0 = 0; r0 < rows; r0 += 4) {
                if (r0) __syncthreads();
                if ((g8 >> 2) == ((r0 >> 2) & 1)) {
                    const int x = r0 >> 3;                       // rows g8 or g8 + 8
                    float* d = s_o + (warp * 4 + (g8 & 3)) * HD + 2 * tq;
#pragma unroll
                    for (int nd = 0; nd < HD / 8; ++nd)
                        *reinterpret_cast<float2*>(d + 8 * nd) =
                            x ? make_float2(oacc[nd][2], oacc[nd][3]) : make_float2(oacc[nd][0], oacc[nd][1]);
                }
                __syncthreads();
                const int r = r0 + tid / CG4, d = (tid % CG4) * 4;
                if (tid >= 4 * CG4 || r >= rows) continue;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(s_o + (w * 4 + (r & 3)) * HD + d);
                    const float f = s_m[w][r];
                    o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
                }
                const int lim = limit(r);
                if (s_bad) {                                     // infinities and NaN taken out of V above
                    for (int k = max(max(lim0, 0), seg_j0 * KU); k < min(lim, (cc.j + 1) * KU); ++k) {
                        const int page = a.block_tables[static_cast<long long>(cc.b) * a.max_pages + (k >> a.page_shift)];
                        if (page < 0 || page >= a.n_pages) continue;
                        float v[4];
                        load4_16<T>(vp + (((static_cast<long long>(page) * a.nkv + cc.g) << a.page_shift) +
                                          (k & ((1 << a.page_shift) - 1))) * HD + d, v);
                        if (!(fabsf(v[0]) < INFINITY)) o.x += v[0];
                        if (!(fabsf(v[1]) < INFINITY)) o.y += v[1];
                        if (!(fabsf(v[2]) < INFINITY)) o.z += v[2];
                        if (!(fabsf(v[3]) < INFINITY)) o.w += v[3];
                    }
                }
                if (whole) {
                    const float inv = lim > 0 ? 1.f / s_l[0][r] : 0.f;
                    if (lim <= 0) o = make_float4(0.f, 0.f, 0.f, 0.f);
                    uint2 y;
                    y.x = pack2<T>(o.x * inv, o.y * inv);
                    y.y = pack2<T>(o.z * inv, o.w * inv);
                    *reinterpret_cast<uint2*>(out_at(r) + d) = y;
                } else {
                    *reinterpret_cast<float4*>(part_o + (static_cast<long long>(slot) * kRows + r) * HD + d) = o;
                }
            }
        } else {
            if (lane == 0) {
#pragma unroll
                for (int x = 0; x < 4; ++x) { s_m[0][4 * warp + x] = mf[x]; s_l[0][4 * warp + x] = lf[x]; }
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < FR; ++x) {
                const int r = fr + x;
                if (r >= rows) break;
                if (whole) {
                    const float inv = s_l[0][r];
                    const bool some = limit(r) > 0;
                    *reinterpret_cast<float4*>(out_at(r) + fc) =
                        some ? make_float4(of[x][0] / inv, of[x][1] / inv, of[x][2] / inv, of[x][3] / inv)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
                } else {
                    *reinterpret_cast<float4*>(part_o + (static_cast<long long>(slot) * kRows + r) * HD + fc) =
                        make_float4(of[x][0], of[x][1], of[x][2], of[x][3]);
                    if (fc == 0) part_ml[slot * kRows + r] = make_float2(s_m[0][r], s_l[0][r]);
                }
            }
        }
        if (!whole) {
            // A tree of groups of kFan: the last of a group to arrive merges it and
            // goes on as its first member; one SM alone would read many partial
            // results from L2 too slowly (few tiles over a long cache: 37
            // contributors of 8 rows took 9 us in one go).
            const int n = cl - cf + 1;
            int k = c - cf, stride = 1;
            for (int* level = counters;; level += 2 * kMaxCtas) {
                const int first = k / (kFan * stride) * (kFan * stride);
                const int members = min(kFan, (n - first + stride - 1) / stride);
                const int x = cf + first;
                __threadfence();
                __syncthreads();
                if (tid == 0) {
                    int* counter = level + 2 * x + (first == 0 ? 1 : 0);
                    s_last = atomicAdd(counter, 1) == members - 1;
                    if (s_last) *counter = 0;
                }
                __syncthreads();
                if (!s_last) break;
                __threadfence();
                const bool top = n <= kFan * stride;
                if (top || members > 1)
                    merge_tile<T, HD>(part_ml, part_o, cf, x, members, stride, rows, top ? out_at(0) : nullptr, lrep,
                                      static_cast<long long>(a.nh) * HD, limit(0));
                if (top) break;
                k = first;
                stride *= kFan;
            }
        }
        if (i + 1 < len) {
            __syncthreads();                      // s_m, s_l, s_q and the flags are reused
            if (cc.j + 1 < cc.nu) ++cc.j; else next_tile(shape, req, a.B, a.nkv, cc);
            start_tile();
            seg_j0 = cc.j;
        }
    }
}

// ---------------------------------------------------------------- host side

template <typename T, int HD>
static int attn_go(const PagedAttnArgs& a, cudaStream_t st) {
    constexpr int KU = kUnitKeys<T>;
    constexpr int ring = kStages * 2 * KU * HD * static_cast<int>(sizeof(T));
    constexpr int scr = sizeof(T) == 2 ? 4 * 4 * HD * 4 : kRows * HD * 4 + kRows * KU * 4;
    // the work list's room, in three sizes so that the occupancy is asked once for each
    constexpr int rooms[3] = {64, 256, kPagedMaxRequests};
    const int bucket = a.B <= rooms[0] ? 0 : a.B <= rooms[1] ? 1 : 2;
    auto smem_of = [](int room) { return ring + scr + (room + 1) * 8 + room * static_cast<int>(sizeof(WorkReq)); };
    const int smem = smem_of(rooms[bucket]);
    auto kern = paged_attn_kernel<T, HD>;
    struct Fit { int sms, resident[3]; };
    static PerDevice<Fit> per_device;
    Fit fit;
    const cudaError_t e = per_device.get(&fit, [&](int dev, Fit* f) {
        cudaError_t r = cudaDeviceGetAttribute(&f->sms, cudaDevAttrMultiProcessorCount, dev);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        for (int i = 0; i < 3 && r == cudaSuccess; ++i) {
            int n = 0;
            r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, smem_of(rooms[i]));
            f->resident[i] = n < 1 ? 1 : n;
        }
        return r;
    });
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(paged_attn_kernel)");
    const int rep = a.nh / a.nkv;
    TileShape shape;
    shape.lr = rep == 1 ? 4 : rep == 2 ? 3 : rep == 4 ? 2 : 1;
    shape.lk = KU == 64 ? 6 : 5;
    // one resident wave, and no more CTAs than the step can have units
    const long long cap = ((static_cast<long long>(a.max_pages) << a.page_shift) + KU - 1) / KU;
    long long grid = static_cast<long long>(fit.sms) * fit.resident[bucket];
    if (grid > kMaxCtas) grid = kMaxCtas;
    const long long most = static_cast<long long>(a.T) * a.nkv * cap;
    if (grid > most) grid = most;
    kern<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a, shape);
    LLB_CHECK_LAUNCH("paged_attn_kernel");
    return LLAMA_OK;
}

template <typename T>
static int attn_hd(const PagedAttnArgs& a, cudaStream_t st) {
    if (a.hd == 32) return attn_go<T, 32>(a, st);
    if (a.hd == 64) return attn_go<T, 64>(a, st);
    return attn_go<T, 128>(a, st);
}

// A call takes the tile kernel when the longest chunk's rows per KV head fill
// more than one 16-row tile (16-bit caches, head_dim 64 or 128).  Measured both
// ways, 8 KV heads, head_dim 128, tile kernel / 16-row kernel, us: 8 tokens of 4
// heads each, 1 request over 300 keys 14 / 19, over 4000 23 / 32, 16 requests over
// 4000 71 / 88; 64 tokens 17 / 25, 38 / 52, 95 / 567.  At 16 rows the 16-row
// kernel is the faster one where there is much to read (4 tokens, 16 requests
// over 4000 keys: 69 / 59), the slower one where there is little (15 / 22).
static bool tile_shape(int nh, int nkv, int hd, int dtype, int max_new) {
    return dtype != LLAMA_F32 && hd != 32 && static_cast<long long>(max_new) * (nh / nkv) > kRows;
}

size_t paged_attention_ws(int nh, int nkv, int hd, int dtype, int max_new) {
    size_t n = ws_bytes(hd);
    if (tile_shape(nh, nkv, hd, dtype, max_new)) {
        const size_t t = paged_attention_tile_ws(hd);
        n = t > n ? t : n;
    }
    return (n + 255) & ~size_t(255);
}

int launch_paged_attention(const PagedAttnArgs& a, int dtype, cudaStream_t st) {
    // the tile kernel scales after its row maximum, which needs a positive factor
    if (tile_shape(a.nh, a.nkv, a.hd, dtype, a.max_new) && a.scale > 0.f) return launch_paged_attention_tile(a, dtype, st);
    if (dtype == LLAMA_BF16) return attn_hd<bf16>(a, st);
    if (dtype == LLAMA_F16) return attn_hd<f16>(a, st);
    return attn_hd<float>(a, st);
}

}  // namespace llb
