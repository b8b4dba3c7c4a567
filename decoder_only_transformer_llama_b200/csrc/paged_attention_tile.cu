// Paged attention of longer chunks on the 5th-generation tensor cores (the
// same operator as paged_attention.cu, for 16-bit caches and head_dim 64 or
// 128): o = softmax_j(q . K[j] * scale) V[j], keys j = 0 .. position.
//
// A tile is 256 query rows that share one KV head (256 n_kv_heads / n_heads
// tokens with their query heads), as two sub-tiles of 128 rows, the lanes of
// TMEM; a unit is 128 keys.  The units of all tiles form one list of which
// each CTA (one per SM) takes an equal run (paged_work.cuh).  Per unit and
// sub-tile t:
//   S_t = Q_t K^T  tcgen05, 128 x 128 over head_dim, from swizzled TMA tiles
//   softmax        one thread per row: scores by tcgen05.ld, running maximum m
//                  and sum l in registers in the log2 domain, P = 2^(s - m)
//                  rounded to 16 bits over the first half of S_t's columns
//   O_t += P_t V   tcgen05 with P_t from TMEM and V read MN-major from its tile
// The two sub-tiles alternate on the tensor core: while one's softmax runs,
// the other's products do.  MMAs of one thread run in order, so S_t of the next
// unit may overwrite P_t once its product is issued.  m moves only when a unit
// raises it by more than 8 (a factor 256): then O_t is rescaled in TMEM.
//
// K and V tiles come by TMA, one box per page (64 columns x min(page, 128)
// rows); pages behind the keys or outside the pool are read at a coordinate
// behind the pool, which fills zeros.
//
// Warps: 0-3 and 4-7 softmax and epilogue of sub-tiles 0 and 1, 8 MMA issuer and
// TMEM owner (S0 | S1 | O0 | O1, 512 columns), 9 TMA producer.  Every wait is
// bounded.  A tile split between CTAs is published, counted and merged per
// sub-tile by the last to arrive, in CTA order.
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "paged.h"
#include "paged_work.cuh"

namespace llb {

namespace {
constexpr int kThreads = 320;
constexpr int kRows = 256;
constexpr int kKeys = 128;
constexpr int kBox = 128 * 128;             // 128 rows of 64 16-bit values
constexpr int kMaxCtas = 160;
constexpr int kMinUnits = 2;
constexpr int kMaxSlots = 8;
constexpr uint32_t kColS = 0, kColO = 256;  // S_t at kColS + 128 t, O_t at kColO + 128 t

constexpr size_t kOffMl = 4096;             // counters: two per CTA
constexpr size_t kOffO = kOffMl + 2ull * kMaxCtas * kRows * sizeof(float2);
constexpr size_t ws_bytes(int hd) { return kOffO + 2ull * kMaxCtas * kRows * hd * sizeof(float); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc]: A's 16-bit values two to a column, K-major.
__device__ __forceinline__ void tc_mma_16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(acc) : "memory");
}
template <typename T> __device__ __forceinline__ bool not_finite16(uint32_t h) {
    constexpr uint32_t e = std::is_same<T, bf16>::value ? 0x7f80u : 0x7c00u;
    return (h & e) == e;
}

// A part of one tile that a CTA works on: units c.j .. c.j + len - 1.
struct Segment {
    WorkCur c;
    int len;
};
}  // namespace

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_tile_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                       const __grid_constant__ CUtensorMap mapV, PagedAttnArgs a, TileShape shape, int nslots) {
    constexpr int NB = HD / 64;                    // boxes per tile
    constexpr int TILE = NB * kBox;                // a [128][HD] tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;                            // 2 tiles
    uint8_t* ring = smem + 2 * TILE;               // K, V, K, V, ...
    long long* cum = reinterpret_cast<long long*>(ring + nslots * TILE);
    WorkReq* req = reinterpret_cast<WorkReq*>(cum + a.B + 1);
    __shared__ uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
    __shared__ uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], mdone;
    __shared__ long long s_scan[2 * kThreads / 32], s_tiles;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_fail, s_bad, s_last[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    build_work<kThreads>(a.cu_new, a.seq_lens, a.B, a.T, cap, a.nkv, shape, req, cum, s_scan, &s_tiles, a.status);
    const long long W = cum[a.B];
    // a CTA for every kMinUnits units or every tile, whichever is more
    const long long parts = max((W + kMinUnits - 1) / kMinUnits, min(s_tiles, W));
    const int P = static_cast<int>(parts < gridDim.x ? parts : gridDim.x), cta = blockIdx.x;
    if (cta >= P) return;                          // the whole CTA, before any barrier or TMEM
    const long long u0 = run_start(cta, W, P), u1 = run_start(cta + 1, W, P);
    const int rep = a.nh / a.nkv, lrep = 8 - shape.lr;
    const int half = 128 >> lrep;                  // tokens of a sub-tile

    if (tid == 0) {
        for (int i = 0; i < nslots; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int t = 0; t < 2; ++t) { mbar_init(&s_full[t], 1); mbar_init(&p_full[t], 128); mbar_init(&o_full[t], 1); }
        mbar_init(&mdone, 1);
        s_fail = 0;
        s_bad = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mapQ);
        tma_prefetch_desc(&mapK);
        tma_prefetch_desc(&mapV);
    }
    if (warp == 8) { tmem_alloc(&tmem_slot, 512); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // every role walks the same segments
    auto first_segment = [&]() {
        Segment s;
        s.c = work_at(shape, req, cum, a.B, a.nkv, u0);
        s.len = static_cast<int>(min(static_cast<long long>(s.c.nu - s.c.j), u1 - u0));
        return s;
    };
    auto next_segment = [&](Segment& s, long long& left) {     // left: units behind this segment
        left -= s.len;
        if (left <= 0) return false;
        next_tile(shape, req, a.B, a.nkv, s.c);
        s.len = static_cast<int>(min(static_cast<long long>(s.c.nu), left));
        return true;
    };
    auto two_halves = [&](const Segment& s) { return req[s.c.b].n - (s.c.tile << shape.lr) > half; };

    int issued = 0;                                // producer: ring slots filled
    int n_q = 0;                                   // and Q tiles asked for
    if (warp == 9) {
        // ---------------- TMA producer: lane p brings page p of a unit
        Segment sg = first_segment();
        long long left = u1 - u0;
        int slot = 0, nseg = 0;
        uint32_t empty_phase = 1;
        bool ok = true;
        const int npg = a.page_shift >= 7 ? 1 : kKeys >> a.page_shift;
        const int prow = kKeys / npg;              // rows per box
        const int none = a.n_pages * a.nkv;        // behind the pool
        do {
            const WorkReq r = req[sg.c.b];
            const int t0 = sg.c.tile << shape.lr;
            const bool two = two_halves(sg);
            ok = __all_sync(0xffffffffu, mbar_wait(&q_empty, (nseg & 1) ^ 1));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&q_full, (two ? 2 : 1) * TILE);
                for (int t = 0; t < (two ? 2 : 1); ++t)
                    for (int x = 0; x < NB; ++x)
                        tma_load_3d(sQ + t * TILE + x * kBox, &mapQ, 64 * x, sg.c.g * rep, r.q0 + t0 + t * half, &q_full);
            }
            ++n_q;
            const int tok_end = min(t0 + (1 << shape.lr), r.n);
            const int kend = min(r.seq, r.seq - r.n + tok_end);
            auto page_of = [&](int j) {            // this lane's page of unit j: a tensor coordinate
                const long long key = static_cast<long long>(j) * kKeys + lane * prow;
                if (lane >= npg || key >= kend) return none;
                const int page = __ldg(a.block_tables + static_cast<long long>(sg.c.b) * a.max_pages + (key >> a.page_shift));
                if (page < 0 || page >= a.n_pages) {
                    report_status(a.status, LLAMA_ERR_INVALID_ARG);
                    return none;
                }
                return page * a.nkv + sg.c.g;
            };
            int z = page_of(sg.c.j);
            for (int j = sg.c.j; ok && j < sg.c.j + sg.len; ++j) {
                const int zn = j + 1 < sg.c.j + sg.len ? page_of(j + 1) : none;
                const int y = a.page_shift > 7 ? (j * kKeys) & ((1 << a.page_shift) - 1) : 0;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[slot], empty_phase));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], TILE);
                    __syncwarp();
                    if (lane < npg)
                        for (int x = 0; x < NB; ++x)
                            tma_load_3d(ring + slot * TILE + x * kBox + lane * prow * 128, kv ? &mapV : &mapK, 64 * x, y, z,
                                        &kv_full[slot]);
                    ++issued;
                    if (++slot == nslots) { slot = 0; empty_phase ^= 1; }
                }
                z = zn;
            }
            ++nseg;
        } while (ok && next_segment(sg, left));
        if (!ok && lane == 0) atomicExch(&s_fail, 1);
    } else if (warp == 8 && lane == 0) {
        // ---------------- MMA issuer
        constexpr uint32_t idesc_s = idesc_16_f32<T>(128, kKeys);
        constexpr uint32_t idesc_o = idesc_16_f32_bmn<T>(128, HD);
        Segment sg = first_segment();
        long long left = u1 - u0;
        int slot = 0, nseg = 0;
        uint32_t full_phase = 0, p_phase[2] = {0, 0};
        bool ok = true;
        const uint32_t q0 = smem_u32(sQ), r0 = smem_u32(ring);
        auto advance = [&]() { if (++slot == nslots) { slot = 0; full_phase ^= 1; } };
        auto scores = [&](int t, int kslot) {
            const uint32_t qb = q0 + t * TILE, kb = r0 + kslot * TILE;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kBox + (kk & 3) * 32;
                tc_mma_16(tmem + kColS + 128 * t, smem_desc_k_sw128(qb + off), smem_desc_k_sw128(kb + off), idesc_s, kk > 0);
            }
            tc_commit(&s_full[t]);
        };
        do {
            const int nt = two_halves(sg) ? 2 : 1;
            ok = mbar_wait(&q_full, nseg & 1) && mbar_wait(&kv_full[slot], full_phase);
            if (!ok) break;
            tc_fence_after();
            for (int t = 0; t < nt; ++t) scores(t, slot);
            tc_commit(&kv_empty[slot]);
            if (sg.len == 1) tc_commit(&q_empty);
            advance();
            for (int i = 0; ok && i < sg.len; ++i) {
                ok = mbar_wait(&kv_full[slot], full_phase);          // V of this unit
                if (!ok) break;
                const int vslot = slot;
                advance();
                const int kslot = slot;                              // K of the next one
                const bool more = i + 1 < sg.len;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= nt || !ok) break;
                    ok = mbar_wait(&p_full[t], p_phase[t]);
                    if (!ok) break;
                    p_phase[t] ^= 1;
                    tc_fence_after();
                    const uint32_t vb = r0 + vslot * TILE;
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        tc_mma_16_ts(tmem + kColO + 128 * t, tmem + kColS + 128 * t + 8 * kk,
                                     smem_desc_mn_sw128(vb + kk * 16 * 128, kBox), idesc_o, i > 0 || kk > 0);
                    tc_commit(&o_full[t]);
                    if (more) {
                        if (t == 0) ok = mbar_wait(&kv_full[kslot], full_phase);
                        if (!ok) break;
                        scores(t, kslot);
                    }
                }
                if (!ok) break;
                tc_commit(&kv_empty[vslot]);
                if (more) {
                    tc_commit(&kv_empty[kslot]);
                    if (i + 2 == sg.len) tc_commit(&q_empty);
                    advance();
                }
            }
            ++nseg;
        } while (ok && next_segment(sg, left));
        if (!ok) atomicExch(&s_fail, 1);
        tc_commit(&mdone);                         // every MMA has finished before TMEM is freed
        if (!mbar_wait(&mdone, 0)) atomicExch(&s_fail, 1);
    } else if (warp < 8) {
        // ---------------- softmax and epilogue: thread = row r of sub-tile t
        const int t = warp >> 2;
        const int r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t colS = tmem + lanes + kColS + 128 * t, colO = tmem + lanes + kColO + 128 * t;
        const float sl2 = a.scale * 1.4426950408889634f;
        int* counters = static_cast<int*>(a.workspace);
        float2* part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(a.workspace) + kOffMl);
        float4* part_o = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.workspace) + kOffO);
        Segment sg = first_segment();
        long long left = u1 - u0;
        long long done = 0;                        // units of earlier segments
        // this half's own barriers count the units it took part in; the ring's
        // V slots (watched by sub-tile 0 only) count all
        uint32_t ph = 0;
        int vslot = 1 % nslots;
        uint32_t v_phase = 0;
        bool stop = false;                         // the same in the 128 threads of this half
        do {
            const WorkReq rq = req[sg.c.b];
            const int t0 = sg.c.tile << shape.lr;
            const bool active = t == 0 || two_halves(sg);
            const int tok = t0 + t * half + (r >> lrep);
            const bool live = tok < rq.n;
            const int lim = live ? min(rq.seq, rq.seq - rq.n + tok + 1) : 0;   // keys this row sees
            const int lim0 = min(rq.seq, rq.seq - rq.n + t0 + 1);              // and the tile's first row
            if (active) {
                float m = -INFINITY, l = 0.f;
                for (int i = 0; i < sg.len; ++i) {
                    const int key0 = (sg.c.j + i) * kKeys;
                    bool ok = mbar_wait(&s_full[t], ph);
                    const bool masked = key0 + kKeys > lim0;
                    if (t == 0 && masked) ok = ok && mbar_wait(&kv_full[vslot], v_phase);
                    if (named_any(1 + t, 128, !ok || *reinterpret_cast<volatile int*>(&s_fail) != 0)) { stop = true; break; }
                    tc_fence_after();
                    if (t == 0 && masked) {
                        // V values that some rows must not see: an infinity or
                        // NaN times a weight of 0 would reach them.  They become
                        // 0 here and are added to the rows that see them at the end.
                        const int from = max(0, lim0 - key0);
                        bool found = false;
                        for (int x = from * 8 * NB + r; x < kKeys * 8 * NB; x += 128) {
                            const int row = x / (8 * NB), ch = x % (8 * NB);
                            uint4* p = reinterpret_cast<uint4*>(ring + vslot * TILE + (ch >> 3) * kBox + row * 128 + (ch & 7) * 16);
                            uint4 v = *p;
                            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
                            bool hit = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const bool lo = not_finite16<T>(w[e] & 0xffffu), hi = not_finite16<T>(w[e] >> 16);
                                if (lo) w[e] &= 0xffff0000u;
                                if (hi) w[e] &= 0x0000ffffu;
                                hit = hit || lo || hi;
                            }
                            if (hit) { *p = v; found = true; }
                        }
                        if (found) *reinterpret_cast<volatile int*>(&s_bad) = 1;   // for the rest of the run
                        fence_proxy_async_smem();
                    }
                    float s[kKeys];
#pragma unroll
                    for (int x = 0; x < kKeys; x += 32) tmem_ld_32x32b_x32(colS + x, *reinterpret_cast<float(*)[32]>(s + x));
                    tc_wait_ld();
                    if (masked) {
                        const int lc = lim - key0;
#pragma unroll
                        for (int x = 0; x < kKeys; ++x) s[x] = x < lc ? s[x] : -INFINITY;
                    }
                    float mx = s[0];
#pragma unroll
                    for (int x = 1; x < kKeys; ++x) mx = fmaxf(mx, s[x]);
                    mx *= sl2;
                    bool rescale = false;
                    float corr = 1.f;
                    if (mx > m + 8.f || m == -INFINITY) {
                        rescale = i > 0 && mx > m;
                        corr = m == -INFINITY ? 0.f : ex2(m - mx);
                        m = mx;
                    }
                    const float ms = m == -INFINITY ? 0.f : m;       // no key so far: every weight is 0
                    float sum0 = 0.f, sum1 = 0.f;
                    uint32_t p[kKeys / 2];
#pragma unroll
                    for (int x = 0; x < kKeys; x += 2) {
                        const float e0 = ex2(fmaf(s[x], sl2, -ms)), e1 = ex2(fmaf(s[x + 1], sl2, -ms));
                        sum0 += e0;
                        sum1 += e1;
                        p[x / 2] = pack2<T>(e0, e1);
                    }
                    l = l * corr + (sum0 + sum1);
#pragma unroll
                    for (int x = 0; x < kKeys / 2; x += 32) {
                        float f[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(p[x + e]);
                        tmem_st_32x32b_x32(colS + x, f);
                    }
                    if (__any_sync(0xffffffffu, rescale)) {
                        // the previous product has to have finished with O
                        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[t], ph ^ 1));
                        tc_fence_after();
                        if (ok) {
#pragma unroll 1
                            for (int x = 0; x < HD; x += 32) {
                                float o[32];
                                tmem_ld_32x32b_x32(colO + x, o);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= corr;
                                tmem_st_32x32b_x32(colO + x, o);
                            }
                        } else if (lane == 0) {
                            atomicExch(&s_fail, 1);                  // seen by all at the next unit or the end
                        }
                    }
                    tc_wait_st();
                    tc_fence_before();
                    mbar_arrive(&p_full[t]);
                    ph ^= 1;
                    vslot += 2;
                    if (vslot >= nslots) { vslot -= nslots; v_phase ^= 1; }
                }
                if (stop) break;
                // ---- end of the tile, or of this CTA's part of it: O holds every unit
                const bool ok = mbar_wait(&o_full[t], ph ^ 1);
                if (named_any(1 + t, 128, !ok || *reinterpret_cast<volatile int*>(&s_fail) != 0)) { stop = true; break; }
                tc_fence_after();
                const bool whole = sg.c.j == 0 && sg.len == sg.c.nu;
                const long long tile_u0 = u0 + done - sg.c.j;
                const int cf = whole ? cta : run_of(tile_u0, W, P), cl = whole ? cta : run_of(tile_u0 + sg.c.nu - 1, W, P);
                const bool bad = *reinterpret_cast<volatile int*>(&s_bad) != 0;
                const int row = t * 128 + r;
                T* dst = static_cast<T*>(a.out) +
                         (static_cast<long long>(rq.q0 + tok) * a.nh + sg.c.g * rep + (r & (rep - 1))) * HD;
                const float inv = lim > 0 ? 1.f / l : 0.f;
                const long long base = static_cast<long long>(2 * cta + (cta == cf ? 1 : 0)) * kRows;
                if (!whole && live) part_ml[base + row] = make_float2(m, l);
#pragma unroll 1
                for (int x = 0; x < HD; x += 32) {
                    float o[32];
                    tmem_ld_32x32b_x32(colO + x, o);
                    tc_wait_ld();
                    if (!live) continue;
                    if (bad) {
                        for (int k = max(lim0 > 0 ? lim0 : 0, sg.c.j * kKeys); k < min(lim, (sg.c.j + sg.len) * kKeys); ++k) {
                            const int page = a.block_tables[static_cast<long long>(sg.c.b) * a.max_pages + (k >> a.page_shift)];
                            if (page < 0 || page >= a.n_pages) continue;
                            const T* v = static_cast<const T*>(a.v_pages) +
                                         (((static_cast<long long>(page) * a.nkv + sg.c.g) << a.page_shift) +
                                          (k & ((1 << a.page_shift) - 1))) * HD + x;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float f = to_f32<T>(v[e]);
                                if (!(fabsf(f) < INFINITY)) o[e] += f;
                            }
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = lim > 0 ? o[e] * inv : 0.f;
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint4 w;
                            w.x = pack2<T>(o[8 * v], o[8 * v + 1]);
                            w.y = pack2<T>(o[8 * v + 2], o[8 * v + 3]);
                            w.z = pack2<T>(o[8 * v + 4], o[8 * v + 5]);
                            w.w = pack2<T>(o[8 * v + 6], o[8 * v + 7]);
                            reinterpret_cast<uint4*>(dst + x)[v] = w;
                        }
                    } else {
                        // four columns of all rows side by side
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            part_o[base * (HD / 4) + static_cast<long long>(x / 4 + v) * kRows + row] =
                                make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    }
                }
                if (!whole) {
                    __threadfence();
                    named_sync(1 + t, 128);
                    if (r == 0) {
                        const int seen = atomicAdd(counters + 2 * cf + t, 1);
                        s_last[t] = seen == cl - cf;
                        if (s_last[t]) counters[2 * cf + t] = 0;
                    }
                    named_sync(1 + t, 128);
                    if (s_last[t] && live) {
                        __threadfence();
                        float M = -INFINITY, L = 0.f;
                        for (int x = cf; x <= cl; ++x)
                            M = fmaxf(M, __ldcg(&part_ml[static_cast<long long>(2 * x + (x == cf)) * kRows + row].x));
                        const float Ms = M == -INFINITY ? 0.f : M;
                        for (int x = cf; x <= cl; ++x) {
                            const float2 ml = __ldcg(part_ml + static_cast<long long>(2 * x + (x == cf)) * kRows + row);
                            L += ml.y * ex2(ml.x - Ms);
                        }
#pragma unroll 1
                        for (int d = 0; d < HD / 4; d += 4) {
                            float4 o[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                            for (int x = cf; x <= cl; ++x) {
                                const long long b = static_cast<long long>(2 * x + (x == cf)) * kRows;
                                const float f = ex2(__ldcg(&part_ml[b + row].x) - Ms);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float4 v = __ldcg(part_o + b * (HD / 4) + static_cast<long long>(d + e) * kRows + row);
                                    o[e].x += v.x * f; o[e].y += v.y * f; o[e].z += v.z * f; o[e].w += v.w * f;
                                }
                            }
                            const float iL = 1.f / L;
                            uint4 w[2];
                            uint32_t* pw = reinterpret_cast<uint32_t*>(w);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                pw[2 * e] = lim > 0 ? pack2<T>(o[e].x * iL, o[e].y * iL) : 0u;
                                pw[2 * e + 1] = lim > 0 ? pack2<T>(o[e].z * iL, o[e].w * iL) : 0u;
                            }
                            reinterpret_cast<uint4*>(dst + 4 * d)[0] = w[0];
                            reinterpret_cast<uint4*>(dst + 4 * d)[1] = w[1];
                        }
                    }
                    named_sync(1 + t, 128);        // s_last is free again
                }
            }
            done += sg.len;
        } while (next_segment(sg, left));
        if (stop && r == 0) atomicExch(&s_fail, 1);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (warp == 9 && *reinterpret_cast<volatile int*>(&s_fail) != 0) {
        if (lane == 0) report_status(a.status, LLAMA_ERR_DEVICE_TIMEOUT);
        // the newest copy of each slot and the last Q land before the CTA exits
        for (int k = issued > nslots ? issued - nslots : 0; k < issued; ++k)
            mbar_wait(&kv_full[k % nslots], (k / nslots) & 1);
        if (n_q > 0) mbar_wait(&q_full, (n_q - 1) & 1);
    }
}

// ---------------------------------------------------------------- host side

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode3 = nullptr;

// A 3-d map of 16-bit values, boxes of 64 x b1 x b2, 128-byte swizzle.
int encode_3d(CUtensorMap* map, const void* base, int dtype, long long d0, long long d1, long long d2, long long s1,
              long long s2, int b1, int b2) {
    if (!g_encode3) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (e != cudaSuccess || fn == nullptr || q != cudaDriverEntryPointSuccess) {
            set_error("cuTensorMapEncodeTiled unavailable");
            return LLAMA_ERR_CUDA;
        }
        g_encode3 = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = g_encode3(map, dtype == LLAMA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                                 const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled failed (%d) for a paged cache", static_cast<int>(r));
        return LLAMA_ERR_CUDA;
    }
    return LLAMA_OK;
}
}  // namespace

template <typename T, int HD>
static int tile_go(const PagedAttnArgs& a, int dtype, cudaStream_t st) {
    constexpr int TILE = 128 * HD * 2;
    const int rep = a.nh / a.nkv, ps = 1 << a.page_shift;
    CUtensorMap mq, mk, mv;
    int rc = encode_3d(&mq, a.q, dtype, HD, a.nh, a.T, HD, static_cast<long long>(a.nh) * HD, rep, 128 / rep);
    const long long heads = static_cast<long long>(a.n_pages) * a.nkv;
    const int rows = ps < 128 ? ps : 128;
    if (rc == LLAMA_OK) rc = encode_3d(&mk, a.k_pages, dtype, HD, ps, heads, HD, static_cast<long long>(ps) * HD, rows, 1);
    if (rc == LLAMA_OK) rc = encode_3d(&mv, a.v_pages, dtype, HD, ps, heads, HD, static_cast<long long>(ps) * HD, rows, 1);
    if (rc != LLAMA_OK) return rc;
    auto kern = paged_attn_tile_kernel<T, HD>;
    const int list = (a.B + 1) * 8 + a.B * static_cast<int>(sizeof(WorkReq));
    constexpr int most = 226 * 1024;               // 227 KB less the static barriers
    int nslots = (most - 1024 - 2 * TILE - list) / TILE;
    if (nslots > kMaxSlots) nslots = kMaxSlots;
    const int smem = 1024 + (2 + nslots) * TILE + list;
    static int sms = 0;
    if (sms == 0) {
        int dev = 0, n = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(paged_attn_tile_kernel)");
        sms = n < kMaxCtas ? n : kMaxCtas;
    }
    TileShape shape;
    shape.lr = rep == 1 ? 8 : rep == 2 ? 7 : rep == 4 ? 6 : 5;
    shape.lk = 7;
    const long long cap = ((static_cast<long long>(a.max_pages) << a.page_shift) + kKeys - 1) / kKeys;
    long long grid = static_cast<long long>(a.T) * a.nkv * cap;
    if (grid > sms) grid = sms;
    kern<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(mq, mk, mv, a, shape, nslots);
    LLB_CHECK_LAUNCH("paged_attn_tile_kernel");
    return LLAMA_OK;
}

size_t paged_attention_tile_ws(int hd) { return ws_bytes(hd); }

int launch_paged_attention_tile(const PagedAttnArgs& a, int dtype, cudaStream_t st) {
    if (dtype == LLAMA_F16) return a.hd == 64 ? tile_go<f16, 64>(a, dtype, st) : tile_go<f16, 128>(a, dtype, st);
    return a.hd == 64 ? tile_go<bf16, 64>(a, dtype, st) : tile_go<bf16, 128>(a, dtype, st);
}

}  // namespace llb
