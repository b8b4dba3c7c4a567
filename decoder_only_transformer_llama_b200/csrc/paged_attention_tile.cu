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
//                  rounded to 16 bits (half a step of P, the size of the
//                  output's own rounding; l sums it unrounded) over the first
//                  half of S_t's columns
//   O_t += P_t V   tcgen05 with P_t from TMEM and V read MN-major from its tile
// The two sub-tiles alternate on the tensor core: while one's softmax runs,
// the other's products do.  MMAs of one thread run in order, so S_t of the next
// unit may overwrite P_t once its product is issued.  m moves only when a unit
// raises it by more than 8 (a factor 256): then O_t is rescaled in TMEM.
//
// Measured: chunks of 1000-2000 tokens over 3000-6000 keys (64/8 heads of 128, bf16)
// 486 us, 1158 TFLOP/s; 560 us under the power cap.  A unit takes about 4000 cycles, of
// which the MMAs are 2048: bound by the chain scores -> softmax -> product of a
// sub-tile, which the other one covers only in part (TMEM has no room for a third).
// 256 rows a tile so that K and V tiles are read once for both sub-tiles; 128 keys a
// unit so that S_t and O_t fill TMEM.
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

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "paged.h"
#include "paged_work.cuh"
#include "per_device.cuh"

namespace llb {

namespace {
constexpr int kThreads = 384;                // three warpgroups; warps 10 and 11 only fill the third
// registers a thread: the launch's 168, of which the third warpgroup gives up
// what the two softmax warpgroups take (2 * 208 + 88 = 3 * 168; 216 + 72 spills in the MMA warp, 1% slower)
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kRows = 256;
constexpr int kKeys = 128;
constexpr int kBox = 128 * 128;             // 128 rows of 64 16-bit values
constexpr int kMaxCtas = 160;
// Units per CTA below which fewer CTAs run: a unit takes about 2 us, a publish
// and a merge of a split tile 5.
constexpr int kMinUnits = 4;
constexpr int kWhole = 5;                   // tiles of so many units stay whole
constexpr int kFan = 4;                     // partial results merged at a time
constexpr int kLevels = 4;                  // kFan^4 contributors: every CTA
constexpr int kMaxSlots = 8;
constexpr uint32_t kColS = 0, kColO = 256;  // S_t at kColS + 128 t, O_t at kColO + 128 t

static_assert(kFan * kFan * kFan * kFan >= kMaxCtas && 4 * kLevels * kMaxCtas * sizeof(int) <= kPagedCounters, "merge tree");
constexpr size_t kOffMl = kPagedCounters;
constexpr size_t kOffO = kOffMl + 2ull * kMaxCtas * kRows * sizeof(float2);
constexpr size_t ws_bytes(int hd) { return kOffO + 2ull * kMaxCtas * kRows * hd * sizeof(float); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pk2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void un2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// 32 lanes x 16 fp32 columns from registers.
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
           "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
// 32 lanes x 32 columns of packed 16-bit pairs from registers.
__device__ __forceinline__ void tmem_st_p(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
           "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]),
           "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]),
           "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// MMAs and commits by one lane of a converged warp (the same lane each time):
// control flow and operands stay uniform over the warp, which keeps the
// descriptors in uniform registers.
__device__ __forceinline__ void warp_mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc) : "memory");
}
// A from TMEM: 16-bit values two to a column, K-major.
__device__ __forceinline__ void warp_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void warp_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit));
}
template <typename T> __device__ __forceinline__ bool not_finite16(uint32_t h) {
    constexpr uint32_t e = std::is_same<T, bf16>::value ? 0x7f80u : 0x7c00u;
    return (h & e) == e;
}

// Merges the partial results of sub-tile t of n <= kFan contributors of a tile, x =
// first, first + stride, ... (contributor x's in slot 2 x, the tile's first one
// cf's in slot 2 cf + 1), in their order: rows_live rows, spread over the 128
// threads with as many columns of a row side by side as there is room for.
// With `out` the rows are finished: row r lies at out + (r >> lrep) * token + (r &
// (2^lrep - 1)) * HD and sees lim0 + (r >> lrep) keys; without it the merged
// partial result takes the place of the first one.
template <typename T, int HD>
__device__ __noinline__ void merge_half(float2* part_ml, float4* part_o, int cf, int first, int n, int stride, int t,
                                        int rows_live, T* out, int lrep, long long token, int lim0) {
    const int tid = threadIdx.x & 127;
    const int lr = rows_live > 1 ? 32 - __clz(rows_live - 1) : 0;    // rows side by side: 2^lr
    const int r = tid & ((1 << lr) - 1), row = t * 128 + r;
    const bool in = r < rows_live;
    long long slot[kFan];
    float f[kFan];
    float M = -INFINITY, L = 0.f;
    float2 ml[kFan];
#pragma unroll
    for (int k = 0; k < kFan; ++k) {
        const int x = first + (k < n ? k : 0) * stride;
        slot[k] = static_cast<long long>(2 * x + (x == cf ? 1 : 0)) * kRows;
        ml[k] = in ? __ldcg(part_ml + slot[k] + row) : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int k = 0; k < kFan; ++k)
        if (k < n) M = fmaxf(M, ml[k].x);
    const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int k = 0; k < kFan; ++k) {
        f[k] = k < n ? ex2(ml[k].x - Ms) : 0.f;
        if (k < n) L += ml[k].y * f[k];
    }
    T* dst = out ? out + (r >> lrep) * token + (r & ((1 << lrep) - 1)) * HD : nullptr;
    const bool some = lim0 + (r >> lrep) > 0;
    if (in) {
#pragma unroll 2
        for (int d = 2 * (tid >> lr); d < HD / 4; d += 256 >> lr) {      // eight columns
            float4 v[kFan][2];
#pragma unroll
            for (int k = 0; k < kFan; ++k)
                if (k < n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        v[k][e] = __ldcg(part_o + slot[k] * (HD / 4) + static_cast<long long>(d + e) * kRows + row);
            float4 o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kFan; ++k) {
                    if (k >= n) break;
                    o[e].x = fmaf(v[k][e].x, f[k], o[e].x); o[e].y = fmaf(v[k][e].y, f[k], o[e].y);
                    o[e].z = fmaf(v[k][e].z, f[k], o[e].z); o[e].w = fmaf(v[k][e].w, f[k], o[e].w);
                }
                if (!out) part_o[slot[0] * (HD / 4) + static_cast<long long>(d + e) * kRows + row] = o[e];
            }
            if (out) {
                const float inv = some ? 1.f / L : 0.f;
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (some) {
                    w.x = pack2<T>(o[0].x * inv, o[0].y * inv); w.y = pack2<T>(o[0].z * inv, o[0].w * inv);
                    w.z = pack2<T>(o[1].x * inv, o[1].y * inv); w.w = pack2<T>(o[1].z * inv, o[1].w * inv);
                }
                *reinterpret_cast<uint4*>(dst + 4 * d) = w;
            }
        }
    }
    if (!out) {
        named_sync(1 + t, 128);                    // every thread has read the first one's (m, l)
        if (in && tid >> lr == 0) part_ml[slot[0] + row] = make_float2(M, L);
    }
}

// Every wait's limit and, in tests of it (llama_debug_stall), the stage of CTA
// 0's run, counted from 1, whose copies never come.
struct Waits {
    uint64_t limit;
    int stalled;
};

// A part of one tile that a CTA works on: units c.j .. c.j + len - 1.
struct Segment {
    WorkCur c;
    int len;
};
}  // namespace

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_tile_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                       const __grid_constant__ CUtensorMap mapV, PagedAttnArgs a, TileShape shape, int nslots,
                       Waits waits) {
    constexpr int NB = HD / 64;                    // boxes per tile
    // fp16 loses relative precision below 2^-14: weights, up to 2^8 before m moves,
    // carry a factor 2^7 there
    constexpr float kLift = std::is_same<T, f16>::value ? 7.f : 0.f;
    constexpr int TILE = NB * kBox;                // a [128][HD] tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;                            // 2 tiles
    uint8_t* ring = smem + 2 * TILE;               // K, V, K, V, ...
    long long* cum = reinterpret_cast<long long*>(ring + nslots * TILE);
    WorkReq* req = reinterpret_cast<WorkReq*>(cum + a.B + 1);
    __shared__ uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
    __shared__ uint64_t q_full, q_empty, s_full[2], p_full[2][2], o_full[2], mdone;
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
    WorkCur start, end;
    const long long u0 = run_bound(shape, req, cum, a.B, a.nkv, run_start(cta, W, P), kWhole, start);
    const long long u1 = run_bound(shape, req, cum, a.B, a.nkv, run_start(cta + 1, W, P), kWhole, end);
    if (u1 <= u0) return;                          // a run inside a tile that its neighbours take
    const int rep = a.nh / a.nkv, lrep = 8 - shape.lr;
    const int half = 128 >> lrep;                  // tokens of a sub-tile

    if (tid == 0) {
        for (int i = 0; i < nslots; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int t = 0; t < 2; ++t) { mbar_init(&s_full[t], 1); mbar_init(&p_full[t][0], 128); mbar_init(&p_full[t][1], 128); mbar_init(&o_full[t], 1); }
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
        s.c = start;
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
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsOther));
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
            ok = __all_sync(0xffffffffu, mbar_wait(&q_empty, (nseg & 1) ^ 1, waits.limit));
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
                    ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[slot], empty_phase, waits.limit));
                    if (!ok) break;
                    const bool comes = cta != 0 || issued + 1 != waits.stalled;
                    if (lane == 0 && comes) mbar_arrive_expect_tx(&kv_full[slot], TILE);
                    __syncwarp();
                    if (lane < npg && comes)
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
    } else if (warp == 8) {
        // ---------------- MMA issuer
        constexpr uint32_t idesc_s = idesc_16_f32<T>(128, kKeys);
        constexpr uint32_t idesc_o = idesc_16_f32_bmn<T>(128, HD);
        Segment sg = first_segment();
        long long left = u1 - u0;
        int slot = 0, nseg = 0;
        uint32_t full_phase = 0, p_phase[2] = {0, 0};
        bool ok = true;
        // Operand descriptors: constant bits once, then one addition per MMA (the
        // address field counts 16 bytes; a single thread issues, so every
        // instruction between two MMAs adds to their spacing).
        const uint64_t q_desc = smem_desc_k_sw128(smem_u32(sQ)), k_desc = smem_desc_k_sw128(smem_u32(ring)),
                       v_desc = smem_desc_mn_sw128(smem_u32(ring), kBox);
        auto advance = [&]() { if (++slot == nslots) { slot = 0; full_phase ^= 1; } };
        auto scores = [&](int t, int kslot) {
            const uint64_t qd = q_desc + t * (TILE >> 4), kd = k_desc + static_cast<uint32_t>(kslot * (TILE >> 4));
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
                warp_mma_ss(tmem + kColS + 128 * t, qd + off, kd + off, idesc_s, kk > 0);
            }
            warp_commit(&s_full[t]);
        };
        // what an early look at a barrier left open
        auto settle = [&](bool seen, uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, seen) || warp_wait(bar, parity, waits.limit);
        };
        do {
            const int nt = two_halves(sg) ? 2 : 1;
            ok = warp_wait(&q_full, nseg & 1, waits.limit) && warp_wait(&kv_full[slot], full_phase, waits.limit);
            if (!ok) break;
            tc_fence_after();
            for (int t = 0; t < nt; ++t) scores(t, slot);
            warp_commit(&kv_empty[slot]);
            if (sg.len == 1) warp_commit(&q_empty);
            advance();
            for (int i = 0; i < sg.len; ++i) {
                // Barriers are asked ahead of the MMAs they gate, while earlier ones
                // run: a wait costs about 130 cycles even if it need not wait.
                const bool more = i + 1 < sg.len;
                const int vslot = slot;
                const uint32_t v_phase = full_phase;
                advance();
                const int kslot = slot;                              // K of the next unit
                bool v_ready = mbar_try_wait(&kv_full[vslot], v_phase);
                bool ready = mbar_try_wait(&p_full[0][0], p_phase[0]);
                bool k_ready = !more || mbar_try_wait(&kv_full[kslot], full_phase);
                ok = settle(v_ready, &kv_full[vslot], v_phase);
                const uint64_t vd = v_desc + static_cast<uint32_t>(vslot * (TILE >> 4));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= nt) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {                    // 64 keys at a time
                        ok = ok && settle(ready, &p_full[t][h], p_phase[t]);
                        if (!ok) break;
                        tc_fence_after();
                        // the next P half: of this sub-tile, or of the other one
                        if (h == 0) ready = mbar_try_wait(&p_full[t][1], p_phase[t]);
                        else if (t == 0 && nt == 2) ready = mbar_try_wait(&p_full[1][0], p_phase[1]);
#pragma unroll
                        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                            warp_mma_ts(tmem + kColO + 128 * t, tmem + kColS + 128 * t + 8 * kk,
                                        vd + (kk * 16 * 128 >> 4), idesc_o, i > 0 || kk > 0);
                    }
                    if (!ok) break;
                    p_phase[t] ^= 1;
                    warp_commit(&o_full[t]);
                    if (more) {
                        if (t == 0) ok = settle(k_ready, &kv_full[kslot], full_phase);
                        if (!ok) break;
                        if (t == 0) tc_fence_after();
                        scores(t, kslot);
                    }
                }
                if (!ok) break;
                warp_commit(&kv_empty[vslot]);
                if (more) {
                    warp_commit(&kv_empty[kslot]);
                    if (i + 2 == sg.len) warp_commit(&q_empty);
                    advance();
                }
            }
            ++nseg;
        } while (ok && next_segment(sg, left));
        if (!ok && lane == 0) atomicExch(&s_fail, 1);
        warp_commit(&mdone);                         // every MMA has finished before TMEM is freed
        if (!warp_wait(&mdone, 0, kWaitLimitNs) && lane == 0) atomicExch(&s_fail, 1);
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegsSoftmax));
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
                bool fail = false;
                for (int i = 0; i < sg.len; ++i) {
                    const int key0 = (sg.c.j + i) * kKeys;
                    const bool masked = key0 + kKeys > lim0;
                    bool ok = mbar_wait(&s_full[t], ph, waits.limit);
                    if (t == 0 && masked) ok = ok && mbar_wait(&kv_full[vslot], v_phase, waits.limit);
                    if (!__all_sync(0xffffffffu, ok)) { fail = true; break; }
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
                    float mx;
                    {
                        float c[4] = {s[0], s[1], s[2], s[3]};       // four chains
#pragma unroll
                        for (int x = 4; x < kKeys; x += 8)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                c[y] = x + 4 + y < kKeys ? fmaxf(c[y], fmaxf(s[x + y], s[x + 4 + y])) : fmaxf(c[y], s[x + y]);
                        mx = fmaxf(fmaxf(c[0], c[1]), fmaxf(c[2], c[3])) * sl2;
                    }
                    bool rescale = false;
                    float corr = 1.f;
                    if (mx > m + 8.f || m == -INFINITY) {
                        rescale = i > 0 && mx > m;
                        corr = m == -INFINITY ? 0.f : ex2(m - mx);
                        m = mx;
                    }
                    if (__any_sync(0xffffffffu, rescale)) {
                        // O holds every earlier unit: these scores came behind its last product
#pragma unroll 1
                        for (int x = 0; x < HD; x += 16) {
                            float o[16];
                            tmem_ld_32x32b_x16(colO + x, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= corr;
                            tmem_st_16(colO + x, o);
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;       // no key so far: every weight is 0
                    const uint64_t scale2 = pk2(sl2, sl2), minus2 = pk2(kLift - ms, kLift - ms);
                    uint64_t sum2[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t p[32];
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            float e0, e1;
                            un2(fma2(pk2(s[64 * h + 2 * x], s[64 * h + 2 * x + 1]), scale2, minus2), e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            sum2[x & 1] = add2(sum2[x & 1], pk2(e0, e1));
                            p[x] = pack2<T>(e0, e1);
                        }
                        tmem_st_p(colS + 32 * h, p);
                        tc_wait_st();
                        tc_fence_before();
                        mbar_arrive(&p_full[t][h]);
                    }
                    {
                        float a0, a1;
                        un2(add2(sum2[0], sum2[1]), a0, a1);
                        l = l * corr + (a0 + a1);
                    }
                    ph ^= 1;
                    vslot += 2;
                    if (vslot >= nslots) { vslot -= nslots; v_phase ^= 1; }
                }
                // ---- end of the tile, or of this CTA's part of it: O holds every unit
                if (!fail) fail = !mbar_wait(&o_full[t], ph ^ 1, waits.limit);
                stop = named_any(1 + t, 128, fail);
                if (stop) break;
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
                    // a tree of groups of kFan, as in the kernel of short tiles
                    const int n = cl - cf + 1, rows_live = min(128, (rq.n - t0 - t * half) << lrep);
                    T* first_row = static_cast<T*>(a.out) +
                                   (static_cast<long long>(rq.q0 + t0 + t * half) * a.nh + sg.c.g * rep) * HD;
                    int k = cta - cf, stride = 1;
                    for (int* level = counters;; level += 4 * kMaxCtas) {
                        const int first = k / (kFan * stride) * (kFan * stride);
                        const int members = min(kFan, (n - first + stride - 1) / stride);
                        const int x = cf + first;
                        __threadfence();
                        named_sync(1 + t, 128);
                        if (r == 0) {
                            int* counter = level + 2 * (2 * x + (first == 0 ? 1 : 0)) + t;
                            s_last[t] = atomicAdd(counter, 1) == members - 1;
                            if (s_last[t]) *counter = 0;
                        }
                        named_sync(1 + t, 128);
                        if (!s_last[t]) break;
                        __threadfence();
                        const bool top = n <= kFan * stride;
                        if (top || members > 1)
                            merge_half<T, HD>(part_ml, part_o, cf, x, members, stride, t, rows_live, top ? first_row : nullptr,
                                              lrep, static_cast<long long>(a.nh) * HD, rq.seq - rq.n + t0 + t * half + 1);
                        if (top) break;
                        k = first;
                        stride *= kFan;
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
            if (cta != 0 || k + 1 != waits.stalled) mbar_wait(&kv_full[k % nslots], (k / nslots) & 1);
        if (n_q > 0) mbar_wait(&q_full, (n_q - 1) & 1);
    }
}

// ---------------------------------------------------------------- host side

namespace {
std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode3{nullptr};
std::atomic<uint64_t> g_stall{0};               // an armed stall: stage + 1 << 32 | wait limit in ns (below 2^32); 0: none

// A 3-d map of 16-bit values, boxes of 64 x b1 x b2, 128-byte swizzle.
int encode_3d(CUtensorMap* map, const void* base, int dtype, long long d0, long long d1, long long d2, long long s1,
              long long s2, int b1, int b2) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = g_encode3.load(std::memory_order_relaxed);
    if (!encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (e != cudaSuccess || fn == nullptr || q != cudaDriverEntryPointSuccess) {
            set_error("cuTensorMapEncodeTiled unavailable");
            return LLAMA_ERR_CUDA;
        }
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        g_encode3.store(encode, std::memory_order_relaxed);
    }
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType type = dtype == LLAMA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = encode(map, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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
    static PerDevice<int> per_device;
    int sms = 0;
    const cudaError_t e = per_device.get(&sms, [&](int dev, int* out) {
        int n = 0;
        cudaError_t r = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        *out = n < kMaxCtas ? n : kMaxCtas;
        return r;
    });
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(paged_attn_tile_kernel)");
    TileShape shape;
    shape.lr = rep == 1 ? 8 : rep == 2 ? 7 : rep == 4 ? 6 : 5;
    shape.lk = 7;
    const long long cap = ((static_cast<long long>(a.max_pages) << a.page_shift) + kKeys - 1) / kKeys;
    long long grid = static_cast<long long>(a.T) * a.nkv * cap;
    if (grid > sms) grid = sms;
    Waits waits = {kWaitLimitNs, 0};
    if (g_stall.load(std::memory_order_relaxed)) {
        const uint64_t s = g_stall.exchange(0);
        if (s) waits = {s & 0xffffffffu, static_cast<int>(s >> 32)};
    }
    kern<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(mq, mk, mv, a, shape, nslots, waits);
    LLB_CHECK_LAUNCH("paged_attn_tile_kernel");
    return LLAMA_OK;
}

size_t paged_attention_tile_ws(int hd) { return ws_bytes(hd); }

void arm_paged_stall(int stage, long long wait_ns) {
    g_stall.store(stage < 0 ? 0 : (static_cast<uint64_t>(stage) + 1) << 32 | static_cast<uint64_t>(wait_ns));
}

int launch_paged_attention_tile(const PagedAttnArgs& a, int dtype, cudaStream_t st) {
    if (dtype == LLAMA_F16) return a.hd == 64 ? tile_go<f16, 64>(a, dtype, st) : tile_go<f16, 128>(a, dtype, st);
    return a.hd == 64 ? tile_go<bf16, 64>(a, dtype, st) : tile_go<bf16, 128>(a, dtype, st);
}

}  // namespace llb
