// Host walk of the paged-attention work list: the closed forms of
// paged_work.cuh against plain loops, and the runs of every CTA count.
#include <cstdio>
#include <cstdlib>

#include "../../decoder_only_transformer_llama_b200/csrc/paged_work.cuh"

using namespace llb;

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

static int plain_units(TileShape s, long long ctx, long long tokens_end) {
    const long long K = 1LL << s.lk;
    return static_cast<int>((ctx + tokens_end + K - 1) / K);
}

int main() {
    srand(1);
    for (int lk = 5; lk <= 7; ++lk)
        for (int lr = 1; lr <= 8; ++lr) {
            const TileShape s = {lr, lk};
            for (int rnd = 0; rnd < 300; ++rnd) {
                const int ctx = rnd < 40 ? rnd : rand() % 5000, n = 1 + (rnd < 60 ? rnd : rand() % 3000);
                const int R = 1 << lr, tiles = (n + R - 1) / R;
                CHECK(tiles_of(s, n) == tiles);
                long long before = 0;
                for (int i = 0; i < tiles; ++i) {
                    CHECK(tiles_units(s, ctx, i) == before);
                    const int end = (i + 1) * R < n ? (i + 1) * R : n;
                    const int u = units_of(s, ctx, n, i);
                    CHECK(u == plain_units(s, ctx, end) && u >= 1);
                    CHECK(tile_at(s, ctx, n, before) == i);
                    CHECK(tile_at(s, ctx, n, before + u - 1) == i);
                    before += u;
                }
                CHECK(request_units(s, ctx, n) == before);
            }
            CHECK(request_units(s, 100, 0) == 0);
            // far positions: 2^30 cached tokens and long chunks stay exact
            const long long far = 1LL << 30;
            const int u0 = units_of(s, static_cast<int>(far), 1, 0);
            CHECK(u0 == plain_units(s, far, 1));
            CHECK(tiles_units(s, far, 3) == plain_units(s, far, 1 << lr) + plain_units(s, far, 2 << lr) +
                                                plain_units(s, far, 3LL << lr));
        }
    for (int rnd = 0; rnd < 4000; ++rnd) {
        const long long P = 1 + rand() % 512;
        const long long W = P + (rnd % 3 ? rand() % 5000 : rand() * 1000LL);
        long long prev = 0;
        for (int c = 0; c < P; ++c) {
            const long long a = run_start(c, W, P), b = run_start(c + 1, W, P);
            CHECK(a == prev && b > a);
            prev = b;
            CHECK(run_of(a, W, P) == c && run_of(b - 1, W, P) == c);
        }
        CHECK(prev == W);
    }
    // whole walks: random requests, every CTA's run between its moved boundaries
    for (int rnd = 0; rnd < 600; ++rnd) {
        const int B = 1 + rand() % 12, nkv = 1 << rand() % 3, lk = 5 + rand() % 3, lr = 1 + rand() % 8;
        const int most = rand() % 2 ? 4 : rand() % 9;
        const TileShape s = {lr, lk};
        WorkReq req[12];
        long long cum[13] = {0};
        for (int b = 0; b < B; ++b) {
            const int n = rand() % 4 ? rand() % (rnd % 3 ? 60 : 900) : rand() % 2;
            req[b].q0 = 0;
            req[b].n = n;
            req[b].seq = rand() % 7 ? n + rand() % (rnd % 5 ? 300 : 4000) : rand() % (n + 1);
            cum[b + 1] = cum[b] + request_units(s, ctx_of(req[b]), n) * nkv;
        }
        const long long W = cum[B];
        if (W == 0) continue;
        const long long P = 1 + rand() % (W < 300 ? W : 300);
        long long prev = 0;
        for (int c = 0; c < P; ++c) {
            WorkCur at, end;
            const long long u0 = run_bound(s, req, cum, B, nkv, run_start(c, W, P), most, at);
            const long long u1 = run_bound(s, req, cum, B, nkv, run_start(c + 1, W, P), most, end);
            CHECK(u0 == prev && u1 >= u0);
            prev = u1;
            WorkCur w = at;
            for (long long u = u0; u < u1;) {
                // the place reached by walking is the place found by searching
                const WorkCur f = work_at(s, req, cum, B, nkv, u);
                CHECK(f.b == w.b && f.g == w.g && f.tile == w.tile && f.j == w.j && f.nu == w.nu);
                const long long len = w.nu - w.j < u1 - u ? w.nu - w.j : u1 - u;
                if (w.j > 0 || w.j + len < w.nu) {
                    // part of a tile: this CTA is one of the contributors that the ends of the tile name
                    CHECK(w.nu > most);
                    const int cf = run_of(u - w.j, W, P), cl = run_of(u - w.j + w.nu - 1, W, P);
                    CHECK(cf < cl && c >= cf && c <= cl);
                    CHECK((c == cf) == (w.j == 0) && (c == cl) == (w.j + len == w.nu));
                    for (int x = cf; x <= cl; ++x) {
                        WorkCur t;
                        const long long a = run_bound(s, req, cum, B, nkv, run_start(x, W, P), most, t);
                        const long long z = run_bound(s, req, cum, B, nkv, run_start(x + 1, W, P), most, t);
                        CHECK(a < u - w.j + w.nu && z > u - w.j && z > a);
                    }
                }
                u += len;
                if (u < u1) next_tile(s, req, B, nkv, w);
            }
        }
        CHECK(prev == W);
    }
    printf("ok\n");
    return 0;
}
