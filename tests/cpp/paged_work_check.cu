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
    printf("ok\n");
    return 0;
}
