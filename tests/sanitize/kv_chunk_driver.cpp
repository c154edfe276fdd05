// The keys of each chunk of a tile (kv_index.h) at the longest sequences, under
// the cuts that attend_plan.h makes there: the chunks of a launch cover the keys
// that the tile sees, each once and in order, and no number overflows.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>

#include "../../quantized_matmul_amd/csrc/attend_plan.h"

using namespace qlin;

#define CHECK(x)                                                    \
    do {                                                            \
        if (!(x)) {                                                 \
            printf("%s:%d: %s\n", __FILE__, __LINE__, #x);          \
            exit(1);                                                \
        }                                                           \
    } while (0)

int main() {
    int calls = 0;
    for (int D : {64, 128, 256})
        for (int heads : {1, 8})
            for (int share : {1, 8})
                for (int64_t B : {1, 3, 64, 4096})
                    for (int page : {16, 1 << 16, 1 << 24})
                        for (int64_t held : {(int64_t)600, (int64_t)1 << 20, (int64_t)(1 << 30) - 16, (int64_t)1 << 30,
                                             (int64_t)2147418112, (int64_t)1 << 31})
                            for (int64_t window : {(int64_t)0, (int64_t)300, (int64_t)1 << 29, (int64_t)1 << 40})
                                for (int n : {1, 5, 700})
                                    for (int causal : {0, 1}) {
                                        KvPool c{};
                                        c.D = D;
                                        c.g = 64;
                                        c.heads = heads;
                                        c.page = page;
                                        c.pages = 1;
                                        AttendArgs a{};
                                        a.B = (int)B;
                                        a.T = B * n;
                                        a.q_heads = heads * share;
                                        a.width = (int)((held + page - 1) / page);
                                        a.causal = causal;
                                        a.window = window;
                                        const AttendPlan p = attend_plan(QLIN_BF16, a.T, a.q_heads, B, a.width, c, window, n == 1);
                                        CHECK(p.path == 1 || p.path == 2);
                                        const int unit = p.path == 1 ? kKvUnit : 64;
                                        for (int64_t length : {held, held - 1, held / 2 + 7, (int64_t)kKvMaxKeys, (int64_t)1}) {
                                            const int64_t most = std::min((int64_t)a.width * page, kKvMaxKeys);
                                            TileWork w{};
                                            int32_t lengths[1] = {(int32_t)std::min(length, (int64_t)0x7FFFFFFF)};
                                            a.lengths = lengths;
                                            w.s.n = n;
                                            w.row0 = 0;
                                            w.rows = std::min(n * share, p.rows);
                                            tile_keys(a, c, w, p.chunk, unit);
                                            CHECK(w.s.keys == std::min((int64_t)lengths[0], most));
                                            CHECK(w.splits >= 0 && w.splits <= p.splits && (w.splits == 0) == (w.lo == w.hi));
                                            int at = w.k0;
                                            for (int split = 0; split < w.splits; ++split) {
                                                const KeyRange k = chunk_of(w, split, p.chunk);
                                                CHECK(k.first == at && k.end > k.first && k.end <= w.hi);
                                                CHECK((k.first - w.k0) % unit == 0 && k.end - k.first <= p.chunk);
                                                at = k.end;
                                            }
                                            CHECK(w.splits == 0 || at == w.hi);
                                            const KeyRange none = chunk_of(w, 0, p.chunk);
                                            CHECK(w.splits || none.first == none.end);
                                            ++calls;
                                        }
                                    }
    CHECK(calls > 10000);
    // what fits the attention's launch fits the join's, too: a wave a row
    int fit = 0;
    for (int share : {1, 20, 64})
        for (int64_t T : {(int64_t)1 << 12, (int64_t)1 << 20, (int64_t)1 << 22, ((int64_t)1 << 23) - 16, (int64_t)1 << 24})
            for (int64_t width : {3, 65, 127})
                for (int64_t B : {T, T / 4}) {
                    KvPool c{};
                    c.D = 64;
                    c.g = 64;
                    c.heads = 1;
                    c.page = 1 << 24;
                    c.pages = 1;
                    const AttendPlan p = attend_plan(QLIN_BF16, T, share, B, width, c, 0, B == T);
                    CHECK(p.path == 1);
                    if (!p.fits || p.splits == 1) continue;
                    CHECK(p.tiles * ((p.rows + 3) / 4) * 256 < (int64_t)1 << 32);
                    ++fit;
                }
    CHECK(fit > 3);
    // decoded keys and values take 8 GiB at most, also for tables without a page
    for (int64_t width : {0, 1, 9, 5000})
        for (int64_t B : {1, 7, 1000, 50000}) {
            KvPool c{};
            c.D = 128;
            c.g = 64;
            c.heads = 8;
            c.page = 64;
            c.pages = 10;
            const AttendPlan p = attend_plan(QLIN_BF16, B * 600, 8, B, width, c, 0, false);
            CHECK(p.present_at <= (size_t)1 << 33);
        }
    printf("ok\n");
    return 0;
}
