// Where rows of q, their keys and their pages lie (kv_index.h) and how a call is
// cut up (attend_plan.h), over random small calls and a few of the largest
// sizes, against statements written here: every row of every sequence in one
// tile and none twice, its keys inside the tile's, pages inside the pool, parts
// inside the workspace; with offsets, lengths and tables that make no sense, all
// of it still inside the buffers.
#include <stdio.h>
#include <stdlib.h>

#include <random>
#include <vector>

#include "../../quantized_matmul_amd/csrc/attend_plan.h"

using namespace qlin;

static std::mt19937 rng(7);
static int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }

#define CHECK(x)                                                    \
    do {                                                            \
        if (!(x)) {                                                 \
            printf("%s:%d: %s\n", __FILE__, __LINE__, #x);          \
            exit(1);                                                \
        }                                                           \
    } while (0)

static void one_call(bool sense) {
    const int dims[] = {64, 96, 128, 192, 256};
    KvPool c{};
    c.D = dims[pick(0, 4)];
    c.mode = (int)pick(0, 2) == 0 ? 1 : 0;
    c.g = c.mode ? 32 : (c.D % 64 ? 32 : 64);
    c.heads = (int)pick(1, 3);
    c.page = 16 * (int)pick(1, 6);
    c.pages = pick(1, 20);
    AttendArgs a{};
    a.B = (int)pick(1, 5);
    a.q_heads = c.heads * (int)pick(1, 20);
    a.width = (int)pick(0, 9);
    a.causal = (int)pick(0, 1);
    a.window = pick(0, 2) ? 0 : pick(1, 200);
    const bool one_row = pick(0, 3) == 0;
    std::vector<int32_t> offsets(a.B + 1), lengths(a.B), table((size_t)a.B * a.width + 1, -7);
    const int most_rows = pick(0, 1) ? 6 : 200;
    int64_t at = one_row ? 0 : pick(0, 5);
    for (int b = 0; b <= a.B; ++b) {
        offsets[b] = (int32_t)at;
        if (b < a.B) at += one_row ? 1 : (pick(0, 3) ? pick(0, most_rows) : 0);
    }
    a.T = at + (one_row ? 0 : pick(0, 4));
    for (auto& l : lengths) l = (int32_t)(pick(0, 5) ? pick(0, (int64_t)a.width * c.page) : (pick(0, 1) ? -3 : 1 << 30));
    for (auto& p : table) p = (int32_t)(pick(0, 6) ? pick(0, c.pages - 1) : (pick(0, 1) ? -1 : c.pages + pick(0, 9)));
    if (!sense && !one_row)
        for (auto& o : offsets) o = pick(0, 2) ? o : (int32_t)(pick(0, 1) ? -pick(0, 1000) : pick(0, 2147483000));
    a.offsets = one_row ? nullptr : offsets.data();
    a.lengths = lengths.data();
    a.table = table.data();
    if (a.T == 0) return;

    const int dt = pick(0, 1) ? QLIN_BF16 : QLIN_F16;
    const AttendPlan p = attend_plan(dt, a.T, a.q_heads, a.B, a.width, c, a.window, one_row);
    CHECK(p.fits && (p.path == 1 || p.path == 2) && p.chunk > 0 && p.splits > 0 && p.rows > 0);
    const int unit = p.path == 1 ? kKvUnit : 64, share = a.q_heads / c.heads;
    const size_t parts = p.splits > 1 ? (size_t)p.tiles * c.heads * p.splits * p.rows * (c.D + 2) * 4 : 0;
    CHECK(p.bytes >= p.part_at + parts);
    if (p.path == 2) {
        CHECK(p.present_at >= (size_t)a.B * p.key_blocks * c.heads * 64 * c.D * 4);
        CHECK(p.part_at >= p.present_at + (size_t)a.B * p.key_blocks * (8 + 8 * c.heads));
    }
    std::vector<int> taken((size_t)a.T * share);
    for (int64_t tile = 0; tile < p.tiles; ++tile) {
        TileWork w = tile_of(a, c, tile, p.rows);
        if (!w.rows) continue;
        CHECK(w.b >= 0 && w.b < a.B && w.rows > 0 && w.rows <= p.rows && w.row0 >= 0);
        tile_keys(a, c, w, p.chunk, unit);
        CHECK(w.splits <= p.splits && w.lo >= 0 && w.lo <= w.hi && w.k0 <= w.lo && w.k0 % unit == 0);
        CHECK((int64_t)w.hi <= (int64_t)a.width * c.page);
        CHECK(p.path == 1 || (int64_t)w.hi <= (int64_t)p.key_blocks * 64);
        for (int i = 0; i < w.rows; ++i) {
            const int64_t token = w.s.first + (w.row0 + i) / share;
            CHECK(token >= 0 && token < a.T);
            if (sense) ++taken[token * share + (w.row0 + i) % share];
            const Seen s = seen_by(a, w.s, (w.row0 + i) / share);
            CHECK(s.lo <= s.hi && (s.lo == s.hi || (s.lo >= w.lo && s.hi <= w.hi)));
            // key by key, from the definition
            const int64_t place = (int64_t)w.s.keys - w.s.n + (w.row0 + i) / share;
            if (i % 7 == 0)
                for (int64_t key = 0; key < w.s.keys; ++key) {
                    bool sees = !a.causal || key <= place;
                    if (a.window && key <= place - a.window) sees = false;
                    CHECK(sees == (key >= s.lo && key < s.hi));
                }
        }
        for (int key = w.k0; key < w.hi; key += kKvUnit) {
            const int32_t page = a.table[(int64_t)w.b * a.width + key / c.page];
            const int h = (int)pick(0, c.heads - 1);
            const int32_t rb = kv_row_block(page, c.pages, c.heads, c.page, h, key / kKvUnit);
            if (page < 0 || page >= c.pages) CHECK(rb == -1);
            else CHECK(rb >= 0 && (int64_t)rb * kKvUnit == ((int64_t)page * c.heads + h) * c.page + key % c.page);
        }
    }
    if (sense)
        for (int64_t t = 0; t < a.T; ++t)
            for (int g = 0; g < share; ++g)
                CHECK(taken[t * share + g] == (one_row || (t >= offsets[0] && t < offsets[a.B]) ? 1 : 0));
}

int main() {
    for (int i = 0; i < 20000; ++i) one_call(i % 4 != 3);
    // the largest sizes: nothing overflows, and what does not fit says so
    KvPool c{};
    c.D = 128;
    c.g = 64;
    c.pages = 1 << 20;
    for (int page : {16, 1 << 24})
        for (int heads : {1, 4096})
            for (int64_t T : {(int64_t)1, (int64_t)1 << 20, ((int64_t)1 << 31) / heads - 1})
                for (int64_t width : {(int64_t)1, (int64_t)1 << 31})
                    for (int64_t window : {(int64_t)0, (int64_t)1000, (int64_t)1 << 60})
                        for (int64_t B : {(int64_t)1, T}) {
                            c.page = page;
                            c.heads = heads;
                            const AttendPlan p = attend_plan(QLIN_BF16, T, heads, B, width, c, window, B == T);
                            CHECK(p.path && p.chunk > 0 && p.splits > 0 && p.tiles > 0);
                            if (p.fits) CHECK(p.tiles * heads * p.splits * 256 < (int64_t)1 << 32);
                        }
    printf("ok\n");
    return 0;
}
