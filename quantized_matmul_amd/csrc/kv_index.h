// kv_index.h -- where a row of q, its keys and their pages lie: everything an
// attention kernel derives from lengths, offsets and page tables. No more than
// integers, so that a CPU build can look at every case.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define QLIN_HD __host__ __device__ __forceinline__
#else
#define QLIN_HD inline
#endif

namespace qlin {

// A pool of pages for keys ([0]) and values ([1]), each [pages, heads, page, D]
// quantized along D to 4 bits. Row (p, h, o) is number (p * heads + h) * page + o.
struct KvPool {
    uint32_t* codes[2];
    void* scales[2];     // AFFINE: of sdt, else bytes
    void* biases[2];     // AFFINE only
    int sdt;             // QLIN_F32, QLIN_F16 or QLIN_BF16
    int mode, g;
    int64_t pages;
    int heads, page, D;
};

constexpr int kKvUnit = 16;      // rows of a page come in runs of this many
constexpr int64_t kKvMaxKeys = 0x7FFFFF00;   // of a sequence: key numbers and those of a block past them fit an int

// Pages [0, pages) exist: the row block (row number over 16) of head h where
// key block `block` (its keys over 16) of a sequence lies, or -1 where its page
// number p is none.
QLIN_HD int32_t kv_row_block(int32_t p, int64_t pages, int heads, int page, int h, int block) {
    if (p < 0 || p >= pages) return -1;
    const int per = page / kKvUnit;
    return (int32_t)(((int64_t)p * heads + h) * per + block % per);
}

struct AttendArgs {
    const void* q;
    void* out;
    int64_t T, q_stride;
    int q_heads;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* offsets;          // null: row b is sequence b's only one
    int B, width;
    float scale;
    int causal;
    int64_t window;                  // 0: none
};

// Last b in [0, B) with value(b) <= x, for a value that never falls; 0 where
// there is none. The loop ends whatever value() gives.
template <class F>
QLIN_HD int last_at_most(int B, int64_t x, F&& value) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (value(mid) <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Rows [first, first + n) of q are sequence b's (kept inside [0, T)), which
// has `keys` keys.
struct Sequence {
    int64_t first;
    int n, keys;
};
QLIN_HD void rows_of(const AttendArgs& a, int b, Sequence& s) {
    int64_t end;
    if (a.offsets) {
        s.first = a.offsets[b];
        end = a.offsets[b + 1];
        s.first = s.first < 0 ? 0 : (s.first > a.T ? a.T : s.first);
        end = end < s.first ? s.first : (end > a.T ? a.T : end);
    } else {
        s.first = b;
        end = b + 1;
    }
    s.n = (int)(end - s.first);
}
QLIN_HD int keys_of(const AttendArgs& a, const KvPool& c, int b) {
    const int64_t held = (int64_t)a.width * c.page, most = held < kKvMaxKeys ? held : kKvMaxKeys;
    const int64_t k = a.lengths[b];
    return (int)(k < 0 ? 0 : (k > most ? most : k));
}
QLIN_HD Sequence sequence_of(const AttendArgs& a, const KvPool& c, int b) {
    Sequence s;
    rows_of(a, b, s);
    s.keys = keys_of(a, c, b);
    return s;
}

// Keys [lo, hi) that row i of a sequence sees: its own place is the key
// keys - n + i, so that the last row stands at the last key.
struct Seen {
    int lo, hi;
};
QLIN_HD Seen seen_by(const AttendArgs& a, const Sequence& s, int i) {
    const int64_t at = (int64_t)s.keys - s.n + i;
    int64_t hi = s.keys, lo = 0;
    if (a.causal && at + 1 < hi) hi = at + 1;
    if (a.window && at + 1 - a.window > 0) lo = at + 1 - a.window;
    if (hi < 0) hi = 0;
    if (lo > hi) lo = hi;
    return {(int)lo, (int)hi};
}

// A tile of rows, and what it has to read: keys [lo, hi), taken from k0 (a
// multiple of `unit`) on in `splits` chunks.
struct TileWork {
    Sequence s;
    int b, row0, rows, lo, hi, k0, splits;       // row0: of the sequence's n * share rows; rows: of this tile
};
QLIN_HD TileWork tile_of(const AttendArgs& a, const KvPool& c, int64_t tile, int tile_rows) {
    const int share = a.q_heads / c.heads;
    TileWork w;
    int64_t rt;
    w.rows = 0;
    if (a.offsets) {
        // sequence b starts at tile floor(offsets[b] * share / tile_rows) + b: a tile more than it needs at most
        auto start = [&](int b) { return (int64_t)a.offsets[b] * share / tile_rows + b; };
        w.b = last_at_most(a.B, tile, start);
        rt = tile - start(w.b);
    } else {
        const uint32_t per = (share + tile_rows - 1) / tile_rows;      // (tiles of a launch number below 2^32)
        w.b = (int)(per == 1 ? (uint32_t)tile : (uint32_t)tile / per);
        rt = tile - (int64_t)w.b * per;
    }
    if (w.b >= a.B || rt < 0) return w;
    rows_of(a, w.b, w.s);
    const int64_t rows = (int64_t)w.s.n * share - rt * tile_rows;
    if (rows <= 0) return w;
    w.row0 = (int)(rt * tile_rows);
    w.rows = rows < tile_rows ? (int)rows : tile_rows;
    return w;
}
QLIN_HD void tile_keys(const AttendArgs& a, const KvPool& c, TileWork& w, int chunk, int unit) {
    const int share = a.q_heads / c.heads;
    w.s.keys = keys_of(a, c, w.b);
    w.lo = seen_by(a, w.s, w.row0 / share).lo;
    w.hi = seen_by(a, w.s, (w.row0 + w.rows - 1) / share).hi;
    w.k0 = w.lo & ~(unit - 1);
    w.splits = w.hi > w.lo ? (w.hi - w.k0 - 1) / chunk + 1 : 0;
}

// Keys of chunk `split` of a tile (of its splits, or the first of none): no sum
// here passes the tile's last key, which a chunk of any length may.
struct KeyRange {
    int first, end;
};
QLIN_HD KeyRange chunk_of(const TileWork& w, int split, int chunk) {
    const int first = w.k0 + split * chunk, left = w.splits ? w.hi - first : 0;
    return {first, first + (left < chunk ? left : chunk)};
}

}  // namespace qlin
