// attend_plan.h -- which attention kernel a call takes and how its keys are
// split, from its sizes alone. Integers only, as kv_index.h.
#pragma once

#include <stddef.h>

#include "../../include/qlin.h"
#include "kv_index.h"

namespace qlin {

struct AttendPlan {
    int path;                        // 0 simple, 1 row tiles, 2 prompt tiles
    int rows;                        // of a tile
    int nt;                          // path 1: runs of 16 columns of a tile
    int codes;                       // path 1: values multiplied as codes (a column for each quant group of a row)
    int64_t tiles;                   // row tiles of all sequences, at most
    int chunk, splits;               // keys a workgroup takes, workgroups along the keys
    int key_blocks;                  // path 2: blocks of 64 keys of a sequence, at most
    size_t part_at, present_at;      // path 2: places in the workspace (its blocks lie at 0)
    size_t bytes;                    // workspace
    bool fits;                       // one launch holds it
};

// Workgroups of the row tiles that a CU holds (waves of a SIMD, what o and q leave
// of the registers; rings of loads, what fits LDS).
constexpr int tile_residents(int D, int NT) { return D * NT <= 128 ? 3 : (D * NT <= 256 ? 2 : 1); }

// f16 prompts take affine keys as two f16 numbers each, whose sum has their bits.
constexpr bool prompt_halves(int dt, int mode) { return dt == QLIN_F16 && mode == 0; }

inline AttendPlan attend_plan(int dt, int64_t T, int q_heads, int64_t B, int64_t width, const KvPool& c, int64_t window,
                              bool one_row) {
    constexpr int64_t kStepKeys = 128;       // keys that the four waves of a workgroup take at a time
    constexpr int64_t kChunkMost = 4096;     // keys a workgroup takes, where that makes no more than kMany of them
    constexpr int64_t kMany = 32768;
    // keys that one workgroup takes sooner than a second launch joins several (500 keys 8.6 us, joined 9.2; 800 11.1 and 9.7)
    constexpr int64_t kOneChunk = 640;
    constexpr int64_t kStart = 768;          // keys that a workgroup could take in the time of its start and end
    // Rows of a sequence and key head, on average, above which a prompt is one: below, the launch that lays the keys out
    // costs more than it saves. us, row tiles and prompts, D 128: 256 rows over 16000 keys 62 and 75, 64 sequences of
    // them 1720 and 2390; 768 rows 141 and 117. D 256: 96 rows 79 and 95, 256 rows 148 and 122.
    const int64_t kPromptRows = c.D <= 128 ? 512 : 192;
    constexpr int64_t kImages = 1LL << 33;   // bytes of decoded keys and values at most
    constexpr int64_t kItems = (1LL << 32) - 1024;     // work-items of a launch
    const int64_t key_bytes = c.D * (prompt_halves(dt, c.mode) ? 6 : 4);     // of a decoded key and its value
    AttendPlan p{};
    const int64_t share = q_heads / c.heads;
    const int64_t held = width > kKvMaxKeys / c.page ? kKvMaxKeys : width * c.page;
    const bool sized = c.D == 64 || c.D == 96 || c.D == 128 || c.D == 192 || c.D == 256;
    if (dt == QLIN_F32 || !sized) {
        p.fits = T * q_heads <= kItems / 64;
        return p;
    }
    const int64_t mean = (T * share + B - 1) / B;
    // keys a tile can see, from the sizes: the table's, or the window before its first row and all behind that row,
    // which without a causal mask are as many as the sequence has rows
    int64_t keys = held;
    if (window && window < keys - T - 64) keys = window + T + 64;
    if (keys < 1) keys = 1;
    const int64_t blocks = held ? (held + 63) / 64 : 1;
    if (mean > kPromptRows && blocks * B <= kImages / (c.heads * key_bytes * 64)) {
        p.path = 2;
        // tiles of 256 rows where they fill the chip (two workgroups a CU), or of 128 (three)
        p.rows = c.D <= 128 && (T * share / 256 + B) * c.heads >= 512 ? 256 : 128;
        p.tiles = T * share / p.rows + B;
        const int64_t base = p.tiles * c.heads, fit = p.rows == 128 && c.D <= 128 ? 768 : 512;
        // keys are split only to fill the chip: each chunk's o goes through the memory twice
        const int64_t splits = base < fit ? fit / base : 1;
        int64_t chunk = ((keys + splits - 1) / splits + 255) / 256 * 256;
        if (splits == 1) chunk = 1 << 30;
        p.chunk = (int)(chunk < (1 << 30) ? chunk : 1 << 30);
        p.splits = (int)((keys + 64 + p.chunk - 1) / p.chunk);
        p.key_blocks = (int)blocks;
        p.present_at = (size_t)(B * p.key_blocks * c.heads * key_bytes * 64);
        p.part_at = (p.present_at + (size_t)B * p.key_blocks * (8 + 8 * c.heads) + 255) / 256 * 256;
        p.bytes = p.part_at + (p.splits > 1 ? (size_t)(base * p.splits * p.rows) * (c.D + 2) * sizeof(float) : 0);
        p.fits = base * p.splits <= kItems / 256;
        return p;
    }
    p.path = 1;
    const int groups = c.mode == 0 && dt == QLIN_BF16 ? c.D / c.g : 0;
    // Values as codes where a sequence's rows fit a tile of 16 / groups: one token of each, or twice the average (D up to
    // 128: there a second tile costs more than decoding). us, decoded and as codes: D 128, groups of 64, 64 sequences of
    // 5000 to 20000 keys 252 and 225, 16 of 1 to 3 rows of four heads over 2000 to 8000 keys 41 and 48; those of D 256,
    // groups of 128, 90 and 73. Four groups of D 128 take more columns than they save (107 and 137), not of D 256.
    p.codes = groups == 1 || (groups >= 2 && (groups <= 3 || (groups == 4 && c.D == 256)) &&
                              (T <= B || c.D > 128 ? mean : 2 * mean) <= 16 / groups);
    const int dup = p.codes ? groups : 1;
    // 32 columns where the rows fill more than 16, as the codes are decoded once for them: 64 sequences of 64 rows over
    // 16000 keys, D 128, 583 us, in tiles of 16 rows 666 (48 columns, of D 64, took 424 for 384: 48 + 16 rows instead of
    // 32 + 32; 33 to 48 rows, which take a second tile that reads and decodes their keys again, were not measured)
    p.nt = mean > 16 && c.D <= 128 ? 2 : 1;
    p.rows = 16 / dup * p.nt;
    p.tiles = one_row ? B * ((share + p.rows - 1) / p.rows) : T * share / p.rows + B;
    const int64_t base = p.tiles * c.heads;
    // Chunks for one to four rounds of the workgroups that the chip holds at once, never a little more than a round,
    // whichever should end first: rounds by the length of a chunk, and a last chunk that starts when all the others are
    // done, as lengths differ. bf16, D 128, us: 32 sequences of 4000 to 16000 keys, always 768 workgroups 111, so 89;
    // 16 sequences of 1 to 5 rows of 32 heads over those keys 124, so 95; 5 sequences of 1 to 3 rows over 2000 to 8000
    // keys 26 and 26.
    const int64_t slots = 256 * tile_residents(c.D, p.nt);     // (an MI355X has 256 CUs)
    const int64_t even = B * ((mean + p.rows - 1) / p.rows), ragged = T * share / p.rows + B / 2;
    const int64_t busy = (one_row ? p.tiles : (even > ragged ? even : ragged)) * c.heads;
    int64_t chunk = keys;
    double best = 0;
    for (int64_t r = 1; keys > kOneChunk && r <= 4; ++r) {
        const int64_t s = r * slots / busy > 1 ? r * slots / busy : 1;
        const int64_t size = ((keys + s - 1) / s + kStepKeys - 1) / kStepKeys * kStepKeys;
        const double time = ((double)busy * (double)s + (double)slots) * (double)(size + kStart);
        if (r == 1 || time < best) best = time, chunk = size;
    }
    if (chunk > kChunkMost) chunk = kChunkMost;
    while (chunk < keys && base * (keys / chunk) > kMany) chunk *= 2;
    if (chunk >= keys) chunk = 1 << 30;
    p.chunk = (int)(chunk < (1 << 30) ? chunk : 1 << 30);
    p.splits = (int)((keys + kKvUnit + p.chunk - 1) / p.chunk);
    if (p.splits > 1) p.bytes = (size_t)(base * p.splits * p.rows) * (c.D + 2) * sizeof(float);
    // (the join takes a wave a row, four a workgroup)
    p.fits = base * p.splits <= kItems / 256 && (p.splits == 1 || p.tiles * ((p.rows + 3) / 4) <= kItems / 256);
    return p;
}

}  // namespace qlin
