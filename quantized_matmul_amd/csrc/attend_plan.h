// attend_plan.h -- which attention kernel a call takes and how its keys are
// split, from its sizes alone. Integers only, as kv_index.h.
#pragma once

#include <stddef.h>

#include "../../include/qlin.h"
#include "kv_index.h"

namespace qlin {

struct AttendPlan {
    int path;                        // 0 simple, 1 row tiles, 2 prompt tiles
    int nt;                          // path 1: runs of 16 rows of a tile
    int64_t tiles;                   // row tiles of all sequences, at most
    int chunk, splits;               // keys a workgroup takes, workgroups along the keys
    int key_blocks;                  // path 2: blocks of 64 keys of a sequence, at most
    size_t part_at, present_at;      // path 2: places in the workspace (its blocks lie at 0)
    size_t bytes;                    // workspace
};

inline AttendPlan attend_plan(int dt, int64_t T, int q_heads, int64_t B, int64_t width, const KvPool& c, int64_t window,
                              bool one_row) {
    constexpr int64_t kStepKeys = 128;       // the waves of a row tile's workgroup take this many keys at a time
    constexpr int64_t kChunkMost = 2048;     // keys such a workgroup takes at most
    constexpr int64_t kWorkgroups = 2048;    // enough of them to fill the chip evenly
    constexpr int64_t kPromptRows = 64;      // rows of a sequence and key head, on average, from which a prompt is one
    constexpr int64_t kImages = 1LL << 33;   // bytes of decoded keys and values at most
    AttendPlan p{};
    const bool sized = c.D == 64 || c.D == 96 || c.D == 128 || c.D == 192 || c.D == 256;
    if (dt == QLIN_F32 || !sized) return p;
    const int64_t share = q_heads / c.heads, held = width * c.page;
    const int64_t mean = (T * share + B - 1) / B;
    // keys a tile can see, from the sizes: the table's, or the window before its first row and all behind that row,
    // which without a causal mask are as many as the sequence has rows
    int64_t keys = held;
    if (window && window < keys - T - 64) keys = window + T + 64;
    if (keys < 1) keys = 1;
    const int64_t blocks = (held + 63) / 64;
    if (mean > kPromptRows && blocks * B <= kImages / ((int64_t)c.heads * c.D * 256)) {
        p.path = 2;
        const int64_t R = c.D <= 128 ? 256 : 128;
        p.tiles = T * share / R + B;
        const int64_t base = p.tiles * c.heads;
        int64_t splits = (512 + base - 1) / base;
        int64_t chunk = ((keys + splits - 1) / splits + 255) / 256 * 256;
        if (splits == 1) chunk = 1 << 30;
        p.chunk = (int)(chunk < (1 << 30) ? chunk : 1 << 30);
        p.splits = (int)((keys + 64 + p.chunk - 1) / p.chunk);
        p.key_blocks = (int)(blocks ? blocks : 1);
        p.present_at = (size_t)B * p.key_blocks * c.heads * c.D * 256;
        p.part_at = (p.present_at + (size_t)B * p.key_blocks * (8 + 4 * c.heads) + 255) / 256 * 256;
        p.bytes = p.part_at + (p.splits > 1 ? (size_t)(base * p.splits * R) * (c.D + 2) * sizeof(float) : 0);
        return p;
    }
    p.path = 1;
    p.nt = mean > 16 ? 2 : 1;
    const int64_t R = 16 * p.nt;
    p.tiles = one_row ? B * ((share + R - 1) / R) : T * share / R + B;
    const int64_t base = p.tiles * c.heads;
    const int64_t splits = (kWorkgroups + base - 1) / base;
    int64_t chunk = ((keys + splits - 1) / splits + kStepKeys - 1) / kStepKeys * kStepKeys;
    if (chunk > kChunkMost) chunk = kChunkMost;
    p.chunk = (int)chunk;
    p.splits = (int)((keys + kKvUnit + chunk - 1) / chunk);
    if (p.splits > 1) p.bytes = (size_t)(base * p.splits * R) * (c.D + 2) * sizeof(float);
    return p;
}

}  // namespace qlin
