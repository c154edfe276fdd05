// attend_plan.cpp -- which attention kernel a call takes and how its keys are
// split, from its sizes alone.
#include "kv_common.h"

namespace qlin {

hipError_t launch_attend_tile_64(const AttendArgs&, const KvPool&, int, const AttendPlan&, void*, hipStream_t);
hipError_t launch_attend_tile_96(const AttendArgs&, const KvPool&, int, const AttendPlan&, void*, hipStream_t);
hipError_t launch_attend_tile_128(const AttendArgs&, const KvPool&, int, const AttendPlan&, void*, hipStream_t);
hipError_t launch_attend_tile_192(const AttendArgs&, const KvPool&, int, const AttendPlan&, void*, hipStream_t);
hipError_t launch_attend_tile_256(const AttendArgs&, const KvPool&, int, const AttendPlan&, void*, hipStream_t);

namespace {
constexpr int64_t kStepKeys = 128;       // a workgroup's waves take this many keys at a time
constexpr int64_t kChunkMost = 2048;     // keys a workgroup takes at most
constexpr int64_t kWorkgroups = 2048;    // enough to fill the chip evenly
}  // namespace

AttendPlan attend_plan(int dt, int64_t T, int q_heads, int64_t B, int64_t width, const KvPool& c, int64_t window,
                       bool one_row) {
    AttendPlan p{};
    const bool sized = c.D == 64 || c.D == 96 || c.D == 128 || c.D == 192 || c.D == 256;
    if (dt == QLIN_F32 || !sized) return p;
    const int64_t share = q_heads / c.heads;
    const int64_t mean = (T * share + B - 1) / B;            // rows of a sequence and key head
    p.path = 1;
    p.nt = mean > 16 ? 2 : 1;
    const int64_t R = 16 * p.nt;
    p.tiles = one_row ? B * ((share + R - 1) / R) : T * share / R + B;
    // keys a tile can see, from the sizes: the table's, or the window before its first row and all behind that row,
    // which without a causal mask are as many as the sequence has rows
    int64_t keys = width * c.page;
    if (window && window < keys - T - kKvUnit) keys = window + T + kKvUnit;
    if (keys < 1) keys = 1;
    const int64_t base = p.tiles * c.heads;
    int64_t splits = (kWorkgroups + base - 1) / base;
    int64_t chunk = (keys + splits - 1) / splits;
    chunk = (chunk + kStepKeys - 1) / kStepKeys * kStepKeys;
    if (chunk > kChunkMost) chunk = kChunkMost;
    p.chunk = (int)chunk;
    p.splits = (int)((keys + kKvUnit + chunk - 1) / chunk);
    if (p.splits > 1) p.bytes = (size_t)(base * p.splits * R) * (c.D + 2) * sizeof(float);
    return p;
}

hipError_t launch_attend(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                         hipStream_t st) {
    if (p.path == 0) return launch_attend_simple(a, c, dt, st);
    switch (c.D) {
    case 64: return launch_attend_tile_64(a, c, dt, p, workspace, st);
    case 96: return launch_attend_tile_96(a, c, dt, p, workspace, st);
    case 128: return launch_attend_tile_128(a, c, dt, p, workspace, st);
    case 192: return launch_attend_tile_192(a, c, dt, p, workspace, st);
    case 256: return launch_attend_tile_256(a, c, dt, p, workspace, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qlin
