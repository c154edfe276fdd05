// mx4_plan.h -- the row plan of the mxfp4 product by experts.
#pragma once

#include "moe_common.h"

namespace qlin {

// Experts of one call: two counters each in the 64 KB of LDS every kernel may ask for.
constexpr int64_t kMx4MaxExperts = 8000;

struct Mx4Plan {
    uint32_t* offsets;      // [E + 2] first place of each group in perm (group E: rows without an expert)
    uint32_t* first_tile;   // [E + 2] first row tile of each group; the last entry is the number of tiles
    uint32_t* tile_group;   // group of each row tile
    uint32_t* perm;         // [R] index rows by group
};

// Row tiles a plan has at most.
inline int64_t mx4_plan_max_tiles(int64_t R, int64_t E, int tile_rows) {
    return R / tile_rows + (E + 1 < R ? E + 1 : R);
}

hipError_t launch_mx4_plan(const int32_t* experts, int64_t R, int64_t E, int tile_rows, void* workspace, Mx4Plan* out,
                           hipStream_t st);

}  // namespace qlin
