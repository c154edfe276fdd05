// attend_tile_64.hip -- the row-tile attention kernels for heads of 64.
#include "attend_tile.h"

namespace qlin {
hipError_t launch_attend_tile_64(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                                 hipStream_t st) {
    return launch_tile_of<64>(a, c, dt, p, workspace, st);
}
}  // namespace qlin
