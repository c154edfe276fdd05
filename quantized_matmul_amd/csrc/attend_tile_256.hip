// attend_tile_256.hip -- the row-tile attention kernels for heads of 256.
#include "attend_tile.h"

namespace qlin {
hipError_t launch_attend_tile_256(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                                 hipStream_t st) {
    return launch_tile_of<256>(a, c, dt, p, workspace, st);
}
}  // namespace qlin
