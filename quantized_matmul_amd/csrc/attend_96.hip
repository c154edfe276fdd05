// attend_96.hip -- the matrix-core attention kernels for heads of 96.
#include "attend_prompt.h"
#include "attend_tile.h"

namespace qlin {
hipError_t launch_attend_96(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                            hipStream_t st) {
    return p.path == 1 ? launch_tile_of<96>(a, c, dt, p, workspace, st) : launch_prompt_of<96>(a, c, dt, p, workspace, st);
}
}  // namespace qlin
