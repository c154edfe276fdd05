// attend.cpp -- the attention kernel that a plan names.
#include "kv_common.h"

namespace qlin {

#define QLIN_ATTEND(D) \
    hipError_t launch_attend_##D(const AttendArgs&, const KvPool&, int, const AttendPlan&, void*, hipStream_t);
QLIN_ATTEND(64) QLIN_ATTEND(96) QLIN_ATTEND(128) QLIN_ATTEND(192) QLIN_ATTEND(256)
#undef QLIN_ATTEND

hipError_t launch_attend(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                         hipStream_t st) {
    if (p.path == 0) return launch_attend_simple(a, c, dt, st);
    switch (c.D) {
    case 64: return launch_attend_64(a, c, dt, p, workspace, st);
    case 96: return launch_attend_96(a, c, dt, p, workspace, st);
    case 128: return launch_attend_128(a, c, dt, p, workspace, st);
    case 192: return launch_attend_192(a, c, dt, p, workspace, st);
    case 256: return launch_attend_256(a, c, dt, p, workspace, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qlin
