// kv_common.h -- the cache of keys and values as the kernels see it, and the
// launcher declarations of the operators around it (rotary positions, writing,
// reading back, attention).
#pragma once

#include "attend_plan.h"
#include "kv_index.h"
#include "qlin_common.h"

namespace qlin {

// Limits of a cache. Row numbers over 16 have to fit 31 bits (the attention
// kernels keep them so), slots an int32.
constexpr int kKvMaxHeads = 4096;
constexpr int kKvMaxPage = 1 << 24;
constexpr int kKvMaxDim = 256;
constexpr int kRotaryMaxDim = 256;

hipError_t launch_kv_write(const KvPool& c, const void* k, const void* v, int dt, int64_t T, int64_t k_stride,
                           int64_t v_stride, const int32_t* slots, hipStream_t st);
hipError_t launch_kv_read(const KvPool& c, const int32_t* slots, int64_t T, void* k, void* v, int dt, hipStream_t st);

struct RotaryArgs {
    const void* x;
    void* y;
    int64_t T, x_stride, y_stride;   // strides of tokens, in elements
    int heads, D, R;
    const int32_t* positions;
    const float* freqs;
    float scale;
    int interleaved, backward;
};
hipError_t launch_rotary(const RotaryArgs& a, int dt, hipStream_t st);

hipError_t launch_attend(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                         hipStream_t st);
hipError_t launch_attend_simple(const AttendArgs& a, const KvPool& c, int dt, hipStream_t st);

}  // namespace qlin
