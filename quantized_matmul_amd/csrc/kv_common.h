// kv_common.h -- the cache of keys and values as the kernels see it, and the
// launcher declarations of the operators around it (rotary positions, writing,
// reading back, attention).
#pragma once

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

// How a call runs, from its sizes alone.
struct AttendPlan {
    int path;                        // 0 simple, 1 row tiles of the matrix cores, 2 prompt tiles
    int nt;                          // path 1: tiles of 16 rows a workgroup takes
    int64_t tiles;                   // row tiles of all sequences, at most
    int chunk, splits;               // keys a workgroup takes, workgroups along the keys
    size_t bytes;                    // workspace
};
AttendPlan attend_plan(int dt, int64_t T, int q_heads, int64_t B, int64_t width, const KvPool& c, int64_t window,
                       bool one_row);
hipError_t launch_attend(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                         hipStream_t st);
hipError_t launch_attend_simple(const AttendArgs& a, const KvPool& c, int dt, hipStream_t st);
hipError_t launch_attend_tile(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                              hipStream_t st);

}  // namespace qlin
