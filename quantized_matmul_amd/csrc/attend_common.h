// attend_common.h -- what the attention kernels share: a row's place among the
// sequences, the keys it sees, decoded values of a word.
#pragma once

#include "kv_common.h"

namespace qlin {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -__builtin_inff();

// Eight numbers of a word of E2M1 codes, times s.
__device__ __forceinline__ void e2m1_values(uint32_t w, float s, float (&v)[8]) {
#define QLIN_PAIR(i)                                                           \
    {                                                                          \
        const auto f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, i);   \
        v[2 * i] = f[0] * s;                                                   \
        v[2 * i + 1] = f[1] * s;                                               \
    }
    QLIN_PAIR(0) QLIN_PAIR(1) QLIN_PAIR(2) QLIN_PAIR(3)
#undef QLIN_PAIR
}

// Scale (and bias) of a group as numbers.
template <int MODE, int SDT>
__device__ __forceinline__ float scale_at(const void* p, int64_t i) {
    if constexpr (MODE == AFFINE) return load_f<SDT>(p, i);
    else if constexpr (MODE == NVFP4) return e4m3_to_f32(((const uint8_t*)p)[i]);
    else return e8m0_to_f32(((const uint8_t*)p)[i]);
}

}  // namespace
}  // namespace qlin
