// mx4_common.h -- what the kernels of the mxfp4 products share: rounding eight
// values of an activation to a packed word, and the row plan of the product by
// experts.
#pragma once

#include "moe_common.h"

namespace qlin {

// ------------------------------------------------------- activation to mxfp4

// Nearest E2M1 code, ties to even, saturated.
__device__ __forceinline__ uint32_t e2m1_code(float v) {
    const float a = fabsf(v);
    const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                       (a > 5.0f);
    return c | ((__float_as_uint(v) >> 28) & 8u);
}

// Eight elements of dtype DT at element i; 16-byte loads where `vec` (the tensor
// is 16-byte aligned and i a multiple of 8).
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, bool vec, float (&v)[8]) {
    if (!vec) {
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = load_f<DT>(p, i + c);
    } else if constexpr (DT == QLIN_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 q = *(const float4*)((const float*)p + i + 4 * h);
            v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
        }
    } else {
        const uint4 q = *(const uint4*)((const uint16_t*)p + i);
        const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[2 * c] = DT == QLIN_BF16 ? bf16_bits_to_f32(d[c] & 0xFFFFu) : f16_bits_to_f32(d[c] & 0xFFFFu);
            v[2 * c + 1] = DT == QLIN_BF16 ? bf16_bits_to_f32(d[c] >> 16) : f16_bits_to_f32(d[c] >> 16);
        }
    }
}

// v = silu(v) * up in fp32, with one IEEE division; no contraction, so that
// every kernel rounds alike.
__device__ __forceinline__ void swiglu8(float (&v)[8], const float (&up)[8]) {
#pragma clang fp contract(off)
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = v[c] / (1.0f + expf(-v[c])) * up[c];
}

// The packed word of eight values; the four lanes of an aligned quad hold a
// block of 32 (all active) and get its scale byte. qlin_quantize's mxfp4 rule:
// shared exponent e = floor(log2 amax) - 2 in [-127, 127], byte e + 127 (0 for
// an all-zero block), codes the nearest E2M1 of v / 2^e. A block with a NaN or
// an infinity gets byte 255, the format's NaN.
__device__ __forceinline__ uint32_t mxfp4_word(const float (&v)[8], uint32_t* byte) {
    float amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        amax = fmaxf(amax, fabsf(v[c]));
        bad |= !(fabsf(v[c]) < INFINITY);
    }
    uint32_t m = bad ? 0x7F800000u : __float_as_uint(amax);      // ordered like the numbers
    m = max_u(m, dpp_u<0xB1>(m));                                // quad_perm 1 0 3 2
    m = max_u(m, dpp_u<0x4E>(m));                                // quad_perm 2 3 0 1
    if (m >= 0x7F800000u) {
        *byte = 255u;
        return 0u;
    }
    int e = m == 0u ? -127 : (m >> 23 ? (int)(m >> 23) - 127 : (31 - __builtin_clz(m)) - 149) - 2;
    e = e < -127 ? -127 : e;
    *byte = (uint32_t)(e + 127);
    uint32_t word = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) word |= e2m1_code(__builtin_ldexpf(v[c], -e)) << (4 * c);
    return word;
}

// ------------------------------------------------------------------ row plan

// Experts of one call: two counters each in the 64 KB of LDS every kernel may ask for.
constexpr int64_t kMx4MaxExperts = 8000;

// Index rows grouped by expert and cut into row tiles. Rows whose expert is
// outside [0, E) form one more group, E, whose tiles write zeros.
struct Mx4Plan {
    uint32_t* offsets;      // [E + 2] first place of each group in perm
    uint32_t* first_tile;   // [E + 2] first row tile of each group; the last entry is the number of tiles
    uint32_t* tile_group;   // group of each row tile
    uint32_t* perm;         // [R] index rows by group
    uint32_t* counts;       // [chunks][E + 1] rows of each group in each chunk of rows
};

constexpr int kPlanMinTile = 64;   // least rows of a row tile

// Row tiles a plan has at most.
inline int64_t mx4_plan_max_tiles(int64_t R, int64_t E, int tile_rows) {
    return R / tile_rows + (E + 1 < R ? E + 1 : R);
}

}  // namespace qlin
