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

// Eight consecutive elements of dtype DT as they lie in memory.
template <int DT>
struct Eight {
    uint32_t d[DT == QLIN_F32 ? 8 : 4];
    __device__ __forceinline__ float at(int c) const {
        if constexpr (DT == QLIN_F32) return __uint_as_float(d[c]);
        const uint32_t h = (d[c / 2] >> (16 * (c & 1))) & 0xFFFFu;
        return DT == QLIN_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
    }
};

// 16-byte loads where `vec` (the tensor is 16-byte aligned and i a multiple of 8); STREAM: past the caches.
template <int DT, bool STREAM = false>
__device__ __forceinline__ Eight<DT> load8(const void* p, int64_t i, bool vec) {
    Eight<DT> r;
    constexpr int N = DT == QLIN_F32 ? 8 : 4;
    if (vec) {
        typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
        const u32x4* q = (const u32x4*)((const char*)p + i * (DT == QLIN_F32 ? 4 : 2));
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
            u32x4 t;
            if constexpr (STREAM) t = __builtin_nontemporal_load(q + h);
            else t = q[h];
            r.d[4 * h] = t[0]; r.d[4 * h + 1] = t[1]; r.d[4 * h + 2] = t[2]; r.d[4 * h + 3] = t[3];
        }
    } else if constexpr (DT == QLIN_F32) {
#pragma unroll
        for (int c = 0; c < 8; ++c) r.d[c] = ((const uint32_t*)p)[i + c];
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            r.d[c] = ((const uint16_t*)p)[i + 2 * c] | (uint32_t)((const uint16_t*)p)[i + 2 * c + 1] << 16;
    }
    return r;
}

// silu(gate) * up in fp32 with the hardware's 2^x and 1 / x, 1 ulp each, and
// the argument of 2^x rounded, which costs more the larger the gate: in all a
// relative error of at most (1.25 |gate| + 7) 2^-24. The result is rounded to
// four bits next, so that decides a code only within as much of a tie (2^-20 at
// a gate of 8, 2^-17 at -80). Below a gate of -87.3 the sigmoid, under 2^-126, is 0.
template <int DT>
__device__ __forceinline__ Eight<QLIN_F32> swiglu8(const Eight<DT>& gate, const Eight<DT>& up) {
    Eight<QLIN_F32> r;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float g = gate.at(c);
        const float s = g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -0x1.715476p+0f));
        r.d[c] = __float_as_uint(s * up.at(c));
    }
    return r;
}

// Bits of the largest magnitude of the eight as an fp32 number (infinity or
// above where one is not finite): integer maxima, since magnitudes order as
// their bits do.
template <int DT>
__device__ __forceinline__ uint32_t amax_bits(const Eight<DT>& v) {
    if constexpr (DT == QLIN_F32) {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) m = max_u(m, v.d[c] & 0x7FFFFFFFu);
        return m;
    } else {
        typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
        u16x2 m = __builtin_bit_cast(u16x2, v.d[0] & 0x7FFF7FFFu);
#pragma unroll
        for (int c = 1; c < 4; ++c)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v.d[c] & 0x7FFF7FFFu));
        const uint32_t h = m[0] > m[1] ? m[0] : m[1];
        if constexpr (DT == QLIN_BF16) return h << 16;
        return h >= 0x7C00u ? 0x7F800000u : __float_as_uint(f16_bits_to_f32(h));
    }
}

// The packed word of eight values; the four lanes of an aligned quad hold a
// block of 32 (all active) and get its scale byte. qlin_quantize's mxfp4 rule:
// shared exponent e = floor(log2 amax) - 2 in [-127, 127], byte e + 127 (0 for
// an all-zero block), codes the nearest E2M1 of v / 2^e, ties to even,
// saturated: what the hardware's conversion gives for every scale of 2^-126 and
// above (checked on the device over ties, their neighbours and random values).
// A block with a NaN or an infinity gets byte 255, the format's NaN.
template <int DT>
__device__ __forceinline__ uint32_t mxfp4_word(const Eight<DT>& v, uint32_t* byte) {
    uint32_t m = amax_bits<DT>(v);
    m = max_u(m, dpp_u<0xB1>(m));                                // quad_perm 1 0 3 2
    m = max_u(m, dpp_u<0x4E>(m));                                // quad_perm 2 3 0 1
    const uint32_t ex = m >> 23;                                 // 0 for an fp32 subnormal: its block is scaled by 2^-127
    *byte = ex >= 255u ? 255u : ex < 2u ? 0u : ex - 2u;
    uint32_t word = 0;
    if (ex < 3u) {                                               // scale 2^-127
#pragma unroll
        for (int c = 0; c < 8; ++c) word |= e2m1_code(__builtin_ldexpf(v.at(c), 127)) << (4 * c);
        return word;
    }
    const float scale = __uint_as_float(*byte << 23);
    if constexpr (DT == QLIN_F32) {
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v.at(0), v.at(1), scale, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v.at(2), v.at(3), scale, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v.at(4), v.at(5), scale, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v.at(6), v.at(7), scale, 3);
    } else if constexpr (DT == QLIN_BF16) {
        typedef __attribute__((ext_vector_type(2))) __bf16 b2;
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(b2, v.d[0]), scale, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(b2, v.d[1]), scale, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(b2, v.d[2]), scale, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(b2, v.d[3]), scale, 3);
    } else {
        typedef __attribute__((ext_vector_type(2))) _Float16 h2;
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, __builtin_bit_cast(h2, v.d[0]), scale, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, __builtin_bit_cast(h2, v.d[1]), scale, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, __builtin_bit_cast(h2, v.d[2]), scale, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, __builtin_bit_cast(h2, v.d[3]), scale, 3);
    }
    return ex >= 255u ? 0u : word;
}

// ------------------------------------------------------------------ row plan

// Experts of one call: two counters each in the 64 KB of LDS every kernel may ask for.
constexpr int64_t kMx4MaxExperts = 8000;
// Index rows of one call: their numbers, rounded up to a chunk of the plan, are 32-bit integers.
constexpr int64_t kMx4MaxRows = (1LL << 31) - (1LL << 14);

// A row tile: everything a workgroup needs to know of it in one 32-byte load.
struct Mx4Tile {
    uint32_t group;         // expert; E: rows without one, whose outputs are zeros
    uint32_t first, count;  // first row tile of the group, row tiles of the group
    uint32_t place, rows;   // first place of the group in perm, rows of the group
    uint32_t unused[3];
};

// Index rows grouped by expert and cut into row tiles. Rows whose expert is
// outside [0, E) form one more group, E, whose tiles write zeros.
struct Mx4Plan {
    Mx4Tile* tiles;
    uint32_t* total;        // [1] row tiles
    uint32_t* perm;         // [R] index rows by group
    uint32_t* counts;       // [chunks][E + 1] rows of each group in each chunk of rows; one more row for the scan
};

constexpr int kPlanMinTile = 64;   // least rows of a row tile

// Row tiles a plan has at most.
inline int64_t mx4_plan_max_tiles(int64_t R, int64_t E, int tile_rows) {
    return R / tile_rows + (E + 1 < R ? E + 1 : R);
}

}  // namespace qlin
