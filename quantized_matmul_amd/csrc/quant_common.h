// quant_common.h -- the arithmetic of group-wise quantization, shared by the
// kernels that quantize weights (quant.hip) and rows of a cache (kv_store.hip):
// a word of codes from its elements, with its group's scale and bias.
//
// Every rounding step is explicit so that codes, scales and biases are
// bit-for-bit reproducible: fp32 subtraction, correctly rounded fp32
// division (__fdiv_rn), nearest-even (rintf), directed rounding into the
// storage dtype done on bit patterns. The files that include this are compiled
// with -ffp-contract=off.
#pragma once

#include <type_traits>

#include "qlin_common.h"

namespace qlin {
namespace {

// ------------------------------------------------- directed rounding (bits)

// bf16: truncation drops the low 16 bits (toward zero); one bf16 step away
// from zero is +1 on the 16-bit pattern for either sign.
__device__ __forceinline__ float bf16_round_down(float v) {
    uint32_t u = __float_as_uint(v);
    uint32_t t = u & 0xFFFF0000u;
    if ((u & 0xFFFFu) && (u >> 31)) t += 0x10000u;  // negative: away from zero is down
    return __uint_as_float(t);
}
__device__ __forceinline__ float bf16_round_up(float v) {
    uint32_t u = __float_as_uint(v);
    uint32_t t = u & 0xFFFF0000u;
    if ((u & 0xFFFFu) && !(u >> 31)) t += 0x10000u;  // positive: away from zero is up
    return __uint_as_float(t);
}

// f16: nearest-even conversion, then one step if it landed on the wrong side.
__device__ __forceinline__ uint32_t f16_step(uint32_t h, bool up) {
    bool neg = h & 0x8000u;
    if ((h & 0x7FFFu) == 0) return up ? 0x0001u : 0x8001u;  // +-0
    return (up != neg) ? h + 1u : h - 1u;                   // away from / toward zero
}
__device__ __forceinline__ float f16_round_dir(float v, bool up) {
    uint32_t h = f32_to_f16_rne(v);
    float hv = f16_bits_to_f32(h);
    if (up ? (hv < v) : (hv > v)) h = f16_step(h, up);
    return f16_bits_to_f32(h);
}

template <int DT>
__device__ __forceinline__ float round_down_to(float v) {
    if constexpr (DT == QLIN_F32) return v;
    else if constexpr (DT == QLIN_BF16) return bf16_round_down(v);
    else return f16_round_dir(v, false);
}
template <int DT>
__device__ __forceinline__ float round_up_to(float v) {
    if constexpr (DT == QLIN_F32) return v;
    else if constexpr (DT == QLIN_BF16) return bf16_round_up(v);
    else return f16_round_dir(v, true);
}

// ------------------------------------------------- small formats (encoding)

// E2M1 nearest-even, saturating at 6, sign kept. The magnitude code is the
// number of rounding boundaries at or below |v|; at a tie the boundary
// counts toward the even code (0.25->0, 0.75->1.0, 1.25->1.0, 1.75->2,
// 2.5->2, 3.5->4, 5->4).
__device__ __forceinline__ uint32_t e2m1_encode(float v) {
    float a = fabsf(v);
    uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
                 (a >= 3.5f) + (a > 5.0f);
    return c | ((__float_as_uint(v) >> 28) & 8u);
}

// E4M3 (FN) nearest-even, saturating at 448, sign kept.
__device__ __forceinline__ uint32_t e4m3_encode(float v) {
    float a = fabsf(v);
    uint32_t mag;
    if (a >= 448.0f) {
        mag = 0x7Eu;
    } else if (a < 0.015625f) {  // below 2^-6: subnormal grid of spacing 2^-9
        mag = (uint32_t)rintf(__builtin_ldexpf(a, 9));
    } else {
        int E = (int)(__float_as_uint(a) >> 23) - 127;   // a is a normal fp32 here
        float t = __builtin_ldexpf(a, 3 - E);             // [8, 16), exact
        mag = (uint32_t)((E + 7) << 3) + ((uint32_t)rintf(t) - 8u);
    }
    return mag | ((__float_as_uint(v) >> 24) & 0x80u);
}

// floor(log2 a) of a positive finite fp32 (normal or subnormal).
__device__ __forceinline__ int floor_log2(float a) {
    uint32_t u = __float_as_uint(a);
    uint32_t e = u >> 23;
    if (e) return (int)e - 127;
    return (31 - __builtin_clz(u & 0x7FFFFFu)) - 149;
}

// PER elements of dtype DT starting at element i (i a multiple of PER).
template <int DT, int PER, bool VEC>
__device__ __forceinline__ void load_chunk(const void* w, int64_t i, float (&v)[PER]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = load_f<DT>(w, i + e);
    } else if constexpr (DT == QLIN_F32) {
        const float4* p = (const float4*)((const float*)w + i);
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) {
            const float4 t = p[q];
            v[4 * q] = t.x; v[4 * q + 1] = t.y; v[4 * q + 2] = t.z; v[4 * q + 3] = t.w;
        }
    } else {
        constexpr int NW = PER / 2;    // dwords of 16-bit elements
        uint32_t d[NW];
        if constexpr (NW % 4 == 0) {
            const uint4* p = (const uint4*)((const uint16_t*)w + i);
#pragma unroll
            for (int q = 0; q < NW / 4; ++q) {
                const uint4 t = p[q];
                d[4 * q] = t.x; d[4 * q + 1] = t.y; d[4 * q + 2] = t.z; d[4 * q + 3] = t.w;
            }
        } else {   // NW == 2
            const uint2 t = *(const uint2*)((const uint16_t*)w + i);
            d[0] = t.x; d[1] = t.y;
        }
#pragma unroll
        for (int q = 0; q < NW; ++q) {
            if constexpr (DT == QLIN_BF16) {
                v[2 * q] = bf16_bits_to_f32(d[q] & 0xFFFFu);
                v[2 * q + 1] = bf16_bits_to_f32(d[q] >> 16);
            } else {
                v[2 * q] = f16_bits_to_f32(d[q] & 0xFFFFu);
                v[2 * q + 1] = f16_bits_to_f32(d[q] >> 16);
            }
        }
    }
}

// The IEEE fp32 quotient d / s from r = 1/s correctly rounded in fp64:
// (float)(d * r) rounds the fp64 product once more, to fp32. The product is
// within 2^-52 (relative) of d / s, and a quotient of two 24-bit
// significands that is not itself an fp32 value lies at least 2^-48 from
// every fp32 rounding boundary in the normal range (a midpoint has 25
// significant bits, and d - s * midpoint is a nonzero multiple of a unit
// 2^-47 of d), so both roundings land on the same fp32 value. Quotients in
// the subnormal range may differ in their last bit; every caller maps such
// a value to code 0 (affine) or to a signed zero (E2M1), as it does the
// exact quotient. One fp64 reciprocal per word replaces a division per
// element, which bound the quantize kernels on VALU issue.
__device__ __forceinline__ float div_by_recip(float d, double r) { return (float)((double)d * r); }

// Min (MIN) or max of v over the LPG adjacent lanes of a group, LPG a power
// of two <= 64. Each stage merges two neighbouring blocks of lanes with the
// lower block's value as the first operand, so among equal values (+0 and
// -0) every lane ends with the first one in element order, as a sequential
// scan with plain comparisons keeps it.
template <int LPG, bool MIN>
__device__ __forceinline__ float group_minmax(float v) {
#pragma unroll
    for (int off = 1; off < LPG; off <<= 1) {
        const float p = __shfl_xor(v, off, 64);
        const bool low = (threadIdx.x & off) == 0;
        const float a = low ? v : p, b = low ? p : v;   // a: lower block, b: upper block
        v = MIN ? ((b < a) ? b : a) : ((b > a) ? b : a);
    }
    return v;
}

// Max of non-negative v over the LPG adjacent lanes of a group.
template <int LPG>
__device__ __forceinline__ float group_amax(float v) {
#pragma unroll
    for (int off = 1; off < LPG; off <<= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

// One packed word of codes from its PER elements v; the LPG lanes of a
// group hold its consecutive words (whole groups are live or not).
template <int DT, int BITS, int LPG>
__device__ __forceinline__ void quantize_affine_word(const float (&v)[32 / BITS], int64_t wid, bool live,
                                                     uint32_t* __restrict__ wq, void* __restrict__ scales,
                                                     void* __restrict__ biases) {
    constexpr int PER = 32 / BITS;
    const int n = (1 << BITS) - 1;
    // group min and max; plain comparisons (not fminf/fmaxf) keep the first
    // of +0/-0 within a lane, and the lanes are combined in element order
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int e = 1; e < PER; ++e) {
        lo = (v[e] < lo) ? v[e] : lo;
        hi = (v[e] > hi) ? v[e] : hi;
    }
    lo = group_minmax<LPG, true>(lo);
    hi = group_minmax<LPG, false>(hi);
    const float z = round_down_to<DT>(lo);
    const float s = round_up_to<DT>(__fdiv_rn(hi - z, (float)n));

    uint32_t word = 0;
    if (s != 0.0f) {
        const double r = 1.0 / (double)s;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            float t = rintf(div_by_recip(v[e] - z, r));
            t = fminf(fmaxf(t, 0.0f), (float)n);
            word |= (uint32_t)t << (e * BITS);
        }
    }
    if (live) {
        wq[wid] = word;
        if ((threadIdx.x & (LPG - 1)) == 0) {
            const int64_t gid = wid / LPG;
            store_f<DT>(scales, gid, s);
            store_f<DT>(biases, gid, z);
        }
    }
}

// Block scale of a microscaled group from its amax ("Emily.QuantizedWeight",
// Microscaled modes; OCP MX shared exponent for mx*, E4M3(amax/6) for
// nvfp4): the scale byte, and the divisor (nvfp4) or exponent (mx*) the
// elements are encoded with.
template <int MODE>
struct MicroScale {
    uint32_t sbyte;
    float sc;   // nvfp4 element divisor
    double rsc; // its fp64 reciprocal (0 when sc is 0)
    int e;      // mx shared exponent
};
template <int MODE>
__device__ __forceinline__ MicroScale<MODE> micro_scale(float amax) {
    MicroScale<MODE> m{0u, 0.0f, 0.0, 0};
    if constexpr (MODE == NVFP4) {
        m.sbyte = e4m3_encode(__fdiv_rn(amax, 6.0f));
        m.sc = e4m3_to_f32(m.sbyte);
        m.rsc = m.sc == 0.0f ? 0.0 : 1.0 / (double)m.sc;
    } else {
        constexpr int EMAX_ELEM = (MODE == MXFP8) ? 8 : 2;
        int e = (amax == 0.0f) ? -127 : floor_log2(amax) - EMAX_ELEM;
        e = e < -127 ? -127 : (e > 127 ? 127 : e);
        m.e = e;
        m.sbyte = (uint32_t)(e + 127);
    }
    return m;
}

// Element code of v under the group's scale.
template <int MODE>
__device__ __forceinline__ uint32_t micro_encode(float v, const MicroScale<MODE>& m) {
    if constexpr (MODE == NVFP4)
        return (m.sc == 0.0f) ? ((__float_as_uint(v) >> 28) & 8u) : e2m1_encode(div_by_recip(v, m.rsc));
    else if constexpr (MODE == MXFP8)
        return e4m3_encode(__builtin_ldexpf(v, -m.e));
    else
        return e2m1_encode(__builtin_ldexpf(v, -m.e));
}

template <int MODE, int LPG>
__device__ __forceinline__ void quantize_micro_word(const float (&v)[MODE == MXFP8 ? 4 : 8], int64_t wid,
                                                    bool live, uint32_t* __restrict__ wq,
                                                    uint8_t* __restrict__ scales) {
    constexpr int BITS = (MODE == MXFP8) ? 8 : 4;
    constexpr int PER = 32 / BITS;
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < PER; ++e) amax = fmaxf(amax, fabsf(v[e]));
    const MicroScale<MODE> m = micro_scale<MODE>(group_amax<LPG>(amax));
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) word |= micro_encode<MODE>(v[k], m) << (k * BITS);
    if (live) {
        wq[wid] = word;
        if ((threadIdx.x & (LPG - 1)) == 0) scales[wid / LPG] = (uint8_t)m.sbyte;
    }
}

template <typename F>
hipError_t dispatch_dtype(int dt, F&& f) {
    switch (dt) {
    case QLIN_F32: return f(std::integral_constant<int, QLIN_F32>{});
    case QLIN_BF16: return f(std::integral_constant<int, QLIN_BF16>{});
    case QLIN_F16: return f(std::integral_constant<int, QLIN_F16>{});
    default: return hipErrorInvalidValue;
    }
}

// lanes per group: g / PER, a power of two from 1 to 32
template <class F>
hipError_t dispatch_lpg(int lpg, F&& f) {
    switch (lpg) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    default: return hipErrorInvalidValue;
    }
}

}  // namespace
}  // namespace qlin
