// kv_store.hip -- rows of keys and values into a 4-bit cache, and back.
//
// Writing is qlin_quantize's rule on each head's row, its place looked up in
// `slots`: the same bytes, by fewer instructions for 4 bits (below). A thread
// owns one packed word, the lanes of a group are neighbours, as in quant.hip.
// Reading decodes a word a thread.
//
// Both are bound by the memory where they are large: 2 D H elements of a token
// on one side, D H bytes of codes and the scales on the other. A head's row is
// D/2 contiguous bytes of a page, the next token's follows it: a block takes WPT
// runs of 256 words, so that neighbouring tokens' rows of a page are written
// (read) together.
//
// Measured, bf16, groups of 64: 32768 tokens of 8 heads of 128 written (172 MB)
// in 55 us, 3.1 TB/s: 23 M vector instructions, 40 us of the units' time, and
// what memory takes before and after them; read back 31 us, 131072 of them 105
// us (684 MB, 6.5 TB/s: the codes of repeated reads lie in the last-level cache).
//
// The arithmetic, bit for bit that of quant_common.h:
//   affine   q = rint(fl(d / s)), d = fl(v - z). The quotient is an fp64 product
//            with 1 / s rounded once more, as there, and so is fl((max - z) / 15):
//            a quotient of two 24-bit numbers lies 2^-48 from any rounding boundary
//            or on it. s is rounded up, so q is in [0, 15] without a clamp, but
//            where an fp32 s is a few of the smallest steps: to nearest it may be
//            half a step short, of 15 steps and less enough for a q of 15.5.
//            v_cvt_pk_u8_f32 rounds it to the nearest even byte, a NaN to zero.
//            Minimum and maximum by the hardware's min and max; only where the
//            minimum is zero does the order of +0 and -0 count, and only where a
//            word's first value is a NaN is it not passed over: plain comparisons
//            decide there, which may leave values of that word outside [z, z + 15 s].
//   mxfp4, nvfp4  the hardware's E2M1 conversion (nearest even, saturating) of
//            v at the block's power of two, or of fl(v / s) at scale one; but not
//            of a NaN, which is no zero there.

#include "kv_common.h"
#include "quant_common.h"

namespace qlin {
namespace {

struct StoreArgs {
    const void* x[2];            // write: rows to take; read: unused
    void* y[2];                  // read: rows to give
    int64_t stride[2];           // write: elements between tokens
    KvPool c;
    const int32_t* slots;
    int64_t T, slots_end;
    FastDiv by_row, by_head, by_page;    // words of a token, words of a head's row, places of a page
};

// Token and place in its row of word `at` past the block's first token.
struct WordPlace {
    int64_t t;
    uint32_t head, w;
};
__device__ __forceinline__ WordPlace word_place(const StoreArgs& a, int64_t t0, uint32_t at) {
    const uint32_t head_words = a.c.D / 8;
    const uint32_t dt = a.by_row(at), r = at - dt * (head_words * a.c.heads), h = a.by_head(r);
    return {t0 + dt, h, r - h * head_words};
}

// Number of the word in the pool, or -1 where the slot names no place.
__device__ __forceinline__ int64_t pool_word(const StoreArgs& a, int32_t slot, const WordPlace& p) {
    if (slot < 0 || slot >= a.slots_end) return -1;
    const uint32_t page = a.by_page((uint32_t)slot), o = (uint32_t)slot - page * (uint32_t)a.c.page;
    return ((int64_t)(page * (uint64_t)a.c.heads + p.head) * a.c.page + o) * (a.c.D / 8) + p.w;
}

// v of the lane that stands for the neighbouring block of OFF lanes, in blocks
// whose lanes all hold one value: a DPP step within a row of 16 lanes.
template <int OFF>
__device__ __forceinline__ float from_neighbour(float v) {
    static_assert(OFF <= 8, "a row of 16 lanes");
    constexpr int CTRL = OFF == 1 ? 0xB1 : (OFF == 2 ? 0x4E : (OFF == 4 ? 0x141 : 0x140));   // quad swaps, mirrors
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LPG, int OFF = 1>
__device__ __forceinline__ float group_most(float v) {
    if constexpr (OFF < LPG) return group_most<LPG, 2 * OFF>(fmaxf(v, from_neighbour<OFF>(v)));
    else return v;
}

// 1 / s for a finite s other than zero: Newton's iteration from the hardware's
// estimate, its error squared twice (under 2^-51).
__device__ __forceinline__ double reciprocal(float s) {
    const double d = s;
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
    return __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
}

template <int DT, int LPG>
__device__ __forceinline__ uint32_t affine_word(const float (&v)[8], float* scale, float* bias) {
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = fminf(lo, v[e]);
        hi = fmaxf(hi, v[e]);
    }
    lo = -group_most<LPG>(-lo);
    hi = group_most<LPG>(hi);
    bool clamp = __any(v[0] != v[0]);
    if (clamp || __any(lo == 0.0f)) {
        float l = v[0], h = v[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) {
            l = (v[e] < l) ? v[e] : l;
            h = (v[e] > h) ? v[e] : h;
        }
        lo = group_minmax<LPG, true>(l);
        hi = group_minmax<LPG, false>(h);
    }
    const float z = round_down_to<DT>(lo);
    const float s = round_up_to<DT>((float)((double)(hi - z) * (1.0 / 15.0)));
    *scale = s;
    *bias = z;
    const double r = s != 0.0f ? reciprocal(s) : 0.0;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = (float)((double)(v[e] - z) * r);
    if constexpr (DT == QLIN_F32) clamp |= __any(s < 0x1p-145f) != 0;      // 16 steps
    if (clamp) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = q[e] > 0.0f ? fminf(q[e], 15.0f) : 0.0f;
    }
    uint32_t even = 0, odd = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        even = __builtin_amdgcn_cvt_pk_u8_f32(q[2 * e], e, even);
        odd = __builtin_amdgcn_cvt_pk_u8_f32(q[2 * e + 1], e, odd);
    }
    return even | (odd << 4);
}

__device__ __forceinline__ uint32_t e2m1_word(const float (&v)[8], float scale) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
}

template <int MODE, int LPG>
__device__ __forceinline__ uint32_t micro_word(const float (&v)[8], uint32_t* byte) {
    float most = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
    const MicroScale<MODE> m = micro_scale<MODE>(group_most<LPG>(most));
    *byte = m.sbyte;
    bool each = MODE == MXFP4 && __any(m.e == -127);         // the conversion's scale has to be a normal number
    each |= __any(__builtin_isunordered(v[0], v[1]) | __builtin_isunordered(v[2], v[3]) | __builtin_isunordered(v[4], v[5]) |
                  __builtin_isunordered(v[6], v[7])) != 0;
    if (each) {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) w |= micro_encode<MODE>(v[k], m) << (4 * k);
        return w;
    }
    if constexpr (MODE == NVFP4) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = m.sc == 0.0f ? __uint_as_float(__float_as_uint(v[e]) & 0x80000000u) : div_by_recip(v[e], m.rsc);
        return e2m1_word(q, 1.0f);
    } else {
        return e2m1_word(v, __uint_as_float(m.sbyte << 23));
    }
}

template <int DT, int MODE, bool VEC, int LPG, int WPT>
__global__ void __launch_bounds__(256) kv_write_kernel(StoreArgs a) {
    const KvPool& c = a.c;
    const int side = blockIdx.y;
    const uint32_t row_words = (uint32_t)(c.D / 8) * c.heads;
    const int64_t first = (int64_t)blockIdx.x * (256 * WPT), t0 = first / row_words;
    const uint32_t r0 = (uint32_t)(first - t0 * row_words) + threadIdx.x;
    float v[WPT][8];
    int64_t word[WPT];
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const WordPlace p = word_place(a, t0, r0 + 256 * j);
        const bool live = p.t < a.T;
        load_chunk<DT, 8, VEC>(a.x[side], live ? p.t * a.stride[side] + p.head * c.D + p.w * 8 : 0, v[j]);
        word[j] = pool_word(a, live ? a.slots[p.t] : -1, p);
    }
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const bool leads = (threadIdx.x & (LPG - 1)) == 0;
        if constexpr (MODE == AFFINE) {
            float s, z;
            const uint32_t w = affine_word<DT, LPG>(v[j], &s, &z);
            if (word[j] < 0) continue;
            c.codes[side][word[j]] = w;
            if (leads) {
                store_f<DT>(c.scales[side], word[j] / LPG, s);
                store_f<DT>(c.biases[side], word[j] / LPG, z);
            }
        } else {
            uint32_t byte;
            const uint32_t w = micro_word<MODE, LPG>(v[j], &byte);
            if (word[j] < 0) continue;
            c.codes[side][word[j]] = w;
            if (leads) ((uint8_t*)c.scales[side])[word[j] / LPG] = (uint8_t)byte;
        }
    }
}

// Two outputs of a 16-bit type, rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == QLIN_BF16) {
        typedef __attribute__((ext_vector_type(2))) __bf16 T2;
        return __builtin_bit_cast(uint32_t, T2{(__bf16)a, (__bf16)b});
    } else {
        return f32_to_f16_rne(a) | (f32_to_f16_rne(b) << 16);
    }
}

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

template <int SDT, int DT, int MODE, int WPT, bool PAST>
__global__ void __launch_bounds__(256) kv_read_kernel(StoreArgs a) {
    const KvPool& c = a.c;
    const int side = blockIdx.y;
    const uint32_t row_words = (uint32_t)(c.D / 8) * c.heads;
    const int64_t first = (int64_t)blockIdx.x * (256 * WPT), t0 = first / row_words;
    const uint32_t r0 = (uint32_t)(first - t0 * row_words) + threadIdx.x;
    const int group_shift = 31 - __builtin_clz((unsigned)c.g / 8);   // words of a group: a power of two
    uint32_t word[WPT];
    float s[WPT], z[WPT];
    bool live[WPT];
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const WordPlace p = word_place(a, t0, r0 + 256 * j);
        live[j] = p.t < a.T;
        const int64_t at = pool_word(a, live[j] ? a.slots[p.t] : -1, p);
        word[j] = 0;
        s[j] = z[j] = 0.0f;
        if (at >= 0) {
            const int64_t group = at >> group_shift;
            word[j] = c.codes[side][at];
            if constexpr (MODE == AFFINE) {
                s[j] = load_f<SDT>(c.scales[side], group);
                z[j] = load_f<SDT>(c.biases[side], group);
            } else {
                const uint32_t b = ((const uint8_t*)c.scales[side])[group];
                s[j] = MODE == NVFP4 ? e4m3_to_f32(b) : e8m0_to_f32(b);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        if (!live[j]) continue;
        const int64_t e = (t0 * row_words + r0 + 256 * j) * 8;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (MODE == AFFINE) {
                v[i] = __builtin_fmaf(s[j], (float)((word[j] >> (4 * i)) & 15u), z[j]);
            } else {
                // two codes an instruction, at scale one: the product with the scale rounds nothing
                const auto f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[j] >> (i / 2 * 8), 1.0f, 0);
                v[i] = f[i & 1] * s[j];
            }
        }
        auto put = [](u32x4 x, u32x4* to) {
            if constexpr (PAST) __builtin_nontemporal_store(x, to);
            else *to = x;
        };
        if constexpr (DT == QLIN_F32) {
            u32x4* y = (u32x4*)((float*)a.y[side] + e);
            put(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, y);
            put(u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])}, y + 1);
        } else {
            put(u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])},
                (u32x4*)((uint16_t*)a.y[side] + e));
        }
    }
}

// Words a thread takes: four runs of 256 keep neighbouring tokens' rows of a
// page in one block; a small call is spread over the CUs instead.
constexpr int64_t kSpreadWords = 256 * 1024;

unsigned blocks(int64_t words, int wpt) { return (unsigned)((words + 256 * wpt - 1) / (256 * wpt)); }

StoreArgs store_args(const KvPool& c, const int32_t* slots, int64_t T) {
    StoreArgs a{};
    a.c = c;
    a.slots = slots;
    a.T = T;
    a.slots_end = c.pages * c.page;
    a.by_row = FastDiv::by((uint32_t)(c.D / 8) * c.heads);
    a.by_head = FastDiv::by((uint32_t)(c.D / 8));
    a.by_page = FastDiv::by((uint32_t)c.page);
    return a;
}

}  // namespace

hipError_t launch_kv_write(const KvPool& c, const void* k, const void* v, int dt, int64_t T, int64_t k_stride,
                           int64_t v_stride, const int32_t* slots, hipStream_t st) {
    StoreArgs a = store_args(c, slots, T);
    a.x[0] = k;
    a.x[1] = v;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    const int64_t words = T * c.heads * (c.D / 8);
    const int elem = dt == QLIN_F32 ? 4 : 2;
    const bool vec = (((uintptr_t)k | (uintptr_t)v | (uintptr_t)(k_stride * elem) | (uintptr_t)(v_stride * elem)) & 15) == 0;
    return dispatch_dtype(dt, [&](auto dtc) -> hipError_t {
        constexpr int DT = decltype(dtc)::value;
        return dispatch_lpg(c.g / 8, [&](auto lpgc) -> hipError_t {
            constexpr int LPG = decltype(lpgc)::value;
            auto go = [&](auto mode, auto vc, auto wpt) -> hipError_t {
                constexpr int M = decltype(mode)::value, W = decltype(wpt)::value;
                kv_write_kernel<DT, M, decltype(vc)::value, LPG, W><<<dim3(blocks(words, W), 2), 256, 0, st>>>(a);
                return hipGetLastError();
            };
            auto sized = [&](auto mode, auto vc) -> hipError_t {
                return words < kSpreadWords ? go(mode, vc, std::integral_constant<int, 1>{})
                                            : go(mode, vc, std::integral_constant<int, 4>{});
            };
            auto moded = [&](auto vc) -> hipError_t {
                if constexpr (LPG == 2) return sized(std::integral_constant<int, NVFP4>{}, vc);
                else if constexpr (LPG == 4 || LPG == 8 || LPG == 16)
                    return c.mode == AFFINE ? sized(std::integral_constant<int, AFFINE>{}, vc)
                                            : sized(std::integral_constant<int, MXFP4>{}, vc);
                else return hipErrorInvalidValue;
            };
            return vec ? moded(std::true_type{}) : moded(std::false_type{});
        });
    });
}

hipError_t launch_kv_read(const KvPool& c, const int32_t* slots, int64_t T, void* k, void* v, int dt, hipStream_t st) {
    StoreArgs a = store_args(c, slots, T);
    a.y[0] = k;
    a.y[1] = v;
    const int64_t words = T * c.heads * (c.D / 8);
    const bool past = words * (2 * 8 * (dt == QLIN_F32 ? 4 : 2) + 2 * 4) >= kStreamBytes;
    return dispatch_dtype(dt, [&](auto dtc) -> hipError_t {
        constexpr int DT = decltype(dtc)::value;
        auto go = [&](auto sdt, auto mode) -> hipError_t {
            constexpr int S = decltype(sdt)::value, M = decltype(mode)::value;
            if (words < kSpreadWords) kv_read_kernel<S, DT, M, 1, false><<<dim3(blocks(words, 1), 2), 256, 0, st>>>(a);
            else if (!past) kv_read_kernel<S, DT, M, 4, false><<<dim3(blocks(words, 4), 2), 256, 0, st>>>(a);
            else kv_read_kernel<S, DT, M, 4, true><<<dim3(blocks(words, 4), 2), 256, 0, st>>>(a);
            return hipGetLastError();
        };
        if (c.mode == MXFP4) return go(std::integral_constant<int, QLIN_F32>{}, std::integral_constant<int, MXFP4>{});
        if (c.mode == NVFP4) return go(std::integral_constant<int, QLIN_F32>{}, std::integral_constant<int, NVFP4>{});
        return dispatch_dtype(c.sdt, [&](auto sdt) { return go(sdt, std::integral_constant<int, AFFINE>{}); });
    });
}

}  // namespace qlin
