// kv_store.hip -- rows of keys and values into a 4-bit cache, and back.
//
// Writing is qlin_quantize's rule on each head's row (quant_common.h: the same
// functions, so the same bytes), the row's place looked up in `slots`. A thread
// owns one packed word, the lanes of a group are neighbours, as in quant.hip.
// Reading decodes a word a thread.
//
// Both are bound by the memory: 2 D H elements of a token on one side, D H
// bytes of codes and the scales on the other. A head's row is D/2 contiguous
// bytes of a page, the next token's follows it: a block of 256 threads takes
// WPT runs of 256 words, so that neighbouring tokens' rows of a page are
// written (read) together and whole lines leave the L2.

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
};

// Token and place in its row of word `at` past the block's first token.
struct WordPlace {
    int64_t t;
    int head, w;
};
__device__ __forceinline__ WordPlace word_place(int64_t t0, uint32_t at, uint32_t row_words, uint32_t head_words) {
    const uint32_t dt = at / row_words, r = at - dt * row_words, h = r / head_words;
    return {t0 + dt, (int)h, (int)(r - h * head_words)};
}

// Number of the word in the pool, or -1 where the slot names no place.
__device__ __forceinline__ int64_t pool_word(const KvPool& c, int32_t slot, int64_t slots_end, const WordPlace& p,
                                             uint32_t head_words) {
    if (slot < 0 || slot >= slots_end) return -1;
    const uint32_t page = (uint32_t)slot / (uint32_t)c.page, o = (uint32_t)slot - page * (uint32_t)c.page;
    return (((int64_t)page * c.heads + p.head) * c.page + o) * head_words + p.w;
}

template <int DT, int MODE, bool VEC, int LPG, int WPT>
__global__ void __launch_bounds__(256) kv_write_kernel(StoreArgs a) {
    const KvPool& c = a.c;
    const int side = blockIdx.y;
    const uint32_t head_words = c.D / 8, row_words = head_words * c.heads;
    const int64_t first = (int64_t)blockIdx.x * (256 * WPT), t0 = first / row_words;
    const uint32_t r0 = (uint32_t)(first - t0 * row_words) + threadIdx.x;
    float v[WPT][8];
    int64_t word[WPT];
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const WordPlace p = word_place(t0, r0 + 256 * j, row_words, head_words);
        const bool live = p.t < a.T;
        load_chunk<DT, 8, VEC>(a.x[side], live ? p.t * a.stride[side] + p.head * c.D + p.w * 8 : 0, v[j]);
        word[j] = pool_word(c, live ? a.slots[p.t] : -1, a.slots_end, p, head_words);
    }
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        if constexpr (MODE == AFFINE)
            quantize_affine_word<DT, 4, LPG>(v[j], word[j], word[j] >= 0, c.codes[side], c.scales[side],
                                             c.biases[side]);
        else
            quantize_micro_word<MODE, LPG>(v[j], word[j], word[j] >= 0, c.codes[side], (uint8_t*)c.scales[side]);
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

template <int SDT, int DT, int MODE, int WPT>
__global__ void __launch_bounds__(256) kv_read_kernel(StoreArgs a) {
    const KvPool& c = a.c;
    const int side = blockIdx.y;
    const uint32_t head_words = c.D / 8, row_words = head_words * c.heads;
    const int64_t first = (int64_t)blockIdx.x * (256 * WPT), t0 = first / row_words;
    const uint32_t r0 = (uint32_t)(first - t0 * row_words) + threadIdx.x;
    const int group_shift = 31 - __builtin_clz((unsigned)c.g / 8);   // words of a group: a power of two
    uint32_t word[WPT];
    float s[WPT], z[WPT];
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const WordPlace p = word_place(t0, r0 + 256 * j, row_words, head_words);
        const int64_t at = pool_word(c, p.t < a.T ? a.slots[p.t] : -1, a.slots_end, p, head_words);
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
        const uint32_t at = r0 + 256 * j;
        if (t0 + at / row_words >= a.T) continue;
        const int64_t e = (t0 * row_words + at) * 8;
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
        if constexpr (DT == QLIN_F32) {
            float4* y = (float4*)((float*)a.y[side] + e);
            y[0] = float4{v[0], v[1], v[2], v[3]};
            y[1] = float4{v[4], v[5], v[6], v[7]};
        } else {
            *(uint4*)((uint16_t*)a.y[side] + e) = uint4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]),
                                                        pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
        }
    }
}

// Words a thread takes: eight runs of 256 keep neighbouring tokens' rows of a
// page in one block; a small call is spread over the CUs instead.
constexpr int64_t kSpreadWords = 256 * 1024;

unsigned blocks(int64_t words, int wpt) { return (unsigned)((words + 256 * wpt - 1) / (256 * wpt)); }

}  // namespace

hipError_t launch_kv_write(const KvPool& c, const void* k, const void* v, int dt, int64_t T, int64_t k_stride,
                           int64_t v_stride, const int32_t* slots, hipStream_t st) {
    const StoreArgs a{{k, v}, {nullptr, nullptr}, {k_stride, v_stride}, c, slots, T, c.pages * c.page};
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
    const StoreArgs a{{nullptr, nullptr}, {k, v}, {0, 0}, c, slots, T, c.pages * c.page};
    const int64_t words = T * c.heads * (c.D / 8);
    return dispatch_dtype(dt, [&](auto dtc) -> hipError_t {
        constexpr int DT = decltype(dtc)::value;
        auto go = [&](auto sdt, auto mode) -> hipError_t {
            constexpr int S = decltype(sdt)::value, M = decltype(mode)::value;
            if (words < kSpreadWords) kv_read_kernel<S, DT, M, 1><<<dim3(blocks(words, 1), 2), 256, 0, st>>>(a);
            else kv_read_kernel<S, DT, M, 4><<<dim3(blocks(words, 4), 2), 256, 0, st>>>(a);
            return hipGetLastError();
        };
        if (c.mode == MXFP4) return go(std::integral_constant<int, QLIN_F32>{}, std::integral_constant<int, MXFP4>{});
        if (c.mode == NVFP4) return go(std::integral_constant<int, QLIN_F32>{}, std::integral_constant<int, NVFP4>{});
        return dispatch_dtype(c.sdt, [&](auto sdt) { return go(sdt, std::integral_constant<int, AFFINE>{}); });
    });
}

}  // namespace qlin
