// quant.hip -- group-wise quantize and dequantize kernels (gfx950).
//
// Quantize follows the affine rule "w ~ scale*q + bias" of the mlx-rs
// quantization.rs quantize/quantized_matmul doc comments, with one scale and
// bias per group of group_size elements along a row, and the microscaled
// modes of the "Emily.QuantizedWeight" Microscaled modes table. Codes are
// packed 32/bits per uint32, lowest element in the lowest bits
// ("Emily.QuantizedWeight", Layout).
//
// Every rounding step is explicit (quant_common.h) so that codes, scales and
// biases are bit-for-bit reproducible. This file is compiled with
// -ffp-contract=off.
//
// All kernels are HBM-streaming: one thread owns one packed word and the
// elements it encodes (the lanes of a group cooperate on its scale).

#include "quant_common.h"

namespace qlin {
namespace {

// ---------------------------------------------------------------- kernels
//
// Quantize: lane l of the grid owns packed word l, i.e. the PER = 32/bits
// consecutive elements it encodes, so a wave reads 64*PER contiguous
// elements (16-byte vector loads when w is 16-byte aligned) and writes 64
// contiguous words. A group is g/PER adjacent lanes of one wave (the flat
// element count is a multiple of g and a group never straddles a row, so
// groups are whole and wave-aligned); its min/max (or amax) is combined
// across those lanes with xor shuffles. Rounding is unchanged: every code
// still takes one correctly rounded fp32 division and rint.

// WPT words per thread, thread t of a block taking words base + t + 256 j:
// every wave-wide load and store stays contiguous and a group's LPG lanes
// stay consecutive; all WPT words' elements are loaded before any is coded.
template <int DT, int BITS, bool VEC, int LPG, int WPT>
__global__ void __launch_bounds__(256) quantize_affine_kernel(
    const void* __restrict__ w, int64_t words, int g, uint32_t* __restrict__ wq,
    void* __restrict__ scales, void* __restrict__ biases) {
    constexpr int PER = 32 / BITS;
    const int64_t base = (int64_t)blockIdx.x * (256 * WPT) + threadIdx.x;
    float v[WPT][PER];
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const int64_t wid = base + 256 * j;
        load_chunk<DT, PER, VEC>(w, (wid < words ? wid : 0) * PER, v[j]);
    }
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const int64_t wid = base + 256 * j;
        quantize_affine_word<DT, BITS, LPG>(v[j], wid, wid < words, wq, scales, biases);
    }
}

template <int DT, int MODE, bool VEC, int LPG, int WPT>
__global__ void __launch_bounds__(256) quantize_micro_kernel(
    const void* __restrict__ w, int64_t words, int g, uint32_t* __restrict__ wq,
    uint8_t* __restrict__ scales) {
    constexpr int BITS = (MODE == MXFP8) ? 8 : 4;
    constexpr int PER = 32 / BITS;
    const int64_t base = (int64_t)blockIdx.x * (256 * WPT) + threadIdx.x;
    float v[WPT][PER];
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const int64_t wid = base + 256 * j;
        load_chunk<DT, PER, VEC>(w, (wid < words ? wid : 0) * PER, v[j]);
    }
#pragma unroll
    for (int j = 0; j < WPT; ++j) {
        const int64_t wid = base + 256 * j;
        quantize_micro_word<MODE, LPG>(v[j], wid, wid < words, wq, scales);
    }
}

// qqmm's activation step (mlx-rs qqmm: x is quantized on the fly): bf16 x
// quantized along its rows with a microscaled mode and decoded straight
// back, xhat = decode(code) * decode(scale byte). Every such value is exact
// in bf16 (at most 6 significant bits), so the matmul kernels then take
// xhat as an ordinary bf16 activation. Lanes and groups as in quantize.
template <int MODE, bool VEC, int LPG>
__global__ void __launch_bounds__(256) qdq_micro_kernel(const void* __restrict__ x, int64_t words,
                                                        uint16_t* __restrict__ xhat) {
    constexpr int BITS = (MODE == MXFP8) ? 8 : 4;
    constexpr int PER = 32 / BITS;
    const int64_t wid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const bool live = wid < words;
    float v[PER];
    load_chunk<QLIN_BF16, PER, VEC>(x, (live ? wid : 0) * PER, v);
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < PER; ++e) amax = fmaxf(amax, fabsf(v[e]));
    const MicroScale<MODE> m = micro_scale<MODE>(group_amax<LPG>(amax));
    const float s = MODE == NVFP4 ? e4m3_to_f32(m.sbyte) : e8m0_to_f32(m.sbyte);
    uint32_t d[PER / 2];
#pragma unroll
    for (int k = 0; k < PER; k += 2) {
        const uint32_t c0 = micro_encode<MODE>(v[k], m), c1 = micro_encode<MODE>(v[k + 1], m);
        const float f0 = (MODE == MXFP8 ? e4m3_to_f32(c0) : e2m1_to_f32(c0)) * s;
        const float f1 = (MODE == MXFP8 ? e4m3_to_f32(c1) : e2m1_to_f32(c1)) * s;
        d[k / 2] = f32_to_bf16_rne(f0) | (f32_to_bf16_rne(f1) << 16);
    }
    if (!live) return;
    if constexpr (VEC) {
        if constexpr (PER == 8) {
            *(uint4*)(xhat + wid * PER) = uint4{d[0], d[1], d[2], d[3]};
        } else {
            *(uint2*)(xhat + wid * PER) = uint2{d[0], d[1]};
        }
    } else {
#pragma unroll
        for (int k = 0; k < PER / 2; ++k) {
            xhat[wid * PER + 2 * k] = (uint16_t)(d[k] & 0xFFFFu);
            xhat[wid * PER + 2 * k + 1] = (uint16_t)(d[k] >> 16);
        }
    }
}

// One packed word; out row-major [rows, cols]. VEC: the word's PER outputs
// go out as 16-byte (or 8-byte) vector stores.
template <int SDT, int ODT, int BITS, int MODE, bool VEC>
__device__ __forceinline__ void dequantize_word(const uint32_t word, int64_t wid,
    const void* __restrict__ scales, const void* __restrict__ biases, int g, void* __restrict__ out);

// WPT packed words per thread, thread t of a block taking words
// base + t + 256 j, so every wave-wide load and store stays contiguous. Four
// words per thread measured faster for 4- and 8-bit codes (W [14336, 4096]
// int4 g64 to bf16, inputs cycled past the Infinity Cache: 39.5 -> 35.7 us;
// int8 54.2 -> 41.7 us; mxfp4 [8192, 8192] 50.1 -> 47.8 us); 2-bit codes
// (16 outputs a word) keep one (38.2 against 41.6 us); loading the four words
// as one 16-byte vector per lane, stores then 64 bytes apart, ran twice as long.
template <int SDT, int ODT, int BITS, int MODE, bool VEC, int WPT>
__global__ void __launch_bounds__(256) dequantize_kernel(
    const uint32_t* __restrict__ wq, const void* __restrict__ scales,
    const void* __restrict__ biases, int64_t words, int g, void* __restrict__ out) {
    const int64_t base = (int64_t)blockIdx.x * (256 * WPT) + threadIdx.x;
    uint32_t wv[WPT];
#pragma unroll
    for (int j = 0; j < WPT; ++j) wv[j] = base + 256 * j < words ? wq[base + 256 * j] : 0u;
#pragma unroll
    for (int j = 0; j < WPT; ++j)
        if (base + 256 * j < words)
            dequantize_word<SDT, ODT, BITS, MODE, VEC>(wv[j], base + 256 * j, scales, biases, g, out);
}

template <int SDT, int ODT, int BITS, int MODE, bool VEC>
__device__ __forceinline__ void dequantize_word(const uint32_t word, int64_t wid,
    const void* __restrict__ scales, const void* __restrict__ biases, int g, void* __restrict__ out) {
    constexpr int PER = 32 / BITS;
    const int64_t k0 = wid * PER;           // flat element index of the word's first code
    const int64_t gidx = k0 / g;            // flat group index (groups never straddle words)
    float s, z = 0.0f;
    if constexpr (MODE == AFFINE) {
        s = load_f<SDT>(scales, gidx);
        z = load_f<SDT>(biases, gidx);
    } else if constexpr (MODE == NVFP4) {
        s = e4m3_to_f32(((const uint8_t*)scales)[gidx]);
    } else {
        s = e8m0_to_f32(((const uint8_t*)scales)[gidx]);
    }
    float v[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        uint32_t q = (word >> (e * BITS)) & ((1u << BITS) - 1u);
        if constexpr (MODE == AFFINE) v[e] = __builtin_fmaf(s, (float)q, z);
        else if constexpr (MODE == MXFP8) v[e] = e4m3_to_f32(q) * s;
        else v[e] = e2m1_to_f32(q) * s;
    }
    if constexpr (!VEC) {
#pragma unroll
        for (int e = 0; e < PER; ++e) store_f<ODT>(out, k0 + e, v[e]);
    } else if constexpr (ODT == QLIN_F32) {
        float4* p = (float4*)((float*)out + k0);
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) p[q] = float4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    } else {
        uint32_t d[PER / 2];
#pragma unroll
        for (int q = 0; q < PER / 2; ++q) {
            const uint32_t a = ODT == QLIN_BF16 ? f32_to_bf16_rne(v[2 * q]) : f32_to_f16_rne(v[2 * q]);
            const uint32_t b = ODT == QLIN_BF16 ? f32_to_bf16_rne(v[2 * q + 1]) : f32_to_f16_rne(v[2 * q + 1]);
            d[q] = a | (b << 16);
        }
        if constexpr (PER / 2 % 4 == 0) {
            uint4* p = (uint4*)((uint16_t*)out + k0);
#pragma unroll
            for (int q = 0; q < PER / 8; ++q) p[q] = uint4{d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
        } else {   // PER == 4
            *(uint2*)((uint16_t*)out + k0) = uint2{d[0], d[1]};
        }
    }
}

inline unsigned nblocks(int64_t n) { return (unsigned)((n + 255) / 256); }

}  // namespace

hipError_t launch_quantize(const void* w, int w_dtype, int64_t rows, int64_t cols, int g,
                           int bits, int mode, uint32_t* wq, void* scales, void* biases,
                           hipStream_t st) {
    const int64_t words = rows * (cols * bits / 32);
    // Words per thread, from rotating-buffer timings over 5 weight copies
    // (14336x4096 affine, 8192x8192 micro; us per call, 1 -> 4 words):
    // affine 8-bit 57.3 -> 54.3, MXFP8 61.0 -> 48.9, MXFP4 45.0 -> 43.0 gain;
    // affine 4-bit 40.1 -> 44.0 and 2-bit 34 -> 41 lose, NVFP4 is flat.
    // Both choices write identical bytes.
    const unsigned nb = nblocks(words), nb4 = nblocks((words + 3) / 4);
    const int per = 32 / bits;
    const bool vec = ((uintptr_t)w & 15) == 0;
    return dispatch_dtype(w_dtype, [&](auto dt) -> hipError_t {
        constexpr int DT = decltype(dt)::value;
        return dispatch_lpg(g / per, [&](auto lpgc) -> hipError_t {
            constexpr int LPG = decltype(lpgc)::value;
            auto go = [&](auto kv) -> hipError_t {
                constexpr bool V = decltype(kv)::value;
                if (mode == AFFINE) {
                    if (bits == 2) quantize_affine_kernel<DT, 2, V, LPG, 1><<<nb, 256, 0, st>>>(w, words, g, wq, scales, biases);
                    else if (bits == 4) quantize_affine_kernel<DT, 4, V, LPG, 1><<<nb, 256, 0, st>>>(w, words, g, wq, scales, biases);
                    else quantize_affine_kernel<DT, 8, V, LPG, 4><<<nb4, 256, 0, st>>>(w, words, g, wq, scales, biases);
                } else if (mode == MXFP4) {
                    quantize_micro_kernel<DT, MXFP4, V, LPG, 4><<<nb4, 256, 0, st>>>(w, words, g, wq, (uint8_t*)scales);
                } else if (mode == MXFP8) {
                    quantize_micro_kernel<DT, MXFP8, V, LPG, 4><<<nb4, 256, 0, st>>>(w, words, g, wq, (uint8_t*)scales);
                } else {
                    quantize_micro_kernel<DT, NVFP4, V, LPG, 1><<<nb, 256, 0, st>>>(w, words, g, wq, (uint8_t*)scales);
                }
                return hipGetLastError();
            };
            return vec ? go(std::true_type{}) : go(std::false_type{});
        });
    });
}

hipError_t launch_qdq_micro(const void* x, int64_t rows, int64_t cols, int g, int mode,
                           void* xhat, hipStream_t st) {
    const int bits = mode == MXFP8 ? 8 : 4;
    const int64_t words = rows * (cols * bits / 32);
    const unsigned nb = nblocks(words);
    const bool vec = (((uintptr_t)x | (uintptr_t)xhat) & 15) == 0;
    return dispatch_lpg(g / (32 / bits), [&](auto lpgc) -> hipError_t {
        constexpr int LPG = decltype(lpgc)::value;
        auto go = [&](auto kv) -> hipError_t {
            constexpr bool V = decltype(kv)::value;
            if (mode == MXFP8) qdq_micro_kernel<MXFP8, V, LPG><<<nb, 256, 0, st>>>(x, words, (uint16_t*)xhat);
            else if (mode == NVFP4) qdq_micro_kernel<NVFP4, V, LPG><<<nb, 256, 0, st>>>(x, words, (uint16_t*)xhat);
            else return hipErrorInvalidValue;
            return hipGetLastError();
        };
        return vec ? go(std::true_type{}) : go(std::false_type{});
    });
}

hipError_t launch_dequantize(const uint32_t* wq, const void* scales, const void* biases,
                             int sdtype, int64_t rows, int64_t cols, int g, int bits, int mode,
                             void* out, int out_dtype, hipStream_t st) {
    const int64_t words = rows * (cols * bits / 32);
    const unsigned nb = nblocks(words), nb4 = nblocks((words + 3) / 4);
    const bool vec = ((uintptr_t)out & 15) == 0;
    return dispatch_dtype(out_dtype, [&](auto odt) -> hipError_t {
        constexpr int ODT = decltype(odt)::value;
        auto go = [&](auto kv) -> hipError_t {
            constexpr bool V = decltype(kv)::value;
            if (mode != AFFINE) {
                if (mode == MXFP4) dequantize_kernel<QLIN_F32, ODT, 4, MXFP4, V, 4><<<nb4, 256, 0, st>>>(wq, scales, biases, words, g, out);
                else if (mode == NVFP4) dequantize_kernel<QLIN_F32, ODT, 4, NVFP4, V, 4><<<nb4, 256, 0, st>>>(wq, scales, biases, words, g, out);
                else dequantize_kernel<QLIN_F32, ODT, 8, MXFP8, V, 4><<<nb4, 256, 0, st>>>(wq, scales, biases, words, g, out);
                return hipGetLastError();
            }
            return dispatch_dtype(sdtype, [&](auto sdt) -> hipError_t {
                constexpr int SDT = decltype(sdt)::value;
                if (bits == 2) dequantize_kernel<SDT, ODT, 2, AFFINE, V, 1><<<nb, 256, 0, st>>>(wq, scales, biases, words, g, out);
                else if (bits == 4) dequantize_kernel<SDT, ODT, 4, AFFINE, V, 4><<<nb4, 256, 0, st>>>(wq, scales, biases, words, g, out);
                else dequantize_kernel<SDT, ODT, 8, AFFINE, V, 4><<<nb4, 256, 0, st>>>(wq, scales, biases, words, g, out);
                return hipGetLastError();
            });
        };
        return vec ? go(std::true_type{}) : go(std::false_type{});
    });
}

}  // namespace qlin
