// mxfp4_act.hip -- activations to mxfp4 on their way into a product, plain or
// through the gated activation silu(gate) * up.
//
// The rule is qlin_quantize's for mxfp4: per 32 values along K a shared
// exponent e = floor(log2 amax) - 2 in [-127, 127] (byte e + 127; 0 for an
// all-zero block), codes the nearest E2M1 of v / 2^e, ties to even, saturated.
// A block that holds a NaN or an infinity gets byte 255, the format's NaN, so
// that it shows in every product that reads it. silu(gate) * up is taken in
// fp32, with one IEEE division, and not rounded before it is quantized.
// Compiled with -ffp-contract=off so that every code is reproducible.
//
// One thread per packed word (8 values), 4 lanes per block; HBM-streaming.

#include "qlin_common.h"
#include "moe_common.h"

namespace qlin {
namespace {

constexpr int ACT_THREADS = 256;

__device__ __forceinline__ uint32_t e2m1_code(float v) {
    const float a = fabsf(v);
    const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                       (a > 5.0f);
    return c | ((__float_as_uint(v) >> 28) & 8u);
}

template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if constexpr (!VEC) {
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

template <int DT, bool VEC, bool SWIGLU>
__global__ void __launch_bounds__(ACT_THREADS) mxfp4_act_kernel(const void* __restrict__ x, int64_t words,
                                                                uint32_t row_words, int64_t sstride,
                                                                uint32_t* __restrict__ xq,
                                                                uint8_t* __restrict__ xs) {
    const int64_t wid = (int64_t)blockIdx.x * ACT_THREADS + threadIdx.x;
    const bool live = wid < words;            // whole blocks of 4 lanes are live or not
    const int64_t w0 = live ? wid : 0;
    const int64_t row = w0 / row_words;
    const uint32_t col = (uint32_t)(w0 - row * row_words);
    float v[8];
    if constexpr (SWIGLU) {
        float up[8];
        load8<DT, VEC>(x, (row * 2 * row_words + col) * 8, v);
        load8<DT, VEC>(x, (row * 2 * row_words + row_words + col) * 8, up);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = v[c] / (1.0f + expf(-v[c])) * up[c];
    } else {
        load8<DT, VEC>(x, w0 * 8, v);
    }
    float amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        amax = fmaxf(amax, fabsf(v[c]));
        bad |= !(fabsf(v[c]) < INFINITY);
    }
    if (bad) amax = INFINITY;
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    uint32_t byte = 255u, word = 0u;
    if (amax < INFINITY) {
        const uint32_t u = __float_as_uint(amax);
        int e = amax == 0.0f ? -127 : (u >> 23 ? (int)(u >> 23) - 127 : (31 - __builtin_clz(u)) - 149) - 2;
        e = e < -127 ? -127 : e;
        byte = (uint32_t)(e + 127);
#pragma unroll
        for (int c = 0; c < 8; ++c) word |= e2m1_code(__builtin_ldexpf(v[c], -e)) << (4 * c);
    }
    if (!live) return;
    xq[wid] = word;
    if ((threadIdx.x & 3) == 0) {
        uint8_t* const s = xs + row * sstride;
        const uint32_t blk = col >> 2;
        s[blk] = (uint8_t)byte;
        if (col + 4 == row_words)
            for (int64_t p = blk + 1; p < sstride; ++p) s[p] = 127;
    }
}

template <int DT>
void run_act(const void* x, int64_t words, uint32_t rw, int swiglu, uint32_t* xq, uint8_t* xs, int64_t sstride,
             hipStream_t st) {
    const unsigned grid = (unsigned)((words + ACT_THREADS - 1) / ACT_THREADS);
    const bool vec = ((uintptr_t)x & 15) == 0;   // rows are whole multiples of 64 bytes
    if (swiglu) {
        if (vec) mxfp4_act_kernel<DT, true, true><<<grid, ACT_THREADS, 0, st>>>(x, words, rw, sstride, xq, xs);
        else mxfp4_act_kernel<DT, false, true><<<grid, ACT_THREADS, 0, st>>>(x, words, rw, sstride, xq, xs);
    } else {
        if (vec) mxfp4_act_kernel<DT, true, false><<<grid, ACT_THREADS, 0, st>>>(x, words, rw, sstride, xq, xs);
        else mxfp4_act_kernel<DT, false, false><<<grid, ACT_THREADS, 0, st>>>(x, words, rw, sstride, xq, xs);
    }
}

}  // namespace

hipError_t launch_mxfp4_activation(const void* x, int dt, int64_t M, int64_t K, int swiglu, uint32_t* xq,
                                   uint8_t* xs, int64_t sstride, hipStream_t st) {
    const int64_t words = M * (K / 8);
    if ((words + ACT_THREADS - 1) / ACT_THREADS > 0x7fffffffLL) return hipErrorInvalidValue;
    const uint32_t rw = (uint32_t)(K / 8);
    if (dt == QLIN_F32) run_act<QLIN_F32>(x, words, rw, swiglu, xq, xs, sstride, st);
    else if (dt == QLIN_BF16) run_act<QLIN_BF16>(x, words, rw, swiglu, xq, xs, sstride, st);
    else run_act<QLIN_F16>(x, words, rw, swiglu, xq, xs, sstride, st);
    return hipGetLastError();
}

}  // namespace qlin
