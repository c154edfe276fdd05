// attend_simple.hip -- attention over the 4-bit cache on the vector units: any
// float type of q, any head size. What the matrix-core kernels do not take
// (fp32, head sizes other than theirs) runs here.
//
// A wave owns one row of q (one head of one token). Its lanes form groups of
// LANES that share a key, a lane holding the eight values of one word: keys are
// taken 64 / LANES at a time, each group with its own running maximum and sum
// (o = sum of p v / sum of p, p = exp(score - maximum)), joined at the end.
// Bound by instructions: about 12 a value, and nothing of a key is shared
// between rows but through the caches.

#include <type_traits>

#include "attend_common.h"

namespace qlin {
namespace {

template <int DT, int MODE, int LANES>
__global__ void __launch_bounds__(256) attend_simple_kernel(AttendArgs a, KvPool c) {
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    const int64_t t = item / a.q_heads;
    const int head = (int)(item - t * a.q_heads), lane = threadIdx.x % 64;
    if (t >= a.T) return;
    int b = (int)t;
    if (a.offsets) {
        b = last_at_most(a.B, t, [&](int i) { return (int64_t)a.offsets[i]; });
        if (a.offsets[b] > t || a.offsets[b + 1] <= t) return;   // a row of no sequence
    }
    const Sequence s = sequence_of(a, c, b);
    const Seen seen = seen_by(a, s, (int)(t - s.first));
    const int h = head / (a.q_heads / c.heads), words = c.D / 8, w = lane % LANES;
    const bool holds = w < words;
    const int wl = holds ? w : 0, per_group = c.g / 8;
    const int32_t* table = a.table + (int64_t)b * a.width;
    float q[8], acc[8], m = kNone, l = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = holds ? load_f<DT>(a.q, t * a.q_stride + (int64_t)head * c.D + 8 * w + i) * (a.scale * kLog2e) : 0.0f;
        acc[i] = 0.0f;
    }
    for (int k0 = seen.lo; k0 < seen.hi; k0 += 64 / LANES) {
        const int key = k0 + lane / LANES;
        int32_t rb = -1;
        if (key < seen.hi) rb = kv_row_block(table[key / c.page], c.pages, c.heads, c.page, h, key / kKvUnit);
        float v[2][8];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            if (rb >= 0) {
                const int64_t row = (int64_t)rb * kKvUnit + key % kKvUnit;
                const uint32_t word = c.codes[side][row * words + wl];
                const int64_t group = row * (words / per_group) + wl / per_group;
                const float sc = scale_at<MODE, DT>(c.scales[side], group);
                if constexpr (MODE == AFFINE) {
                    const float z = load_f<DT>(c.biases[side], group);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[side][i] = __builtin_fmaf(sc, (float)((word >> (4 * i)) & 15u), z);
                } else {
                    e2m1_values(word, sc, v[side]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[side][i] = 0.0f;
            }
        }
        float score = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) score = __builtin_fmaf(q[i], holds ? v[0][i] : 0.0f, score);
#pragma unroll
        for (int off = LANES / 2; off; off /= 2) score += __shfl_xor(score, off, 64);
        if (rb >= 0) {
            const float top = fmaxf(m, score), old = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
            const float p = __builtin_amdgcn_exp2f(score - top);
            m = top;
            l = __builtin_fmaf(l, old, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(acc[i], old, p * v[1][i]);
        }
    }
#pragma unroll
    for (int off = LANES; off < 64; off *= 2) {
        const float m2 = __shfl_xor(m, off, 64), l2 = __shfl_xor(l, off, 64);
        const float top = fmaxf(m, m2);
        const float f1 = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        const float f2 = m2 == kNone ? 0.0f : __builtin_amdgcn_exp2f(m2 - top);
        m = top;
        l = l * f1 + l2 * f2;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = acc[i] * f1 + __shfl_xor(acc[i], off, 64) * f2;
    }
    if (lane < words) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // a row that sees no key: zeros
#pragma unroll
        for (int i = 0; i < 8; ++i) store_f<DT>(a.out, (t * a.q_heads + head) * c.D + 8 * lane + i, acc[i] * inv);
    }
}

}  // namespace

hipError_t launch_attend_simple(const AttendArgs& a, const KvPool& c, int dt, hipStream_t st) {
    const int64_t items = a.T * a.q_heads;
    const unsigned nb = (unsigned)((items + 3) / 4);
    auto sized = [&](auto dtc, auto mode) -> hipError_t {
        constexpr int DT = decltype(dtc)::value, M = decltype(mode)::value;
        if (c.D <= 64) attend_simple_kernel<DT, M, 8><<<nb, 256, 0, st>>>(a, c);
        else if (c.D <= 128) attend_simple_kernel<DT, M, 16><<<nb, 256, 0, st>>>(a, c);
        else attend_simple_kernel<DT, M, 32><<<nb, 256, 0, st>>>(a, c);
        return hipGetLastError();
    };
    auto moded = [&](auto dtc) -> hipError_t {
        if (c.mode == AFFINE) return sized(dtc, std::integral_constant<int, AFFINE>{});
        if (c.mode == MXFP4) return sized(dtc, std::integral_constant<int, MXFP4>{});
        return sized(dtc, std::integral_constant<int, NVFP4>{});
    };
    if (dt == QLIN_F32) return moded(std::integral_constant<int, QLIN_F32>{});
    if (dt == QLIN_F16) return moded(std::integral_constant<int, QLIN_F16>{});
    return moded(std::integral_constant<int, QLIN_BF16>{});
}

}  // namespace qlin
