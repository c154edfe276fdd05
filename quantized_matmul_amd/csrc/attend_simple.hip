// attend_simple.hip -- attention over the 4-bit cache on the vector units: any
// float type of q, any head size. What the matrix-core kernels do not take
// (fp32, head sizes other than theirs) runs here.
//
// WAVES waves own one row of q (one head of one token) and take its keys in
// turn. A wave's lanes form groups of LANES that share a key, a lane holding the
// eight values of one word: keys are taken 64 / LANES at a time, AHEAD such steps
// on their way together, each group with its own running maximum and sum (o = sum
// of p v / sum of p, p = exp(score - maximum)), joined at the end.
// Bound by instructions: about 12 a value, and nothing of a key is shared
// between rows but through the caches. fp32, D 128: a row each of 32 sequences of
// 32 heads over 4000 to 16000 keys 0.87 ms (a wave a row and a step at a time
// 5.8), of one sequence of 1500 32 us (326), 2048 rows of 32 heads 3.4 ms.

#include <type_traits>

#include "attend_common.h"

namespace qlin {
namespace {

constexpr int kAhead = 4;

template <int DT, int MODE, int LANES, int WAVES>
__global__ void __launch_bounds__(WAVES < 4 ? 256 : 64 * WAVES) attend_simple_kernel(AttendArgs a, KvPool c) {
    constexpr int ROWS = WAVES < 4 ? 4 / WAVES : 1, KEYS = 64 / LANES;       // rows of a workgroup; keys of a step
    __shared__ float part[WAVES > 1 ? WAVES : 1][LANES * 8 + 2];
    const int64_t item = (int64_t)blockIdx.x * ROWS + (WAVES == 1 ? threadIdx.x / 64 : 0);
    const int64_t t = item / a.q_heads;
    const int head = (int)(item - t * a.q_heads), wave = WAVES == 1 ? 0 : threadIdx.x / 64, lane = threadIdx.x % 64;
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
    for (int64_t k0 = seen.lo + (int64_t)wave * (KEYS * kAhead); k0 < seen.hi; k0 += WAVES * KEYS * kAhead) {
        bool live[kAhead];
        uint32_t word[2][kAhead];
        float sc[2][kAhead], z[2][kAhead], score[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t at = k0 + u * KEYS + lane / LANES;
            const int key = (int)(at < seen.hi ? at : seen.hi - 1);
            const int32_t rb = kv_row_block(table[key / c.page], c.pages, c.heads, c.page, h, key / kKvUnit);
            live[u] = rb >= 0 && at < seen.hi;
            const int64_t row = (int64_t)(rb < 0 ? 0 : rb) * kKvUnit + key % kKvUnit;
            const int64_t group = row * (words / per_group) + wl / per_group;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                word[side][u] = c.codes[side][row * words + wl];
                sc[side][u] = scale_at<MODE, DT>(c.scales[side], group);
                z[side][u] = MODE == AFFINE ? load_f<DT>(c.biases[side], group) : 0.0f;
            }
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int side = 0; side < 2; ++side) {       // what is not there is no number
                sc[side][u] = live[u] && (holds || side) ? sc[side][u] : 0.0f;
                z[side][u] = live[u] && (holds || side) ? z[side][u] : 0.0f;
            }
            float v[8];
            word_values<MODE>(word[0][u], sc[0][u], z[0][u], v);
            score[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) score[u] = __builtin_fmaf(q[i], v[i], score[u]);
#pragma unroll
            for (int off = LANES / 2; off; off /= 2) score[u] += __shfl_xor(score[u], off, 64);
            if (live[u]) top = fmaxf(top, score[u]);
        }
        const float old = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= old;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] *= old;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float p = live[u] ? __builtin_amdgcn_exp2f(score[u] - m) : 0.0f;
            float v[8];
            word_values<MODE>(word[1][u], sc[1][u], z[1][u], v);
            l += p;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(p, v[i], acc[i]);
        }
    }
    auto join = [&](float m2, float l2, auto&& acc2) {
        const float top = fmaxf(m, m2);
        const float f1 = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        const float f2 = m2 == kNone ? 0.0f : __builtin_amdgcn_exp2f(m2 - top);
        m = top;
        l = l * f1 + l2 * f2;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = acc[i] * f1 + acc2(i) * f2;
    };
#pragma unroll
    for (int off = LANES; off < 64; off *= 2)
        join(__shfl_xor(m, off, 64), __shfl_xor(l, off, 64), [&](int i) { return __shfl_xor(acc[i], off, 64); });
    if constexpr (WAVES > 1) {
        if (lane < LANES) {
#pragma unroll
            for (int i = 0; i < 8; ++i) part[wave][lane * 8 + i] = acc[i];
            part[wave][LANES * 8] = m;
            part[wave][LANES * 8 + 1] = l;
        }
        __syncthreads();
        if (wave) return;
        for (int o = 1; o < WAVES; ++o)
            join(part[o][LANES * 8], part[o][LANES * 8 + 1], [&](int i) { return part[o][w * 8 + i]; });
    }
    if (lane < words) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // a row that sees no key: zeros
#pragma unroll
        for (int i = 0; i < 8; ++i) store_f<DT>(a.out, (t * a.q_heads + head) * c.D + 8 * lane + i, acc[i] * inv);
    }
}

}  // namespace

hipError_t launch_attend_simple(const AttendArgs& a, const KvPool& c, int dt, hipStream_t st) {
    // Sixteen waves to a row where there are few rows, or rather few and many keys. Measured, one wave and sixteen (fp32,
    // D 128, us): 1024 rows of 300 keys 45 and 54, of 4000 keys 474 and 290; 2048 rows of 4000 584 and 554, 4096 rows 942
    // and 1057
    const int64_t items = a.T * a.q_heads;
    const bool shared = items <= 512 || (items <= 2048 && (int64_t)a.width * c.page > 1024);
    auto sized = [&](auto dtc, auto mode) -> hipError_t {
        constexpr int DT = decltype(dtc)::value, M = decltype(mode)::value;
        auto go = [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            if (!shared) attend_simple_kernel<DT, M, L, 1><<<(unsigned)((items + 3) / 4), 256, 0, st>>>(a, c);
            else attend_simple_kernel<DT, M, L, 16><<<(unsigned)items, 1024, 0, st>>>(a, c);
        };
        if (c.D <= 64) go(std::integral_constant<int, 8>{});
        else if (c.D <= 128) go(std::integral_constant<int, 16>{});
        else go(std::integral_constant<int, 32>{});
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
