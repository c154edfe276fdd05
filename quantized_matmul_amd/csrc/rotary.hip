// rotary.hip -- rotary positions: the first R values of each head are taken as
// R/2 pairs (i, i + R/2), or (2i, 2i + 1) interleaved, and pair i of token t is
// turned by the angle positions[t] * freqs[i]:
//     (a, b) -> scale * (a cos - b sin, a sin + b cos)
// The gradient is the same with the angle's sign changed (the transpose).
//
// Bound by the memory: x is read and y written once. A thread owns 16 bytes of
// a head's row and walks the heads, so that its angles (fp64 product and
// reduction, polynomials of degree 9 and 10 for sine and cosine) are taken once
// a token. The partners come from the same row, which the wave's neighbouring
// lanes read in the same instruction. All of a row's lanes belong to one wave
// and load before any of them stores, so y may be x.
// 32768 tokens of 40 heads of 128 (bf16, 671 MB) 140 us, 4.8 TB/s, what a copy
// reaches; 8191 tokens of 20 heads of 96, 64 turned (f16, 63 MB) 12.7 us; 1 token 3.4 us,
// the launch.

#include <type_traits>

#include "kv_common.h"

namespace qlin {
namespace {

// Sine and cosine of 2 pi r for an fp64 number of turns: the turn's fraction
// is exact in fp64 up to the rounding of r itself, the eighth of a turn around
// the nearest quarter is left to Taylor polynomials (below 2 * 10^-9 off).
__device__ __forceinline__ void sincos_turns(double r, float* s, float* c) {
    const double q = rint(r * 4.0);
    const float x = (float)((r - q * 0.25) * 6.283185307179586476925);
    const float x2 = x * x;
    float p = __builtin_fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
    p = __builtin_fmaf(x2, p, 1.0f / 120.0f);
    p = __builtin_fmaf(x2, p, -1.0f / 6.0f);
    const float sn = __builtin_fmaf(x * x2, p, x);
    p = __builtin_fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    p = __builtin_fmaf(x2, p, -1.0f / 720.0f);
    p = __builtin_fmaf(x2, p, 1.0f / 24.0f);
    p = __builtin_fmaf(x2, p, -0.5f);
    const float cs = __builtin_fmaf(x2, p, 1.0f);
    const int k = (int)(q - 4.0 * floor(q * 0.25));
    const float a = (k & 1) ? cs : sn, b = (k & 1) ? sn : cs;
    *s = (k & 2) ? -a : a;
    *c = (k == 1 || k == 2) ? -b : b;
}

// NV elements (16 bytes) at element i; VEC: one 16-byte load.
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

template <int DT, int NV, bool VEC>
__device__ __forceinline__ void load_run(const void* p, int64_t i, float (&v)[NV]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int e = 0; e < NV; ++e) v[e] = load_f<DT>(p, i + e);
    } else if constexpr (DT == QLIN_F32) {
        const float4 t = *(const float4*)((const float*)p + i);
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
        const uint4 t = *(const uint4*)((const uint16_t*)p + i);
        const uint32_t d[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = DT == QLIN_BF16 ? __uint_as_float(d[e] << 16) : f16_bits_to_f32(d[e] & 0xFFFFu);
            v[2 * e + 1] = DT == QLIN_BF16 ? __uint_as_float(d[e] & 0xFFFF0000u) : f16_bits_to_f32(d[e] >> 16);
        }
    }
}

// PAST: past the caches.
template <int DT, int NV, bool VEC, bool PAST>
__device__ __forceinline__ void store_run(void* p, int64_t i, const float (&v)[NV]) {
    auto put = [](u32x4 x, void* to) {
        if constexpr (PAST) __builtin_nontemporal_store(x, (u32x4*)to);
        else *(u32x4*)to = x;
    };
    if constexpr (!VEC) {
#pragma unroll
        for (int e = 0; e < NV; ++e) store_f<DT>(p, i + e, v[e]);
    } else if constexpr (DT == QLIN_F32) {
        put(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, (float*)p + i);
    } else {
        uint32_t d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (DT == QLIN_BF16) {
                typedef __attribute__((ext_vector_type(2))) __bf16 T2;
                d[e] = __builtin_bit_cast(uint32_t, T2{(__bf16)v[2 * e], (__bf16)v[2 * e + 1]});
            } else {
                d[e] = f32_to_f16_rne(v[2 * e]) | (f32_to_f16_rne(v[2 * e + 1]) << 16);
            }
        }
        put(u32x4{d[0], d[1], d[2], d[3]}, (uint16_t*)p + i);
    }
}

// PAIR 0: interleaved, the partner is a neighbour; 1: half a rotated row away,
// a whole number of runs; 2: half a row away, anywhere.
// LANES lanes (a power of two) take a head's row; a block of 256 threads takes
// 256 / LANES (token, head part) items, part = heads / parts of them.
template <int DT, int PAIR, bool VEC, int LANES, bool PAST>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryArgs a, int parts, int part_heads) {
    constexpr int NV = DT == QLIN_F32 ? 4 : 8;
    const int64_t item = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    const int64_t t = item / parts;
    const int h0 = (int)(item - t * parts) * part_heads;
    const int e = (threadIdx.x % LANES) * NV;
    const bool live = t < a.T && e < a.D;
    if (!live) return;
    const int half = a.R / 2;
    const double turns = (double)a.positions[t] * 0.15915494309189533577;
    float c[NV], s[NV];
    int partner[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = e + i;
        const bool turned = d < a.R;
        const bool second = PAIR == 0 ? d & 1 : d >= half;
        const int f = PAIR == 0 ? d >> 1 : (second ? d - half : d);
        partner[i] = !turned ? d : (PAIR == 0 ? d ^ 1 : (second ? d - half : d + half));
        float sn = 0.0f, cs = 1.0f;
        if (turned) {
            sincos_turns(turns * (double)a.freqs[f], &sn, &cs);
            sn *= a.scale;
            cs *= a.scale;
        }
        s[i] = second != (a.backward != 0) ? sn : -sn;
        c[i] = cs;
    }
    const int run = PAIR == 1 ? partner[0] : 0;
    const int h1 = min(h0 + part_heads, a.heads);
    // HB heads' loads at once: a store may not be passed by a later load, as y may be x
    constexpr int HB = 4;
    for (int h = h0; h < h1; h += HB) {
        float v[HB][NV], w[HB][NV];
#pragma unroll
        for (int u = 0; u < HB; ++u) {
            const int64_t row = t * a.x_stride + (int64_t)min(h + u, h1 - 1) * a.D;
            load_run<DT, NV, VEC>(a.x, row + e, v[u]);
            if constexpr (PAIR == 1) {
                load_run<DT, NV, VEC>(a.x, row + run, w[u]);
            } else if constexpr (PAIR == 2) {
#pragma unroll
                for (int i = 0; i < NV; ++i) w[u][i] = load_f<DT>(a.x, row + partner[i]);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) w[u][i] = v[u][i ^ 1];
            }
        }
#pragma unroll
        for (int u = 0; u < HB; ++u) {
            if (h + u >= h1) break;
            float y[NV];
            // the product with the sine rounds first, then the sum: 2^-23 of the pair's size at most
#pragma unroll
            for (int i = 0; i < NV; ++i) y[i] = e + i < a.R ? __builtin_fmaf(v[u][i], c[i], w[u][i] * s[i]) : v[u][i];
            store_run<DT, NV, VEC, PAST>(a.y, t * a.y_stride + (int64_t)(h + u) * a.D + e, y);
        }
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, int dt, hipStream_t st) {
    const int elem = dt == QLIN_F32 ? 4 : 2, nv = 16 / elem;
    const bool vec = (((uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)(a.x_stride * elem) | (uintptr_t)(a.y_stride * elem)) & 15) == 0;
    const int pair = a.interleaved ? 0 : ((a.R / 2) % nv == 0 ? 1 : 2);
    int lanes = 1;
    while (lanes * nv < a.D) lanes *= 2;
    // heads of a thread: all of them where the tokens alone fill the chip
    const int64_t want = 4096 * (256 / lanes) / 4;
    int parts = a.T >= want ? 1 : (int)((want + a.T - 1) / a.T);
    if (parts > a.heads) parts = a.heads;
    const int part_heads = (a.heads + parts - 1) / parts;
    parts = (a.heads + part_heads - 1) / part_heads;
    const int64_t per = 256 / lanes;
    // tokens of a launch, whose work-items stay below 2^32
    const int64_t most = ((1LL << 31) / 256) * per / parts;
    const bool past = a.x != a.y && 2 * a.T * a.heads * a.D * elem >= kStreamBytes;
    RotaryArgs part = a;
    unsigned nb = 0;
    auto go = [&](auto dtc, auto pc, auto vc) -> hipError_t {
        constexpr int DT = decltype(dtc)::value, P = decltype(pc)::value;
        constexpr bool V = decltype(vc)::value;
        auto run = [&](auto lc) {
            constexpr int L = decltype(lc)::value;
            if (V && past) rotary_kernel<DT, P, V, L, V><<<nb, 256, 0, st>>>(part, parts, part_heads);
            else rotary_kernel<DT, P, V, L, false><<<nb, 256, 0, st>>>(part, parts, part_heads);
        };
        for (int64_t t = 0; t < a.T; t += most) {
            part.T = a.T - t < most ? a.T - t : most;
            part.x = (const char*)a.x + t * a.x_stride * elem;
            part.y = (char*)a.y + t * a.y_stride * elem;
            part.positions = a.positions + t;
            nb = (unsigned)((part.T * parts + per - 1) / per);
            switch (lanes) {
            case 1: run(std::integral_constant<int, 1>{}); break;
            case 2: run(std::integral_constant<int, 2>{}); break;
            case 4: run(std::integral_constant<int, 4>{}); break;
            case 8: run(std::integral_constant<int, 8>{}); break;
            case 16: run(std::integral_constant<int, 16>{}); break;
            case 32: run(std::integral_constant<int, 32>{}); break;
            case 64: run(std::integral_constant<int, 64>{}); break;
            default: return hipErrorInvalidValue;
            }
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    auto paired = [&](auto dtc, auto vc) -> hipError_t {
        if (pair == 0) return go(dtc, std::integral_constant<int, 0>{}, vc);
        if (pair == 1) return go(dtc, std::integral_constant<int, 1>{}, vc);
        return go(dtc, std::integral_constant<int, 2>{}, vc);
    };
    auto typed = [&](auto dtc) -> hipError_t {
        return vec ? paired(dtc, std::true_type{}) : paired(dtc, std::false_type{});
    };
    if (dt == QLIN_F32) return typed(std::integral_constant<int, QLIN_F32>{});
    if (dt == QLIN_F16) return typed(std::integral_constant<int, QLIN_F16>{});
    return typed(std::integral_constant<int, QLIN_BF16>{});
}

}  // namespace qlin
