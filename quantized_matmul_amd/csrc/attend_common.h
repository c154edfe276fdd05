// attend_common.h -- what the attention kernels share: a row's place among the
// sequences, the keys it sees, decoded values of a word.
#pragma once

#include "kv_common.h"

namespace qlin {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -__builtin_inff();
constexpr float kSlack = 8.0f;                  // log2 of how far scores may pass the running maximum

// Eight numbers of a word of E2M1 codes, times s (POWER: a power of two, or
// zero, which the conversion takes for a very small one).
template <bool POWER = false>
__device__ __forceinline__ void e2m1_values(uint32_t w, float s, float (&v)[8]) {
#define QLIN_PAIR(i)                                                                        \
    {                                                                                       \
        const auto f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, POWER ? s : 1.0f, i);    \
        v[2 * i] = POWER ? f[0] : f[0] * s;                                                 \
        v[2 * i + 1] = POWER ? f[1] : f[1] * s;                                             \
    }
    QLIN_PAIR(0) QLIN_PAIR(1) QLIN_PAIR(2) QLIN_PAIR(3)
#undef QLIN_PAIR
}

template <int MODE>
__device__ __forceinline__ void word_values(uint32_t w, float s, float z, float (&v)[8]) {
    if constexpr (MODE == AFFINE) {
        const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __builtin_fmaf(s, (float)(((i & 1 ? odd : even) >> (i / 2 * 8)) & 0xFFu), z);
    } else {
        e2m1_values(w, s, v);
    }
}

// Scale (and bias) of a group as numbers.
template <int MODE, int SDT>
__device__ __forceinline__ float scale_at(const void* p, int64_t i) {
    if constexpr (MODE == AFFINE) return load_f<SDT>(p, i);
    else if constexpr (MODE == NVFP4) return e4m3_to_f32(((const uint8_t*)p)[i]);
    else return e8m0_to_f32(((const uint8_t*)p)[i]);
}

// floor(log2 |x|) of a finite number other than zero.
__device__ __forceinline__ int ilogb_of(float x) { return __builtin_amdgcn_frexp_expf(x) - 1; }

// Two numbers rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t round2(float a, float b) {
    if constexpr (DT == QLIN_BF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}

// sum plus the two numbers of a pair that round2 made, exact but for the sums' own
// rounding (subnormal f16 numbers among them).
template <int DT>
__device__ __forceinline__ float add2(uint32_t pair, float sum) {
    if constexpr (DT == QLIN_BF16)
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), bf16x2{(__bf16)1.0f, (__bf16)1.0f}, sum, false);
    else
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, pair), f16x2{(_Float16)1.0f, (_Float16)1.0f}, sum, false);
}

struct TileArgs {
    AttendArgs a;
    KvPool c;
    int chunk, splits;           // keys of a workgroup; splits of the grid
    float* part_o;               // [tile, head, split, row, D]
    float* part_ml;              // [tile, head, split, row, 2]: maximum (of scores times log2 e), sum
    const uint8_t* images;       // prompt tiles: dense keys and values of kImageKeys keys, [sequence, key block, head]
    uint64_t* present;           // [sequence, key block]: which of its keys are there
    float* key_scale;            // [sequence, key block, head]: what its keys are to be multiplied by
    int32_t* value_power;        // [sequence, key block, head]: the power of two that its values are to be multiplied by
    int key_blocks;              // of a sequence
};

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, f32x4 v) {
    *(uint2*)((uint16_t*)p + i) = uint2{round2<DT>(v[0], v[1]), round2<DT>(v[2], v[3])};
}

// Joins the chunks of each row, out = sum f o / sum f l with f = exp2(m - largest
// m): WAVES waves a row, D / 4 lanes a chunk, the others the next chunks; sums
// in one fixed order. unit: as the chunks were cut.
template <int DT, int D, int WAVES>
__global__ void __launch_bounds__(256) attend_join_kernel(TileArgs t, int tile_rows, int unit) {
    constexpr int L4 = D / 4, AT_ONCE = 64 / L4, ROWS = 4 / WAVES, STRIDE = AT_ONCE * WAVES;
    __shared__ f32x4 part_x[WAVES][WAVES > 1 ? L4 : 1];
    __shared__ float part_l[WAVES];
    const AttendArgs& a = t.a;
    const KvPool& c = t.c;
    const int groups = (tile_rows + ROWS - 1) / ROWS, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int row = (int)(blockIdx.x % groups) * ROWS + wave / WAVES, h = blockIdx.y;
    const int64_t tile = blockIdx.x / groups;
    if (row >= tile_rows) return;
    const int64_t part = ((tile * c.heads + h) * t.splits) * tile_rows + row;
    const float2* const ml = (const float2*)t.part_ml + part;
    // the first chunks' numbers, before the lengths say how many there are
    const float2 early = ml[(int64_t)min(lane, t.splits - 1) * tile_rows];
    TileWork w = tile_of(a, c, tile, tile_rows);
    if (row >= w.rows) return;
    tile_keys(a, c, w, t.chunk, unit);
    if (w.splits <= 1) return;
    float top = lane < w.splits ? early.x : kNone;
    for (int i = lane + 64; i < w.splits; i += 64) top = fmaxf(top, ml[(int64_t)i * tile_rows].x);
#pragma unroll
    for (int off = 32; off; off /= 2) top = fmaxf(top, __shfl_xor(top, off, 64));
    const int mine = wave % WAVES * AT_ONCE + lane / L4, d = lane % L4 * 4;
    f32x4 x{0, 0, 0, 0};
    float l = 0.0f;
    if (lane / L4 < AT_ONCE) {
        const float* const o = t.part_o + part * D + d;
#pragma unroll 4
        for (int i = mine; i < w.splits; i += STRIDE) {
            const float2 e = ml[(int64_t)i * tile_rows];
            const float f = e.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(e.x - top);
            l = __builtin_fmaf(f, e.y, l);
            x += f * *(const f32x4*)(o + (int64_t)i * tile_rows * D);
        }
    }
    const f32x4 own = x;                         // what the lane itself has: sums in between would count twice
    const float own_l = l;
#pragma unroll
    for (int i = 1; i < AT_ONCE; ++i) {
        l += __shfl(own_l, lane + i * L4, 64);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += __shfl(own[e], lane + i * L4, 64);
    }
    if constexpr (WAVES > 1) {
        if (lane < L4) part_x[wave][lane] = x;
        if (lane == 0) part_l[wave] = l;
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int i = 1; i < WAVES; ++i) {
            if (lane < L4) x += part_x[i][lane];
            l += part_l[i];
        }
    }
    if (lane >= L4) return;
    x *= l == 0.0f ? 0.0f : 1.0f / l;
    const int share = a.q_heads / c.heads, rr = w.row0 + row;
    store4<DT>(a.out, ((w.s.first + rr / share) * a.q_heads + h * share + rr % share) * D + d, x);
}

// A wave a row, or four where few rows have many chunks (65 chunks of 32 rows, D
// 128: 6.7 and 3.8 us; 10 chunks of 2048 rows: 7.8 and 11.1 us).
template <int DT, int D>
hipError_t launch_join(const TileArgs& t, int64_t tiles, int tile_rows, int unit, hipStream_t st) {
    if (t.splits > 8 && tiles * tile_rows * t.c.heads <= 2048)
        attend_join_kernel<DT, D, 4><<<dim3((unsigned)(tiles * tile_rows), (unsigned)t.c.heads), 256, 0, st>>>(t, tile_rows, unit);
    else
        attend_join_kernel<DT, D, 1><<<dim3((unsigned)(tiles * ((tile_rows + 3) / 4)), (unsigned)t.c.heads), 256, 0, st>>>(t, tile_rows, unit);
    return hipGetLastError();
}

}  // namespace
}  // namespace qlin
