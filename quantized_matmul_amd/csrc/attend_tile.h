// attend_tile.h -- attention over the 4-bit cache on the matrix cores, for the
// rows of q that share few keys' reads: decode and drafted tokens. One head
// size a translation unit (attend_tile_*.hip).
//
// A sequence's rows of one key head (n tokens by q_heads / heads query heads)
// form tiles of 16 NT rows; a workgroup takes a tile and `chunk` keys, its four
// waves every fourth step of 32 keys, each with its own running maximum m, sum l
// and o (o = sum of p v, p = exp2(score - m)), joined through LDS at the end.
// Workgroups of other chunks of the same rows leave o, m and l in the workspace
// and attend_join adds them up.
//
// Everything of a step stays in registers, no key or value passes through LDS:
//   scores^T = K q^T: lane (r = lane % 16, j = lane / 16) of an A operand holds
//     key r's codes, eight of them a word as they lie in memory; q's operand has
//     its values in the same order. Keys stay codes: affine ones become 16 + c
//     (bf16) by a shift and one and-or for two of them, the accumulator starts
//     at -16 sum(q), and scale and bias join in fp32: score = s acc + z sum(q).
//   o^T = V^T p^T: the scores leave the matrix cores as p's operand wants them
//     (lane (q row, j) has keys 4j..4j+3 of both sub-tiles), so lane (r, j) of V's
//     operand takes word r of those eight keys: its eight codes are eight rows of
//     V^T, decoded in fp32 and rounded in pairs of keys.
// Scales and biases go through LDS once, as numbers (a lane there needs those of
// eight keys); keys outside the sequence get zeros there, whatever their page holds.
//
// Bound by the memory: D/2 bytes and the scales of a key and of a value, read
// once for the tile's rows.
#pragma once

#include <type_traits>

#include "attend_common.h"

namespace qlin {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;                       // keys of a wave's step
constexpr int kMaxChunk = 4096;                 // keys of a workgroup, a multiple of kWaves * kStep
constexpr int kScaleRow = kStep + 4;            // floats of a group's scales of a step in LDS: rows on other banks

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == QLIN_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A word's eight codes as an MFMA operand: AFFINE 16 + c, pairs (i, i + 4);
// else the code's number, pairs (2i, 2i + 1).
template <int DT, int MODE>
__device__ __forceinline__ u32x4 code_operand(uint32_t w) {
    if constexpr (MODE == AFFINE) {
        if constexpr (DT == QLIN_BF16)
            return u32x4{((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                         ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u};
        else
            return u32x4{((w << 6) & 0x03C003C0u) | 0x4C004C00u, ((w << 2) & 0x03C003C0u) | 0x4C004C00u,
                         ((w >> 2) & 0x03C003C0u) | 0x4C004C00u, ((w >> 6) & 0x03C003C0u) | 0x4C004C00u};
    } else if constexpr (DT == QLIN_BF16) {
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3))};
    } else {
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3))};
    }
}
// Value of q in the half-word e (0..7) of that operand.
template <int MODE>
__device__ __forceinline__ constexpr int operand_place(int e) {
    return MODE == AFFINE ? (e / 2) + 4 * (e % 2) : e;
}

// Largest (sum) over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float across_max(float v) {
    uint32_t u = __float_as_uint(v);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    u = __float_as_uint(v);
    a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float across_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// LDS writes of a wave before its own reads, without a barrier for the others.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// GQ: a quant group's words over 4 (AFFINE 32/64/128: 1/2/4; MXFP4: 1; NVFP4: unused)
template <int DT, int MODE, int D, int GQ, int NT>
__global__ void __launch_bounds__(256, D * NT <= 256 ? 2 : 1) attend_tile_kernel(TileArgs t) {
    constexpr int HW = D / 8;                              // words of a head's row
    constexpr int NM = D / 32;                             // MFMAs along D for 16 keys
    constexpr int G = MODE == NVFP4 ? 16 : 32 * GQ;
    constexpr int NG = D / G;                              // quant groups of a row
    constexpr int VC = (HW + 15) / 16;                     // words of a value a lane takes
    constexpr int R = 16 * NT;
    constexpr bool AFF = MODE == AFFINE;
    constexpr int ARR = AFF ? 4 : 2;                       // scale arrays of a step
    constexpr int SCALES = kWaves * ARR * NG * kScaleRow, OBUF = R * (D + 4);
    __shared__ int32_t blocks[kMaxChunk / kKvUnit];
    __shared__ float buf[SCALES > OBUF ? SCALES : OBUF];
    __shared__ float wave_ml[kWaves][R][2];

    const AttendArgs& a = t.a;
    const KvPool& c = t.c;
    const int split = blockIdx.x % t.splits, h = blockIdx.x / t.splits % c.heads;
    const int64_t tile = blockIdx.x / t.splits / c.heads;
    const TileWork w = tile_work(a, c, tile, R, t.chunk, kKvUnit);
    if (!w.rows || (split && split >= w.splits)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64, r = lane % 16, j = lane / 16;
    const int share = a.q_heads / c.heads;
    const int k0 = w.k0 + split * t.chunk, k1 = w.splits ? min(w.hi, k0 + t.chunk) : k0;
    const int steps = (k1 - k0 + kStep - 1) / kStep;
    {
        const int32_t* table = a.table + (int64_t)w.b * a.width;
        for (int i = tid; i < steps * (kStep / kKvUnit); i += 256) {
            const int key = k0 + i * kKvUnit;
            blocks[i] = key < k1 ? kv_row_block(table, c.pages, c.heads, c.page, h, key / kKvUnit) : -1;
        }
    }

    // rows of q: their place, the keys they see, their operand
    Seen seen[NT];
    u32x4 q[NT][NM];
    f32x4 start[NT][AFF ? NG : 1];
    float qsum[NT][AFF ? NG : 1];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int rr = min(w.row0 + n * 16 + r, w.row0 + w.rows - 1);     // rows past the end repeat the last
        seen[n] = seen_by(a, w.s, rr / share);
        const uint16_t* qp = (const uint16_t*)a.q + (w.s.first + rr / share) * a.q_stride + (int64_t)(h * share + rr % share) * D;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const int word = MODE == NVFP4 ? m * 4 + j : m / GQ * (4 * GQ) + j * GQ + m % GQ;
            uint32_t e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = qp[word * 8 + operand_place<MODE>(i)];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[n][m][i] = e[2 * i] | (e[2 * i + 1] << 16);
        }
        if constexpr (AFF) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float sum = 0.0f;
#pragma unroll
                for (int m = 0; m < GQ; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t d = q[n][g * GQ + m][i];
                        sum += DT == QLIN_BF16 ? __uint_as_float(d << 16) : f16_bits_to_f32(d & 0xFFFFu);
                        sum += DT == QLIN_BF16 ? __uint_as_float(d & 0xFFFF0000u) : f16_bits_to_f32(d >> 16);
                    }
                sum = across_sum(sum);
                qsum[n][g] = sum;
                start[n][g] = f32x4{-16.0f * sum, -16.0f * sum, -16.0f * sum, -16.0f * sum};
            }
        }
    }
    __syncthreads();

    f32x4 o[NT][VC * 8];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kNone;
        l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < VC * 8; ++i) o[n][i] = f32x4{0, 0, 0, 0};
    }
    const float scale = a.scale * kLog2e;
    float* const sl = buf + wave * (ARR * NG * kScaleRow);               // this wave's scales: [array, group, key]
    constexpr int SE = (kStep * NG + 63) / 64;                           // a lane's numbers of an array
    constexpr int VROW = HW < 16 ? HW : 16;

    uint32_t kw[2][NM], vw[8][VC];
    float sraw[ARR][SE];
    int32_t rb[2];

    auto load = [&](int step) {
#pragma unroll
        for (int st = 0; st < 2; ++st) rb[st] = __builtin_amdgcn_readfirstlane(blocks[step * 2 + st]);
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const int64_t row = (int64_t)max(rb[st], 0) * kKvUnit;
            const uint32_t* kp = c.codes[0] + row * HW;
            const uint32_t* vp = c.codes[1] + row * HW;
            if constexpr (MODE == NVFP4) {
#pragma unroll
                for (int i = 0; i < NM; ++i) kw[st][i] = kp[r * HW + i * 4 + j];
            } else {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t* p = kp + r * HW + g * (4 * GQ) + j * GQ;
                    if constexpr (GQ == 4) {
                        const uint4 v = *(const uint4*)p;
                        kw[st][4 * g] = v.x; kw[st][4 * g + 1] = v.y; kw[st][4 * g + 2] = v.z; kw[st][4 * g + 3] = v.w;
                    } else if constexpr (GQ == 2) {
                        const uint2 v = *(const uint2*)p;
                        kw[st][2 * g] = v.x; kw[st][2 * g + 1] = v.y;
                    } else {
                        kw[st][g] = *p;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    const int word = v * 16 + r;
                    vw[st * 4 + i][v] = vp[(4 * j + i) * HW + (word < HW ? word : word - VROW)];
                }
        }
#pragma unroll
        for (int e = 0; e < SE; ++e) {
            const int at = lane + 64 * e, key = at / NG, g = at % NG;
            const bool second = key >= kKvUnit;
            const int32_t b = second ? rb[1] : rb[0];
            const bool live = b >= 0 && k0 + step * kStep + key < k1 && at < kStep * NG;
            const int64_t i = ((int64_t)max(b, 0) * kKvUnit + key % kKvUnit) * NG + g;
#pragma unroll
            for (int s = 0; s < ARR; ++s) {
                const void* p = s < 2 ? c.scales[s] : c.biases[s - 2];
                const float x = AFF ? load_f<DT>(p, i) : scale_at<MODE, DT>(p, i);
                sraw[s][e] = live ? x : 0.0f;
            }
        }
    };

    if (wave < steps) load(wave);
    for (int step = wave; step < steps; step += kWaves) {
        const int key0 = k0 + step * kStep;
        // the step's scales where the lanes find those of their keys
#pragma unroll
        for (int e = 0; e < SE; ++e) {
            const int at = lane + 64 * e;
            if (kStep * NG % 64 == 0 || at < kStep * NG)
#pragma unroll
                for (int s = 0; s < ARR; ++s) sl[(s * NG + at % NG) * kScaleRow + at / NG] = sraw[s][e];
        }
        wave_fence();
        f32x4 sc[NT][2];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if constexpr (MODE == NVFP4) {
#pragma unroll
                for (int n = 0; n < NT; ++n) sc[n][st] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NM; ++i) {
                    // the word's group is not its MFMA's only one: its codes take their scale here, exact in both types
                    const float s = sl[(2 * i + j / 2) * kScaleRow + st * 16 + r];
                    float v[8];
                    e2m1_values(kw[st][i], s, v);
                    const u32x4 k{round2<DT>(v[0], v[1]), round2<DT>(v[2], v[3]), round2<DT>(v[4], v[5]), round2<DT>(v[6], v[7])};
#pragma unroll
                    for (int n = 0; n < NT; ++n) sc[n][st] = mfma16<DT>(k, q[n][i], sc[n][st]);
                }
            } else {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const f32x4 s = *(const f32x4*)(sl + g * kScaleRow + st * 16 + 4 * j);
                    f32x4 z{0, 0, 0, 0};
                    if constexpr (AFF) z = *(const f32x4*)(sl + (2 * NG + g) * kScaleRow + st * 16 + 4 * j);
                    u32x4 k[GQ];
#pragma unroll
                    for (int i = 0; i < GQ; ++i) k[i] = code_operand<DT, MODE>(kw[st][g * GQ + i]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        f32x4 acc = AFF ? start[n][g] : f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int i = 0; i < GQ; ++i) acc = mfma16<DT>(k[i], q[n][g * GQ + i], acc);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x = g ? sc[n][st][i] : 0.0f;
                            if constexpr (AFF) x = g ? __builtin_fmaf(z[i], qsum[n][g], x) : z[i] * qsum[n][g];
                            sc[n][st][i] = (AFF || g) ? __builtin_fmaf(s[i], acc[i], x) : s[i] * acc[i];
                        }
                    }
                }
            }
        }
        const bool whole[2] = {rb[0] >= 0, rb[1] >= 0};
        u32x4 p[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = sc[n][e / 4][e % 4] * scale;
            const bool inside = key0 >= seen[n].lo && key0 + kStep <= seen[n].hi && whole[0] && whole[1];
            if (__any(!inside)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int key = key0 + e / 4 * 16 + 4 * j + e % 4;
                    if (key < seen[n].lo || key >= seen[n].hi || !whole[e / 4]) x[e] = kNone;
                }
            }
            float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            top = fmaxf(across_max(top), m[n]);
            if (__any(top > m[n])) {
                const float f = m[n] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m[n] - top);
                m[n] = top;
                l[n] *= f;
#pragma unroll
                for (int i = 0; i < VC * 8; ++i) o[n][i] *= f;
            }
            const float base = m[n] == kNone ? 0.0f : m[n];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = __builtin_amdgcn_exp2f(x[e] - base);
                l[n] += x[e];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) p[n][i] = round2<DT>(x[2 * i], x[2 * i + 1]);
        }
        // values: word v*16 + r of the lane's eight keys
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            const int word = v * 16 + r, g = (word < HW ? word : word - VROW) / (G / 8);
            const f32x4 s0 = *(const f32x4*)(sl + (NG + g) * kScaleRow + 4 * j);
            const f32x4 s1 = *(const f32x4*)(sl + (NG + g) * kScaleRow + 16 + 4 * j);
            if constexpr (AFF) {
                const f32x4 z0 = *(const f32x4*)(sl + (3 * NG + g) * kScaleRow + 4 * j);
                const f32x4 z1 = *(const f32x4*)(sl + (3 * NG + g) * kScaleRow + 16 + 4 * j);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t even = vw[e][v] & 0x0F0F0F0Fu, odd = (vw[e][v] >> 4) & 0x0F0F0F0Fu;
                        const float code = (float)(((i & 1 ? odd : even) >> (i / 2 * 8)) & 0xFFu);
                        x[e] = __builtin_fmaf(e < 4 ? s0[e & 3] : s1[e & 3], code, e < 4 ? z0[e & 3] : z1[e & 3]);
                    }
                    const u32x4 vt{round2<DT>(x[0], x[1]), round2<DT>(x[2], x[3]), round2<DT>(x[4], x[5]), round2<DT>(x[6], x[7])};
#pragma unroll
                    for (int n = 0; n < NT; ++n) o[n][v * 8 + i] = mfma16<DT>(vt, p[n], o[n][v * 8 + i]);
                }
            } else {
                float x[8][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) e2m1_values(vw[e][v], e < 4 ? s0[e & 3] : s1[e & 3], x[e]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const u32x4 vt{round2<DT>(x[0][i], x[1][i]), round2<DT>(x[2][i], x[3][i]),
                                   round2<DT>(x[4][i], x[5][i]), round2<DT>(x[6][i], x[7][i])};
#pragma unroll
                    for (int n = 0; n < NT; ++n) o[n][v * 8 + i] = mfma16<DT>(vt, p[n], o[n][v * 8 + i]);
                }
            }
        }
        wave_fence();                                        // scales are read before the next step's come
        if (step + kWaves < steps) load(step + kWaves);
    }

    // the waves' sums: a common maximum, then o added up in LDS in the order of the waves
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        l[n] = across_sum(l[n]);
        if (j == 0) {
            wave_ml[wave][n * 16 + r][0] = m[n];
            wave_ml[wave][n * 16 + r][1] = l[n];
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float top = kNone;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) top = fmaxf(top, wave_ml[i][n * 16 + r][0]);
        const float f = m[n] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m[n] - top);
#pragma unroll
        for (int i = 0; i < VC * 8; ++i) o[n][i] *= f;
    }
    for (int turn = 0; turn < kWaves; ++turn) {
        if (turn == wave) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n * 16 + r >= w.rows) continue;
#pragma unroll
                for (int v = 0; v < VC; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int word = v * 16 + 4 * j + i;
                        if (word >= HW) continue;
                        f32x4* at = (f32x4*)(buf + (n * 16 + r) * (D + 4) + word * 8);
                        f32x4 x0{o[n][v * 8][i], o[n][v * 8 + 1][i], o[n][v * 8 + 2][i], o[n][v * 8 + 3][i]};
                        f32x4 x1{o[n][v * 8 + 4][i], o[n][v * 8 + 5][i], o[n][v * 8 + 6][i], o[n][v * 8 + 7][i]};
                        if (turn) {
                            x0 += at[0];
                            x1 += at[1];
                        }
                        at[0] = x0;
                        at[1] = x1;
                    }
            }
        }
        __syncthreads();
    }
    const int64_t part = (tile * c.heads + h) * t.splits + split;
    for (int e = tid; e < w.rows * (D / 4); e += 256) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        float top = kNone, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) top = fmaxf(top, wave_ml[i][row][0]);
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
            sum += wave_ml[i][row][0] == kNone ? 0.0f : wave_ml[i][row][1] * __builtin_amdgcn_exp2f(wave_ml[i][row][0] - top);
        f32x4 x = *(const f32x4*)(buf + row * (D + 4) + d);
        if (w.splits <= 1) {
            x *= sum == 0.0f ? 0.0f : 1.0f / sum;                        // a row that sees no key: zeros
            const int rr = w.row0 + row;
            store4<DT>(a.out, ((w.s.first + rr / share) * a.q_heads + h * share + rr % share) * D + d, x);
        } else {
            *(f32x4*)(t.part_o + (part * R + row) * D + d) = x;
            if (d == 0) {
                t.part_ml[(part * R + row) * 2] = top;
                t.part_ml[(part * R + row) * 2 + 1] = sum;
            }
        }
    }
}

template <int D>
hipError_t launch_tile_of(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                          hipStream_t st) {
    const int R = 16 * p.nt;
    TileArgs t{a, c, p.chunk, p.splits, (float*)workspace, nullptr, nullptr, nullptr, nullptr, 0};
    t.part_ml = t.part_o + p.tiles * c.heads * p.splits * R * D;
    const unsigned grid = (unsigned)(p.tiles * c.heads * p.splits);
    auto run = [&](auto dtc, auto mode, auto gq) -> hipError_t {
        constexpr int DT = decltype(dtc)::value, M = decltype(mode)::value, GQ = decltype(gq)::value;
        if constexpr (M == AFFINE && D % (32 * GQ) != 0) {
            return hipErrorInvalidValue;
        } else {
            if (p.nt == 1) attend_tile_kernel<DT, M, D, GQ, 1><<<grid, 256, 0, st>>>(t);
            else if (p.nt == 2) attend_tile_kernel<DT, M, D, GQ, 2><<<grid, 256, 0, st>>>(t);
            else return hipErrorInvalidValue;
            hipError_t e = hipGetLastError();
            if (e != hipSuccess || p.splits == 1) return e;
            return launch_join<DT, D>(t, p.tiles, R, kKvUnit, st);
        }
    };
    auto moded = [&](auto dtc) -> hipError_t {
        using I1 = std::integral_constant<int, 1>;
        using I2 = std::integral_constant<int, 2>;
        using I4 = std::integral_constant<int, 4>;
        if (c.mode == MXFP4) return run(dtc, std::integral_constant<int, MXFP4>{}, I1{});
        if (c.mode == NVFP4) return run(dtc, std::integral_constant<int, NVFP4>{}, I1{});
        using A = std::integral_constant<int, AFFINE>;
        return c.g == 32 ? run(dtc, A{}, I1{}) : (c.g == 64 ? run(dtc, A{}, I2{}) : run(dtc, A{}, I4{}));
    };
    return dt == QLIN_BF16 ? moded(std::integral_constant<int, QLIN_BF16>{}) : moded(std::integral_constant<int, QLIN_F16>{});
}

}  // namespace
}  // namespace qlin
