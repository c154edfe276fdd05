// attend_prompt.h -- attention over the 4-bit cache where many rows share the
// keys: (parts of) prompts. Two launches, a third where keys are split.
//
// attend_lay_kernel decodes the keys that any row sees once, into blocks of 64
// keys and a head laid out as the second kernel's LDS wants them: keys as
// [8 values][key], values as [8 keys][value], 16 bytes each, so that a wave's
// operands are contiguous (no bank is met twice) and blocks go from memory to
// LDS as they are. The eight keys of a piece are those that a lane's scores come
// out as: 4 hb .. 4 hb + 3 and 8 + 4 hb .. (hb = lane / 32).
// Keys, values, q and p are multiplied as f16 for either type, a block's keys
// divided by a power of two that takes their largest into [1, 2), its values and
// a row of q likewise: bf16 keys put 2^-9 of |q| |k| on a score, which a sharp
// softmax passes on, and bf16 values and p as much on the output (errors of a
// bf16 output, whose own rounding is 0.0017: 0.0051; with f16 keys 0.0025, with
// all in f16 0.0018). No value leaves f16's range; what is 2^-14 of the largest
// of its block and less is held to 2^-25 of that. o is kept in units of a power
// of two that follows the blocks': up to any larger one, and down where a block's
// lies 2^4 and more below, so that p, divided by what is left between the two, is
// held to 2^-21 at least (blocks within 2^64 of the largest; rows may see none but
// small ones). A block without values has no power. f16 rows add up p as it
// multiplies the values, rounded, so that their weights make one (equal values come
// out as they are; in bf16 that does not show, and cost 2 %).
// f16 prompts take affine keys as two f16 numbers, the second the first one's rest,
// and two products: with one, scores made outputs 2.5 times as far off as their own
// rounding, with both 1.43 (p's and the values' rounding). 8192 rows over 16384
// keys (D 128) 1.75 and 2.28 ms, 4096 over 8192 of D 256 0.91 and 1.18.
// Decoding inside the attention kernel would cost every workgroup again what
// this does once: 190 of about 560 vector instructions of 64 keys (D 128), where
// the matrix cores need the time of 512.
//
// attend_prompt_kernel: a workgroup takes 128 RT rows (a sequence's rows of one
// key head, as in attend_tile.h), a wave 32 RT of them, with blocks of keys in
// two LDS buffers, the next one on its way while one is used:
//   scores^T = K q^T, 32 keys by 32 rows; p = exp2(score - m) for the lane's row;
//   o^T += V^T p^T, p's operand being the lane's own scores, rounded.
// The running maximum m follows the scores only where they pass it by 2^8, so
// that o is rarely scaled. A wave reads each operand of K and V once for its
// 32 RT rows: RT = 2 keeps LDS below the matrix cores' time, for D up to 128 (o
// would not fit the registers above) and where tiles of 256 rows fill the chip;
// otherwise RT = 1, in buffers of 32 keys, which three workgroups (two above 128)
// hold at once.
//
// 8192 rows of 32 heads over 16384 keys of 8 (D 128, bf16): 1.53 to 1.66 ms, 1.0
// to 1.08 PFLOP/s; laying the keys out is 29 us of that. The matrix cores are
// busy for half the cycles and the vector units (softmax) for as many, two waves
// of a SIMD in turn, at 2.0 of 2.4 GHz. Priorities for either part, and barriers
// that keep the compiler from mixing the two, cost 2 %. 4096 rows over 8192 keys:
// D 64 0.66 PFLOP/s, 96 0.79, 192 0.87, 256 0.94.
#pragma once

#include <type_traits>

#include "attend_common.h"

namespace qlin {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;

constexpr int kImageKeys = 64;
constexpr int kNoPower = -1000;                  // of zeros: below any number's
constexpr int kFall = 4;                         // how far a block's power may lie below o's
constexpr int kReach = 64;                       // how far o's may lie below the largest so far: o stays inside fp32

__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A block of 256 threads: the 64 keys of one image, in parts of BK keys.
template <int DT, int MODE, int D, int BK>
__global__ void __launch_bounds__(256) attend_lay_kernel(TileArgs t, uint8_t* images) {
    constexpr bool LO = prompt_halves(DT, MODE);
    constexpr int HW = D / 8, KEYS = BK * D * (LO ? 4 : 2), PART = KEYS + BK * D * 2;      // (LO: their rests behind the keys)
    const AttendArgs& a = t.a;
    const KvPool& c = t.c;
    const int h = blockIdx.x % c.heads, kb = blockIdx.x / c.heads % t.key_blocks, b = blockIdx.x / c.heads / t.key_blocks;
    const Sequence s = sequence_of(a, c, b);
    if (!s.n) return;
    const int lo = seen_by(a, s, 0).lo, hi = seen_by(a, s, s.n - 1).hi, key0 = kb * kImageKeys;
    if (key0 >= hi || key0 + kImageKeys <= lo) return;
    __shared__ int32_t blocks[kImageKeys / kKvUnit];
    __shared__ float largest[2][4];
    const int tid = threadIdx.x;
    if (tid < kImageKeys / kKvUnit)
        blocks[tid] = key0 + tid * kKvUnit < s.keys
                          ? kv_row_block(a.table[(int64_t)b * a.width + (key0 + tid * kKvUnit) / c.page], c.pages, c.heads,
                                         c.page, h, key0 / kKvUnit + tid)
                          : -1;
    __syncthreads();
    const int per = c.g / 8, groups = D / c.g;
    uint8_t* const image = images + (((int64_t)b * t.key_blocks + kb) * c.heads + h) * (kImageKeys / BK * PART);
    auto row_of = [&](int key) -> int64_t {      // -1: not there, or no row sees it
        const int32_t rb = blocks[key / kKvUnit];
        return rb >= 0 && key0 + key >= lo && key0 + key < hi ? (int64_t)rb * kKvUnit + key % kKvUnit : -1;
    };
    // power of two of the largest value of a side's keys, kNoPower where they are all zero or not there
    auto power = [&](int side) {
        const int64_t row = row_of(tid % 64);
        float most = 0.0f;
        for (int g = tid / 64; g < groups; g += 4)
            if (row >= 0) {
                const float sc = scale_at<MODE, DT>(c.scales[side], row * groups + g);
                const float z = MODE == AFFINE ? load_f<DT>(c.biases[side], row * groups + g) : 0.0f;
                most = fmaxf(most, MODE == AFFINE ? fmaxf(fabsf(z), fabsf(__builtin_fmaf(sc, 15.0f, z))) : 6.0f * fabsf(sc));
            }
#pragma unroll
        for (int off = 32; off; off /= 2) most = fmaxf(most, __shfl_xor(most, off, 64));
        if (tid % 64 == 0) largest[side][tid / 64] = most;
        __syncthreads();
        most = fmaxf(fmaxf(largest[side][0], largest[side][1]), fmaxf(largest[side][2], largest[side][3]));
        return most > 0.0f ? ilogb_of(most) : kNoPower;
    };
    {
        const int key = tid % 64;
        const int64_t row = row_of(key);
        if (h == 0) {
            const uint64_t there = __ballot(row >= 0);
            if (tid == 0) t.present[(int64_t)b * t.key_blocks + kb] = there;
        }
        int e = power(0);
        if (e == kNoPower) e = 0;
        if (tid == 0) t.key_scale[((int64_t)b * t.key_blocks + kb) * c.heads + h] = __builtin_ldexpf(1.0f, e);
        for (int w = tid / 64; w < HW; w += 4) {
            u32x4 out{0, 0, 0, 0}, rest{0, 0, 0, 0};
            if (row >= 0) {
                const int64_t g = row * groups + w / per;
                float v[8];
                word_values<MODE>(c.codes[0][row * HW + w], scale_at<MODE, DT>(c.scales[0], g),
                                  MODE == AFFINE ? load_f<DT>(c.biases[0], g) : 0.0f, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __builtin_ldexpf(v[i], -e);
                out = u32x4{round2<QLIN_F16>(v[0], v[1]), round2<QLIN_F16>(v[2], v[3]), round2<QLIN_F16>(v[4], v[5]),
                            round2<QLIN_F16>(v[6], v[7])};
                if constexpr (LO) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        rest[i] = round2<QLIN_F16>(v[2 * i] - f16_bits_to_f32(out[i] & 0xFFFFu), v[2 * i + 1] - f16_bits_to_f32(out[i] >> 16));
                }
            }
            uint8_t* const to = image + key / BK * PART + w * (BK * 16) + key % BK * 16;
            *(u32x4*)to = out;
            if constexpr (LO) *(u32x4*)(to + BK * D * 2) = rest;
        }
    }
    const int ve = power(1);
    if (tid == 0) t.value_power[((int64_t)b * t.key_blocks + kb) * c.heads + h] = ve;
    for (int e = tid; e < 8 * HW; e += 256) {
        const int w = e % HW, piece = e / HW;    // keys 16 (piece / 2) + 4 (piece % 2) + {0..3, 8..11}
        float v[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = row_of(16 * (piece / 2) + 4 * (piece % 2) + i % 4 + 8 * (i / 4));
            if (row >= 0) {
                const int64_t g = row * groups + w / per;
                word_values<MODE>(c.codes[1][row * HW + w], scale_at<MODE, DT>(c.scales[1], g),
                                  MODE == AFFINE ? load_f<DT>(c.biases[1], g) : 0.0f, v[i]);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[i][k] = __builtin_ldexpf(v[i][k], -ve);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
            }
        }
        uint8_t* const to = image + piece / (BK / 8) * PART + KEYS + (piece % (BK / 8) * D + w * 8) * 16;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            *(u32x4*)(to + k * 16) = u32x4{round2<QLIN_F16>(v[0][k], v[1][k]), round2<QLIN_F16>(v[2][k], v[3][k]),
                                           round2<QLIN_F16>(v[4][k], v[5][k]), round2<QLIN_F16>(v[6][k], v[7][k])};
    }
}

// Waves of a SIMD that the registers hold.
constexpr int prompt_residents(int D, int RT) { return D <= 128 && RT == 1 ? 3 : 2; }
// Keys of a buffer: two (three) workgroups' pairs of them fit a CU's LDS.
constexpr int prompt_keys(int D, int RT, bool LO) { return D <= 128 && RT == 2 && !LO ? 64 : 32; }
// Buffers of a workgroup: of two with one each, the other computes while one's keys come (D 256, 4096 rows over 8192 keys:
// 1.64 ms by one workgroup with two buffers, 1.18 so).
constexpr int prompt_buffers(int D, bool LO) { return D == 256 && LO ? 1 : 2; }

// LO: keys come with their rests.
template <int DT, int D, int RT, bool LO>
__global__ void __launch_bounds__(256, prompt_residents(D, RT)) attend_prompt_kernel(TileArgs t, int64_t tiles) {
    constexpr int R = 128 * RT, KS = D / 16, DTILES = D / 32, BK = prompt_keys(D, RT, LO), KEYS = BK * D * (LO ? 4 : 2);
    constexpr int PART = KEYS + BK * D * 2, ROUNDS = (PART + 4095) / 4096, PARTS = kImageKeys / BK, IMAGE = PARTS * PART;
    constexpr int BUFS = prompt_buffers(D, LO);
    __shared__ __attribute__((aligned(16))) uint8_t lds[BUFS][PART];
    const AttendArgs& a = t.a;
    const KvPool& c = t.c;
    // heads over the XCDs, so that each L2 keeps its head's keys; the last tiles, which see most, first
    const int h = blockIdx.x % c.heads, split = blockIdx.x / c.heads % t.splits;
    const int64_t tile = tiles - 1 - blockIdx.x / c.heads / t.splits;
    TileWork w = tile_of(a, c, tile, R);
    if (!w.rows) return;
    tile_keys(a, c, w, t.chunk, kImageKeys);
    if (split && split >= w.splits) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64, r = lane % 32, hb = lane / 32;
    const int share = a.q_heads / c.heads;
    const KeyRange keys = chunk_of(w, split, t.chunk);
    const int k0 = keys.first, k1 = keys.end;
    const int kb0 = k0 / BK, kb1 = (k1 + BK - 1) / BK;

    auto row_at = [&](int i) { return min(w.row0 + i, w.row0 + w.rows - 1); };   // rows past the end repeat the last
    const int first = wave * 32 * RT;
    const Seen see_first = seen_by(a, w.s, row_at(first) / share), see_last = seen_by(a, w.s, row_at(first + 32 * RT - 1) / share);
    const bool idle = first >= w.rows;
    Seen seen[RT];
    u32x4 q[RT][KS];
    float row_scale[RT];
    // the sign of scale goes into q, so that maxima stay maxima, and so does a scale of zero, so that a masked -infinity
    // times it is none
    const float size = fabsf(a.scale) * kLog2e, scale = size == 0.0f ? 1.0f : size;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, keep = size == 0.0f ? 0u : ~0u;
#pragma unroll
    for (int n = 0; n < RT; ++n) {
        const int rr = row_at(first + n * 32 + r);
        seen[n] = seen_by(a, w.s, rr / share);
        const uint16_t* qp = (const uint16_t*)a.q + (w.s.first + rr / share) * a.q_stride + (int64_t)(h * share + rr % share) * D;
        const bool aligned = ((uintptr_t)qp & 15) == 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            u32x4 v;
            if (aligned) {
                v = *(const u32x4*)(qp + k * 16 + hb * 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = qp[k * 16 + hb * 8 + 2 * i] | ((uint32_t)qp[k * 16 + hb * 8 + 2 * i + 1] << 16);
            }
            q[n][k] = (v ^ flip) & keep;
        }
        uint32_t most = 0;                       // both types' sizes order as their patterns do
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) most = max(most, max(q[n][k][i] & 0x7FFFu, q[n][k][i] >> 16 & 0x7FFFu));
        most = max(most, (uint32_t)__shfl_xor((int)most, 32, 64));
        const int e = most ? ilogb_of(DT == QLIN_BF16 ? bf16_bits_to_f32(most) : f16_bits_to_f32(most)) : 0;
        row_scale[n] = __builtin_ldexpf(scale, e);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t d = q[n][k][i];
                const float x = DT == QLIN_BF16 ? bf16_bits_to_f32(d & 0xFFFFu) : f16_bits_to_f32(d & 0xFFFFu);
                const float y = DT == QLIN_BF16 ? bf16_bits_to_f32(d >> 16) : f16_bits_to_f32(d >> 16);
                q[n][k][i] = round2<QLIN_F16>(__builtin_ldexpf(x, -e), __builtin_ldexpf(y, -e));
            }
    }

    f32x16 o[RT][DTILES];
    float m[RT], l[RT];
    int unit = kNoPower, least = kNoPower;       // o's power of two; kReach below the largest so far
#pragma unroll
    for (int n = 0; n < RT; ++n) {
        m[n] = kNone;
        l[n] = 0.0f;
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[n][d][i] = 0.0f;
    }

    const uint8_t* const images = t.images + ((int64_t)w.b * t.key_blocks * c.heads + h) * IMAGE;
    auto fetch = [&](int kb, int buf) {
        const uint8_t* from = images + (int64_t)(kb / PARTS) * c.heads * IMAGE + kb % PARTS * PART + tid * 16;
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            if (PART % 4096 && i == ROUNDS - 1 && wave >= PART % 4096 / 1024) break;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + i * 4096),
                                             (__attribute__((address_space(3))) void*)(lds[buf] + i * 4096 + wave * 1024),
                                             16, 0, 0);
        }
    };

    if (BUFS == 2 && kb0 < kb1) fetch(kb0, 0);
    for (int kb = kb0; kb < kb1; ++kb) {
        const int buf = (kb - kb0) & (BUFS - 1);
        if constexpr (BUFS == 1) {
            __syncthreads();                     // the last block is read
            fetch(kb, 0);
        }
        const int64_t ib = (int64_t)w.b * t.key_blocks + kb / PARTS;          // waited for with the block:
        const uint64_t there = PARTS == 1 ? t.present[ib] : ((const uint32_t*)t.present)[ib * 2 + kb % 2] | 0xFFFFFFFF00000000ull;
        const float key_scale = t.key_scale[ib * c.heads + h];
        const int value_power = t.value_power[ib * c.heads + h];
        __syncthreads();                         // this block has landed, the other buffer is read
        if (BUFS == 2 && kb + 1 < kb1) fetch(kb + 1, buf ^ 1);
        const int key0 = kb * BK;
        if (idle || key0 >= see_last.hi || key0 + BK <= see_first.lo) continue;
        const int up = __builtin_amdgcn_readfirstlane(value_power);
        least = max(least, up - kReach);
        const int to = max(up, least);
        if (__builtin_expect((unsigned)(unit - to) > (unsigned)kFall, 0) && up != kNoPower) {     // (1580 us, 1571 so)
            const float f = __builtin_ldexpf(1.0f, unit == kNoPower ? 0 : unit - to);
            unit = to;
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int d = 0; d < DTILES; ++d) o[n][d] *= f;
        }
        // p is multiplied by 2^down, its sum back; where that is nothing beside the largest block (or there are no values),
        // by no less than 2^-64
        const int fall = max(up - unit, -kReach);
        const float down = (float)fall, back = __builtin_ldexpf(1.0f, -fall);
        const bool whole = there == ~0ull && key0 >= see_last.lo && key0 + BK <= see_first.hi;
        const uint8_t* const kl = lds[buf] + hb * (BK * 16) + r * 16;
        const uint8_t* const vl = lds[buf] + KEYS + hb * (D * 16) + r * 16;
#pragma unroll 1
        for (int kt = 0; kt < BK / 32; ++kt) {
            f32x16 s[RT];
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[n][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const u32x4 ka = *(const u32x4*)(kl + k * (2 * BK * 16) + kt * 512);
#pragma unroll
                for (int n = 0; n < RT; ++n) s[n] = mfma32(ka, q[n][k], s[n]);
                if constexpr (LO) {
                    const u32x4 kr = *(const u32x4*)(kl + BK * D * 2 + k * (2 * BK * 16) + kt * 512);
#pragma unroll
                    for (int n = 0; n < RT; ++n) s[n] = mfma32(kr, q[n][k], s[n]);
                }
            }
            u32x4 p[RT][2];
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                if (!whole) {
                    // the lane's keys are 8 (i / 4) + i % 4 past this one
                    const int from = key0 + kt * 32 + 4 * hb;
                    const int lo = seen[n].lo - from, hi = seen[n].hi - from;
                    const uint32_t bits = (uint32_t)(there >> (kt * 32)) >> (4 * hb);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int at = 8 * (i / 4) + i % 4;
                        if (at < lo || at >= hi || !(bits & (1u << at))) s[n][i] = kNone;
                    }
                }
                float top = fmaxf(s[n][0], s[n][1]);
#pragma unroll
                for (int i = 2; i < 16; i += 2) top = fmaxf(fmaxf(top, s[n][i]), s[n][i + 1]);
                const uint32_t u = __float_as_uint(top);
                const auto both = __builtin_amdgcn_permlane32_swap(u, u, false, false);
                // (above zero whatever the two are: a masked -infinity stays one)
                const float to_log2 = fmaxf(row_scale[n] * key_scale, 1.17549435e-38f);
                top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * to_log2;
                if (__any(top > m[n] + kSlack)) {
                    const float next = fmaxf(top, m[n]), f = m[n] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m[n] - next);
                    m[n] = next;
                    l[n] *= f;
#pragma unroll
                    for (int d = 0; d < DTILES; ++d) o[n][d] *= f;
                }
                const float base = (m[n] == kNone ? 0.0f : m[n]) - down;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[n][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][i], to_log2, -base));
                    if constexpr (DT == QLIN_BF16) sum += s[n][i];
                }
                if constexpr (DT == QLIN_BF16) l[n] = __builtin_fmaf(sum, back, l[n]);
#pragma unroll
                for (int i = 0; i < 8; ++i) p[n][i / 4][i % 4] = round2<QLIN_F16>(s[n][2 * i], s[n][2 * i + 1]);
                if constexpr (DT == QLIN_F16) {      // of p as it multiplies the values, unless that is nothing
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum = add2<QLIN_F16>(p[n][i / 4][i % 4], sum);
                    if (__builtin_expect(fall < -kFall, 0)) {
                        sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum += s[n][i];
                    }
                    l[n] = __builtin_fmaf(sum, back, l[n]);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int d = 0; d < DTILES; ++d) {
                    const u32x4 va = *(const u32x4*)(vl + (kt * 4 + k * 2) * (D * 16) + d * 512);
#pragma unroll
                    for (int n = 0; n < RT; ++n) o[n][d] = mfma32(va, p[n][k], o[n][d]);
                }
        }
    }

    const int64_t part = ((tile * c.heads + h) * t.splits + split) * R;
#pragma unroll
    for (int n = 0; n < RT; ++n) {
        l[n] += __shfl_xor(l[n], 32, 64);
        const float of = unit == kNoPower ? 1.0f : __builtin_ldexpf(1.0f, unit);
        const int row = first + n * 32 + r;
        if (row >= w.rows) continue;
        if (w.splits <= 1) {
            const float inv = l[n] == 0.0f ? 0.0f : of / l[n];            // a row that sees no key: zeros
            const int rr = w.row0 + row;
            const int64_t to = ((w.s.first + rr / share) * a.q_heads + h * share + rr % share) * D + 4 * hb;
#pragma unroll
            for (int d = 0; d < DTILES; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store4<DT>(a.out, to + d * 32 + i * 8,
                               f32x4{o[n][d][4 * i], o[n][d][4 * i + 1], o[n][d][4 * i + 2], o[n][d][4 * i + 3]} * inv);
        } else {
            if (hb == 0) {
                t.part_ml[(part + row) * 2] = m[n];
                t.part_ml[(part + row) * 2 + 1] = l[n];
            }
#pragma unroll
            for (int d = 0; d < DTILES; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *(f32x4*)(t.part_o + (part + row) * D + 4 * hb + d * 32 + i * 8) =
                        f32x4{o[n][d][4 * i], o[n][d][4 * i + 1], o[n][d][4 * i + 2], o[n][d][4 * i + 3]} * of;
        }
    }
}

template <int D, int RT>
hipError_t launch_prompt_rows(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                              hipStream_t st) {
    constexpr int R = 128 * RT;
    char* const ws = (char*)workspace;
    TileArgs t{a, c, p.chunk, p.splits, (float*)(ws + p.part_at), nullptr, (uint8_t*)ws, (uint64_t*)(ws + p.present_at),
               (float*)(ws + p.present_at) + (int64_t)a.B * p.key_blocks * 2, nullptr, p.key_blocks};
    t.value_power = (int32_t*)t.key_scale + (int64_t)a.B * p.key_blocks * c.heads;
    t.part_ml = t.part_o + p.tiles * c.heads * p.splits * R * D;
    auto run = [&](auto dtc, auto mode) -> hipError_t {
        constexpr int DT = decltype(dtc)::value, M = decltype(mode)::value;
        constexpr bool LO = prompt_halves(DT, M);
        constexpr int BK = prompt_keys(D, RT, LO);
        attend_lay_kernel<DT, M, D, BK><<<(unsigned)((int64_t)a.B * p.key_blocks * c.heads), 256, 0, st>>>(t, (uint8_t*)ws);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        attend_prompt_kernel<DT, D, RT, LO><<<(unsigned)(p.tiles * c.heads * p.splits), 256, 0, st>>>(t, p.tiles);
        e = hipGetLastError();
        if (e != hipSuccess || p.splits == 1) return e;
        return launch_join<DT, D>(t, p.tiles, R, kImageKeys, st);
    };
    auto moded = [&](auto dtc) -> hipError_t {
        if (c.mode == MXFP4) return run(dtc, std::integral_constant<int, MXFP4>{});
        if (c.mode == NVFP4) return run(dtc, std::integral_constant<int, NVFP4>{});
        return run(dtc, std::integral_constant<int, AFFINE>{});
    };
    return dt == QLIN_BF16 ? moded(std::integral_constant<int, QLIN_BF16>{}) : moded(std::integral_constant<int, QLIN_F16>{});
}

template <int D>
hipError_t launch_prompt_of(const AttendArgs& a, const KvPool& c, int dt, const AttendPlan& p, void* workspace,
                            hipStream_t st) {
    if constexpr (D <= 128)
        if (p.rows == 256) return launch_prompt_rows<D, 2>(a, c, dt, p, workspace, st);
    return p.rows == 128 ? launch_prompt_rows<D, 1>(a, c, dt, p, workspace, st) : hipErrorInvalidValue;
}

}  // namespace
}  // namespace qlin
