// attend_tile.h -- attention over the 4-bit cache on the matrix cores, for the
// rows of q that share few keys' reads: decode and drafted tokens. One head
// size a translation unit (attend_64.hip and its neighbours).
//
// A sequence's rows of one key head (n tokens by q_heads / heads query heads)
// form tiles; a workgroup takes a tile and `chunk` keys, its four waves (three
// where D is 256) every fourth step of 32 keys, each with its own running maximum
// m, sum l and o (o = sum of p v, p = exp2(score - m)), joined through LDS at the
// end. Workgroups of other chunks of the same rows leave o, m and l in the
// workspace and attend_join adds them up.
//
// Loads. Codes and scales go from memory straight into a ring of a wave's own in
// LDS, one to three steps ahead, without a barrier: a wave waits for the count of
// its own loads alone. What is ahead costs no registers that way, so that three
// workgroups fit a CU: 64 x 8192 to 32768 keys, D 128, loads into registers 363
// us, through the ring 344, three workgroups 294 (two 310). Not so for affine
// groups of 32 in 32 columns of D 64 and 128: 5 to 28 registers of o, q and the
// scales do not fit (1 to 3 in 16 columns of D 96 and 192), and their reloads wait
// for the ring.
//
// Products, 16 x 16 x 32:
//   scores^T = K q^T. Lane (r = lane % 16, j = lane / 16) of K's operand holds
//     eight codes of key r, a word as it lies in memory; q's operand has its values
//     in the same order. Keys stay codes, and scales join in fp32. Affine codes
//     become 16 + c by a shift and one and-or for two of them (a nibble put at the
//     top of the mantissa of 16), which the bias makes up for: score = s acc +
//     (z - 16 s) sum(q). E2M1 codes are the hardware's conversion; nvfp4's groups
//     of 16 are shorter than the product's 32, so its codes take their scale
//     before, in f16, which holds every product of the two exactly.
//   o^T = V^T p^T. The scores leave the matrix cores as p's operand wants them
//     (lane (q row, j) has keys 4j..4j+3 of both halves of the step), so lane
//     (r, j) of V's operand takes word r of those eight keys: its eight codes are
//     eight rows of V^T. Two ways to make them numbers:
//     - decoded: fl(s c + z) as f16 by packed instructions, two keys each. bf16
//       values are in units of a power of two that follows the largest of a step
//       (a wave's; o is scaled where it moves), up by 2^15, down by 2^6: no value
//       leaves f16's range, and what is small beside the step's largest keeps 2^-19
//       of it (steps within 2^64 of the largest so far). In bf16, p and the
//       values put 0.0015 on outputs that round by 0.0017 themselves; in f16 nothing
//       that shows, in the same time (64 rows, groups of 32: 82 us for 75).
//     - as codes (PS; bf16 affine): p takes the scale and the codes stay 16 + c,
//       2.5 instructions a pair instead of 4 and more. A column of p belongs to a
//       single group then, so a row of q has as many columns as a row has groups
//       (DUP), and 16 columns hold 16 / groups rows. What is left of each value is
//       z + 8 s (summed in fp32) and 8 s too many of 16 + c - 8, taken off at the
//       end as 24 times the sum of the rounded p s, which a product with ones
//       gives: what p s lost by rounding multiplies c - 8, not 16 + c. p s is f16 in
//       units that follow the largest scale of a step, as those of decoded values
//       do: outputs are off by their own rounding, 0.0017, where p s in bf16 made it
//       0.0021 (64 x 8192 to 32768 keys 295 us, in bf16 294; 500 keys 9.7 and 9.4).
//       64 x 5000 to 20000 keys, D 128, groups of 64: 252 us decoded, 228 as codes.
//   Rounded on the way: p s (as codes), p and decoded values to f16; mxfp4's p to the
//   type, its values not at all, nor nvfp4's. Sums, m and l are fp32; l adds up p as
//   it multiplies the values, rounded, so that a row's weights make one (bf16 mxfp4:
//   outputs off by 1.15 times their own rounding where exact p had 1.27).
//
// Scales go through LDS a second time, as numbers (a lane there needs those of
// eight keys); keys that no row of the tile sees (behind its end, before its
// window) get zeros there, whatever their page holds, and the lowest score.
//
// Bound by the memory: D/2 bytes and the scales of a key and of a value, read
// once for the tile's rows. 64 sequences of 8192 to 32768 keys (D 128, 8 heads,
// groups of 64) are 1.48 GB, 295 us with the join: 5.0 TB/s of the 6.2 that a
// plain read reaches; the vector units are busy for three quarters of that time.
#pragma once

#include <type_traits>

#include "attend_common.h"

namespace qlin {
namespace {

constexpr int kStep = 32;                       // keys of a wave's step
constexpr int kWindow = 4096;                   // keys whose pages are looked up at once
constexpr int kScaleRow = kStep + 4;            // floats of a group's scales of a step in LDS: rows on other banks

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == QLIN_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A word's eight E2M1 codes as numbers, in their order.
template <int DT>
__device__ __forceinline__ u32x4 code_operand(uint32_t w) {
    if constexpr (DT == QLIN_BF16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3))};
    else
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3))};
}

// A number twice, and the four pairs of an operand times it.
__device__ __forceinline__ f16x2 both(float s) { return f16x2{(_Float16)s, (_Float16)s}; }
__device__ __forceinline__ u32x4 times(u32x4 a, f16x2 s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = a[i];                          // (a bit cast of the element itself reads the first)
        a[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, pair) * s);
    }
    return a;
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
// Largest of a wave's numbers, in every lane (steps within rows of 16 lanes first).
__device__ __forceinline__ float wave_max(float v) {
    auto with = [&](auto ctrl) {
        v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true)));
    };
    with(std::integral_constant<int, 0xB1>{});               // neighbours, pairs, halves of 8, of 16
    with(std::integral_constant<int, 0x4E>{});
    with(std::integral_constant<int, 0x141>{});
    with(std::integral_constant<int, 0x140>{});
    return across_max(v);
}
__device__ __forceinline__ float across_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// 16 (4) bytes a lane from memory into LDS, 64 lanes one after the other from
// byte `to` on. As statements the compiler would take any later read of LDS for
// a read of what they bring and wait for all of them there; written out, the
// waits are wait_loads'. They have no register to write but M0, which nothing
// else here uses, and the wait state before its use is theirs.
__device__ __forceinline__ uint32_t lds_byte(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}
__device__ __forceinline__ void to_lds16(uint32_t to, const uint8_t* base, uint32_t offset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void to_lds16(uint32_t to, const uint8_t* from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory");
}
__device__ __forceinline__ void to_lds4(uint32_t to, const uint8_t* from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "memory");
}

// s_waitcnt vmcnt(N). Field layout: vmcnt [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8].
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}

// s_waitcnt lgkmcnt(0).
__device__ __forceinline__ void wait_reads() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}

// LDS writes of a wave before its own reads, without a barrier for the others.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Bits that hide a constant's or a number's value from the compiler, which
// else takes masks apart again into more instructions.
__device__ __forceinline__ uint32_t scalar_bits(uint32_t x) {
    asm("" : "+s"(x));
    return x;
}
__device__ __forceinline__ uint32_t vector_bits(uint32_t x) {
    asm("" : "+v"(x));
    return x;
}

// Keeps a rare branch a branch: what follows is not done beforehand.
__device__ __forceinline__ void out_of_line() { asm volatile(""); }

// Nibble I of both halves of w as a pair of 16 + c.
template <int DT, int I>
__device__ __forceinline__ uint32_t sixteen_plus(uint32_t w, uint32_t mask, uint32_t sixteen) {
    constexpr int UP = (DT == QLIN_BF16 ? 3 : 6) - 4 * I;      // from the nibble's place to the highest bits of a mantissa
    if constexpr (UP >= 0) return ((w << UP) & mask) | sixteen;
    else return ((w >> -UP) & mask) | sixteen;
}

// How a kernel's rows are laid out: see the top.
template <int DT, int MODE, int D, int GQ, int NT, bool PS>
struct TileShape {
    static constexpr int G = MODE == NVFP4 ? 16 : 32 * GQ;   // values of a quant group
    static constexpr int NG = D / G;                         // quant groups of a row
    static constexpr int DUP = PS ? NG : 1;                  // columns of a row of q
    static constexpr int PER = 16 / DUP;                     // rows of q in 16 columns
    static constexpr int R = PER * NT;
};

// Waves of a workgroup: two workgroups' rings of loads fit a CU's LDS.
constexpr int tile_waves(int D) { return D == 256 ? 3 : 4; }

// GQ: a quant group's words over 4 (AFFINE 32/64/128: 1/2/4; MXFP4: 1; NVFP4: unused)
// PS: values stay codes, see the top (AFFINE, at most four groups).
template <int DT, int MODE, int D, int GQ, int NT, bool PS>
__global__ void __launch_bounds__(64 * tile_waves(D), tile_residents(D, NT)) attend_tile_kernel(TileArgs t) {
    constexpr int WAVES = tile_waves(D);
    using S = TileShape<DT, MODE, D, GQ, NT, PS>;
    constexpr int HW = D / 8;                              // words of a head's row
    constexpr int NM = D / 32;                             // MFMAs along D for 16 keys
    constexpr int G = S::G, NG = S::NG, R = S::R, PER = S::PER;
    constexpr bool HALF = HW == 8;                         // 8 words for 16 lanes: each takes half of one
    constexpr int VC = (HW + 15) / 16;                     // words of a value a lane takes
    constexpr int CL = HALF ? 4 : 8, OT = VC * CL;         // codes of a word it takes; tiles of o
    constexpr bool AFF = MODE == AFFINE;
    // types of the products' operands: all of nvfp4 fits f16; bf16 values (or p times their scales) are f16 in a power of two
    constexpr int KT = MODE == NVFP4 ? (int)QLIN_F16 : DT;
    constexpr bool UNIT = AFF && DT == QLIN_BF16;
    constexpr int VT = UNIT ? (int)QLIN_F16 : KT;
    static_assert(!PS || (AFF && NG <= 4 && DT == QLIN_BF16), "values as codes");
    constexpr int ARR = AFF ? 4 : 2;                       // scale arrays of a step: keys', values', biases in the same order
    constexpr int WSCALES = ARR * NG * kScaleRow;          // a wave's scales as numbers
    constexpr int CH = D / 32;                             // 16-byte chunks of a head's row
    constexpr int ES = AFF ? 2 : 1;                        // bytes of a scale
    constexpr int U = 16 * NG * ES / 4;                    // dwords of 16 keys' scales
    constexpr int NC = D / 32, NI = (ARR * 2 * U + 63) / 64;     // loads of a step: codes, scales
    constexpr int STAGE = 32 * D + NI * 256;
    // LDS of a workgroup, so that as many fit a CU
    constexpr int ROOM = (tile_residents(D, NT) == 3 ? 52 : 78) * 1024 - WAVES * WSCALES * 4;
    constexpr int ST = WAVES * 4 * STAGE <= ROOM ? 4 : (WAVES * 3 * STAGE <= ROOM ? 3 : 2);
    constexpr int ROW = D + 4;                             // floats of a row of o in LDS, rows on other banks
    constexpr int RING = WAVES * ST * STAGE, SUMS = WAVES * R * ROW * 4, BUF = RING > SUMS ? RING : SUMS;
    static_assert(SUMS <= 72 * 1024, "two workgroups a CU");
    __shared__ int32_t blocks[kWindow / kKvUnit];
    __shared__ __attribute__((aligned(16))) uint8_t ring[BUF];
    __shared__ __attribute__((aligned(16))) float numbers[WAVES * WSCALES];
    __shared__ float wave_ml[WAVES][R][2];

    const AttendArgs& a = t.a;
    const KvPool& c = t.c;
    const int h = blockIdx.y, split = t.splits == 1 ? 0 : blockIdx.x % t.splits;
    const int64_t tile = t.splits == 1 ? blockIdx.x : blockIdx.x / t.splits;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64, r = lane % 16, j = lane / 16;
    const int share = a.q_heads / c.heads;
    TileWork w = tile_of(a, c, tile, R);
    if (!w.rows) return;
    // Ahead of the lengths, which say whether they count: the page of the thread's first row block, known without a
    // window; and the rows of q.
    int32_t guess = -1;
    if (!a.window && a.width) {
        const uint32_t page = ((uint32_t)split * (uint32_t)t.chunk + tid * kKvUnit) / (uint32_t)c.page;
        guess = a.table[(int64_t)w.b * a.width + min(page, (uint32_t)a.width - 1)];
    }
    u32x4 q[NT][NM];
    int at_row[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int rr = min(w.row0 + n * PER + r % PER, w.row0 + w.rows - 1);     // rows past the end repeat the last
        at_row[n] = rr / share;
        const uint16_t* qp = (const uint16_t*)a.q + (w.s.first + at_row[n]) * a.q_stride + (int64_t)(h * share + rr % share) * D;
        const bool aligned = (((uintptr_t)a.q | (uintptr_t)(a.q_stride * 2)) & 15) == 0;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const int word = MODE == NVFP4 ? m * 4 + j : m / GQ * (4 * GQ) + j * GQ + m % GQ;
            if (aligned) {
                q[n][m] = *(const u32x4*)(qp + word * 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) q[n][m][i] = qp[word * 8 + 2 * i] | ((uint32_t)qp[word * 8 + 2 * i + 1] << 16);
            }
        }
    }
    tile_keys(a, c, w, t.chunk, kKvUnit);
    if (split && split >= w.splits) return;
    const KeyRange keys = chunk_of(w, split, t.chunk);
    const int k0 = keys.first, k1 = keys.end;
    const int steps = (k1 - k0 + kStep - 1) / kStep;
    const int32_t* const table = a.table + (int64_t)w.b * a.width;
    auto look_up = [&](int first) {                        // row blocks of the keys of a window
        const int n = min(steps * (kStep / kKvUnit) - first, kWindow / kKvUnit);
        for (int i = tid; i < n; i += 64 * WAVES) {
            const int key = k0 + (first + i) * kKvUnit;
            int32_t p = guess;
            if (a.window || first || i != tid) p = key < k1 ? table[key / c.page] : -1;
            blocks[i] = key < k1 ? kv_row_block(p, c.pages, c.heads, c.page, h, key / kKvUnit) : -1;
        }
    };
    look_up(0);
    // keys that every row of the tile sees
    const int all_lo = seen_by(a, w.s, (w.row0 + w.rows - 1) / share).lo, all_hi = seen_by(a, w.s, w.row0 / share).hi;
    Seen seen[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) seen[n] = seen_by(a, w.s, at_row[n]);

    f32x4 o[NT][OT], ones[NT];
    // p = exp2(score - base), base being m + kUnder, or 0 while there is no m. kUnder keeps sums of bf16's largest values
    // inside fp32; f16, whose values cannot leave it, has no bits to give for that.
    constexpr float kUnder = VT == QLIN_BF16 || PS ? kSlack : 0.0f;
    float m[NT], l[NT], zsum[NT], base[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kNone;
        base[n] = 0.0f;
        l[n] = zsum[n] = 0.0f;
        ones[n] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < OT; ++i) o[n][i] = f32x4{0, 0, 0, 0};
    }
    // UNIT: o and the values (PS: the scales) are in units of 2^unit, which follows the largest of a step: up where that
    // would leave f16 (of the value, of p times the scale), down where little of it would be left
    constexpr int kHead = PS ? 6 : 0, kUp = PS ? 8 : 15, kDown = 6, kReach = 64;     // (p is 2^-kUnder at first)
    float largest = 0.0f, least = -1.0f, to_unit = 1.0f;
    int unit = 0, unit_least = -120;                         // (2^-unit is a number; o stays inside fp32)
    const float scale = a.scale * kLog2e;
    float* const sl = numbers + wave * WSCALES;                          // this wave's scales: [array, group, key]
    constexpr int SE = (kStep * NG + 63) / 64;                           // a lane's numbers of an array
    constexpr int VROW = HW < 16 ? HW : 16;
    const uint32_t mask = scalar_bits(DT == QLIN_BF16 ? 0x00780078u : 0x03C003C0u);
    const uint32_t sixteen = vector_bits(DT == QLIN_BF16 ? 0x41804180u : 0x4C004C00u);
    const uint32_t value_mask = UNIT ? scalar_bits(0x03C003C0u) : mask, value_sixteen = UNIT ? vector_bits(0x4C004C00u) : sixteen;

    // A stage of the ring: the codes of the step's keys and values, [16 keys of them, K or V][row][chunk], then the bytes
    // of their scales. Key 4 y + x lies in row 4 x + y, its chunks by x further round, so that neither K's reads (16
    // keys, one chunk) nor V's (keys 4 j + i, 16 words) meet in a bank.
    uint8_t* const mine = ring + wave * (ST * STAGE);
    auto turn_of = [](int x) { return (CH & (CH - 1)) ? 0 : x & (CH - 1); };
    auto word_at = [&](int st, int side, int key, int word) -> int {
        const int x = key % 4, row = x * 4 + key / 4;
        return (st * 2 + side) * (8 * D) + row * (D / 2) + (((word / 4) ^ turn_of(x)) * 16) + word % 4 * 4;
    };
    // what the lane fetches of each load, past the 16 keys' place in its pool
    uint32_t code_from[NC];
    const uint8_t* scale_from[NI];
    bool scale_second[NI];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int at = (i * 64 + lane) % (D / 2), row = at / CH, x = row / 4, key = row % 4 * 4 + x;
        code_from[i] = key * (D / 2) + ((at % CH) ^ turn_of(x)) * 16;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int at = min(i * 64 + lane, ARR * 2 * U - 1), s = at / U % ARR;
        const void* p = c.scales[0];
#pragma unroll
        for (int e = 1; e < ARR; ++e)
            if (s == e) p = e < 2 ? c.scales[e] : c.biases[e - 2];
        scale_from[i] = (const uint8_t*)p + at % U * 4;
        scale_second[i] = at / U >= ARR;
    }
    auto fetch = [&](int at, int stage) {                    // step `at` of the window
        int32_t b[2];
#pragma unroll
        for (int st = 0; st < 2; ++st) b[st] = max(__builtin_amdgcn_readfirstlane(blocks[at * 2 + st]), 0);
        const uint32_t to = lds_byte(mine) + stage * STAGE;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if constexpr (D == 128) {                        // a load is 16 keys' rows of one side
                to_lds16(to + i * 1024, (const uint8_t*)c.codes[i % 2] + (int64_t)b[i / 2] * (8 * D), code_from[i]);
            } else {
                const int part = (i * 64 + lane) / (D / 2);
                const uint8_t* const k = (const uint8_t*)c.codes[part % 2];
                to_lds16(to + i * 1024, k + (int64_t)(part / 2 ? b[1] : b[0]) * (8 * D) + code_from[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
            to_lds4(to + 32 * D + i * 256, scale_from[i] + (int64_t)(scale_second[i] ? b[1] : b[0]) * (U * 4));
    };

    // ST - 1 steps of a window on their way; past its end the last one again, so that the counts of loads stay the same
    auto begin = [&](int n_steps) {
        if (wave < n_steps) {
#pragma unroll
            for (int i = 0; i < ST - 1; ++i) fetch(min(wave + i * WAVES, n_steps - 1), i);
        }
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)                             // q has come: no later wait for it is one for those loads
#pragma unroll
        for (int m = 0; m < NM; ++m) asm volatile("" : "+v"(q[n][m]));
    __syncthreads();
    begin(min(steps, kWindow / kStep));

    float qsum[NT][AFF ? NG : 1];
    if constexpr (AFF) {                                     // q's values 0..7 to the order of the codes: 0 4 1 5 2 6 3 7; sums
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float sum = 0.0f;
#pragma unroll
                for (int m = 0; m < GQ; ++m) {
                    const u32x4 v = q[n][g * GQ + m];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sum += DT == QLIN_BF16 ? __uint_as_float(v[i] << 16) : f16_bits_to_f32(v[i] & 0xFFFFu);
                        sum += DT == QLIN_BF16 ? __uint_as_float(v[i] & 0xFFFF0000u) : f16_bits_to_f32(v[i] >> 16);
                    }
                    q[n][g * GQ + m] = u32x4{(v[0] & 0xFFFFu) | (v[2] << 16), (v[0] >> 16) | (v[2] & 0xFFFF0000u),
                                             (v[1] & 0xFFFFu) | (v[3] << 16), (v[1] >> 16) | (v[3] & 0xFFFF0000u)};
                }
                qsum[n][g] = across_sum(sum);
            }
    }

    float scale_of[NT];                                      // of scores of these operands
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        scale_of[n] = scale;
        if constexpr (MODE == NVFP4 && DT == QLIN_BF16) {    // a row as f16 in a power of two of its largest value,
            // which holds all but what is below 2^-17 of that, and that to 2^-25 of it
            uint32_t most = 0;
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = max(most, max(q[n][m][i] & 0x7FFFu, q[n][m][i] >> 16 & 0x7FFFu));
            most = max(most, (uint32_t)__shfl_xor((int)most, 16, 64));
            most = max(most, (uint32_t)__shfl_xor((int)most, 32, 64));
            const int e = most ? ilogb_of(bf16_bits_to_f32(most)) : 0;
            scale_of[n] = __builtin_ldexpf(scale, e);
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[n][m][i] = round2<QLIN_F16>(__builtin_ldexpf(bf16_bits_to_f32(q[n][m][i] & 0xFFFFu), -e),
                                                  __builtin_ldexpf(bf16_bits_to_f32(q[n][m][i] >> 16), -e));
        }
    }

    for (int first = 0; first < steps; first += kWindow / kStep) {
        const int n_steps = min(steps - first, kWindow / kStep);
        if (first) {                                         // another window: its row blocks take the place of the last ones
            __syncthreads();
            look_up(first * (kStep / kKvUnit));
            __syncthreads();
            begin(n_steps);
        }
        auto run = [&](int step, auto stage_c) {
            constexpr int stage = decltype(stage_c)::value;
            const int key0 = k0 + (first + step) * kStep;
            const int32_t rb[2] = {__builtin_amdgcn_readfirstlane(blocks[step * 2]), __builtin_amdgcn_readfirstlane(blocks[step * 2 + 1])};
            fetch(min(step + (ST - 1) * WAVES, n_steps - 1), (stage + ST - 1) % ST);
            // every row sees all the step's keys, and they are there
            const bool whole = key0 >= all_lo && key0 + kStep <= all_hi && (rb[0] | rb[1]) >= 0;
            wait_loads<(ST - 1) * (NC + NI)>();              // this step's have landed
            const uint8_t* const in = mine + stage * STAGE;
            // the scales as numbers where the lanes find those of their keys; the keys' take the softmax's scale along,
            // and their biases what 16 + c has too much
            float x[SE][ARR];
#pragma unroll
            for (int e = 0; e < SE; ++e) {
                const int at = lane + 64 * e, key = min(at / NG, kStep - 1), g = at % NG, st = key / kKvUnit;
                const uint8_t* const raw = in + 32 * D + st * (ARR * U * 4) + (key % kKvUnit * NG + g) * ES;
#pragma unroll
                for (int s = 0; s < ARR; ++s) x[e][s] = scale_at<MODE, DT>(raw + s * (U * 4), 0);
                if (MODE != NVFP4) x[e][0] *= scale;
                if (AFF) x[e][ARR - 2] = __builtin_fmaf(x[e][0], -16.0f, x[e][ARR - 2] * scale);
                if (PS) x[e][ARR - 1] = __builtin_fmaf(x[e][1], 8.0f, x[e][ARR - 1]);
                if (!whole) {                                // what is not there is no number
                    out_of_line();
                    const bool live = (st ? rb[1] : rb[0]) >= 0 && key0 + key >= w.lo && key0 + key < k1;
#pragma unroll
                    for (int s = 0; s < ARR; ++s) x[e][s] = live ? x[e][s] : 0.0f;
                }
            }
            if constexpr (UNIT) {
                float most = 0.0f;
#pragma unroll
                for (int e = 0; e < SE; ++e)
                    most = fmaxf(most, PS ? fabsf(x[e][1]) : __builtin_fmaf(fabsf(x[e][1]), 15.0f, fabsf(x[e][3])));
                if (__any(most > largest) || !__any(most > least)) {
                    out_of_line();
                    most = wave_max(most);
                    const int of = __builtin_amdgcn_readfirstlane(ilogb_of(most)), to = max(of - kHead, unit_least);
                    if (__any(most > 0.0f) && (largest == 0.0f || to != unit)) {
                        const float f = largest == 0.0f ? 1.0f : __builtin_ldexpf(1.0f, unit - to);
                        unit = to;
                        unit_least = max(unit_least, to - kReach);
                        to_unit = __builtin_ldexpf(1.0f, -to);
                        largest = __builtin_ldexpf(1.0f, to + kHead + kUp);
                        least = to == unit_least ? -1.0f : __builtin_ldexpf(1.0f, to + kHead - kDown);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if constexpr (PS) ones[n] *= f;
#pragma unroll
                            for (int i = 0; i < OT; ++i) o[n][i] *= f;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < SE; ++e) {
                    x[e][1] *= to_unit;
                    if constexpr (!PS) x[e][3] *= to_unit;
                }
            }
#pragma unroll
            for (int e = 0; e < SE; ++e) {
                const int at = lane + 64 * e, key = min(at / NG, kStep - 1), g = at % NG;
                if (kStep * NG % 64 == 0 || at < kStep * NG)
#pragma unroll
                    for (int s = 0; s < ARR; ++s) sl[(s * NG + g) * kScaleRow + key] = x[e][s];
            }
            wave_fence();
            uint32_t vw[8][VC];
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    const int word = HALF ? r / 2 : v * 16 + r;
                    vw[e][v] = *(const uint32_t*)(in + word_at(e / 4, 1, 4 * j + e % 4, word < HW ? word : word - VROW));
                }
            f32x4 sc[NT][2];
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                if constexpr (MODE == NVFP4) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) sc[n][st] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < NM; ++i) {
                        // the word's group is not its MFMA's only one: its codes take their scale here, exact in f16
                        const f16x2 s = both(sl[(2 * i + j / 2) * kScaleRow + st * 16 + r]);
                        const u32x4 k = times(code_operand<QLIN_F16>(*(const uint32_t*)(in + word_at(st, 0, r, i * 4 + j))), s);
#pragma unroll
                        for (int n = 0; n < NT; ++n) sc[n][st] = mfma16<KT>(k, q[n][i], sc[n][st]);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const f32x4 s = *(const f32x4*)(sl + g * kScaleRow + st * 16 + 4 * j);
                        f32x4 z{0, 0, 0, 0};
                        if constexpr (AFF) z = *(const f32x4*)(sl + (2 * NG + g) * kScaleRow + st * 16 + 4 * j);
                        uint32_t kw[GQ];
                        const uint8_t* const kp = in + word_at(st, 0, r, g * (4 * GQ) + j * GQ);
                        if constexpr (GQ == 4) {
                            const uint4 x = *(const uint4*)kp;
                            kw[0] = x.x; kw[1] = x.y; kw[2] = x.z; kw[3] = x.w;
                        } else if constexpr (GQ == 2) {
                            const uint2 x = *(const uint2*)kp;
                            kw[0] = x.x; kw[1] = x.y;
                        } else {
                            kw[0] = *(const uint32_t*)kp;
                        }
                        u32x4 k[GQ];
#pragma unroll
                        for (int i = 0; i < GQ; ++i) {
                            const uint32_t x = kw[i];
                            if constexpr (AFF)
                                k[i] = u32x4{sixteen_plus<DT, 0>(x, mask, sixteen), sixteen_plus<DT, 1>(x, mask, sixteen),
                                             sixteen_plus<DT, 2>(x, mask, sixteen), sixteen_plus<DT, 3>(x, mask, sixteen)};
                            else k[i] = code_operand<DT>(x);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            f32x4 acc{0, 0, 0, 0};
#pragma unroll
                            for (int i = 0; i < GQ; ++i) acc = mfma16<DT>(k[i], q[n][g * GQ + i], acc);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float x = g ? sc[n][st][i] : -base[n];
                                if constexpr (AFF) x = __builtin_fmaf(z[i], qsum[n][g], x);
                                sc[n][st][i] = __builtin_fmaf(s[i], acc[i], x);
                            }
                        }
                    }
                }
            }
            u32x4 p[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = MODE == NVFP4 ? __builtin_fmaf(sc[n][e / 4][e % 4], scale_of[n], -base[n]) : sc[n][e / 4][e % 4];
                if (!whole) {
                    out_of_line();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int key = key0 + e / 4 * 16 + 4 * j + e % 4;
                        if (key < seen[n].lo || key >= seen[n].hi || rb[e / 4] < 0) x[e] = kNone;
                    }
                }
                float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
                top = across_max(top);
                // the maximum follows where a score passes it by 2^8, or the first number comes
                if (__any(top > (m[n] == kNone ? kNone : kSlack - kUnder))) {
                    out_of_line();
                    const float to = fmaxf(top + base[n], m[n]), f = m[n] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m[n] - to);
                    const float more = to == kNone ? 0.0f : to + kUnder - base[n];
                    m[n] = to;
                    base[n] += more;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] -= more;
                    l[n] *= f;
                    if constexpr (PS) {
                        zsum[n] *= f;
                        ones[n] *= f;
                    }
#pragma unroll
                    for (int i = 0; i < OT; ++i) o[n][i] *= f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = __builtin_amdgcn_exp2f(x[e]);
                    if constexpr (PS) l[n] += x[e];
                }
                if constexpr (PS) {                          // p times the scales of the column's group; the biases' part
                    const int group = min(r / PER, NG - 1);
                    const float* const vs = sl + (NG + group) * kScaleRow + 4 * j;
                    const float* const vz = sl + (3 * NG + group) * kScaleRow + 4 * j;
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const f32x4 s = *(const f32x4*)(vs + 16 * st), z = *(const f32x4*)(vz + 16 * st);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            zsum[n] = __builtin_fmaf(x[4 * st + i], z[i], zsum[n]);
                            x[4 * st + i] *= s[i];
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[n][i] = round2<VT>(x[2 * i], x[2 * i + 1]);
                    if constexpr (!PS) l[n] = add2<VT>(p[n][i], l[n]);     // as it multiplies the values: see the top
                }
                if constexpr (PS) ones[n] = mfma16<VT>(u32x4{0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u}, p[n], ones[n]);
            }
            // values: word v*16 + r of the lane's eight keys
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                if constexpr (PS) {
                    auto four = [&](uint32_t halves, int to) {       // the low or high halves: four codes of each key
                        u32x4 x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = __builtin_amdgcn_perm(vw[2 * e + 1][v], vw[2 * e][v], halves);
                        auto one = [&](auto ic) {
                            constexpr int I = decltype(ic)::value;
                            const u32x4 vt{sixteen_plus<VT, I>(x[0], value_mask, value_sixteen), sixteen_plus<VT, I>(x[1], value_mask, value_sixteen),
                                           sixteen_plus<VT, I>(x[2], value_mask, value_sixteen), sixteen_plus<VT, I>(x[3], value_mask, value_sixteen)};
#pragma unroll
                            for (int n = 0; n < NT; ++n) o[n][v * CL + to + I] = mfma16<VT>(vt, p[n], o[n][v * CL + to + I]);
                        };
                        one(std::integral_constant<int, 0>{});
                        one(std::integral_constant<int, 1>{});
                        one(std::integral_constant<int, 2>{});
                        one(std::integral_constant<int, 3>{});
                    };
                    if constexpr (HALF) {
                        four(r & 1 ? 0x07060302u : 0x05040100u, 0);
                    } else {
                        four(0x05040100u, 0);
                        four(0x07060302u, 4);
                    }
                } else {
                    const int word = HALF ? r / 2 : v * 16 + r, g = (word < HW ? word : word - VROW) / (G / 8);
                    const f32x4 s0 = *(const f32x4*)(sl + (NG + g) * kScaleRow + 4 * j);
                    const f32x4 s1 = *(const f32x4*)(sl + (NG + g) * kScaleRow + 16 + 4 * j);
                    if constexpr (AFF) {
                        const f32x4 z0 = *(const f32x4*)(sl + (3 * NG + g) * kScaleRow + 4 * j);
                        const f32x4 z1 = *(const f32x4*)(sl + (3 * NG + g) * kScaleRow + 16 + 4 * j);
                        // fl(s c + z) by packed instructions, two keys each
                        f16x2 s2[4], z2[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s2[e] = __builtin_convertvector((e < 2 ? f32x2{s0[2 * e], s0[2 * e + 1]} : f32x2{s1[2 * e - 4], s1[2 * e - 3]}), f16x2);
                            z2[e] = __builtin_convertvector((e < 2 ? f32x2{z0[2 * e], z0[2 * e + 1]} : f32x2{z1[2 * e - 4], z1[2 * e - 3]}), f16x2);
                        }
                        auto four = [&](uint32_t halves, int to) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] = __builtin_amdgcn_perm(vw[2 * e + 1][v], vw[2 * e][v], halves);
                            auto one = [&](auto ic) {
                                constexpr int I = decltype(ic)::value;
                                u32x4 vt;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const f16x2 c2 = __builtin_bit_cast(f16x2, sixteen_plus<QLIN_F16, I>(x[e], value_mask, value_sixteen)) - (f16x2){16, 16};
                                    vt[e] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c2, s2[e], z2[e]));
                                }
#pragma unroll
                                for (int n = 0; n < NT; ++n) o[n][v * CL + to + I] = mfma16<VT>(vt, p[n], o[n][v * CL + to + I]);
                            };
                            one(std::integral_constant<int, 0>{});
                            one(std::integral_constant<int, 1>{});
                            one(std::integral_constant<int, 2>{});
                            one(std::integral_constant<int, 3>{});
                        };
                        if constexpr (HALF) {
                            four(r & 1 ? 0x07060302u : 0x05040100u, 0);
                        } else {
                            four(0x05040100u, 0);
                            four(0x07060302u, 4);
                        }
                    } else if constexpr (MODE == NVFP4) {     // exact in f16; pairs of values to pairs of keys
#pragma unroll
                        for (int half = 0; half < CL / 4; ++half) {
                            u32x4 vt[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t pair[2][2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int key = 2 * e + k;
                                    const uint32_t w4 = HALF ? vw[key][v] >> (16 * (r & 1)) : vw[key][v] >> (16 * half);
                                    const f16x2 s = both(key < 4 ? s0[key & 3] : s1[key & 3]);
                                    pair[k][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w4, 1.0f, 0) * s);
                                    pair[k][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w4, 1.0f, 1) * s);
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    vt[i][e] = __builtin_amdgcn_perm(pair[1][i / 2], pair[0][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    o[n][v * CL + half * 4 + i] = mfma16<VT>(vt[i], p[n], o[n][v * CL + half * 4 + i]);
                        }
                    } else {
                        float x[8][8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            e2m1_values<true>(HALF ? vw[e][v] >> (16 * (r & 1)) : vw[e][v], e < 4 ? s0[e & 3] : s1[e & 3], x[e]);
#pragma unroll
                        for (int i = 0; i < CL; ++i) {
                            const u32x4 vt{round2<DT>(x[0][i], x[1][i]), round2<DT>(x[2][i], x[3][i]),
                                           round2<DT>(x[4][i], x[5][i]), round2<DT>(x[6][i], x[7][i])};
#pragma unroll
                            for (int n = 0; n < NT; ++n) o[n][v * CL + i] = mfma16<DT>(vt, p[n], o[n][v * CL + i]);
                        }
                    }
                }
            }
            wait_reads();                                    // this stage is read before another takes its place
        };
        for (int step = wave; step < n_steps; step += ST * WAVES) {
            run(step, std::integral_constant<int, 0>{});
            if (step + WAVES >= n_steps) break;
            run(step + WAVES, std::integral_constant<int, 1>{});
            if constexpr (ST > 2) {
                if (step + 2 * WAVES >= n_steps) break;
                run(step + 2 * WAVES, std::integral_constant<int, 2>{});
            }
            if constexpr (ST > 3) {
                if (step + 3 * WAVES >= n_steps) break;
                run(step + 3 * WAVES, std::integral_constant<int, 3>{});
            }
        }
        wait_loads<0>();                                     // the loads past the end have landed, too
    }

    // the waves' sums: a common maximum, then o added up in the order of the waves
    float* const buf = (float*)ring;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        l[n] = across_sum(l[n]);
        if constexpr (PS) zsum[n] = across_sum(zsum[n]);
        if (j == 0 && r < PER) {
            wave_ml[wave][n * PER + r][0] = m[n];
            wave_ml[wave][n * PER + r][1] = l[n];
        }
    }
    __syncthreads();                                         // (the ring is read)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float too_much = PS ? 24.0f * ones[n][0] : 0.0f;            // all rows of `ones` are the column's sum
        const float one = UNIT ? __builtin_ldexpf(1.0f, unit) : 1.0f;
#pragma unroll
        for (int i = 0; i < OT; ++i) o[n][i] = PS ? (o[n][i] - too_much) * one + zsum[n] : (UNIT ? o[n][i] * one : o[n][i]);
        if (n * PER + r % PER >= w.rows) continue;
#pragma unroll
        for (int v = 0; v < VC; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int word = v * 16 + 4 * j + i;           // HALF: half-word
                if (word >= D / CL || (PS && word * CL / G != r / PER)) continue;
                f32x4* const at = (f32x4*)(buf + (wave * R + n * PER + r % PER) * ROW + word * CL);
#pragma unroll
                for (int u = 0; u < CL / 4; ++u)
                    at[u] = f32x4{o[n][v * CL + 4 * u][i], o[n][v * CL + 4 * u + 1][i], o[n][v * CL + 4 * u + 2][i],
                                  o[n][v * CL + 4 * u + 3][i]};
            }
    }
    __syncthreads();
    const int64_t part = (tile * c.heads + h) * t.splits + split;
    for (int e = tid; e < w.rows * (D / 4); e += 64 * WAVES) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        float top = kNone, sum = 0.0f, f[WAVES];
#pragma unroll
        for (int i = 0; i < WAVES; ++i) top = fmaxf(top, wave_ml[i][row][0]);
        f32x4 x{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            f[i] = wave_ml[i][row][0] == kNone ? 0.0f : __builtin_amdgcn_exp2f(wave_ml[i][row][0] - top);
            sum = __builtin_fmaf(f[i], wave_ml[i][row][1], sum);
        }
#pragma unroll
        for (int i = 0; i < WAVES; ++i) x += *(const f32x4*)(buf + (i * R + row) * ROW + d) * f[i];
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
    TileArgs t{a, c, p.chunk, p.splits, (float*)workspace, nullptr, nullptr, nullptr, nullptr, nullptr, 0};
    t.part_ml = t.part_o + p.tiles * c.heads * p.splits * p.rows * D;
    const dim3 grid((unsigned)(p.tiles * p.splits), (unsigned)c.heads);
    auto run = [&](auto dtc, auto mode, auto gq) -> hipError_t {
        constexpr int DT = decltype(dtc)::value, M = decltype(mode)::value, GQ = decltype(gq)::value;
        if constexpr (M == AFFINE && D % (32 * GQ) != 0) {
            return hipErrorInvalidValue;
        } else {
            constexpr int GROUPS = D / (32 * GQ);
            constexpr bool CAN = M == AFFINE && DT == QLIN_BF16 && (GROUPS <= 3 || (GROUPS == 4 && D == 256));   // as the plan has it
            auto go = [&](auto ntc, auto psc) {
                attend_tile_kernel<DT, M, D, GQ, decltype(ntc)::value, decltype(psc)::value><<<grid, 64 * tile_waves(D), 0, st>>>(t);
            };
            constexpr bool ALL = CAN && D == 32 * GQ;               // a single group: codes for any number of rows
            auto sized = [&](auto ntc) -> hipError_t {
                constexpr int NT = decltype(ntc)::value;
                constexpr bool PS = NT == 1 ? CAN : ALL;
                if (p.codes && !PS) return hipErrorInvalidValue;
                if (PS && p.codes) go(ntc, std::integral_constant<bool, PS>{});
                else if constexpr (!ALL) go(ntc, std::false_type{});
                else return hipErrorInvalidValue;
                return hipGetLastError();
            };
            hipError_t e;
            if (p.nt == 1) e = sized(std::integral_constant<int, 1>{});
            else if constexpr (D <= 128) {
                e = p.nt == 2 ? sized(std::integral_constant<int, 2>{}) : hipErrorInvalidValue;
            } else e = hipErrorInvalidValue;
            if (e != hipSuccess || p.splits == 1) return e;
            return launch_join<DT, D>(t, p.tiles, p.rows, kKvUnit, st);
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
