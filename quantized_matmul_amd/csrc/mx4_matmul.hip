// mx4_matmul.hip -- product of two mxfp4 operands on the CDNA4 scaled MFMA,
// dense or by experts.
//
//   y[m][n] = sum over blocks b of 32 along K of
//             2^(ex[m][b] + ew[n][b]) * sum_k cx[m][k] cw[n][k]
//
// with E2M1 codes c and E8M0 exponents e: the scaled MFMA's own input format,
// so no operand is ever decoded. Accumulation is fp32; y is rounded once.
//
// Operand layout of the 4-bit instructions (checked on the device with a
// one-wave probe against a host model): a lane holds 32 consecutive codes of
// one row (column) -- one block -- in 16 bytes, and the scale byte of that
// block is the byte op_sel names of its scale register. 32x32x64: row lane % 32,
// block lane / 32; 16x16x128: row lane % 16, block lane / 16. Since every lane
// brings its own block and scale, the blocks an instruction multiplies need not
// be neighbours along K: lane piece q takes blocks 4q .. 4q + 3 of a run in
// four instructions, so its codes are 64 contiguous bytes, its scales one
// dword, and op_sel alone steps through them.
//
// Two kernels:
//  * streaming (few rows): bound by reading W once. 16 NT weight rows per
//    workgroup, K split over its waves, both operands straight from memory
//    into the instruction's registers, partial sums joined through LDS.
//  * tiled (many rows): bound by the matrix cores and LDS. See mx4_tiled_kernel.

#include "mx4_plan.h"

#include <atomic>
#include <cstdlib>
#include <type_traits>

namespace qlin {
namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

constexpr uint32_t ONES = 0x7F7F7F7Fu;   // four scale bytes of 2^0

__device__ __forceinline__ i32x8 frag(u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

template <int S>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(a), frag(b), c, 4, 4, S, (int)sa, S, (int)sb);
}
template <int S>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(a), frag(b), c, 4, 4, S, (int)sa, S, (int)sb);
}

// Four scale bytes at any alignment; bytes past `left` read as 2^0 (their codes are zero).
__device__ __forceinline__ uint32_t scale4(const uint8_t* p, int left) {
    uint32_t v = ONES;
    if (left >= 4) {
        __builtin_memcpy(&v, p, 4);
    } else {
        for (int b = 0; b < left; ++b) v = (v & ~(0xFFu << (8 * b))) | ((uint32_t)p[b] << (8 * b));
    }
    return v;
}

// Four consecutive outputs at element i (a multiple of 4, y aligned to four of them).
template <int YDT>
__device__ __forceinline__ void store4(void* y, int64_t i, float a, float b, float c, float d) {
    if constexpr (YDT == QLIN_F32) {
        *(float4*)((float*)y + i) = float4{a, b, c, d};
    } else if constexpr (YDT == QLIN_BF16) {
        typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
        *(uint2*)((uint16_t*)y + i) = __builtin_bit_cast(uint2, bf16x4{(__bf16)a, (__bf16)b, (__bf16)c, (__bf16)d});
    } else {
        typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
        *(uint2*)((uint16_t*)y + i) =
            __builtin_bit_cast(uint2, f16x4{(_Float16)a, (_Float16)b, (_Float16)c, (_Float16)d});
    }
}

// ------------------------------------------------------------- streaming

enum Rows : int { DENSE = 0, DIRECT = 1, PLAN = 2 };

struct StreamArgs {
    Mx4Args a;
    Mx4Plan plan;
    uint32_t per_entry;    // index rows per row of x
    int tile_n;            // blocks along N
};

// Where the tile's local row m comes from and goes to; false past the tile.
struct RowMap {
    int64_t src, dst;
    bool ok;
};

template <int NT, int MT, int YDT, int ROWS>
__global__ void __launch_bounds__(512) mx4_stream_kernel(StreamArgs s) {
    extern __shared__ float red[];                 // [waves][16 MT][16 NT]
    const Mx4Args& a = s.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    const int i = lane & 15, q = lane >> 4;
    const uint32_t tile = blockIdx.x / (uint32_t)s.tile_n;
    const int64_t n0 = (int64_t)(blockIdx.x - tile * (uint32_t)s.tile_n) * (16 * NT);
    int64_t first = 0, rows = 0;                   // places of the tile's rows
    uint32_t expert = 0;
    bool zero = false;
    if constexpr (ROWS == DENSE) {
        first = (int64_t)tile * (16 * MT);
        rows = a.M - first;
    } else if constexpr (ROWS == DIRECT) {
        first = tile;
        rows = 1;
        expert = (uint32_t)a.experts[tile];
        zero = expert >= (uint32_t)a.E;
    } else {
        if (tile >= s.plan.first_tile[a.E + 1]) return;
        expert = s.plan.tile_group[tile];
        zero = expert == (uint32_t)a.E;
        first = (int64_t)s.plan.offsets[expert] + (int64_t)(tile - s.plan.first_tile[expert]) * (16 * MT);
        rows = (int64_t)s.plan.offsets[expert + 1] - first;
    }
    auto map = [&](int m) {
        RowMap r{0, 0, m < rows};
        if (!r.ok) return r;
        if constexpr (ROWS == PLAN) {
            const uint32_t row = s.plan.perm[first + m];
            r.dst = row;
            r.src = row / s.per_entry;
        } else {
            r.dst = first + m;
            r.src = ROWS == DIRECT ? (int64_t)((uint32_t)first / s.per_entry) : first + m;
        }
        return r;
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (!zero) {
        const int KB = (int)(a.K / 32);            // blocks per row
        const int64_t half = a.K / 2;
        const uint8_t *wp[NT], *wsp[NT], *xp[MT], *xsp[MT];
        bool xok[MT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            int64_t n = n0 + 16 * t + i;
            n = n < a.N ? n : a.N - 1;             // rows past N are computed and not stored
            wp[t] = a.wq + ((int64_t)expert * a.N + n) * half + 64 * q;
            wsp[t] = a.ws + ((int64_t)expert * a.N + n) * a.wsstride + 4 * q;
        }
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const RowMap r = map(16 * u + i);
            xok[u] = r.ok;
            xp[u] = a.xq + r.src * half + 64 * q;
            xsp[u] = a.xs + r.src * a.xsstride + 4 * q;
        }
        const int runs = (KB + 15) / 16;           // runs of 16 blocks: 4 per lane piece
        for (int run = wave; run < runs; run += waves) {
            const int left = KB - run * 16 - 4 * q;          // blocks of this lane piece
            u32x4 w[NT][4], x[MT][4];
            uint32_t sw[NT], sx[MT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                sw[t] = scale4(wsp[t] + run * 16, left);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    w[t][c] = c < left ? *(const u32x4*)(wp[t] + (int64_t)run * 256 + 16 * c) : u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                const int l = xok[u] ? left : 0;
                sx[u] = scale4(xsp[u] + run * 16, l);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    x[u][c] = c < l ? *(const u32x4*)(xp[u] + (int64_t)run * 256 + 16 * c) : u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < MT; ++u) {
                    acc[t][u] = mfma16<0>(w[t][0], x[u][0], acc[t][u], sw[t], sx[u]);
                    acc[t][u] = mfma16<1>(w[t][1], x[u][1], acc[t][u], sw[t], sx[u]);
                    acc[t][u] = mfma16<2>(w[t][2], x[u][2], acc[t][u], sw[t], sx[u]);
                    acc[t][u] = mfma16<3>(w[t][3], x[u][3], acc[t][u], sw[t], sx[u]);
                }
        }
    }
    // D[n][m]: n = 4 q + r, m = i
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
            *(f32x4*)(red + ((wave * MT + u) * 16 + i) * (16 * NT) + 16 * t + 4 * q) = acc[t][u];
    __syncthreads();
    for (int o = tid; o < 256 * NT * MT; o += blockDim.x) {
        const int m = o / (16 * NT), n = o - m * (16 * NT);
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += red[w * (256 * NT * MT) + o];
        const RowMap r = map(m);
        if (r.ok && n0 + n < a.N) store_f<YDT>(a.y, r.dst * a.N + n0 + n, v);
    }
}

// ------------------------------------------------------------------ tiled

struct TiledArgs {
    Mx4Args a;
    Mx4Plan plan;
    uint32_t per_entry;
    int tiles_n;
    int xcds;
    int lds_nan;
    int wide;          // outputs can be stored 16 bytes at a time
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// 16-byte chunk c of row r sits in slot c ^ swz(r) of its LDS row of 128 or 64
// bytes: any 8 neighbouring rows then keep a chunk in 8 different 16-byte
// columns of the 128-byte bank line.
template <int BKB>
__device__ __forceinline__ int swz(int r) {
    return BKB == 128 ? (r & 7) ^ ((r >> 3) & 1) : (r >> 1) & 3;
}

// s_waitcnt vmcnt(N) lgkmcnt(0). Field layout: vmcnt [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8].
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
}

// Contiguous run of ids for each XCD (ids are dealt to the XCDs round-robin); a bijection on [0, n).
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n, uint32_t xcds) {
    const uint32_t x = b % xcds, per = n / xcds, more = n % xcds;
    return x * per + (x < more ? x : more) + b / xcds;
}

#ifndef SPREAD
#define SPREAD 1
#endif
constexpr uint32_t NOWHERE = 0x80000000u;   // past every buffer range: reads zeros

// Tile of BN weight rows (n) by BM activation rows (m), WN x WM waves of
// TN x TM 32x32 accumulators, K in steps of BKB bytes (2 BKB codes) a row:
//  * code rows go global -> LDS by buffer -> LDS loads, ST - 1 steps ahead
//    through a ring of ST stages; one wave instruction moves 1 KB of whole row
//    pieces, swizzled so that a fragment read meets no bank conflict;
//  * scale rows go the same way, 16 bytes (SG steps) at a time, issued with
//    the codes of the step that first needs them;
//  * a step is KH instructions deep along K; the fragments of the next one
//    are read while the current one multiplies;
//  * the outputs go through LDS, so that they leave in whole lines.
// Rows past the tile and chunks past K read zeros (buffer range checks).
template <int BN, int BM, int WN, int WM, int ST, int BKB>
struct Shape {
    static constexpr int NW = WN * WM, TN = BN / WN / 32, TM = BM / WM / 32;
    static constexpr int CH = BKB / 16, KH = CH / 2;               // chunks of a row and step; instructions along K
    static constexpr int WSTAGE = BN * BKB, STAGE = (BN + BM) * BKB;
    static constexpr int RPL = 1024 / BKB;                         // rows one load moves
    static constexpr int ND = (BN + BM) / RPL / NW;                // code loads per wave and step
    static constexpr int NSI = (BN + BM) / 64;                     // scale loads per batch
    static constexpr int NS = (NSI + NW - 1) / NW;                 // ... per wave
    static constexpr int SG = 256 / BKB;                           // steps per batch of 16 scale bytes
    static constexpr int LA = ST - 1;                              // steps ahead
    static constexpr int SST = (LA + SG - 1) / SG + 1;             // scale stages
    static constexpr int SSTAGE = (BN + BM) * 16;
    static constexpr int LOOP = ST * STAGE + SST * SSTAGE;         // LDS of the loop
    // LDS of the outputs: per wave 32 rows of TN 32 values, rows 16 bytes longer against conflicts
    static constexpr int orow(int size) { return TN * 32 * size + 16; }
    static constexpr int lds(int size) { return LOOP > NW * 32 * orow(size) ? LOOP : NW * 32 * orow(size); }
    static_assert((BN / RPL) % NW == 0 && (BM / RPL) % NW == 0, "whole loads per wave");
    // loads issued after those of a step of phase ph (its number mod SG) when it starts: the LA - 1
    // steps after it, of which those that open a batch brought its scales
    static constexpr int after(int ph) {
        int n = 0;
        for (int u = 1; u < LA; ++u) n += ND + ((ph + u) % SG == 0 ? NS : 0);
        return n;
    }
};

template <int BN, int BM, int WN, int WM, int ST, int BKB, int YDT, bool GATHER>
__global__ void __launch_bounds__(64 * WN * WM) mx4_tiled_kernel(TiledArgs p) {
    using S = Shape<BN, BM, WN, WM, ST, BKB>;
    constexpr int NW = S::NW, TN = S::TN, TM = S::TM;
    constexpr int YS = YDT == QLIN_F32 ? 4 : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char* const slds = smem + ST * S::STAGE;
    const Mx4Args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wv / WM, wm = wv % WM;
    const int i = lane & 31, j = lane >> 5;

    int64_t m0, rows;
    int n0;
    uint32_t expert = 0;
    if constexpr (GATHER) {
        const uint32_t total = p.plan.first_tile[a.E + 1] * (uint32_t)p.tiles_n;
        if (blockIdx.x >= total) return;
        const uint32_t b = xcd_run(blockIdx.x, total, p.xcds);
        expert = p.plan.tile_group[b / (uint32_t)p.tiles_n];
        const uint32_t f = p.plan.first_tile[expert], cnt = p.plan.first_tile[expert + 1] - f;
        const uint32_t in = b - f * (uint32_t)p.tiles_n;         // within the expert: m fastest
        n0 = (int)(in / cnt) * BN;
        m0 = (int64_t)p.plan.offsets[expert] + (int64_t)(in % cnt) * BM;
        rows = (int64_t)p.plan.offsets[expert + 1] - m0;
    } else {
        const uint32_t b = xcd_run(blockIdx.x, gridDim.x, p.xcds);
        const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM);
        // bands of 8 row tiles, n outer and m inner within a band
        const uint32_t band = b / (8 * (uint32_t)p.tiles_n), in = b - band * 8 * (uint32_t)p.tiles_n;
        const uint32_t h = tm - band * 8 < 8 ? tm - band * 8 : 8;
        n0 = (int)(in / h) * BN;
        m0 = (int64_t)(band * 8 + in % h) * BM;
        rows = a.M - m0;
    }
    if (rows > BM) rows = BM;
    const int nrows = (int)(a.N - n0 < BN ? a.N - n0 : BN);

    f32x16 acc[TN][TM];
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[tn][tm][r] = 0.f;

    if (!GATHER || expert < (uint32_t)a.E) {
        if (p.lds_nan) {   // debug: every LDS byte of the tile starts as NaN
            for (int o = tid * 16; o < S::lds(YS); o += 64 * NW * 16) *(u32x4*)(smem + o) = u32x4{~0u, ~0u, ~0u, ~0u};
            __syncthreads();
        }
        const uint32_t half = (uint32_t)(a.K / 2);
        const int KB = (int)(a.K / 32);
        const int64_t wrow = (int64_t)expert * a.N + n0;
        const __amdgpu_buffer_rsrc_t wr = rsrc(a.wq + wrow * half, (uint32_t)nrows * half);
        const __amdgpu_buffer_rsrc_t wsr = rsrc(a.ws + wrow * a.wsstride, (uint32_t)(nrows * a.wsstride));
        const int64_t xrow = GATHER ? 0 : m0, xrows = GATHER ? a.B : rows;
        const __amdgpu_buffer_rsrc_t xr = rsrc(a.xq + xrow * half, (uint32_t)(xrows * half));
        const __amdgpu_buffer_rsrc_t xsr = rsrc(a.xs + xrow * a.xsstride, (uint32_t)(xrows * a.xsstride));
        auto src = [&](int r) -> uint32_t {        // x row of local row r, NOWHERE past the tile
            if (r >= rows) return NOWHERE;
            if constexpr (GATHER) return p.plan.perm[m0 + r] / p.per_entry;
            else return (uint32_t)r;
        };

        uint32_t doff[S::ND], dchunk[S::ND];
#pragma unroll
        for (int d = 0; d < S::ND; ++d) {
            const int blk = d * NW + wv;           // W's row blocks first, then x's
            const bool isw = blk < BN / S::RPL;
            const int r = (isw ? blk : blk - BN / S::RPL) * S::RPL + lane / S::CH;
            dchunk[d] = (uint32_t)((lane & (S::CH - 1)) ^ swz<BKB>(r));
            const uint32_t row = isw ? (r < nrows ? (uint32_t)r : NOWHERE) : src(r);
            doff[d] = row == NOWHERE ? NOWHERE : row * half + dchunk[d] * 16u;
        }
        const int nk = (KB + S::CH - 1) / S::CH;
        // load d of step kt (past the end: of the last step, so that the counts stay the same)
        auto dma = [&](int kt, int d) {
            const int k = kt < nk ? kt : nk - 1;
            const bool isw = d < BN / S::RPL / NW;
            uint32_t off = doff[d];
            if (k == nk - 1 && KB % S::CH != 0 && (uint32_t)(k * S::CH) + dchunk[d] >= (uint32_t)KB) off = NOWHERE;
            unsigned char* to = smem + (kt % ST) * S::STAGE + (d * NW + wv) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(isw ? wr : xr, (__attribute__((address_space(3))) void*)to, 16,
                                                     (int)off, k * BKB, 0, 0);
        };
        uint32_t soff[S::NS];
#pragma unroll
        for (int d = 0; d < S::NS; ++d) {
            const int blk = (d * NW + wv) % S::NSI;   // a wave without a load of its own repeats another's
            const int r = (blk < BN / 64 ? blk : blk - BN / 64) * 64 + lane;
            const uint32_t row = blk < BN / 64 ? (r < nrows ? (uint32_t)r : NOWHERE) : src(r);
            soff[d] = row == NOWHERE ? NOWHERE : row * (uint32_t)(blk < BN / 64 ? a.wsstride : a.xsstride);
        }
        auto dma_scales = [&](int stage, int g) {
#pragma unroll
            for (int d = 0; d < S::NS; ++d) {
                const int blk = (d * NW + wv) % S::NSI;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    blk < BN / 64 ? wsr : xsr,
                    (__attribute__((address_space(3))) void*)(slds + stage * S::SSTAGE + blk * 1024), 16, (int)soff[d],
                    g * 16, 0, 0);
            }
        };
        const int ng = (nk + S::SG - 1) / S::SG;
        // the batch of scales that step kt opens, if it opens one
        auto open_scales = [&](int kt) {
            if (kt % S::SG == 0) {
                const int g = kt / S::SG;
                dma_scales(g % S::SST, g < ng ? g : ng - 1);
            }
        };
#pragma unroll
        for (int u = 0; u < S::LA; ++u) {
            open_scales(u);
#pragma unroll
            for (int d = 0; d < S::ND; ++d) dma(u, d);
        }

        // the lane's place in a stage: row i of a 32-row tile, its first chunk;
        // swz repeats every 16 rows and chunk h of the lane's piece differs in
        // the low bits only
        const uint32_t wlane = (uint32_t)(32 * TN * wn + i) * BKB + (((S::KH * j) ^ swz<BKB>(i)) << 4);
        const uint32_t xlane = (uint32_t)(S::WSTAGE + (32 * TM * wm + i) * BKB) + (((S::KH * j) ^ swz<BKB>(i)) << 4);
        const uint32_t slane = (uint32_t)i * 16 + (S::SG == 2 ? 4 * j : 0);
        auto step = [&](int kt) {
            __builtin_amdgcn_s_barrier();
            const unsigned char* const stage = smem + (kt % ST) * S::STAGE;
            // the scale bytes of the lane's blocks: its own dword of the step's 8
            // bytes a row, or its half of 4
            const unsigned char* const st = slds + (kt / S::SG % S::SST) * S::SSTAGE + (kt % S::SG) * (16 / S::SG) + slane;
            const int shift = S::SG == 2 ? 0 : 16 * j;
            uint32_t sw[TN], sx[TM];
            u32x4 fa[2][TN], fb[2][TM];
            auto read = [&](int h) {
#pragma unroll
                for (int t = 0; t < TN; ++t) fa[h & 1][t] = *(const u32x4*)(stage + (wlane ^ (h << 4)) + t * 32 * BKB);
#pragma unroll
                for (int t = 0; t < TM; ++t) fb[h & 1][t] = *(const u32x4*)(stage + (xlane ^ (h << 4)) + t * 32 * BKB);
            };
            read(0);
#pragma unroll
            for (int t = 0; t < TN; ++t) sw[t] = *(const uint32_t*)(st + 32 * (TN * wn + t) * 16) >> shift;
#pragma unroll
            for (int t = 0; t < TM; ++t) sx[t] = *(const uint32_t*)(st + (BN + 32 * (TM * wm + t)) * 16) >> shift;
            open_scales(kt + S::LA);
            // the loads of step kt + LA go into the stage read one step ago, a few
            // after each product so that none waits for the others to be taken
            int d = 0;
#pragma unroll
            for (int h = 0; h < S::KH; ++h) {
                if (h + 1 < S::KH) read(h + 1);
                __builtin_amdgcn_sched_barrier(0);   // keeps those reads ahead of this round's products
#pragma unroll
                for (int q = 0; q < TN * TM; ++q) {
                    const u32x4 A = fa[h & 1][q / TM], B = fb[h & 1][q % TM];
                    f32x16& c = acc[q / TM][q % TM];
                    const uint32_t sa = sw[q / TM], sb = sx[q % TM];
                    if (h == 0) c = mfma32<0>(A, B, c, sa, sb);
                    else if (h == 1) c = mfma32<1>(A, B, c, sa, sb);
                    else if (h == 2) c = mfma32<2>(A, B, c, sa, sb);
                    else c = mfma32<3>(A, B, c, sa, sb);
                    if (d < S::ND && q % SPREAD == SPREAD - 1) {
                        dma(kt + S::LA, d++);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        };
        for (int kt = 0; kt < nk; kt += S::SG) {
            wait_loads<S::after(0)>();
            step(kt);
            if (kt + 1 < nk) {
                wait_loads<S::after(1)>();
                step(kt + 1);
            }
            if constexpr (S::SG == 4) {
                if (kt + 2 < nk) {
                    wait_loads<S::after(2)>();
                    step(kt + 2);
                }
                if (kt + 3 < nk) {
                    wait_loads<S::after(3)>();
                    step(kt + 3);
                }
            }
        }
        wait_loads<0>();                           // every load has landed ...
        __syncthreads();                           // ... and every read is done: LDS is free for the outputs
    }

    // acc[tn][tm][r] = D[n][m]: m = lane % 32, n = 8 (r / 4) + 4 (lane / 32) + r % 4.
    // Each wave lays 32 rows m of its TN * 32 columns out in LDS and stores
    // them by rows; no other wave reads them.
    constexpr int OROW = S::orow(YS), PER = 16 / YS, LPR = TN * 32 / PER;   // values and lanes of a 16-byte store
    unsigned char* const ot = smem + wv * 32 * OROW;
    const int nw0 = n0 + 32 * TN * wn;
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
        const int mb = 32 * (TM * wm + tm);
        if (mb >= rows) break;
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x16& c = acc[tn][tm];
                store4<YDT>(ot + i * OROW, 32 * tn + 8 * g + 4 * j, c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (p.wide) {
#pragma unroll 4
            for (int r = lane / LPR; r < 32; r += 64 / LPR) {
                const int c = (lane % LPR) * PER, n = nw0 + c;
                if (mb + r >= rows || n >= a.N) continue;      // N is a multiple of PER
                const int64_t dst = GATHER ? (int64_t)p.plan.perm[m0 + mb + r] : m0 + mb + r;
                *(u32x4*)((unsigned char*)a.y + (dst * a.N + n) * YS) = *(const u32x4*)(ot + r * OROW + c * YS);
            }
        } else {
            for (int r = 0; r < 32; ++r) {
                if (mb + r >= rows) break;
                const int64_t dst = GATHER ? (int64_t)p.plan.perm[m0 + mb + r] : m0 + mb + r;
                for (int c = lane; c < TN * 32; c += 64) {
                    if (nw0 + c >= a.N) break;
                    if constexpr (YS == 4) ((uint32_t*)a.y)[dst * a.N + nw0 + c] = *(const uint32_t*)(ot + r * OROW + c * 4);
                    else ((uint16_t*)a.y)[dst * a.N + nw0 + c] = *(const uint16_t*)(ot + r * OROW + c * 2);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

__global__ void __launch_bounds__(256) pad_scales_kernel(const uint8_t* __restrict__ s, int64_t n, uint32_t KS,
                                                         uint8_t* __restrict__ out, uint32_t stride) {
    const int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (o >= n) return;
    const int64_t row = o / stride;
    const uint32_t c = (uint32_t)(o - row * stride);
    out[o] = c < KS ? s[row * KS + c] : (uint8_t)127;
}

// ---------------------------------------------------------------- dispatch

template <int NT, int MT, int YDT, int ROWS>
void stream_launch(const StreamArgs& s, int64_t tiles, hipStream_t st) {
    const int64_t runs = (s.a.K + 511) / 512;
    const int waves = runs >= 8 ? 8 : runs >= 4 ? 4 : runs >= 2 ? 2 : 1;
    const size_t shm = (size_t)waves * 256 * NT * MT * sizeof(float);
    mx4_stream_kernel<NT, MT, YDT, ROWS><<<(unsigned)(tiles * s.tile_n), 64 * waves, shm, st>>>(s);
}

template <int YDT, int ROWS>
hipError_t stream_rows(StreamArgs s, int mt, int64_t tiles, hipStream_t st) {
    s.tile_n = (int)((s.a.N + 15) / 16);
    if (tiles * s.tile_n > 0x7fffffffLL) return hipErrorInvalidValue;
    if (mt == 1) stream_launch<1, 1, YDT, ROWS>(s, tiles, st);
    else if (mt == 2) stream_launch<1, 2, YDT, ROWS>(s, tiles, st);
    else stream_launch<1, 4, YDT, ROWS>(s, tiles, st);
    return hipGetLastError();
}

template <int BN, int BM, int WN, int WM, int ST, int BKB, int YDT, bool GATHER>
hipError_t tiled_launch(TiledArgs p, hipStream_t st) {
    const Mx4Args& a = p.a;
    p.tiles_n = (int)((a.N + BN - 1) / BN);
    const int64_t tm = GATHER ? mx4_plan_max_tiles(a.M, a.E, BM) : (a.M + BM - 1) / BM;
    if (tm * p.tiles_n > 0x7fffffffLL) return hipErrorInvalidValue;
    constexpr size_t shm = Shape<BN, BM, WN, WM, ST, BKB>::lds(YDT == QLIN_F32 ? 4 : 2);
    static_assert(shm <= 160 * 1024, "LDS of a compute unit");
    const auto kernel = mx4_tiled_kernel<BN, BM, WN, WM, ST, BKB, YDT, GATHER>;
    static std::atomic<bool> attr{false};
    if (!attr.load(std::memory_order_acquire)) {
        const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)shm);
        if (e != hipSuccess) return e;
        attr.store(true, std::memory_order_release);
    }
    kernel<<<(unsigned)(tm * p.tiles_n), 64 * WN * WM, shm, st>>>(p);
    return hipGetLastError();
}

constexpr int64_t kStreamRows = 64;    // rows (of one expert, on average) up to which W is streamed

int forced_tile() {
    const char* e = getenv("QLIN_MXFP4_TILE");
    return e && *e ? atoi(e) : -1;
}

template <int YDT, bool GATHER>
hipError_t tiled_rows(const Mx4Args& a, const Mx4Plan& plan, uint32_t per, int tile, hipStream_t st) {
    const TiledArgs p{a, plan, per, 0, device_shape().xcds, debug_lds_nan() ? 1 : 0,
                      a.N % (YDT == QLIN_F32 ? 4 : 8) == 0 && (uintptr_t)a.y % 16 == 0 ? 1 : 0};
    if (tile == 1) return tiled_launch<256, 256, 2, 2, 2, 128, YDT, GATHER>(p, st);
    if (tile == 2) return tiled_launch<256, 256, 2, 4, 4, 64, YDT, GATHER>(p, st);
    if (tile == 3) return tiled_launch<256, 128, 2, 2, 3, 64, YDT, GATHER>(p, st);
    if (tile == 4) return tiled_launch<128, 128, 2, 2, 2, 128, YDT, GATHER>(p, st);
    if (tile == 8) return tiled_launch<256, 128, 4, 2, 3, 128, YDT, GATHER>(p, st);
    if (tile == 9) return tiled_launch<128, 64, 2, 2, 2, 128, YDT, GATHER>(p, st);
    if (tile == 10) return tiled_launch<128, 64, 2, 2, 3, 128, YDT, GATHER>(p, st);
    if (tile == 11) return tiled_launch<64, 64, 2, 2, 4, 128, YDT, GATHER>(p, st);
    if (tile == 5) return tiled_launch<256, 256, 2, 2, 4, 64, YDT, GATHER>(p, st);
    if (tile == 6) return tiled_launch<256, 256, 2, 4, 2, 128, YDT, GATHER>(p, st);
    if (tile == 7) return tiled_launch<128, 128, 2, 2, 4, 64, YDT, GATHER>(p, st);
    return tiled_launch<128, 128, 2, 2, 4, 128, YDT, GATHER>(p, st);
}

template <int YDT>
hipError_t launch(const Mx4Args& a, hipStream_t st, const char** path) {
    int tile = forced_tile();
    if (tile < 0) tile = 4;
    if (!a.experts) {
        if (!mx4_tiled(a.M, a.N, a.K, 1, false)) {
            *path = "mxfp4_stream";
            const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
            return stream_rows<YDT, DENSE>(StreamArgs{a, Mx4Plan{}, 1, 0}, mt, (a.M + 16 * mt - 1) / (16 * mt), st);
        }
        *path = "mxfp4_tiled";
        return tiled_rows<YDT, false>(a, Mx4Plan{}, 1, tile, st);
    }
    const uint32_t per = (uint32_t)(a.M / a.B);
    if (2 * a.M <= a.E) {
        *path = "mxfp4_gather_direct";
        return stream_rows<YDT, DIRECT>(StreamArgs{a, Mx4Plan{}, per, 0}, 1, a.M, st);
    }
    Mx4Plan plan{};
    const bool tiled = mx4_tiled(a.M, a.N, a.K, a.E, true);
    const int mt = a.M <= 16 * a.E ? 1 : a.M <= 32 * a.E ? 2 : 4;
    const int rows = tiled ? (tile >= 9 ? 64 : tile == 0 || tile == 3 || tile == 4 || tile == 7 || tile == 8 ? 128 : 256) : 16 * mt;
    hipError_t e = launch_mx4_plan(a.experts, a.M, a.E, rows, a.plan, &plan, st);
    if (e != hipSuccess) return e;
    if (!tiled) {
        *path = "mxfp4_gather_stream";
        return stream_rows<YDT, PLAN>(StreamArgs{a, plan, per, 0}, mt, mx4_plan_max_tiles(a.M, a.E, rows), st);
    }
    *path = "mxfp4_gather_tiled";
    return tiled_rows<YDT, true>(a, plan, per, tile, st);
}

}  // namespace

bool mx4_tiled(int64_t M, int64_t N, int64_t K, int64_t E, bool gather) {
    const char* e = getenv("MX4S"); const int64_t kr = e ? atoi(e) : kStreamRows; return M > kr * (gather ? E : 1);
}

hipError_t launch_mx4_matmul(const Mx4Args& a, hipStream_t st, const char** path) {
    if (a.ydt == QLIN_BF16) return launch<QLIN_BF16>(a, st, path);
    if (a.ydt == QLIN_F16) return launch<QLIN_F16>(a, st, path);
    return launch<QLIN_F32>(a, st, path);
}

hipError_t launch_mx4_pad_scales(const uint8_t* s, int64_t rows, int64_t KS, uint8_t* out, int64_t stride,
                                 hipStream_t st) {
    const int64_t n = rows * stride, grid = (n + 255) / 256;
    if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
    pad_scales_kernel<<<(unsigned)grid, 256, 0, st>>>(s, n, (uint32_t)KS, out, (uint32_t)stride);
    return hipGetLastError();
}

}  // namespace qlin
