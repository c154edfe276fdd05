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
//  * streaming (few rows): bound by reading W. 16 weight rows per workgroup, K
//    split over its waves, W straight from memory into the instruction's
//    registers, partial sums joined through LDS. Blocks of 16 rows of codes, 4 of
//    a float x, which each wave quantizes for its own part of K, or by experts
//    one index row: each block reads W for itself, which costs less than the
//    launch it saves while W is small. One row, N 14336, K 4096: 8.4 us (3.7 TB/s
//    with the launch); one token by 8 experts, N 1536, K 2048: 7.0 us; 16 rows
//    of codes, N = K = 8192: 11.8 us.
//  * tiled (many rows): bound by power, which holds the clock (matrix cores alone
//    5.9 PFLOP/s; a step of 256 codes takes a 256 x 256 tile 2.1 us with random
//    codes, 1.35 with zeros), and at small K by the start and outputs of a tile.
//    8192 rows, N 12288, K 4096: 219 us (3.8 PFLOP/s); N = K = 8192: 284 us (3.9);
//    65536 rows by 64 experts, N 4096, K 2048: 415 us (2.7); 512 tokens by 8 of
//    64 experts, N 1536, K 2048: 34 us, 3.2 TB/s of W.

#include "mx4_common.h"

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

constexpr int STREAM_ROWS = 16;        // rows of x of a workgroup
constexpr int STREAM_FLOAT_ROWS = 4;   // ... of a float x
constexpr int STREAM_WAVES = 16;

struct StreamArgs {
    Mx4Args a;
    uint32_t per_entry;    // index rows per row of x (DIRECT)
    int tiles_n;           // workgroups of a block of rows
    FastDiv by_tiles;      // workgroup / tiles_n
    int vec;               // a float x is 16-byte aligned
};

// A run is 512 values along K, 16 blocks: lane piece q of an operand's row holds
// blocks 4q .. 4q + 3, 64 bytes of codes and a dword of scales.
struct Piece {
    u32x4 c[4];
    uint32_t s;
};

// Lane piece of whole run `run` of a row whose piece of run 0 starts at c and s.
__device__ __forceinline__ Piece load_piece(const uint8_t* c, const uint8_t* s, int run) {
    Piece p;
    __builtin_memcpy(&p.s, s + run * 16, 4);
#pragma unroll
    for (int b = 0; b < 4; ++b) p.c[b] = *(const u32x4*)(c + (int64_t)run * 256 + 16 * b);
    return p;
}
// The same of a run of which the piece has `left` blocks; the others are zeros.
__device__ __forceinline__ Piece load_piece(const uint8_t* c, const uint8_t* s, int run, int left) {
    Piece p;
    p.s = scale4(s + run * 16, left);
#pragma unroll
    for (int b = 0; b < 4; ++b)
        p.c[b] = b < left ? *(const u32x4*)(c + (int64_t)run * 256 + 16 * b) : u32x4{0, 0, 0, 0};
    return p;
}

// Rows of a workgroup: by experts (DIRECT) one index row, with its expert's W.
template <int XDT, bool DIRECT>
constexpr int stream_block() { return DIRECT ? 1 : XDT == QLIN_U8 ? STREAM_ROWS : STREAM_FLOAT_ROWS; }

// XDT QLIN_U8: x's codes; else a float x, quantized here.
template <int YDT, int XDT, bool DIRECT>
__global__ void __launch_bounds__(64 * STREAM_WAVES) mx4_stream_kernel(StreamArgs s) {
    constexpr bool FLOAT = XDT != QLIN_U8;
    constexpr int XR = stream_block<XDT, DIRECT>();
    extern __shared__ __align__(16) uint32_t lds[];     // partial sums [waves][16][16]; codes of a float x
    const Mx4Args& a = s.a;
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, q = lane >> 4;
    const uint32_t tile = s.by_tiles(blockIdx.x);                       // block of rows
    const int64_t n0 = (int64_t)(blockIdx.x - tile * (uint32_t)s.tiles_n) * 16;
    const int64_t m0 = (int64_t)tile * XR;                              // first row of y
    const int rows = (int)(a.M - m0 < XR ? a.M - m0 : XR);
    const int64_t src = DIRECT ? (int64_t)(tile / s.per_entry) : m0;    // ... and of x
    const uint32_t expert = DIRECT ? (uint32_t)a.experts[tile] : 0;

    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (!DIRECT || expert < (uint32_t)a.E) {            // else the row is zeros
        const int KB = (int)(a.K / 32);                 // blocks of a row
        const int64_t half = a.K / 2;
        const int64_t n = (int64_t)expert * a.N + (n0 + i < a.N ? n0 + i : a.N - 1);   // rows past N are not stored
        const uint8_t* const wp = a.wq + n * half + 64 * q;
        const uint8_t* const wsp = a.ws + n * a.wsstride + 4 * q;
        const int64_t xrow = src + (i < rows ? i : 0);  // columns past the rows repeat the first and are not stored
        const int whole = KB / 16;                      // whole runs; one more of KB % 16 blocks
        const uint8_t* const xp = a.xq + xrow * half + 64 * q;
        const uint8_t* const xsp = a.xs + xrow * a.xsstride + 4 * q;
        // x's piece of a run: from its codes, or rounded here
        auto x_piece = [&](int run) {
            if constexpr (!FLOAT) {
                return load_piece(xp, xsp, run);
            } else {
                // lane l rounds values 8 l .. 8 l + 7 of the run, a row at a time; the wave's own LDS
                // turns words into pieces
                uint32_t* const words = lds + waves * 256 + wave * XR * 68;      // [XR][64] words, [XR][4] scales
                uint8_t* const bytes = (uint8_t*)(words + XR * 64);
                const int64_t k = (int64_t)run * 512 + 8 * lane;
                const bool live = k < a.K;                                       // whole blocks of 4 lanes
#pragma unroll
                for (int r = 0; r < XR; ++r) {
                    if (r >= rows) break;
                    const int64_t at = (src + r) * a.K * (a.swiglu ? 2 : 1) + (live ? k : 0);
                    uint32_t byte, word;
                    if (a.swiglu)
                        word = mxfp4_word<QLIN_F32>(
                            swiglu8<XDT>(load8<XDT>(a.x, at, s.vec), load8<XDT>(a.x, at + a.K, s.vec)), &byte);
                    else
                        word = mxfp4_word<XDT>(load8<XDT>(a.x, at, s.vec), &byte);
                    words[r * 64 + lane] = live ? word : 0u;
                    if ((lane & 3) == 0) bytes[r * 16 + (lane >> 2)] = live ? (uint8_t)byte : (uint8_t)127;
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const int r = i < rows ? i : 0;
                Piece x;
#pragma unroll
                for (int b = 0; b < 4; ++b) x.c[b] = *(const u32x4*)(words + r * 64 + 16 * q + 4 * b);
                x.s = *(const uint32_t*)(bytes + r * 16 + 4 * q);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                return x;
            }
        };
        auto multiply = [&](const Piece& w, const Piece& x) {
            acc = mfma16<0>(w.c[0], x.c[0], acc, w.s, x.s);
            acc = mfma16<1>(w.c[1], x.c[1], acc, w.s, x.s);
            acc = mfma16<2>(w.c[2], x.c[2], acc, w.s, x.s);
            acc = mfma16<3>(w.c[3], x.c[3], acc, w.s, x.s);
        };
        // two runs at a time, both pieces of W on their way before x is looked at (an odd last one loads twice)
        for (int run = wave; run < whole; run += 2 * waves) {
            const bool two = run + waves < whole;
            const Piece w0 = load_piece(wp, wsp, run), w1 = load_piece(wp, wsp, two ? run + waves : run);
            if constexpr (FLOAT) {
                __builtin_amdgcn_sched_barrier(0);
                multiply(w0, x_piece(run));
                if (two) multiply(w1, x_piece(run + waves));
            } else {
                const Piece x0 = x_piece(run), x1 = x_piece(two ? run + waves : run);
                __builtin_amdgcn_sched_barrier(0);
                multiply(w0, x0);
                if (two) multiply(w1, x1);
            }
        }
        if (KB % 16 && whole % waves == wave) {
            const int left = KB - whole * 16 - 4 * q;
            const Piece w = load_piece(wp, wsp, whole, left);
            if constexpr (FLOAT) multiply(w, x_piece(whole));
            else multiply(w, load_piece(xp, xsp, whole, left));
        }
    }
    // D[n][m]: n = 4 q + r, m = i
    float* const red = (float*)lds;
    *(f32x4*)(red + (wave * 16 + i) * 16 + 4 * q) = acc;
    __syncthreads();
    for (int o = tid; o < 16 * rows; o += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += red[w * 256 + o];
        const int m = o >> 4, n = o & 15;
        if (n0 + n < a.N) store_f<YDT>(a.y, (m0 + m) * a.N + n0 + n, v);
    }
}

// ------------------------------------------------------------------ tiled

struct TiledArgs {
    Mx4Args a;
    Mx4Plan plan;
    FastDiv per_entry;     // index row / index rows per row of x
    int tiles_n;
    int xcds;
    int lds_nan;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

constexpr int BKB = 128;                    // bytes of a row a step takes: 256 codes, 8 blocks
constexpr int CH = BKB / 16, KH = CH / 2;   // chunks (blocks) of a row and step; instructions along K
constexpr int SG = 2;                       // steps whose scales one 16-byte load of a row brings

// 16-byte chunk c of row r sits in slot c ^ swz(r) of its LDS row of 128 bytes:
// any 8 neighbouring rows then keep a chunk in 8 different 16-byte columns of
// the 128-byte bank line.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

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

constexpr uint32_t NOWHERE = 0x80000000u;   // past every buffer range: reads zeros

// Where a workgroup's tile lies. `b` numbers the tiles: by experts an expert's row
// tiles run fastest, dense ones in bands of 8 row tiles, n outer and m inner in a
// band, so that neighbours share W or x in their XCD's L2.
struct TilePlace {
    int64_t m0;            // first place (dense: row) of the tile
    int rows, n0, nrows;
    uint32_t expert;       // E: zeros
};

template <int BN, int BM, bool GATHER>
__device__ __forceinline__ TilePlace tile_place(const TiledArgs& p, uint32_t b) {
    const Mx4Args& a = p.a;
    const uint32_t tn = (uint32_t)p.tiles_n;
    TilePlace t;
    int64_t rows;
    if constexpr (GATHER) {
        // one scalar load: the plan does not change while the kernel runs
        typedef __attribute__((ext_vector_type(8))) uint32_t u32x8;
        const Mx4Tile g = __builtin_bit_cast(
            Mx4Tile, *(const __attribute__((address_space(4))) u32x8*)(p.plan.tiles + b / tn));
        const uint32_t in = b - g.first * tn;
        t.expert = g.group;
        t.n0 = (int)(in / g.count) * BN;
        const uint32_t m = in % g.count * BM;
        t.m0 = (int64_t)g.place + m;
        rows = (int64_t)g.rows - m;
    } else {
        const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM);
        const uint32_t band = b / (8 * tn), in = b - band * 8 * tn, h = tm - band * 8 < 8 ? tm - band * 8 : 8;
        t.expert = 0;
        t.n0 = (int)(in / h) * BN;
        t.m0 = (int64_t)(band * 8 + in % h) * BM;
        rows = a.M - t.m0;
    }
    t.rows = (int)(rows < BM ? rows : BM);
    t.nrows = (int)(a.N - t.n0 < BN ? a.N - t.n0 : BN);
    return t;
}

// Tiles in all.
template <int BM, bool GATHER>
__device__ __forceinline__ uint32_t tiles_total(const TiledArgs& p) {
    const uint32_t tm =
        GATHER ? *(const __attribute__((address_space(4))) uint32_t*)p.plan.total : (uint32_t)((p.a.M + BM - 1) / BM);
    return tm * (uint32_t)p.tiles_n;
}

// Tile of BN weight rows (n) by BM activation rows (m), WN x WM waves of
// TN x TM 32x32 accumulators, K in steps of BKB bytes a row:
//  * code rows go global -> LDS by buffer -> LDS loads, ST - 1 steps ahead
//    through a ring of ST stages; one wave instruction moves 1 KB of whole row
//    pieces, swizzled so that a fragment read meets no bank conflict;
//  * scale rows go the same way, 16 bytes (SG steps) at a time, issued with
//    the codes of the step that first needs them;
//  * a step is KH instructions deep along K; the fragments of the next one
//    are read while the current one multiplies;
//  * the outputs go through LDS, so that they leave in whole lines.
// Rows past the tile and chunks past K read zeros (buffer range checks).
template <int BN, int BM, int WN, int WM, int ST>
struct Shape {
    static constexpr int NW = WN * WM, TN = BN / WN / 32, TM = BM / WM / 32;
    static constexpr int WSTAGE = BN * BKB, STAGE = (BN + BM) * BKB;
    static constexpr int RPL = 1024 / BKB;                         // rows one load moves
    static constexpr int ND = (BN + BM) / RPL / NW;                // code loads per wave and step
    static constexpr int NSI = (BN + BM) / 64;                     // scale loads per batch
    static constexpr int NS = (NSI + NW - 1) / NW;                 // ... per wave
    static constexpr int LA = ST - 1;                              // steps ahead
    static constexpr int SST = (LA + SG - 1) / SG + 1;             // scale stages
    static constexpr int SSTAGE = (BN + BM) * 16;
    static constexpr int LOOP = ST * STAGE + SST * SSTAGE;         // LDS of the loop
    // LDS of the outputs: per wave 32 rows of TN 32 values, rows 16 bytes longer against conflicts
    static constexpr int orow(int size) { return TN * 32 * size + 16; }
    static constexpr int lds(int size) { return LOOP > NW * 32 * orow(size) ? LOOP : NW * 32 * orow(size); }
    // products between two code loads of a step; all of them go out in it
    static constexpr int EVERY = 2 * ND <= KH * TN * TM && TN * TM % 2 == 0 ? 2 : 1;
    static_assert(ND * EVERY <= KH * TN * TM, "a step issues all its loads");
    static_assert((BN / RPL) % NW == 0 && (BM / RPL) % NW == 0, "whole loads per wave");
    // loads issued after those of a step of phase ph (its number mod SG) when it starts: the LA - 1
    // steps after it, of which those that open a batch brought its scales
    static constexpr int after(int ph) {
        int n = 0;
        for (int u = 1; u < LA; ++u) n += ND + ((ph + u) % SG == 0 ? NS : 0);
        return n;
    }
};

template <int BN, int BM, int WN, int WM, int ST, int YDT, bool GATHER>
__global__ void __launch_bounds__(64 * WN * WM) mx4_tiled_kernel(TiledArgs p) {
    using S = Shape<BN, BM, WN, WM, ST>;
    constexpr int NW = S::NW, TN = S::TN, TM = S::TM;
    constexpr int YS = YDT == QLIN_F32 ? 4 : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char* const slds = smem + ST * S::STAGE;
    const Mx4Args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wv / WM, wm = wv % WM;
    const int i = lane & 31, j = lane >> 5;

    const uint32_t total = tiles_total<BM, GATHER>(p);
    if (blockIdx.x >= total) return;
    const TilePlace t = tile_place<BN, BM, GATHER>(p, xcd_run(blockIdx.x, total, p.xcds));
    const int64_t m0 = t.m0;
    const int rows = t.rows, n0 = t.n0, nrows = t.nrows;
    const uint32_t expert = t.expert;

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
            if constexpr (GATHER) return p.per_entry(p.plan.perm[m0 + r]);
            else return (uint32_t)r;
        };

        uint32_t doff[S::ND], dchunk[S::ND];
#pragma unroll
        for (int d = 0; d < S::ND; ++d) {
            const int blk = d * NW + wv;           // W's row blocks first, then x's
            const bool isw = blk < BN / S::RPL;
            const int r = (isw ? blk : blk - BN / S::RPL) * S::RPL + lane / CH;
            dchunk[d] = (uint32_t)((lane & (CH - 1)) ^ swz(r));
            const uint32_t row = isw ? (r < nrows ? (uint32_t)r : NOWHERE) : src(r);
            doff[d] = row == NOWHERE ? NOWHERE : row * half + dchunk[d] * 16u;
        }
        const int nk = (KB + CH - 1) / CH;
        // load d of step kt (past the end: of the last step, so that the counts stay the same)
        auto dma = [&](int kt, int d) {
            const int k = kt < nk ? kt : nk - 1;
            const bool isw = d < BN / S::RPL / NW;
            uint32_t off = doff[d];
            if (k == nk - 1 && KB % CH != 0 && (uint32_t)(k * CH) + dchunk[d] >= (uint32_t)KB) off = NOWHERE;
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
        const int ng = (nk + SG - 1) / SG;
        // the batch of scales that step kt opens, if it opens one
        auto open_scales = [&](int kt) {
            if (kt % SG == 0) {
                const int g = kt / SG;
                dma_scales(g % S::SST, g < ng ? g : ng - 1);
            }
        };
#pragma unroll
        for (int u = 0; u < S::LA; ++u) {
#pragma unroll
            for (int d = 0; d < S::ND; ++d) {
                if (d == BN / S::RPL / NW) open_scales(u);   // W's codes first: they wait for no row numbers
                dma(u, d);
            }
        }

        // the lane's place in a stage: row i of a 32-row tile, its first chunk;
        // swz repeats every 16 rows and chunk h of the lane's piece differs in
        // the low bits only
        const uint32_t wlane = (uint32_t)(32 * TN * wn + i) * BKB + (((KH * j) ^ swz(i)) << 4);
        const uint32_t xlane = (uint32_t)(S::WSTAGE + (32 * TM * wm + i) * BKB) + (((KH * j) ^ swz(i)) << 4);
        const uint32_t slane = (uint32_t)i * 16 + 4 * j;
        auto step = [&](int kt) {
            __builtin_amdgcn_s_barrier();
            const unsigned char* const stage = smem + (kt % ST) * S::STAGE;
            // the scale bytes of the lane's blocks: a dword of the step's 8 bytes a row
            const unsigned char* const st = slds + (kt / SG % S::SST) * S::SSTAGE + (kt % SG) * (16 / SG) + slane;
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
            for (int t = 0; t < TN; ++t) sw[t] = *(const uint32_t*)(st + 32 * (TN * wn + t) * 16);
#pragma unroll
            for (int t = 0; t < TM; ++t) sx[t] = *(const uint32_t*)(st + (BN + 32 * (TM * wm + t)) * 16);
            open_scales(kt + S::LA);
            // the loads of step kt + LA go into the stage read one step ago, a few
            // after each product so that none waits for the others to be taken
            int d = 0;
#pragma unroll
            for (int h = 0; h < KH; ++h) {
                if (h + 1 < KH) read(h + 1);
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
                    if (d < S::ND && q % S::EVERY == S::EVERY - 1) dma(kt + S::LA, d++);
                }
            }
        };
        for (int kt = 0; kt < nk; kt += SG) {
            wait_loads<S::after(0)>();
            step(kt);
            if (kt + 1 < nk) {
                wait_loads<S::after(1)>();
                step(kt + 1);
            }
        }
        wait_loads<0>();                           // every load has landed ...
        __syncthreads();                           // ... and every read is done: LDS is free for the outputs
    }

    // acc[tn][tm][r] = D[n][m]: m = lane % 32, n = 8 (r / 4) + 4 (lane / 32) + r % 4.
    // Each wave lays 32 rows m of its TN * 32 columns out in LDS and stores
    // them by rows; no other wave reads them.
    // In large calls y goes past the caches, which otherwise lose x and W to it
    // just when the next tiles start.
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
        auto rows_out = [&](auto stream) {     // a loop each: in one, the two kinds of store would be merged
#pragma unroll 4
            for (int r = lane / LPR; r < 32; r += 64 / LPR) {
                const int c = (lane % LPR) * PER, n = nw0 + c;
                if (mb + r >= rows || n >= a.N) continue;
                const int64_t dst = GATHER ? (int64_t)p.plan.perm[m0 + mb + r] : m0 + mb + r;
                unsigned char* const to = (unsigned char*)a.y + (dst * a.N + n) * YS;
                if (n + PER <= a.N) {
                    const u32x4 v = *(const u32x4*)(ot + r * OROW + c * YS);
                    typedef u32x4 __attribute__((aligned(2))) any_u32x4;   // a row of an odd N starts at any element
                    if constexpr (decltype(stream)::value) __builtin_nontemporal_store(v, (any_u32x4*)to);
                    else *(any_u32x4*)to = v;
                } else {
                    for (int q = 0; n + q < a.N; ++q) {
                        if constexpr (YS == 4) ((uint32_t*)to)[q] = *(const uint32_t*)(ot + r * OROW + (c + q) * 4);
                        else ((uint16_t*)to)[q] = *(const uint16_t*)(ot + r * OROW + (c + q) * 2);
                    }
                }
            }
        };
        if (a.stream) rows_out(std::true_type());
        else rows_out(std::false_type());
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// ---------------------------------------------------------------- dispatch

// Reads of W by a float x's blocks of rows.
int64_t stream_reads(int64_t M, bool gather) { return gather ? M : (M + STREAM_FLOAT_ROWS - 1) / STREAM_FLOAT_ROWS; }

// Waves of a workgroup: a wave takes one run, or two where that lets all of W's loads be in flight at once (four waves
// a SIMD). Codes take as many as a float x, so that both give the same bits.
int stream_waves(int64_t reads, int64_t N, int64_t K) {
    int64_t runs = (K + 511) / 512;
    if (reads * ((N + 15) / 16) * runs > 16 * (int64_t)device_shape().cus) runs = (runs + 1) / 2;
    return (int)(runs < STREAM_WAVES ? runs : STREAM_WAVES);
}

template <int YDT, int XDT, bool DIRECT>
hipError_t stream_launch(const Mx4Args& a, hipStream_t st) {
    constexpr int ROWS = stream_block<XDT, DIRECT>();
    const int64_t tiles_m = (a.M + ROWS - 1) / ROWS;
    const int waves = stream_waves(stream_reads(a.M, DIRECT), a.N, a.K);
    const int tiles_n = (int)((a.N + 15) / 16);
    StreamArgs s{a, DIRECT ? (uint32_t)(a.M / a.B) : 1, tiles_n, FastDiv::by((uint32_t)tiles_n), ((uintptr_t)a.x & 15) == 0};
    const size_t floats = XDT == QLIN_U8 ? 0 : ROWS * 68;
    mx4_stream_kernel<YDT, XDT, DIRECT>
        <<<(unsigned)(tiles_m * s.tiles_n), 64 * waves, (size_t)waves * (256 + floats) * sizeof(uint32_t), st>>>(s);
    return hipGetLastError();
}

template <int YDT, int XDT>
hipError_t stream_rows(const Mx4Args& a, hipStream_t st) {
    return a.experts ? stream_launch<YDT, XDT, true>(a, st) : stream_launch<YDT, XDT, false>(a, st);
}

template <int BN, int BM, int WN, int WM, int ST, int YDT, bool GATHER>
hipError_t tiled_launch(TiledArgs p, hipStream_t st) {
    const Mx4Args& a = p.a;
    p.tiles_n = (int)((a.N + BN - 1) / BN);
    const int64_t tm = GATHER ? mx4_plan_max_tiles(a.M, a.E, BM) : (a.M + BM - 1) / BM;
    constexpr size_t shm = Shape<BN, BM, WN, WM, ST>::lds(YDT == QLIN_F32 ? 4 : 2);
    static_assert(shm <= 160 * 1024, "LDS of a compute unit");
    const auto kernel = mx4_tiled_kernel<BN, BM, WN, WM, ST, YDT, GATHER>;
    static std::atomic<bool> attr{false};
    if (!attr.load(std::memory_order_acquire)) {
        const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)shm);
        if (e != hipSuccess) return e;
        attr.store(true, std::memory_order_release);
    }
    kernel<<<(unsigned)(tm * p.tiles_n), 64 * WN * WM, shm, st>>>(p);
    return hipGetLastError();
}

// Shapes of the tiled kernel's workgroup: weight rows x activation rows, how
// many of it fit a CU, and what a round of them takes, in us: `start` for a
// tile's first loads and its outputs, `step` for each step of 256 codes with
// every place of the CU taken, `alone` with one workgroup a CU. Measured at N =
// K = 8192 and N = 12288, K = 4096 with 128 to 8192 rows.
//  0: 8 waves of 64 x 128: the least LDS and L2 traffic a product.
//  1: 4 waves of 64 x 64, two stages: one workgroup's outputs leave under the other's products.
//  2, 3: for few rows: more workgroups and more loads in flight for each byte of W.
//  4: 1 with four stages, where there is one workgroup a CU at most and nothing else hides the loads (497 rows, N = K =
//     8192: 26.1 us; 31.3 with 1, 33.7 with 2).
constexpr int kTiles = 5;
struct TileShape {
    int n, m, threads, per_cu;
    float start, step, alone;
};
constexpr TileShape kTile[kTiles] = {{256, 256, 512, 1, 9.5f, 1.72f, 1.72f},
                                     {128, 128, 256, 2, 3.4f, 1.28f, 0.90f},
                                     {128, 64, 256, 2, 3.0f, 0.78f, 0.38f},
                                     {64, 64, 256, 2, 2.5f, 0.56f, 0.20f},
                                     {128, 128, 256, 1, 3.4f, 0.68f, 0.68f}};

template <int YDT, bool GATHER>
hipError_t tiled_rows(const Mx4Args& a, const Mx4Plan& plan, int tile, hipStream_t st) {
    const TiledArgs p{a, plan, FastDiv::by(GATHER ? (uint32_t)(a.M / a.B) : 1), 0, device_shape().xcds,
                      debug_lds_nan() ? 1 : 0};
    switch (tile) {
    case 0: return tiled_launch<256, 256, 4, 2, 2, YDT, GATHER>(p, st);
    case 1: return tiled_launch<128, 128, 2, 2, 2, YDT, GATHER>(p, st);
    case 2: return tiled_launch<128, 64, 2, 2, 3, YDT, GATHER>(p, st);
    case 3: return tiled_launch<64, 64, 2, 2, 4, YDT, GATHER>(p, st);
    default: return tiled_launch<128, 128, 2, 2, 4, YDT, GATHER>(p, st);
    }
}

template <int YDT>
hipError_t launch(const Mx4Args& a, const Mx4Choice& c, const Mx4Plan* plan, hipStream_t st) {
    if (c.path == Mx4Path::kStreamFloat) {
        if (a.xdt == QLIN_F32) return stream_rows<YDT, QLIN_F32>(a, st);
        if (a.xdt == QLIN_F16) return stream_rows<YDT, QLIN_F16>(a, st);
        return stream_rows<YDT, QLIN_BF16>(a, st);
    }
    if (c.path == Mx4Path::kStream) return stream_rows<YDT, QLIN_U8>(a, st);
    return a.experts ? tiled_rows<YDT, true>(a, *plan, c.tile, st) : tiled_rows<YDT, false>(a, Mx4Plan{}, c.tile, st);
}

// QLIN_MXFP4_TILE=0..4 forces the tiled kernel and its tile (tests run every one on the same inputs).
int forced_tile() {
    const char* e = getenv("QLIN_MXFP4_TILE");
    return e && e[0] >= '0' && e[0] < '0' + kTiles && !e[1] ? e[0] - '0' : -1;
}

}  // namespace

// Few rows stream, each (dense: each 4) with a read of W of its own and x
// rounded on the way, where that costs less than the launch and the plan that it
// saves: up to 12 MB of such reads dense and 24 MB by experts (measured around
// them, us streamed and not: 13 rows, N 653, K 3712 6.5 and 8.8; 36 rows, N
// 5578, K 800, 20 MB 13.7 and 9.0; 51 by 10 experts, N 462, K 1952 7.3 and 9.6;
// 210 by 32, N 393, K 768, 32 MB 11.4 and 9.5). Dense, up to 16 rows stream from
// codes. By experts index rows stream also while they are no more than experts:
// each reads its expert's W, so this wins while few share one and loses where
// many do. Top 8 of E, K 2048, us streamed and with the best tile, experts in
// even demand and (in brackets) in a log-normal one of deviation 2:
//   64, N 1536:   16 rows 7.8, 11.0 (7.5, 10.7)  32 11.2, 14.4 (10.9, 11.7)  64 19.2, 19.6 (18.3, 14.7)
//   64, N 4096:   16 rows 14.0, 16.6 (13.7, 15.3)  32 25.9, 28.5 (23.3, 20.0)  64 46.3, 44.1 (42.6, 28.0)
//   256, N 4096:  64 rows 50.5, 55.0 (43.1, 35.8)  128 93.8, 89.9 (82.4, 53.1)  256 181, 132 (161, 78.5)
// The sizes alone do not tell the demand, and a bound by bytes would have to
// weigh the repeats; this one does not.
// Beyond, the tile whose rounds over the CUs take least. An expert's last row
// tile is half empty on average, so R rows make R / m + E / 2 tiles, or one an
// expert if that is more. Over 223 drawn sizes the choice costs 1.3% more than
// the best of the five tiles on average and 18% at most.
Mx4Choice mx4_choose(int64_t M, int64_t N, int64_t K, int64_t E, bool gather, bool codes) {
    int tile = forced_tile();
    const int64_t reads = stream_reads(M, gather);
    const bool again = reads == 1 || (double)reads * N * K * 0.5 <= (gather ? 24e6 : 12e6);
    if (tile < 0 && (gather ? M <= E || again : M <= STREAM_ROWS || again))
        return {codes || (!gather && !again) ? Mx4Path::kStream : Mx4Path::kStreamFloat, -1, 0};
    if (tile < 0) {
        const int64_t cus = device_shape().cus, steps = (K + 255) / 256;
        double best = 0;
        for (int t = 0; t < kTiles; ++t) {
            const TileShape& s = kTile[t];
            int64_t m = (M + s.m - 1) / s.m;
            if (gather) {
                const int64_t hit = E < M ? E : M;
                m = M / s.m + hit / 2 > hit ? M / s.m + hit / 2 : hit;
            }
            const int64_t tiles = m * ((N + s.n - 1) / s.n), places = cus * s.per_cu, rest = tiles % places;
            double us = (double)(tiles / places) * (s.start + s.step * steps);
            if (rest) us += s.start + (rest > cus ? s.step : s.alone) * steps;
            if (t == 0 || us < best) {
                best = us;
                tile = t;
            }
        }
    }
    return {Mx4Path::kTiled, tile, kTile[tile].m};
}

bool mx4_fits(int64_t M, int64_t N, int64_t K, int64_t E, bool gather, const Mx4Choice& c) {
    if (c.path != Mx4Path::kTiled) {
        const int rows = gather ? 1 : c.path == Mx4Path::kStream ? STREAM_ROWS : STREAM_FLOAT_ROWS;
        return (M + rows - 1) / rows * ((N + 15) / 16) <=
               2 * kLaunchItems / (64 * stream_waves(stream_reads(M, gather), N, K)) - 1;
    }
    const TileShape& s = kTile[c.tile];
    const int64_t m = gather ? mx4_plan_max_tiles(M, E, s.m) : (M + s.m - 1) / s.m;
    return m * ((N + s.n - 1) / s.n) <= 2 * kLaunchItems / s.threads - 1;
}

hipError_t launch_mx4_matmul(const Mx4Args& a, const Mx4Choice& c, const Mx4Plan* plan, hipStream_t st) {
    if (a.ydt == QLIN_BF16) return launch<QLIN_BF16>(a, c, plan, st);
    if (a.ydt == QLIN_F16) return launch<QLIN_F16>(a, c, plan, st);
    return launch<QLIN_F32>(a, c, plan, st);
}

}  // namespace qlin
