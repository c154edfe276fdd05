// mx4_prepare.hip -- what an mxfp4 product needs before its tiles can run: the
// activation's codes and scales, by experts the row plan, and scale rows in
// whole 16-byte units where K / 32 is no multiple of 16 or their address none.
// All of it comes from one launch where the index rows fit one chunk, so that
// the plan's round trips hide behind the rest.
//
// Activation: one thread per packed word (8 values), 4 lanes per block; bound
// by HBM (65536 rows of 2 x 2048 bf16 values with swiglu: 103 us, 5.9 TB/s;
// 8192 of 4096: 20 us; with the plan of 512 tokens by 8 experts 5.1 us).
// Scale rows: one thread per 16-byte unit.
// Plan: workgroups of their own at the front of the launch, bound by latency
// (a few barriers and memory round trips). More than one chunk of rows takes a
// second launch (65536 rows: 6.8 us): first counts per chunk, then each chunk
// scans all counts for its own places. The order of rows inside a group is
// free: each output row depends on its own inputs only.

#include "mx4_common.h"

namespace qlin {
namespace {

constexpr int THREADS = 512;
constexpr int PLAN_PER = 8;                          // index rows of a thread ...
constexpr int PLAN_CHUNK = THREADS * PLAN_PER;       // ... and of a workgroup, a chunk
// A plan of up to two chunks of rows is one of twice the size: longer than a chunk's, but in the first launch (4872
// rows 17.6 -> 14.7 us for the product; chunks of that size throughout 39.0 -> 42.5 at 16000 rows).
constexpr int PLAN_ONE = 2;
// Above this many chunks a launch between the two scans the counts, which every chunk otherwise does for itself.
constexpr int PLAN_SCAN = 64;

struct PrepareArgs {
    // activation
    const void* x;
    int64_t words;          // packed words in all; 0: codes are given
    uint32_t row_words;     // packed words of a row
    FastDiv by_row;         // word / row_words
    int swiglu, vec;
    uint32_t* xq;
    uint8_t* xs;
    int64_t sstride;
    int act_blocks;
    // scale rows to lay out: W's (0) and given codes' (1)
    Mx4Scales pad[2];
    FastDiv by_unit;        // 16-byte unit / units of a row
    int pad_blocks[2];
    // plan
    const int32_t* experts; // null: dense
    int R, E, chunks, tile_rows;
    int scanned;            // counts hold the sums of the chunks before, and of all in a last row
    Mx4Plan plan;
};

__device__ __forceinline__ uint32_t group_of(int32_t e, uint32_t E) { return (uint32_t)e < E ? (uint32_t)e : E; }

// Rows of each group in chunk `chunk`, to counts.
__device__ __forceinline__ void plan_count(const PrepareArgs& a, int chunk, uint32_t* cnt) {
    for (int e = threadIdx.x; e <= a.E; e += THREADS) cnt[e] = 0;
    __syncthreads();
    const int r0 = chunk * PLAN_CHUNK + threadIdx.x;
#pragma unroll
    for (int c = 0; c < PLAN_PER; ++c)
        if (r0 + c * THREADS < a.R) atomicAdd(&cnt[group_of(a.experts[r0 + c * THREADS], a.E)], 1u);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += THREADS) a.plan.counts[(size_t)chunk * (a.E + 1) + e] = cnt[e];
}

// Places of the rows of chunk `chunk`; chunk 0 writes the tables too. A single
// chunk counts its rows itself. PER: rows of a thread.
template <int PER>
__device__ __forceinline__ void plan_place(const PrepareArgs& a, int chunk, uint32_t* sh) {
    const int E = a.E, tid = threadIdx.x;
    uint32_t* const tot = sh;                        // [E + 1] rows of the group
    uint32_t* const cur = sh + E + 1;                // [E + 1] next place of this chunk's rows
    __shared__ uint32_t wsum[THREADS / 64][2], carry[2];
    const int r0 = chunk * THREADS * PER + tid;
    if (tid < 2) carry[tid] = 0;
    uint32_t g[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        const int r = r0 + c * THREADS;
        g[c] = group_of(a.experts[r < a.R ? r : a.R - 1], E);
    }
    if (a.chunks == 1) {
        for (int e = tid; e <= E; e += THREADS) tot[e] = cur[e] = 0;
        __syncthreads();
#pragma unroll
        for (int c = 0; c < PER; ++c)
            if (r0 + c * THREADS < a.R) atomicAdd(&tot[g[c]], 1u);
    } else {
        for (int e = tid; e <= E; e += THREADS) {
            if (a.scanned) {
                tot[e] = a.plan.counts[(size_t)a.chunks * (E + 1) + e];
                cur[e] = a.plan.counts[(size_t)chunk * (E + 1) + e];
                continue;
            }
            uint32_t all = 0, before = 0;
#pragma unroll 4
            for (int q = 0; q < a.chunks; ++q) {
                const uint32_t n = a.plan.counts[(size_t)q * (E + 1) + e];
                before += q < chunk ? n : 0u;
                all += n;
            }
            tot[e] = all;
            cur[e] = before;
        }
    }
    __syncthreads();
    // exclusive scans over the groups: places, and row tiles
    for (int base = 0; base <= E; base += THREADS) {
        const int e = base + tid;
        const uint32_t n = e <= E ? tot[e] : 0u;
        const uint32_t nt = (n + a.tile_rows - 1) / a.tile_rows;
        uint32_t vn = n, vt = nt;
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t un = __shfl_up(vn, off, 64), ut = __shfl_up(vt, off, 64);
            if ((tid & 63) >= off) {
                vn += un;
                vt += ut;
            }
        }
        if ((tid & 63) == 63) {
            wsum[tid >> 6][0] = vn;
            wsum[tid >> 6][1] = vt;
        }
        __syncthreads();
        uint32_t pn = carry[0], pt = carry[1];
        for (int w = 0; w < (tid >> 6); ++w) {
            pn += wsum[w][0];
            pt += wsum[w][1];
        }
        const uint32_t first = pn + vn - n, ftile = pt + vt - nt;
        if (e <= E) {
            cur[e] += first;
            if (chunk == 0) {
                for (uint32_t u = 0; u < nt; ++u)
                    a.plan.tiles[ftile + u] = Mx4Tile{(uint32_t)e, ftile, nt, first, n, {0, 0, 0}};
                if (e == E) *a.plan.total = ftile + nt;
            }
        }
        __syncthreads();
        if (tid == THREADS - 1) {
            carry[0] = pn + vn;
            carry[1] = pt + vt;
        }
        __syncthreads();
    }
    uint32_t at[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c) at[c] = r0 + c * THREADS < a.R ? atomicAdd(&cur[g[c]], 1u) : 0u;
#pragma unroll
    for (int c = 0; c < PER; ++c)
        if (r0 + c * THREADS < a.R) a.plan.perm[at[c]] = (uint32_t)(r0 + c * THREADS);
}

template <int DT, bool STREAM>
__device__ __forceinline__ void activation(const PrepareArgs& a, int64_t wid) {
    const bool live = wid < a.words;                 // whole blocks of 4 lanes are live or not
    const int64_t w0 = live ? wid : 0;
    const int64_t row = a.by_row((uint32_t)w0);
    const uint32_t col = (uint32_t)(w0 - row * a.row_words);
    uint32_t byte, word;
    if (a.swiglu) {
        const int64_t at = (row * a.row_words + w0) * 8;
        const Eight<DT> gate = load8<DT, STREAM>(a.x, at, a.vec),
                         up = load8<DT, STREAM>(a.x, at + (int64_t)a.row_words * 8, a.vec);
        word = mxfp4_word<QLIN_F32>(swiglu8<DT>(gate, up), &byte);
    } else {
        word = mxfp4_word<DT>(load8<DT, STREAM>(a.x, w0 * 8, a.vec), &byte);
    }
    uint8_t* const s = a.xs + row * a.sstride;
    const uint32_t blk = col >> 2;
    if (live) a.xq[wid] = word;
    if (a.row_words % 16 == 0) {
        // 16 lanes hold four blocks of one row: their bytes leave as a dword
        uint32_t four = byte << (8 * (blk & 3));
        four |= dpp_u<0x124>(four);                  // row_ror 4 and 8
        four |= dpp_u<0x128>(four);
        if (live && (threadIdx.x & 15) == 0) *(uint32_t*)(s + blk) = four;
    } else if (live && (threadIdx.x & 3) == 0) {
        s[blk] = (uint8_t)byte;
    }
    if (live && col + 4 == a.row_words)              // the row's last block
        for (int64_t p = blk + 1; p < a.sstride; ++p) s[p] = 127;
}

// One 16-byte unit of a scale row; bytes past the row are 127.
__device__ __forceinline__ void pad_unit(const Mx4Scales& p, const FastDiv& by_unit, int64_t u) {
    const int64_t units = (p.KS + 15) / 16;
    if (u >= p.rows * units) return;
    const int64_t row = by_unit((uint32_t)u);
    const int64_t c = (u - row * units) * 16;
    const uint8_t* const from = p.from + row * p.KS + c;
    uint32_t d[4] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
    if (c + 16 <= p.KS) {
        __builtin_memcpy(d, from, 16);                // rows start at any byte
    } else {
        const int left = (int)(p.KS - c);
#pragma unroll
        for (int b = 0; b < 16; ++b)
            if (b < left) d[b / 4] = (d[b / 4] & ~(0xFFu << (8 * (b & 3)))) | (uint32_t)from[b] << (8 * (b & 3));
    }
    *(uint4*)(p.to + u * 16) = uint4{d[0], d[1], d[2], d[3]};
}

// Workgroups in order: the plan (with several chunks, its counts), the activation, scale rows.
template <int DT, bool STREAM, int PER>
__global__ void __launch_bounds__(THREADS) mx4_prepare_kernel(PrepareArgs a) {
    extern __shared__ uint32_t sh[];
    int b = blockIdx.x;
    if (a.experts) {
        if (b < a.chunks) {
            if (a.chunks == 1) plan_place<PER>(a, 0, sh);
            else plan_count(a, b, sh);
            return;
        }
        b -= a.chunks;
    }
    if (b < a.act_blocks) return activation<DT, STREAM>(a, (int64_t)b * THREADS + threadIdx.x);
    b -= a.act_blocks;
    const int which = b < a.pad_blocks[0] ? 0 : 1;
    if (which) b -= a.pad_blocks[0];
    pad_unit(which ? a.pad[1] : a.pad[0], a.by_unit, (int64_t)b * THREADS + threadIdx.x);
}

__global__ void __launch_bounds__(THREADS) mx4_place_kernel(PrepareArgs a) {
    extern __shared__ uint32_t sh[];
    plan_place<PLAN_PER>(a, blockIdx.x, sh);
}

template <int DT>
auto prepare_kernel(bool stream, bool wide) {
    if (wide) return stream ? mx4_prepare_kernel<DT, true, PLAN_ONE * PLAN_PER> : mx4_prepare_kernel<DT, false, PLAN_ONE * PLAN_PER>;
    return stream ? mx4_prepare_kernel<DT, true, PLAN_PER> : mx4_prepare_kernel<DT, false, PLAN_PER>;
}

// A thread for each group sums its counts over the chunks.
__global__ void __launch_bounds__(THREADS) mx4_scan_kernel(PrepareArgs a) {
    const int e = blockIdx.x * THREADS + threadIdx.x;
    if (e > a.E) return;
    uint32_t sum = 0;
#pragma unroll 8
    for (int q = 0; q < a.chunks; ++q) {
        uint32_t* const at = a.plan.counts + (size_t)q * (a.E + 1) + e;
        const uint32_t n = *at;
        *at = sum;
        sum += n;
    }
    a.plan.counts[(size_t)a.chunks * (a.E + 1) + e] = sum;
}

}  // namespace

size_t mx4_plan_bytes(int64_t R, int64_t E) {
    const int64_t chunks = (R + PLAN_CHUNK - 1) / PLAN_CHUNK;
    return (size_t)(R / kPlanMinTile + E + 1) * sizeof(Mx4Tile) + (size_t)(1 + R + (chunks + 1) * (E + 1)) * sizeof(uint32_t);
}

hipError_t launch_mx4_prepare(const Mx4Prepare& q, Mx4Plan* plan, hipStream_t st) {
    PrepareArgs a{};
    a.row_words = (uint32_t)(q.K / 8);
    a.by_row = FastDiv::by(a.row_words);
    a.swiglu = q.swiglu;
    a.vec = ((uintptr_t)q.x & 15) == 0;              // rows are whole multiples of 64 bytes
    a.sstride = q.sstride;
    const int64_t units = (q.K / 32 + 15) / 16;
    a.by_unit = FastDiv::by((uint32_t)units);
    size_t shm = 0;
    bool wide = false;                               // one chunk of PLAN_ONE
    if (q.experts) {
        const int64_t R = q.R, E = q.E;
        if (R < 1 || R > kMx4MaxRows || E < 1 || E > kMx4MaxExperts || q.tile_rows < kPlanMinTile)
            return hipErrorInvalidValue;
        a.experts = q.experts;
        a.R = (int)R;
        a.E = (int)E;
        wide = R > PLAN_CHUNK && R <= PLAN_ONE * PLAN_CHUNK;
        a.chunks = wide ? 1 : (int)((R + PLAN_CHUNK - 1) / PLAN_CHUNK);
        a.tile_rows = q.tile_rows;
        a.plan.tiles = (Mx4Tile*)q.plan;
        a.plan.total = (uint32_t*)(a.plan.tiles + (R / kPlanMinTile + E + 1));
        a.plan.perm = a.plan.total + 1;
        a.plan.counts = a.plan.perm + R;
        *plan = a.plan;
        shm = (size_t)2 * (E + 1) * sizeof(uint32_t);
    }
    // the first launch takes the plan and up to a part of everything else; few calls have more
    const int64_t part = kLaunchItems / 4;           // items: words, 16-byte units
    const int64_t row_bytes = q.K * (q.swiglu ? 2 : 1) * (q.dt == QLIN_F32 ? 4 : 2);
    int64_t done = 0, padded[2] = {0, 0};            // rows
    for (bool more = true; more;) {
        more = false;
        int64_t blocks = a.chunks;
        // up to `part` items of the rows left: rows of this launch
        auto take = [&](int64_t& at, int64_t rows, int64_t items, int* grid) {
            const int64_t most = part / items, n = rows - at < most ? rows - at : most;
            *grid = (int)((n * items + THREADS - 1) / THREADS);
            blocks += *grid;
            at += n;
            more |= at < rows;
            return n;
        };
        a.x = (const char*)q.x + done * row_bytes;
        a.xq = q.xq + done * a.row_words;
        a.xs = q.xs + done * q.sstride;
        a.words = q.x ? take(done, q.rows, a.row_words, &a.act_blocks) * a.row_words : 0;
        for (int w = 0; w < 2; ++w) {
            if (!q.pad[w].to) continue;
            a.pad[w] = q.pad[w];
            a.pad[w].from += padded[w] * q.pad[w].KS;
            a.pad[w].to += padded[w] * units * 16;
            a.pad[w].rows = take(padded[w], q.pad[w].rows, units, &a.pad_blocks[w]);
        }
        if (blocks) {
            const auto kernel = q.dt == QLIN_F32 ? prepare_kernel<QLIN_F32>(q.stream, wide)
                              : q.dt == QLIN_F16 ? prepare_kernel<QLIN_F16>(q.stream, wide)
                                                 : prepare_kernel<QLIN_BF16>(q.stream, wide);
            kernel<<<(unsigned)blocks, THREADS, shm, st>>>(a);
        }
        if (a.chunks > PLAN_SCAN) {
            mx4_scan_kernel<<<(unsigned)((a.E + THREADS) / THREADS), THREADS, 0, st>>>(a);
            a.scanned = 1;
        }
        if (a.chunks > 1) mx4_place_kernel<<<(unsigned)a.chunks, THREADS, shm, st>>>(a);
        a.experts = nullptr;                         // the plan is on its way
        a.chunks = 0;
    }
    return hipGetLastError();
}

}  // namespace qlin
