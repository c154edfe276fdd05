// mx4_plan.hip -- the row plan of the mxfp4 product by experts: index rows
// grouped by expert and cut into row tiles, made on the device.
//
// Rows whose expert is outside [0, E) form one more group, E, whose tiles
// write zeros. The order of rows inside a group is free: each output row
// depends on its own inputs only.
//
// Two launches for many rows (counts per chunk of rows; then each chunk scans
// the counts for its own places), one where a single chunk holds all rows.
// Both are latency-bound: a few barriers and memory round trips.

#include "mx4_plan.h"

namespace qlin {
namespace {

constexpr int PLAN_THREADS = 256;
constexpr int PLAN_CHUNK = 4096;                         // rows per workgroup
constexpr int PLAN_PER = PLAN_CHUNK / PLAN_THREADS;

__device__ __forceinline__ uint32_t group_of(int32_t e, uint32_t E) { return (uint32_t)e < E ? (uint32_t)e : E; }

__global__ void __launch_bounds__(PLAN_THREADS) plan_count_kernel(const int32_t* __restrict__ experts, int R, int E,
                                                                  uint32_t* __restrict__ counts) {
    extern __shared__ uint32_t cnt[];                    // [E + 1]
    for (int e = threadIdx.x; e <= E; e += PLAN_THREADS) cnt[e] = 0;
    __syncthreads();
    const int r0 = blockIdx.x * PLAN_CHUNK;
#pragma unroll
    for (int c = 0; c < PLAN_PER; ++c) {
        const int r = r0 + c * PLAN_THREADS + threadIdx.x;
        if (r < R) atomicAdd(&cnt[group_of(experts[r], E)], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += PLAN_THREADS) counts[(size_t)blockIdx.x * (E + 1) + e] = cnt[e];
}

// chunks == 1: counts its rows itself and reads no counts.
__global__ void __launch_bounds__(PLAN_THREADS) plan_place_kernel(const int32_t* __restrict__ experts, int R, int E,
                                                                  int chunks, int tile_rows,
                                                                  const uint32_t* __restrict__ counts, Mx4Plan p) {
    extern __shared__ uint32_t sh[];
    uint32_t* const tot = sh;                            // [E + 1] rows of the group
    uint32_t* const cur = sh + E + 1;                    // [E + 1] next place of this chunk's rows
    __shared__ uint32_t wsum[PLAN_THREADS / 64][2], carry[2];
    const int tid = threadIdx.x, chunk = blockIdx.x;
    const int r0 = chunk * PLAN_CHUNK;
    if (tid < 2) carry[tid] = 0;
    uint32_t g[PLAN_PER];
#pragma unroll
    for (int c = 0; c < PLAN_PER; ++c) {
        const int r = r0 + c * PLAN_THREADS + tid;
        g[c] = r < R ? group_of(experts[r], E) : 0u;
    }
    if (chunks == 1) {
        for (int e = tid; e <= E; e += PLAN_THREADS) tot[e] = cur[e] = 0;
        __syncthreads();
#pragma unroll
        for (int c = 0; c < PLAN_PER; ++c)
            if (r0 + c * PLAN_THREADS + tid < R) atomicAdd(&tot[g[c]], 1u);
    } else {
        for (int e = tid; e <= E; e += PLAN_THREADS) {
            uint32_t all = 0, before = 0;
            for (int q = 0; q < chunks; ++q) {
                const uint32_t n = counts[(size_t)q * (E + 1) + e];
                if (q < chunk) before += n;
                all += n;
            }
            tot[e] = all;
            cur[e] = before;
        }
    }
    __syncthreads();
    // exclusive scans over the groups: places, and row tiles
    for (int base = 0; base <= E; base += PLAN_THREADS) {
        const int e = base + tid;
        const uint32_t n = e <= E ? tot[e] : 0u;
        const uint32_t nt = (n + tile_rows - 1) / tile_rows;
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
                p.offsets[e] = first;
                p.first_tile[e] = ftile;
                for (uint32_t u = 0; u < nt; ++u) p.tile_group[ftile + u] = (uint32_t)e;
                if (e == E) {
                    p.offsets[E + 1] = first + n;
                    p.first_tile[E + 1] = ftile + nt;
                }
            }
        }
        __syncthreads();
        if (tid == PLAN_THREADS - 1) {
            carry[0] = pn + vn;
            carry[1] = pt + vt;
        }
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < PLAN_PER; ++c) {
        const int r = r0 + c * PLAN_THREADS + tid;
        if (r < R) p.perm[atomicAdd(&cur[g[c]], 1u)] = (uint32_t)r;
    }
}

}  // namespace

size_t mx4_plan_bytes(int64_t R, int64_t E) {
    const int64_t chunks = (R + PLAN_CHUNK - 1) / PLAN_CHUNK;
    // offsets, first tiles, tile groups (tiles of 16 rows or more), perm, counts
    const int64_t words = 2 * (E + 2) + (R / 16 + E + 1) + R + chunks * (E + 1);
    return (size_t)words * sizeof(uint32_t);
}

hipError_t launch_mx4_plan(const int32_t* experts, int64_t R, int64_t E, int tile_rows, void* workspace, Mx4Plan* out,
                           hipStream_t st) {
    if (tile_rows < 16 || R < 1 || R >= (1LL << 31) || E < 1 || E > kMx4MaxExperts) return hipErrorInvalidValue;
    const int chunks = (int)((R + PLAN_CHUNK - 1) / PLAN_CHUNK);
    uint32_t* w = (uint32_t*)workspace;
    Mx4Plan p{};
    p.offsets = w;
    p.first_tile = p.offsets + (E + 2);
    p.tile_group = p.first_tile + (E + 2);
    p.perm = p.tile_group + (R / 16 + E + 1);
    uint32_t* const counts = p.perm + R;
    const size_t shm = (size_t)(E + 1) * sizeof(uint32_t);
    if (chunks > 1) plan_count_kernel<<<chunks, PLAN_THREADS, shm, st>>>(experts, (int)R, (int)E, counts);
    plan_place_kernel<<<chunks, PLAN_THREADS, 2 * shm, st>>>(experts, (int)R, (int)E, chunks, tile_rows, counts, p);
    *out = p;
    return hipGetLastError();
}

}  // namespace qlin
