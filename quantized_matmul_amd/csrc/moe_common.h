// moe_common.h -- wave-wide helpers and launcher declarations of the
// mixture-of-experts operators (routing, mxfp4 products, combine).
#pragma once

#include "qlin_common.h"

namespace qlin {

// One step of a wave reduction over DPP lanes: lanes without a source keep
// `id`. row_shr 1, 2, 4, 8 reduce each row of 16 into its last lane; row_bcast
// 15 and 31 carry rows into the next ones; lane 63 then holds the result.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float id, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(id), __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// Value of v in a lane every lane names (wave-uniform result).
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Largest v of the wave's 64 lanes, all active (0 is the identity, so each
// step is one instruction).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t min_u(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_u(v, dpp_u<0x111>(v));
    v = max_u(v, dpp_u<0x112>(v));
    v = max_u(v, dpp_u<0x114>(v));
    v = max_u(v, dpp_u<0x118>(v));
    v = max_u(v, dpp_u<0x142>(v));
    v = max_u(v, dpp_u<0x143>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Sum of v over the wave's 64 lanes, all active, in one fixed order. Only lane
// 63 ends with the whole sum: row_bcast 15 gives it rows 2 + 3 and lane 31
// rows 0 + 1, which row_bcast 31 adds.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f<0x111>(0.0f, v);
    v += dpp_f<0x112>(0.0f, v);
    v += dpp_f<0x114>(0.0f, v);
    v += dpp_f<0x118>(0.0f, v);
    v += dpp_f<0x142>(0.0f, v);
    v += dpp_f<0x143>(0.0f, v);
    return lane_value(v, 63);
}

// Largest expert count and choice of the router: 64 lanes of 16 experts, one
// lane per place.
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxChoice = 64;
constexpr int kRouteMaxGroups = 64;

// An operator that touches this much and more reads and writes what it touches
// once past the caches (non-temporal loads and stores): three quarters of the
// 256 MB in front of the memory, which then keep what is read again. Outputs of
// smaller calls are better left there. Measured (us, through the caches and
// past them): 8192 bf16 rows, N 12288, K 4096 250 and 231; 65536 rows of 8 of 64
// experts, N 1536, K 2048 184 and 162; 4096 fp32 rows, N 8192, K 2048, 147 MB
// in all: 56 and 63.
constexpr int64_t kStreamBytes = 192LL << 20;

// Work-items of one launch at most: a launch of 2^32 or more loses those beyond
// a multiple of it without an error, so larger work takes several launches.
constexpr int64_t kLaunchItems = 1LL << 31;

hipError_t launch_moe_route(const void* logits, int dt, int64_t T, int E, int k, const float* bias,
                            int sigmoid, int renorm, float scale, int groups, int kept, int group_top,
                            float* weights, int32_t* experts, hipStream_t st);
hipError_t launch_moe_route_grad(const void* logits, int dt, int64_t T, int E, int k, const int32_t* experts,
                                 const float* grad_w, int sigmoid, int renorm, float scale, void* grad,
                                 hipStream_t st);

hipError_t launch_moe_combine(const void* h, int dt, int64_t T, int k, int64_t D, const float* weights,
                              const int32_t* experts, void* y, hipStream_t st);
hipError_t launch_moe_combine_grad(const void* gy, const void* h, int dt, int64_t T, int k, int64_t D,
                                   const float* weights, const int32_t* experts, void* gh, float* gw,
                                   hipStream_t st);

// Product of two mxfp4 operands; gather form with experts != null.
struct Mx4Args {
    const uint8_t* xq;        // codes [B, K/2 bytes]
    const uint8_t* xs;        // scale rows, xsstride bytes apart
    const uint8_t* wq;        // codes [E, N, K/2 bytes]
    const uint8_t* ws;        // scale rows [E, N], wsstride bytes apart
    void* y;                  // [M, N] (gather: [R, N])
    int64_t M, N, K;          // gather: M = R
    int64_t xsstride, wsstride;
    int ydt;
    int stream;               // y goes past the caches
    // a float x, quantized inside the kernel (streaming kernel, few rows)
    const void* x;
    int xdt, swiglu;
    // gather form
    const int32_t* experts;   // [R] or null
    int64_t B, E;             // row r reads x row r / (R / B)
};

// How a product runs.
enum class Mx4Path {
    kStreamFloat,             // streaming kernel, x quantized inside it
    kStream,                  // streaming kernel on x's codes
    kTiled                    // tiled kernel on x's codes; reads scale rows in 16-byte units
};
struct Mx4Choice {
    Mx4Path path;
    int tile;                 // kTiled: index of the tile's shape
    int tile_rows;            // its rows
};
bool mx4_fits(int64_t M, int64_t N, int64_t K, int64_t E, bool gather, const Mx4Choice& c);   // one launch holds it
Mx4Choice mx4_choose(int64_t M, int64_t N, int64_t K, int64_t E, bool gather, bool codes);
hipError_t launch_mx4_matmul(const Mx4Args& a, const Mx4Choice& c, const struct Mx4Plan* plan, hipStream_t st);

// Scale rows of KS bytes to copy to rows of whole 16-byte units, filled with 127.
struct Mx4Scales {
    const uint8_t* from;
    int64_t rows, KS;
    uint8_t* to;              // null: none
};

// x's codes and scale rows `sstride` bytes apart (bytes past K / 32 get 127) from a
// float x [rows, K] (swiglu: [rows, 2K]), unless x is null; the row plan for
// R experts, unless experts is null; scale rows to lay out.
struct Mx4Prepare {
    const void* x;
    int dt;
    int64_t rows, K;
    int swiglu;
    int stream;               // x goes past the caches
    uint32_t* xq;
    uint8_t* xs;
    int64_t sstride;
    const int32_t* experts;
    int64_t R, E;
    int tile_rows;
    void* plan;               // mx4_plan_bytes(R, E)
    Mx4Scales pad[2];
};
size_t mx4_plan_bytes(int64_t R, int64_t E);
hipError_t launch_mx4_prepare(const Mx4Prepare& q, struct Mx4Plan* plan, hipStream_t st);

}  // namespace qlin
