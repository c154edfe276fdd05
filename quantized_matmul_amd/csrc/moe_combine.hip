// moe_combine.hip -- joins the experts' rows of each token, and its gradient.
//
//   y[t] = sum_j w[t, j] h[t, j]            h [T, k, D], w [T, k]
//   dh[t, j] = w[t, j] dy[t]
//   dw[t, j] = sum_d dy[t, d] h[t, j, d]
//
// Places whose expert is negative (dropped by the router) are left out: what
// their rows of h hold does not matter (the sum loads them all the same, without
// a branch), dh and dw get zeros. Sums are fp32 in a
// fixed order; each output is rounded once. Both kernels are bound by HBM, and
// by one round trip where there are few tokens: so all rows of a token are on
// their way before any is used. 8192 tokens of 8 rows of 4096 bf16 values: 108
// us (5.6 TB/s), the gradient 191 us (6.0 TB/s); 515 tokens of 6 rows of 2568:
// 5.5 us; one token 2.6 us.

#include "qlin_common.h"
#include "mx4_common.h"

namespace qlin {
namespace {

// VEC elements of dtype DT at element i (16-byte aligned unless VEC is 1).
template <int DT, int VEC>
__device__ __forceinline__ void load_v(const void* p, int64_t i, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = load_f<DT>(p, i);
    } else if constexpr (DT == QLIN_F32) {
        const float4 q = *(const float4*)((const float*)p + i);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
        const uint4 q = *(const uint4*)((const uint16_t*)p + i);
        const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[2 * c] = DT == QLIN_BF16 ? bf16_bits_to_f32(d[c] & 0xFFFFu) : f16_bits_to_f32(d[c] & 0xFFFFu);
            v[2 * c + 1] = DT == QLIN_BF16 ? bf16_bits_to_f32(d[c] >> 16) : f16_bits_to_f32(d[c] >> 16);
        }
    }
}

// The same to memory; STREAM: past the caches.
template <int DT, int VEC, bool STREAM>
__device__ __forceinline__ void store_v(void* p, int64_t i, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        store_f<DT>(p, i, v[0]);
    } else if constexpr (DT == QLIN_F32) {
        typedef __attribute__((ext_vector_type(4))) float f32x4;
        const f32x4 d = {v[0], v[1], v[2], v[3]};
        f32x4* const to = (f32x4*)((float*)p + i);
        if constexpr (STREAM) __builtin_nontemporal_store(d, to);
        else *to = d;
    } else {
        typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
        u32x4 d;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t lo = DT == QLIN_BF16 ? f32_to_bf16_rne(v[2 * c]) : f32_to_f16_rne(v[2 * c]);
            const uint32_t hi = DT == QLIN_BF16 ? f32_to_bf16_rne(v[2 * c + 1]) : f32_to_f16_rne(v[2 * c + 1]);
            d[c] = lo | (hi << 16);
        }
        u32x4* const to = (u32x4*)((uint16_t*)p + i);
        if constexpr (STREAM) __builtin_nontemporal_store(d, to);
        else *to = d;
    }
}

struct CombineArgs {
    const void* h;
    const float* w;
    const int32_t* experts;   // [T, k] or null
    int64_t T, D;
    int k;
    void* y;
    const void* gy;
    void* gh;
    float* gw;
    int64_t first;           // first token (gradient: row) of the launch; the launch ends before `end`
    int64_t end;
    FastDiv by_row;          // thread / threads of a token (gradient: row / k)
};

constexpr int COMBINE_THREADS = 256;

// Each thread owns VEC consecutive outputs of one token and has KC rows of h in
// flight; places past k read the token's first row again and count nothing, so
// that no branch stands between the loads.
template <int DT, int VEC, int KC, bool STREAM>
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(CombineArgs a) {
    const int64_t per = a.D / VEC;
    const uint32_t i = blockIdx.x * COMBINE_THREADS + threadIdx.x, own = a.by_row(i);
    const int64_t t = a.first + own, d = (i - own * per) * VEC;
    if (t >= a.end) return;
    const float* const w = a.w + t * a.k;
    const int32_t* const e = (a.experts ? a.experts : (const int32_t*)a.w) + t * a.k;
    const int64_t h = t * a.k * a.D + d;
    float acc[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] = 0.0f;
    const uint32_t k = (uint32_t)a.k;
    for (uint32_t j0 = 0; j0 < k; j0 += KC) {
        float v[KC][VEC], wj[KC];
        int32_t ej[KC];
#pragma unroll
        for (int q = 0; q < KC; ++q) {
            const uint32_t j = j0 + q < k ? j0 + q : 0;
            load_v<DT, VEC>(a.h, h + (int64_t)j * a.D, v[q]);
            wj[q] = w[j];
            ej[q] = e[j];
        }
#pragma unroll
        for (int q = 0; q < KC; ++q) {
            const bool live = j0 + q < k && (!a.experts || ej[q] >= 0);
            const float f = live ? wj[q] : 0.0f;
#pragma unroll
            for (int c = 0; c < VEC; ++c) acc[c] += f * (live ? v[q][c] : 0.0f);
        }
    }
    store_v<DT, VEC, STREAM>(a.y, t * a.D + d, acc);
}

// One wave per row (t, j).
template <int DT, int VEC, bool STREAM>
__global__ void __launch_bounds__(COMBINE_THREADS) combine_grad_kernel(CombineArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t r = a.first + (int64_t)blockIdx.x * (COMBINE_THREADS / 64) + (threadIdx.x >> 6);
    if (r >= a.end) return;
    const int64_t t = a.by_row((uint32_t)r);      // rows are below 2^31
    const bool dead = a.experts && a.experts[r] < 0;
    const float w = dead ? 0.0f : a.w[r];
    float sum = 0.0f;
    for (int64_t d = (int64_t)lane * VEC; d < a.D; d += 64 * VEC) {
        float g[VEC], v[VEC], o[VEC];
        if (dead) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) o[c] = 0.0f;
        } else {
            load_v<DT, VEC>(a.gy, t * a.D + d, g);
            load_v<DT, VEC>(a.h, r * a.D + d, v);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                sum += g[c] * v[c];
                o[c] = w * g[c];
            }
        }
        store_v<DT, VEC, STREAM>(a.gh, r * a.D + d, o);
    }
    sum = wave_sum(sum);
    if (lane == 0) a.gw[r] = sum;
}

// Whether a call of `rows` rows of D values in all goes past the caches.
bool past_caches(int dt, double rows, int64_t D) { return rows * (double)D * (dt == QLIN_F32 ? 4 : 2) >= (double)kStreamBytes; }

bool wide(int dt, int64_t D, const void* a, const void* b, const void* c) {
    const int64_t per = dt == QLIN_F32 ? 4 : 8;
    return D % per == 0 && (((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) & 15) == 0;
}

template <int DT, int WIDE, bool STREAM>
void run_combine(CombineArgs a, bool vec, hipStream_t st) {
    const int64_t per = vec ? a.D / WIDE : a.D, most = kLaunchItems / per;   // threads of a token; tokens of a launch
    a.by_row = FastDiv::by((uint32_t)per);
    for (a.first = 0; a.first < a.T; a.first = a.end) {
        a.end = a.T - a.first < most ? a.T : a.first + most;
        const unsigned grid = (unsigned)(((a.end - a.first) * per + COMBINE_THREADS - 1) / COMBINE_THREADS);
        if (!vec) combine_kernel<DT, 1, 8, false><<<grid, COMBINE_THREADS, 0, st>>>(a);
        else if (a.k <= 2) combine_kernel<DT, WIDE, 2, STREAM><<<grid, COMBINE_THREADS, 0, st>>>(a);
        else if (a.k <= 4) combine_kernel<DT, WIDE, 4, STREAM><<<grid, COMBINE_THREADS, 0, st>>>(a);
        else if (a.k <= 6) combine_kernel<DT, WIDE, 6, STREAM><<<grid, COMBINE_THREADS, 0, st>>>(a);
        else combine_kernel<DT, WIDE, 8, STREAM><<<grid, COMBINE_THREADS, 0, st>>>(a);
    }
}

template <int DT, int WIDE, bool STREAM>
void run_combine_grad(CombineArgs a, bool vec, hipStream_t st) {
    const int64_t rows = a.T * a.k, most = kLaunchItems / 64;
    a.by_row = FastDiv::by((uint32_t)a.k);
    for (a.first = 0; a.first < rows; a.first = a.end) {
        a.end = rows - a.first < most ? rows : a.first + most;
        const unsigned grid = (unsigned)((a.end - a.first + COMBINE_THREADS / 64 - 1) / (COMBINE_THREADS / 64));
        if (vec) combine_grad_kernel<DT, WIDE, STREAM><<<grid, COMBINE_THREADS, 0, st>>>(a);
        else combine_grad_kernel<DT, 1, false><<<grid, COMBINE_THREADS, 0, st>>>(a);
    }
}

template <int DT, int WIDE, bool STREAM>
void run(const CombineArgs& a, bool vec, hipStream_t st, bool grad) {
    if (grad) run_combine_grad<DT, WIDE, STREAM>(a, vec, st);
    else run_combine<DT, WIDE, STREAM>(a, vec, st);
}
template <bool STREAM>
void by_type(int dt, const CombineArgs& a, bool vec, hipStream_t st, bool grad) {
    if (dt == QLIN_F32) run<QLIN_F32, 4, STREAM>(a, vec, st, grad);
    else if (dt == QLIN_BF16) run<QLIN_BF16, 8, STREAM>(a, vec, st, grad);
    else run<QLIN_F16, 8, STREAM>(a, vec, st, grad);
}

}  // namespace

hipError_t launch_moe_combine(const void* h, int dt, int64_t T, int k, int64_t D, const float* weights,
                              const int32_t* experts, void* y, hipStream_t st) {
    CombineArgs a{};
    a.h = h; a.w = weights; a.experts = experts; a.T = T; a.D = D; a.k = k; a.y = y;
    const bool vec = wide(dt, D, h, y, nullptr);
    if (past_caches(dt, (double)T * (k + 1.0), D)) by_type<true>(dt, a, vec, st, false);
    else by_type<false>(dt, a, vec, st, false);
    return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const void* gy, const void* h, int dt, int64_t T, int k, int64_t D,
                                   const float* weights, const int32_t* experts, void* gh, float* gw,
                                   hipStream_t st) {
    CombineArgs a{};
    a.h = h; a.w = weights; a.experts = experts; a.T = T; a.D = D; a.k = k; a.gy = gy; a.gh = gh; a.gw = gw;
    const bool vec = wide(dt, D, h, gy, gh);
    if (past_caches(dt, (double)T * (2.0 * k + 1.0), D)) by_type<true>(dt, a, vec, st, true);
    else by_type<false>(dt, a, vec, st, true);
    return hipGetLastError();
}

}  // namespace qlin
