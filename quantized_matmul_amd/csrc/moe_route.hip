// moe_route.hip -- routing tokens to experts, and the gradient of the logits.
//
// For a token's logits x[0..E):
//   score  s = softmax(x) or 1 / (1 + exp(-x)), over the finite logits;
//   key    x itself without a balance bias (the order of s, with no rounding
//          between them), s + b with one;
//   groups E split into G runs of E/G experts; a group's key is its largest
//          key (score with group_top 1) or the sum of its two largest
//          s (+ b); the `kept` best groups stay in the choice;
//   choice the k largest keys, descending, equal keys by ascending index;
//   weight w_i = c s_i, or c s_i / (sum_chosen s + 1e-20).
// An expert whose logit is not finite (or whose key is NaN) cannot be chosen;
// places that stay empty get expert -1 and weight 0.
//
// Gradient for g = dL/dw, S = the renormalizing sum:
//   ds_i = c g_i, or (c g_i - sum_j g_j w_j) / S;
//   sigmoid  dx_i = ds_i s_i (1 - s_i), with 1 - s_i = 1 / (1 + exp(x_i));
//   softmax  dx_j = s_j (ds_j - sum_i ds_i s_i); with renormalization the sum
//            is exactly 0 (w does not change when every logit of the choice
//            moves together), so only the chosen logits get a gradient.
//
// One wave per token, four tokens per workgroup. Lane l holds experts
// l V .. l V + V - 1 (V = 1, 2, 4, 8 or 16), so that a ballot of equal keys
// orders them by index. Everything is fp32.

#include "qlin_common.h"
#include "moe_common.h"

#include <cmath>

namespace qlin {
namespace {

constexpr int ROUTE_WAVES = 4;

struct RouteArgs {
    const void* logits;
    const float* bias;       // [E] or null
    int64_t T;
    int E, k;
    int sigmoid, renorm;
    int groups, kept, group_top;
    float scale;
    float* weights;          // [T, k]
    int32_t* experts;        // [T, k]
};

// The lane's V logits; experts past E and logits that are not finite are -inf.
template <int DT, int V>
__device__ __forceinline__ void load_logits(const void* p, int64_t base, int e0, int E, float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = e0 + v;
        const float f = e < E ? load_f<DT>(p, base + e) : -INFINITY;
        x[v] = isfinite(f) ? f : -INFINITY;
    }
}

// Scores of the lane's logits (0 where the logit is -inf).
template <int V>
__device__ __forceinline__ void scores_of(const float (&x)[V], int sigmoid, float (&s)[V]) {
    if (sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = x[v] == -INFINITY ? 0.0f : 1.0f / (1.0f + expf(-x[v]));
        return;
    }
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = wave_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[v] = x[v] == -INFINITY ? 0.0f : expf(x[v] - m);
        sum += s[v];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = sum > 0.0f ? s[v] / sum : 0.0f;
}

template <int DT, int V>
__global__ void __launch_bounds__(64 * ROUTE_WAVES) route_kernel(RouteArgs a) {
    extern __shared__ float lds[];               // [waves][E], only with groups
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + wv;
    const bool live = t < a.T;                   // the other waves only keep the barrier company
    const int e0 = lane * V;
    float x[V], s[V], key[V];
    load_logits<DT, V>(a.logits, (live ? t : 0) * a.E, e0, a.E, x);
    scores_of<V>(x, a.sigmoid, s);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        key[v] = x[v];
        if (a.bias && x[v] != -INFINITY) {
            const float b = s[v] + a.bias[e0 + v];
            key[v] = b == b ? b : -INFINITY;
        }
    }
    if (a.kept < a.groups) {
        float* const row = lds + wv * a.E;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e0 + v < a.E) row[e0 + v] = x[v] == -INFINITY ? -INFINITY : (a.bias ? key[v] : s[v]);
        __syncthreads();
        const int per = a.E / a.groups;
        float g = -INFINITY;
        if (lane < a.groups) {
            float m1 = -INFINITY, m2 = -INFINITY;
            for (int e = 0; e < per; ++e) {
                const float f = row[lane * per + e];
                m2 = fmaxf(m2, fminf(m1, f));
                m1 = fmaxf(m1, f);
            }
            g = a.group_top == 2 ? m1 + m2 : m1;
        }
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
            const float f = lane_value(g, o);
            rank += (f > g || (f == g && o < lane)) ? 1 : 0;
        }
        const uint64_t keep = __ballot(lane < a.groups && rank < a.kept);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int gr = (e0 + v) / per;
            if (gr >= a.groups || !((keep >> gr) & 1)) key[v] = -INFINITY;
        }
    }
    // k rounds: the wave's largest key, its lowest index
    float my_s = 0.0f;
    int my_e = -1;
    for (int j = 0; j < a.k; ++j) {
        float b = key[0], bs = s[0];
        int bv = 0;
#pragma unroll
        for (int v = 1; v < V; ++v)
            if (key[v] > b) {
                b = key[v];
                bs = s[v];
                bv = v;
            }
        const float top = wave_max(b);
        if (top == -INFINITY) break;
        const int win = __builtin_ctzll(__ballot(b == top));
        const float ws = lane_value(bs, win);
        const int we = lane_value(bv, win) + win * V;
        if (lane == j) {
            my_s = ws;
            my_e = we;
        }
        if (lane == win) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v == bv) key[v] = -INFINITY;
        }
    }
    float w = a.scale * my_s;
    if (a.renorm) w = w / (wave_sum(my_s) + 1e-20f);
    if (live && lane < a.k) {
        a.weights[t * a.k + lane] = w;
        a.experts[t * a.k + lane] = my_e;
    }
}

struct RouteGradArgs {
    const void* logits;
    const int32_t* experts;
    const float* grad_w;
    int64_t T;
    int E, k;
    int sigmoid, renorm;
    float scale;
    void* grad;              // [T, E], the logits' dtype
};

template <int DT, int V>
__global__ void __launch_bounds__(64 * ROUTE_WAVES) route_grad_kernel(RouteGradArgs a) {
    extern __shared__ float lds[];               // [waves][2][E]: scores, then ds of the chosen
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + wv;
    const bool live = t < a.T;
    const int e0 = lane * V;
    float* const srow = lds + wv * 2 * a.E;
    float* const drow = srow + a.E;
    float x[V], s[V];
    load_logits<DT, V>(a.logits, (live ? t : 0) * a.E, e0, a.E, x);
    scores_of<V>(x, a.sigmoid, s);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (e0 + v < a.E) {
            srow[e0 + v] = s[v];
            drow[e0 + v] = 0.0f;
        }
    __syncthreads();
    int id = -1;
    float g = 0.0f, sc = 0.0f;
    if (live && lane < a.k) {
        id = a.experts[t * a.k + lane];
        if (id < 0 || id >= a.E) id = -1;
        if (id >= 0) {
            g = a.grad_w[t * a.k + lane];
            sc = srow[id];
        }
    }
    float ds = a.scale * g;
    if (a.renorm) {
        const float total = wave_sum(sc) + 1e-20f;
        ds = (a.scale * g - wave_sum(g * (a.scale * sc / total))) / total;
    }
    const float dot = (!a.sigmoid && !a.renorm) ? wave_sum(ds * sc) : 0.0f;
    if (id >= 0) drow[id] = ds;
    __syncthreads();
    if (!live) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (e0 + v >= a.E) continue;
        const float d = drow[e0 + v];
        float r;
        if (a.sigmoid) r = d == 0.0f ? 0.0f : d * s[v] * (1.0f / (1.0f + expf(x[v])));
        else r = s[v] * (d - dot);
        if (x[v] == -INFINITY) r = 0.0f;
        store_f<DT>(a.grad, t * a.E + e0 + v, r);
    }
}

template <int DT, int V>
struct Route {
    static void run(const RouteArgs& a, unsigned grid, size_t shm, hipStream_t st) {
        route_kernel<DT, V><<<grid, 64 * ROUTE_WAVES, shm, st>>>(a);
    }
};
template <int DT, int V>
struct RouteGrad {
    static void run(const RouteGradArgs& a, unsigned grid, size_t shm, hipStream_t st) {
        route_grad_kernel<DT, V><<<grid, 64 * ROUTE_WAVES, shm, st>>>(a);
    }
};

template <template <int, int> class F, int DT, typename A>
void by_width(int E, const A& a, unsigned grid, size_t shm, hipStream_t st) {
    if (E <= 64) F<DT, 1>::run(a, grid, shm, st);
    else if (E <= 128) F<DT, 2>::run(a, grid, shm, st);
    else if (E <= 256) F<DT, 4>::run(a, grid, shm, st);
    else if (E <= 512) F<DT, 8>::run(a, grid, shm, st);
    else F<DT, 16>::run(a, grid, shm, st);
}

template <template <int, int> class F, typename A>
hipError_t by_type(int dt, int E, const A& a, size_t shm, hipStream_t st) {
    const unsigned grid = (unsigned)((a.T + ROUTE_WAVES - 1) / ROUTE_WAVES);
    if (dt == QLIN_F32) by_width<F, QLIN_F32>(E, a, grid, shm, st);
    else if (dt == QLIN_BF16) by_width<F, QLIN_BF16>(E, a, grid, shm, st);
    else by_width<F, QLIN_F16>(E, a, grid, shm, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const void* logits, int dt, int64_t T, int E, int k, const float* bias,
                            int sigmoid, int renorm, float scale, int groups, int kept, int group_top,
                            float* weights, int32_t* experts, hipStream_t st) {
    const RouteArgs a{logits, bias, T, E, k, sigmoid, renorm, groups, kept, group_top, scale, weights, experts};
    const size_t shm = kept < groups ? (size_t)ROUTE_WAVES * E * sizeof(float) : 0;
    return by_type<Route>(dt, E, a, shm, st);
}

hipError_t launch_moe_route_grad(const void* logits, int dt, int64_t T, int E, int k, const int32_t* experts,
                                 const float* grad_w, int sigmoid, int renorm, float scale, void* grad,
                                 hipStream_t st) {
    const RouteGradArgs a{logits, experts, grad_w, T, E, k, sigmoid, renorm, scale, grad};
    return by_type<RouteGrad>(dt, E, a, (size_t)ROUTE_WAVES * 2 * E * sizeof(float), st);
}

}  // namespace qlin
