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
// An expert whose logit is not finite (or whose key is NaN or -inf) cannot be
// chosen; places that stay empty get expert -1 and weight 0.
//
// Gradient for g = dL/dw, S = the renormalizing sum:
//   ds_i = c g_i, or (c g_i - sum_j g_j w_j) / S, taken as
//          c (sum_j (g_i - g_j) s_j + 1e-20 g_i) / S^2;
//   sigmoid  dx_i = ds_i s_i (1 - s_i), with 1 - s_i = 1 / (1 + exp(x_i));
//   softmax  dx_j = s_j (ds_j - sum_i ds_i s_i); with renormalization the sum
//            is c 1e-20 (sum_i g_i s_i) / S^2: nothing in fp32, and no gradient
//            outside the choice, unless the chosen scores sum to about 1e-20.
//
// A token takes L lanes, 16 (a DPP row, four tokens a wave) up to 256 experts
// and a wave beyond; lane l holds experts l V .. l V + V - 1 (V = 1, 2, 4, 8
// or 16), so that the first of the lanes with equal keys has the lowest index.
// A lane sorts its keys once, then each of k rounds takes the largest head of
// the lanes: at 16384 tokens of 256 experts in groups 28 us with a wave a token
// and k passes over all values, 11.2 so. Everything is fp32.
// Bound by instructions there (1000 for four tokens; its bytes would take 3.7
// us), by the launch for few tokens (one token 2.7 us; 8191 of 60 experts 3.8).

#include "qlin_common.h"
#include "moe_common.h"

#include <cmath>

namespace qlin {
namespace {

constexpr int ROUTE_WAVES = 4;
constexpr int64_t ROUTE_TOKENS = kLaunchItems / 64;   // tokens of a launch, a wave each at most

struct RouteArgs {
    const void* logits;
    const float* bias;       // [E] or null
    int64_t T;
    int E, k;
    int sigmoid, renorm;
    int groups, kept, group_top;
    int seg;                 // lanes of a group where that is a power of two of whole lanes, else 0
    int vec;                 // rows can be loaded V elements at a time
    float scale;
    float* weights;          // [T, k]
    int32_t* experts;        // [T, k]
};

// exp(x) for x <= 0 within 2 ulp: 2^(x log2 e), with what the product's
// rounding lost put back to first order. Results below 2^-126 (x < -87.34) are
// 0, as the hardware's 2^x gives no subnormal numbers; the argument is held at
// -104 (-inf and NaN too).
__device__ __forceinline__ float exp_of(float x) {
    const float hi = 0x1.715476p+0f, lo = 0x1.4ae0cp-26f;   // log2 e = hi + lo
    x = fmaxf(x, -104.0f);
    const float t = x * hi;
    const float e = __builtin_amdgcn_exp2f(t);
    const float d = __builtin_fmaf(x, hi, -t) + x * lo;     // |d| < 2^-16: 2^d = 1 + d ln 2
    return __builtin_fmaf(e, d * 0x1.62e43p-1f, e);
}

// 1 / (1 + exp(-x)) from e = exp(-|x|): 1 / (1 + e), or e / (1 + e) for
// negative x (0 for -inf). The reciprocal is the hardware's estimate and one
// step of Newton's iteration.
__device__ __forceinline__ float sigmoid_of(float x) {
    const float e = exp_of(-fabsf(x)), d = 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
    return x >= 0.0f ? r : e * r;
}

__device__ __forceinline__ float finite_or_none(float f) {
    return fabsf(f) < INFINITY ? f : -INFINITY;   // NaN fails the comparison too
}

// The lane's V values of a row of E; values past E, and with FINITE those that are not finite, are -inf.
template <int DT, int V, bool FINITE = true>
__device__ __forceinline__ void load_logits(const void* p, int64_t base, int e0, int E, int vec, float (&x)[V]) {
    constexpr int SIZE = DT == QLIN_F32 ? 4 : 2, BYTES = V * SIZE;
    if (V > 1 && vec) {
        struct __attribute__((aligned(BYTES < 16 ? BYTES : 16))) Raw {
            uint32_t d[BYTES < 4 ? 1 : BYTES / 4];
        } raw;
        if (e0 < E) raw = *(const Raw*)((const char*)p + (base + e0) * SIZE);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f;
            if constexpr (DT == QLIN_F32) f = __uint_as_float(raw.d[v]);
            else {
                const uint32_t h = (raw.d[v / 2] >> (16 * (v & 1))) & 0xFFFFu;
                f = DT == QLIN_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
            }
            x[v] = e0 < E ? (FINITE ? finite_or_none(f) : f) : -INFINITY;
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = e0 + v;
        const float f = load_f<DT>(p, base + (e < E ? e : E - 1));   // no branch between the loads
        x[v] = e < E ? (FINITE ? finite_or_none(f) : f) : -INFINITY;
    }
}

// exp of the lane's logits against the row's largest (0 for -inf, also where no logit is finite) and
// their sum over the wave.
template <int V>
__device__ __forceinline__ float softmax_terms(const float (&x)[V], float top, float (&s)[V]) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[v] = exp_of(x[v] - top);
        sum += s[v];
    }
    return wave_sum(sum);
}

// Floats as unsigned numbers of the same order, so that a step of a maximum
// over lanes is one instruction: 0 below every number, for "none"; -0 counts
// as +0.
__device__ __forceinline__ uint32_t order_of_sum(float f) {   // f is not -0
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t order_of(float f) { return order_of_sum(f + 0.0f); }
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o ^ ((uint32_t)(~(int32_t)o >> 31) | 0x80000000u));
}
constexpr uint32_t NONE = 0;            // below order_of(-inf)

template <int V>
__device__ __forceinline__ uint32_t largest(const uint32_t (&x)[V]) {
    uint32_t m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = max_u(m, x[v]);
    return m;
}

template <int V>
__device__ __forceinline__ float row_max(const float (&x)[V]) {
    uint32_t o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = order_of(x[v]);
    return value_of(wave_max(largest<V>(o)));
}

// (m1, m2) the two largest of themselves and x.
__device__ __forceinline__ void insert2(uint32_t& m1, uint32_t& m2, uint32_t x) {
    m2 = max_u(min_u(m1, m2), min_u(max_u(m1, m2), x));    // the median: one instruction
    m1 = max_u(m1, x);
}

// (m1, m2) the two largest of the lane's and a partner's two largest.
__device__ __forceinline__ void merge2(uint32_t& m1, uint32_t& m2, uint32_t p1, uint32_t p2) {
    m2 = max_u(min_u(m1, p1), max_u(m2, p2));
    m1 = max_u(m1, p1);
}

// What a token's L lanes know together. Every lane gets the result; `row` is the lane's place among
// the L.
template <int L>
struct Lanes;

template <>
struct Lanes<64> {
    __device__ static uint32_t max_all(uint32_t v) { return wave_max(v); }
    __device__ static float sum_all(float v) { return wave_sum(v); }
    // first of the token's lanes for which p holds (one does)
    __device__ static int first(bool p, int lane) { return __builtin_ctzll(__ballot(p)); }
};

template <>
struct Lanes<16> {
    // rotations inside the row of 16: each step joins two sets of lanes whose results agree
    __device__ static uint32_t max_all(uint32_t v) {
        v = max_u(v, dpp_u<0x128>(v));
        v = max_u(v, dpp_u<0x124>(v));
        v = max_u(v, dpp_u<0x122>(v));
        return max_u(v, dpp_u<0x121>(v));
    }
    __device__ static float sum_all(float v) {
        v += dpp_f<0x128>(0.0f, v);
        v += dpp_f<0x124>(0.0f, v);
        v += dpp_f<0x122>(0.0f, v);
        return v + dpp_f<0x121>(0.0f, v);
    }
    __device__ static int first(bool p, int lane) {
        const uint64_t m = __ballot(p);
        const uint32_t half = lane & 32 ? (uint32_t)(m >> 32) : (uint32_t)m;
        return __builtin_ctz((half >> (lane & 16)) | 0x10000u) & 15;
    }
};

// A group's key from its two largest: -inf where it has fewer experts to choose from than count.
__device__ __forceinline__ uint32_t group_key(const RouteArgs& a, uint32_t m1, uint32_t m2) {
    if (a.group_top == 1) return m1 == NONE ? order_of(-INFINITY) : m1;
    return order_of(m2 == NONE ? -INFINITY : value_of(m1) + value_of(m2));
}

// Whether the lane's group is among the `kept` best, for groups of a.seg whole
// lanes. f holds the lane's V values.
template <int L, int V>
__device__ __forceinline__ bool in_best_groups(const RouteArgs& a, const uint32_t (&f)[V], int lane) {
    uint32_t m1 = NONE, m2 = NONE;
    // join the lanes' two largest over DPP inside rows of 16 lanes (each step
    // joins two blocks that already agree), by shuffles beyond
#pragma unroll
    for (int v = 0; v < V; ++v) insert2(m1, m2, f[v]);
    if (a.seg > 1) merge2(m1, m2, dpp_u<0xB1>(m1), dpp_u<0xB1>(m2));      // quad_perm 1 0 3 2
    if (a.seg > 2) merge2(m1, m2, dpp_u<0x4E>(m1), dpp_u<0x4E>(m2));      // quad_perm 2 3 0 1
    if (a.seg > 4) merge2(m1, m2, dpp_u<0x141>(m1), dpp_u<0x141>(m2));    // row_half_mirror
    if (a.seg > 8) merge2(m1, m2, dpp_u<0x140>(m1), dpp_u<0x140>(m2));    // row_mirror
    if constexpr (L == 64) {
        if (a.seg > 16) merge2(m1, m2, (uint32_t)__shfl_xor((int)m1, 16, 64), (uint32_t)__shfl_xor((int)m2, 16, 64));
        if (a.seg > 32) merge2(m1, m2, (uint32_t)__shfl_xor((int)m1, 32, 64), (uint32_t)__shfl_xor((int)m2, 32, 64));
    }
    const int row = lane & (L - 1);
    uint32_t g = row < a.groups * a.seg ? group_key(a, m1, m2) : NONE;
    bool in = false;
    for (int r = 0; r < a.kept; ++r) {
        const int win = Lanes<L>::first(g == Lanes<L>::max_all(g), lane);      // the first lane of its group
        const bool mine = (uint32_t)(row - win) < (uint32_t)a.seg;
        in |= mine;
        g = mine ? NONE : g;
    }
    return in && row < a.groups * a.seg;
}

// Bits of the `kept` best groups where they are not whole lanes: through LDS,
// one lane of the wave per group.
template <int V>
__device__ __forceinline__ uint64_t best_groups(const RouteArgs& a, const uint32_t (&f)[V], int lane, uint32_t* row) {
    const int per = a.E / a.groups;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (lane * V + v < a.E) row[lane * V + v] = f[v];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    uint32_t m1 = NONE, m2 = NONE, g = NONE;
    if (lane < a.groups) {
        for (int e = 0; e < per; ++e) insert2(m1, m2, row[lane * per + e]);
        g = group_key(a, m1, m2);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    uint64_t in = 0;
    for (int r = 0; r < a.kept; ++r) {
        const int win = __builtin_ctzll(__ballot(g == wave_max(g)));
        in |= 1ull << win;
        g = lane == win ? NONE : g;
    }
    return in;
}

// Batcher's odd-even merge sort of n = 2^i values as a list of comparisons.
struct Sorter {
    int n;
    uint8_t a[64], b[64];
};
constexpr Sorter sorter(int n) {
    Sorter s{0, {}, {}};
    for (int p = 1; p < n; p *= 2)
        for (int k = p; k >= 1; k /= 2)
            for (int j = k % p; j + k < n; j += 2 * k)
                for (int i = 0; i < k && i + j + k < n; ++i)
                    if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        s.a[s.n] = (uint8_t)(i + j);
                        s.b[s.n] = (uint8_t)(i + j + k);
                        ++s.n;
                    }
    return s;
}

// Larger and smaller of two finite numbers, one instruction each.
__device__ __forceinline__ double max_f64(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double min_f64(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// LDS of a wave, in words: the chosen experts of its tokens; then each lane's
// sorted keys and places (the first is in registers; none for one key), or the
// row of a group choice (used before them, by whole waves only).
constexpr int kPlaces = kRouteMaxChoice;
constexpr int route_lds(int L, int V) { return 64 / L * kPlaces + (V > 1 ? 2 * V * 64 : L == 64 ? 64 : 0); }

template <int DT, int L, int V>
__global__ void __launch_bounds__(64 * ROUTE_WAVES) route_kernel(RouteArgs a) {
    __shared__ __align__(8) uint32_t lds[ROUTE_WAVES][route_lds(L, V)];
    static_assert(L != 64 || route_lds(L, V) >= kPlaces + 64 * V, "the row of a group choice lies in the wave's own LDS");
    static_assert(V == 1 || route_lds(L, V) >= 64 / L * kPlaces + 2 * 64 * V, "so do the lanes' lists");
    using G = Lanes<L>;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, row = lane & (L - 1);
    const int64_t mine_t = ((int64_t)blockIdx.x * ROUTE_WAVES + wv) * (64 / L) + lane / L;
    if (__ballot(mine_t < a.T) == 0) return;     // waves share nothing
    const int64_t t = mine_t < a.T ? mine_t : a.T - 1;
    const int e0 = row * V;
    float x[V], s[V];
    uint32_t key[V];
    load_logits<DT, V>(a.logits, t * a.E, e0, a.E, a.vec, x);
    float bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = 0.0f;
    if (a.bias) load_logits<QLIN_F32, V, false>(a.bias, 0, e0, a.E, a.vec, bias);
    // scores of all experts only where the choice needs them
    const bool grouped = a.kept < a.groups;
    const bool scored = a.bias || (grouped && a.group_top == 2);
    float top = 0.0f, inv = 0.0f;
    if (!a.sigmoid) {
        uint32_t o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = order_of(x[v]);
        top = value_of(G::max_all(largest<V>(o)));
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += s[v] = exp_of(x[v] - top);
        sum = G::sum_all(sum);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] *= inv;
    } else if (scored) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = sigmoid_of(x[v]);
    }
    // NaN fails the comparison
    if (a.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = __builtin_fmaf(x[v], 0.0f, s[v] + bias[v]);    // NaN where the logit is -inf
            key[v] = b > -INFINITY ? order_of_sum(b) : NONE;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = x[v] > -INFINITY ? order_of(x[v]) : NONE;
    }
    uint32_t* const chosen = lds[wv] + lane / L * kPlaces;
    uint2* const list = (uint2*)(lds[wv] + 64 / L * kPlaces) + lane;          // [V][64]
    if (grouped) {
        uint32_t f[V];
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = key[v];
        if (!a.bias && a.group_top == 2) {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = key[v] == NONE ? NONE : order_of_sum(s[v]);
        }
        if (a.seg) {
            const bool in = in_best_groups<L, V>(a, f, lane);
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = in ? key[v] : NONE;
        } else if constexpr (L == 64) {
            const uint64_t keep = best_groups<V>(a, f, lane, lds[wv] + kPlaces);
            const int per = a.E / a.groups;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int gr = (e0 + v) / per;
                if (gr >= a.groups || !((keep >> gr) & 1)) key[v] = NONE;
            }
        }
    }
    // Each lane sorts its keys, of equal ones the lower place first, and keeps
    // the best at hand. Then k rounds: the best of the token's lanes, of equal
    // ones the first lane's; that lane notes it and takes its next.
    uint32_t head = key[0], place = 0;
    if constexpr (V > 1) {
        // key and place as one positive fp64 number of the same order (bits 2^60 + 256 key + V - 1 - place, all
        // of one exponent), so that a comparison of the network is a maximum and a minimum
        double kp[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            kp[v] = __hiloint2double((int)__builtin_amdgcn_alignbit(0x00100000u, key[v], 24),
                                     (int)(key[v] << 8 | (uint32_t)(V - 1 - v)));
        constexpr Sorter net = sorter(V);
#pragma unroll
        for (int c = 0; c < net.n; ++c) {
            const double p = kp[net.a[c]], q = kp[net.b[c]];
            kp[net.a[c]] = max_f64(p, q);
            kp[net.b[c]] = min_f64(p, q);
        }
        auto entry = [&](int v) {
            const uint32_t hi = (uint32_t)__double2hiint(kp[v]), lo = (uint32_t)__double2loint(kp[v]);
            return uint2{hi << 24 | lo >> 8, (uint32_t)(V - 1) - (lo & 255u)};
        };
#pragma unroll
        for (int v = 1; v < V; ++v) list[64 * v] = entry(v);
        head = entry(0).x;
        place = entry(0).y;
    }
    for (int j = row; j < a.k; j += L) chosen[j] = 0xFFFFFFFFu;
    int taken = 0;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t best = G::max_all(head);
        if (L == 64 && best == NONE) break;
        if (row == G::first(head == best, lane) && best != NONE) {
            chosen[j] = (uint32_t)e0 + place;
            ++taken;
            if (V > 1 && taken < V) {
                const uint2 n = list[64 * taken];
                head = n.x;
                place = n.y;
            } else {
                head = NONE;
            }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float sum = 0.0f;
    constexpr int PER = kRouteMaxChoice / L;       // places of a lane
    float sc[PER];
    int id[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        id[p] = -1;
        sc[p] = 0.0f;
        if (p * L < a.k) {
            if (row + p * L < a.k) id[p] = (int)chosen[row + p * L];
            if (id[p] >= 0) {
                const float l = load_f<DT>(a.logits, t * a.E + id[p]);
                sc[p] = a.sigmoid ? sigmoid_of(l) : exp_of(l - top) * inv;
            }
            sum += sc[p];
        }
    }
    const float by = a.renorm ? a.scale / (G::sum_all(sum) + 1e-20f) : a.scale;
#pragma unroll
    for (int p = 0; p < PER; ++p)
        if (row + p * L < a.k && mine_t < a.T) {
            a.weights[t * a.k + row + p * L] = sc[p] * by;
            a.experts[t * a.k + row + p * L] = id[p];
        }
}

struct RouteGradArgs {
    const void* logits;
    const int32_t* experts;
    const float* grad_w;
    int64_t T;
    int E, k;
    int sigmoid, renorm;
    int vec;
    float scale;
    void* grad;              // [T, E], the logits' dtype
};

// Lane j works out the gradient of place j's logit; LDS carries it to the
// lane that writes that logit. Only softmax needs the whole row of logits.
// Latency-bound: 8191 tokens of 60 experts, 4 chosen, 4.0 us.
template <int DT, int V>
__global__ void __launch_bounds__(64 * ROUTE_WAVES) route_grad_kernel(RouteGradArgs a) {
    extern __shared__ float lds[];               // [waves][64 V]
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + wv;
    if (t >= a.T) return;                        // waves share nothing
    const int e0 = lane * V;
    float* const row = lds + wv * 64 * V;
    int id = -1;
    float g = 0.0f, l = 0.0f;
    if (lane < a.k) {
        id = a.experts[t * a.k + lane];
        if ((uint32_t)id < (uint32_t)a.E) {
            l = finite_or_none(load_f<DT>(a.logits, t * a.E + id));
            if (l == -INFINITY) id = -1;
            else g = a.grad_w[t * a.k + lane];
        } else {
            id = -1;
        }
    }
    float x[V], s[V];
    float sc = 0.0f;
    if (a.sigmoid) {
        if (id >= 0) sc = sigmoid_of(l);
    } else {
        load_logits<DT, V>(a.logits, t * a.E, e0, a.E, a.vec, x);
        const float top = row_max<V>(x);
        const float sum = softmax_terms<V>(x, top, s);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] *= inv;
        if (id >= 0) sc = exp_of(l - top) * inv;
    }
    float ds = a.scale * g, dot = 0.0f;
    if (a.renorm) {
        // differences from one place's g: what all of them share cancels exactly
        const uint64_t places = __ballot(id >= 0);
        const float g0 = lane_value(g, places ? __builtin_ctzll(places) : 0), dg = id >= 0 ? g - g0 : 0.0f;
        const float sum = wave_sum(sc), total = sum + 1e-20f;
        const float extra = total - sum;   // 1e-20, or 0 where that is lost in the sum
        ds = (dg * sum - wave_sum(dg * sc) + extra * g) / total / total * a.scale;
        if (!a.sigmoid) dot = extra / total * (wave_sum(g * sc) / total) * a.scale;   // no factor is near 1e-40
    } else if (!a.sigmoid) {
        dot = wave_sum(ds * sc);
    }
    const float r = a.sigmoid ? ds * sc * sigmoid_of(-l) : sc * (ds - dot);
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) row[e0 + v] = a.sigmoid ? 0.0f : 0.0f - s[v] * dot;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (id >= 0) row[id] = r;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = row[e0 + v];
    constexpr int SIZE = DT == QLIN_F32 ? 4 : 2, BYTES = V * SIZE;
    if (V > 1 && a.vec) {
        struct __attribute__((aligned(BYTES < 16 ? BYTES : 16))) Raw {
            uint32_t d[BYTES < 4 ? 1 : BYTES / 4];
        } raw;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (DT == QLIN_F32) raw.d[v] = __float_as_uint(o[v]);
            else {
                const uint32_t h = DT == QLIN_BF16 ? f32_to_bf16_rne(o[v]) : f32_to_f16_rne(o[v]);
                raw.d[v / 2] = v & 1 ? raw.d[v / 2] | (h << 16) : h;
            }
        }
        if (e0 < a.E) *(Raw*)((char*)a.grad + (t * a.E + e0) * SIZE) = raw;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e0 + v < a.E) store_f<DT>(a.grad, t * a.E + e0 + v, o[v]);
    }
}

// Experts a lane for E of them over L lanes.
inline int lane_width(int E, int L) {
    int V = 1;
    while (V * L < E) V *= 2;
    return V;
}

// Lanes of a group of `per` experts where that is a power of two of whole lanes, else 0.
inline int group_lanes(int per, int L, int V) {
    const int lanes = per % V ? 0 : per / V;
    return lanes >= 1 && lanes <= L && (lanes & (lanes - 1)) == 0 ? lanes : 0;
}

// Whether every lane's V elements of every row are aligned and inside or outside the row as a whole.
inline int whole_lanes(int dt, int E, int V, const void* a, const void* b) {
    const int bytes = V * (dt == QLIN_F32 ? 4 : 2);
    return E % V == 0 && (((uintptr_t)a | (uintptr_t)b) & (uintptr_t)((bytes < 16 ? bytes : 16) - 1)) == 0;
}

template <int DT, int L, int V>
void route_launch(const RouteArgs& a, hipStream_t st) {
    constexpr int per = ROUTE_WAVES * (64 / L);
    RouteArgs part = a;
    for (int64_t t = 0; t < a.T; t += ROUTE_TOKENS) {
        part.T = a.T - t < ROUTE_TOKENS ? a.T - t : ROUTE_TOKENS;
        part.logits = (const char*)a.logits + t * a.E * (DT == QLIN_F32 ? 4 : 2);
        part.weights = a.weights + t * a.k;
        part.experts = a.experts + t * a.k;
        route_kernel<DT, L, V><<<(unsigned)((part.T + per - 1) / per), 64 * ROUTE_WAVES, 0, st>>>(part);
    }
}
template <int DT>
void route_by_width(const RouteArgs& a, int L, int V, hipStream_t st) {
    if (L == 16) {
        switch (V) {
        case 1: return route_launch<DT, 16, 1>(a, st);
        case 2: return route_launch<DT, 16, 2>(a, st);
        case 4: return route_launch<DT, 16, 4>(a, st);
        case 8: return route_launch<DT, 16, 8>(a, st);
        default: return route_launch<DT, 16, 16>(a, st);
        }
    }
    switch (V) {
    case 1: return route_launch<DT, 64, 1>(a, st);
    case 2: return route_launch<DT, 64, 2>(a, st);
    case 4: return route_launch<DT, 64, 4>(a, st);
    case 8: return route_launch<DT, 64, 8>(a, st);
    default: return route_launch<DT, 64, 16>(a, st);
    }
}
template <int DT, int V>
void route_grad_launch(const RouteGradArgs& a, hipStream_t st) {
    RouteGradArgs part = a;
    for (int64_t t = 0; t < a.T; t += ROUTE_TOKENS) {
        part.T = a.T - t < ROUTE_TOKENS ? a.T - t : ROUTE_TOKENS;
        part.logits = (const char*)a.logits + t * a.E * (DT == QLIN_F32 ? 4 : 2);
        part.grad = (char*)a.grad + t * a.E * (DT == QLIN_F32 ? 4 : 2);
        part.experts = a.experts + t * a.k;
        part.grad_w = a.grad_w + t * a.k;
        route_grad_kernel<DT, V><<<(unsigned)((part.T + ROUTE_WAVES - 1) / ROUTE_WAVES), 64 * ROUTE_WAVES,
                                   ROUTE_WAVES * 64 * V * sizeof(float), st>>>(part);
    }
}
template <int DT>
void route_grad_by_width(const RouteGradArgs& a, int V, hipStream_t st) {
    switch (V) {
    case 1: return route_grad_launch<DT, 1>(a, st);
    case 2: return route_grad_launch<DT, 2>(a, st);
    case 4: return route_grad_launch<DT, 4>(a, st);
    case 8: return route_grad_launch<DT, 8>(a, st);
    default: return route_grad_launch<DT, 16>(a, st);
    }
}

}  // namespace

hipError_t launch_moe_route(const void* logits, int dt, int64_t T, int E, int k, const float* bias,
                            int sigmoid, int renorm, float scale, int groups, int kept, int group_top,
                            float* weights, int32_t* experts, hipStream_t st) {
    const int per = E / groups;
    int L = 16, V = lane_width(E, L), seg = group_lanes(per, L, V);
    if (E > 256 || (kept < groups && !seg)) {
        L = 64;
        V = lane_width(E, L);
        seg = group_lanes(per, L, V);
    }
    const RouteArgs a{logits, bias, T, E, k, sigmoid, renorm, groups, kept, group_top, seg,
                      whole_lanes(dt, E, V, logits, nullptr) && whole_lanes(QLIN_F32, E, V, bias, nullptr), scale,
                      weights, experts};
    if (dt == QLIN_F32) route_by_width<QLIN_F32>(a, L, V, st);
    else if (dt == QLIN_BF16) route_by_width<QLIN_BF16>(a, L, V, st);
    else route_by_width<QLIN_F16>(a, L, V, st);
    return hipGetLastError();
}

hipError_t launch_moe_route_grad(const void* logits, int dt, int64_t T, int E, int k, const int32_t* experts,
                                 const float* grad_w, int sigmoid, int renorm, float scale, void* grad,
                                 hipStream_t st) {
    const int V = lane_width(E, 64);
    const RouteGradArgs a{logits, experts, grad_w, T, E, k, sigmoid, renorm, whole_lanes(dt, E, V, logits, grad), scale, grad};
    if (dt == QLIN_F32) route_grad_by_width<QLIN_F32>(a, V, st);
    else if (dt == QLIN_BF16) route_grad_by_width<QLIN_BF16>(a, V, st);
    else route_grad_by_width<QLIN_F16>(a, V, st);
    return hipGetLastError();
}

}  // namespace qlin
