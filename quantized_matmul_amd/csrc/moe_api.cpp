// moe_api.cpp -- the C ABI of the mixture-of-experts operators: argument
// validation, workspace layout and launches. As everywhere in the library, a
// rejected call launches nothing.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/qlin.h"
#include "api_common.h"
#include "moe_common.h"
#include "mx4_common.h"

using qlin::device_status;
using qlin::fail;
using qlin::is_float_dtype;
using qlin::ok;

namespace {

constexpr int64_t kMaxIndex = (1LL << 31) - 1;

qlin_status check_score(const char* score, double scale, int* sigmoid) {
    if (!score) return fail(QLIN_ERR_INVALID_ARGUMENT, "score is NULL");
    if (!strcmp(score, "softmax")) *sigmoid = 0;
    else if (!strcmp(score, "sigmoid")) *sigmoid = 1;
    else return fail(QLIN_ERR_INVALID_ARGUMENT, "unknown score \"%s\" (softmax, sigmoid)", score);
    if (!std::isfinite((float)scale)) return fail(QLIN_ERR_INVALID_ARGUMENT, "scale must be finite in fp32");
    return QLIN_OK;
}

qlin_status check_route(int dtype, int64_t T, int64_t E, int64_t k) {
    if (!is_float_dtype(dtype)) return fail(QLIN_ERR_INVALID_ARGUMENT, "logits must be f32, f16 or bf16");
    if (E < 1 || E > qlin::kRouteMaxExperts)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "E must be in [1, %d] (got %lld)", qlin::kRouteMaxExperts, (long long)E);
    if (k < 1 || k > E || k > qlin::kRouteMaxChoice)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "k must be in [1, min(E, %d)] (got %lld)", qlin::kRouteMaxChoice,
                    (long long)k);
    if (T < 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "T must be >= 0");
    if (T > kMaxIndex) return fail(QLIN_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens are not supported");
    return QLIN_OK;
}

qlin_status check_aligned(const void* p, uintptr_t align, const char* what) {
    if ((uintptr_t)p % align) return fail(QLIN_ERR_INVALID_ARGUMENT, "%s must be %d-byte aligned", what, (int)align);
    return QLIN_OK;
}

uintptr_t elem(int dtype) { return dtype == QLIN_F32 ? 4 : 2; }

size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }

// Scale rows as the tiled kernel reads them.
int64_t scale_stride(int64_t K) { return (int64_t)up((size_t)(K / 32), 16); }

// Pieces of a product's workspace, each 256-byte aligned: x's codes and
// scales (or, for given codes, their scales in 16-byte rows), W's scales in
// 16-byte rows (used where they do not lie so already; the sizes do not tell
// their address), the row plan. A streamed float x needs none.
struct Layout {
    size_t xq, xs, ws, plan, bytes;
};
Layout layout(const qlin::Mx4Choice& c, int64_t rows, int64_t R, int64_t K, int64_t E, int64_t N, bool codes,
              bool gather) {
    Layout l{};
    const bool tiled = c.path == qlin::Mx4Path::kTiled;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t p = at;
        at += up(n, 256);
        return p;
    };
    const bool quantized = !codes && c.path != qlin::Mx4Path::kStreamFloat;
    l.xq = take(quantized ? (size_t)rows * (size_t)(K / 2) : 0);
    l.xs = take(quantized || (codes && tiled) ? (size_t)rows * (size_t)scale_stride(K) : 0);
    l.ws = take(tiled ? (size_t)E * (size_t)N * (size_t)scale_stride(K) : 0);
    l.plan = take(gather && tiled ? qlin::mx4_plan_bytes(R, E) : 0);
    l.bytes = at;
    return l;
}

bool product_sizes_ok(int64_t rows, int64_t K, int64_t N) {
    return rows >= 0 && K >= 32 && K % 32 == 0 && K <= (1LL << 22) && N >= 1 && rows <= kMaxIndex && N <= kMaxIndex;
}

// Everything the dense and the gathered product share. rows: rows of x.
qlin_status product(const void* x, int x_dtype, const void* x_scales, const char* activation, int64_t rows, int64_t K,
                    const uint32_t* wq, const void* scales, int64_t E, int64_t N, const int32_t* experts, int64_t R,
                    bool gather, void* workspace, size_t workspace_bytes, void* y, int y_dtype, hipStream_t st,
                    const char* what) {
    int swiglu = 0;
    if (activation && !strcmp(activation, "swiglu")) swiglu = 1;
    else if (activation && strcmp(activation, "none"))
        return fail(QLIN_ERR_INVALID_ARGUMENT, "unknown activation \"%s\" (none, swiglu)", activation);
    const bool codes = x_dtype == QLIN_U8;
    if (!codes && !is_float_dtype(x_dtype))
        return fail(QLIN_ERR_INVALID_ARGUMENT, "x must be f32, f16, bf16 or mxfp4 words");
    if (!is_float_dtype(y_dtype)) return fail(QLIN_ERR_INVALID_ARGUMENT, "y must be f32, f16 or bf16");
    if (codes && swiglu) return fail(QLIN_ERR_INVALID_ARGUMENT, "mxfp4 words take no activation");
    if (rows < 0 || R < 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "negative size");
    if (N <= 0 || K <= 0 || E <= 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "N, K and E must be positive");
    if (K % 32) return fail(QLIN_ERR_INVALID_ARGUMENT, "K must be a multiple of 32 (got %lld)", (long long)K);
    if (!product_sizes_ok(rows, K, N))
        return fail(QLIN_ERR_UNSUPPORTED, "rows and N above 2^31 - 1 or K above 2^22 are not supported");
    if (gather) {
        if (R > qlin::kMx4MaxRows) return fail(QLIN_ERR_UNSUPPORTED, "more than 2^31 - 2^14 index rows are not supported");
        if (E > qlin::kMx4MaxExperts)
            return fail(QLIN_ERR_UNSUPPORTED, "more than %lld experts are not supported",
                        (long long)qlin::kMx4MaxExperts);
        if (rows == 0 ? R != 0 : R % rows != 0)
            return fail(QLIN_ERR_INVALID_ARGUMENT, "R (%lld) must be a multiple of the rows of x (%lld)", (long long)R,
                        (long long)rows);
    }
    if (R == 0) return ok();
    if (!x || !wq || !scales || !y || (gather && !experts)) return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if (codes && !x_scales) return fail(QLIN_ERR_INVALID_ARGUMENT, "mxfp4 words need x_scales");
    if (!codes && x_scales) return fail(QLIN_ERR_INVALID_ARGUMENT, "x_scales go with mxfp4 words only");
    qlin_status s;
    if ((s = check_aligned(x, codes ? 16 : elem(x_dtype), "x"))) return s;
    if ((s = check_aligned(wq, 16, "wq"))) return s;
    if ((s = check_aligned(y, elem(y_dtype), "y"))) return s;
    if ((s = check_aligned(experts, 4, "experts"))) return s;
    // the tiled kernel's row offsets are 32 bits: tiles of W and (by experts) all of x's codes
    const qlin::Mx4Choice c = qlin::mx4_choose(R, N, K, E, gather, codes);
    const bool tiled = c.path == qlin::Mx4Path::kTiled;
    if (gather && tiled && rows * (K / 2) >= (1LL << 31))
        return fail(QLIN_ERR_UNSUPPORTED, "x has more than 2^32 values: split its rows over several calls");
    if (!qlin::mx4_fits(R, N, K, E, gather, c))
        return fail(QLIN_ERR_UNSUPPORTED, "more output tiles than one launch holds: split the rows over several calls");
    const Layout l = layout(c, rows, R, K, E, N, codes, gather);
    if (l.bytes) {
        if (!workspace || workspace_bytes < l.bytes)
            return fail(QLIN_ERR_INVALID_ARGUMENT, "workspace of %zu bytes needed (got %zu)", l.bytes,
                        workspace ? workspace_bytes : (size_t)0);
        if ((s = check_aligned(workspace, 16, "workspace"))) return s;
    }
    char* const w = (char*)workspace;
    const int64_t KS = K / 32, stride = scale_stride(K);
    qlin::Mx4Args a{};
    a.xq = (const uint8_t*)x;
    a.xs = (const uint8_t*)x_scales;
    a.wq = (const uint8_t*)wq;
    a.ws = (const uint8_t*)scales;
    a.y = y;
    a.M = R;
    a.N = N;
    a.K = K;
    a.xsstride = a.wsstride = KS;
    a.ydt = y_dtype;
    a.x = x;
    a.xdt = x_dtype;
    a.swiglu = swiglu;
    a.experts = experts;
    a.B = rows;
    a.E = E;
    const bool quantized = !codes && c.path != qlin::Mx4Path::kStreamFloat;
    // what the call touches: x, its codes, the experts met, y
    const double touched = (double)rows * K * (codes ? 0.5 : (double)elem(x_dtype) * (swiglu ? 2 : 1) + 0.5) +
                           (double)(E < R ? E : R) * N * K * 0.5 + (double)R * N * elem(y_dtype);
    const bool large = touched >= (double)qlin::kStreamBytes;
    // 16-byte stores off their alignment split lines, which the caches join (8192 rows, N 13001, K 4096: 298 us through
    // them, 305 past them)
    a.stream = large && N * elem(y_dtype) % 16 == 0 && (uintptr_t)y % 16 == 0;
    qlin::Mx4Plan plan{};
    hipError_t e;
    qlin::Mx4Prepare q{};
    q.dt = x_dtype;
    q.K = K;
    bool prepare = false;
    if (quantized) {
        prepare = true;
        q.x = x;
        q.rows = rows;
        q.swiglu = swiglu;
        q.stream = large;
        q.xq = (uint32_t*)(w + l.xq);
        q.xs = (uint8_t*)(w + l.xs);
        q.sstride = stride;
        a.xq = (const uint8_t*)(w + l.xq);
        a.xs = (const uint8_t*)(w + l.xs);
        a.xsstride = stride;
    }
    if (gather && tiled) {
        prepare = true;
        q.experts = experts;
        q.R = R;
        q.E = E;
        q.tile_rows = c.tile_rows;
        q.plan = w + l.plan;
    }
    if (tiled) {
        // the tiled kernel reads scale rows 16 bytes at a time
        if (KS % 16 || (uintptr_t)scales % 16) {
            prepare = true;
            q.pad[0] = {a.ws, E * N, KS, (uint8_t*)(w + l.ws)};
            a.ws = (const uint8_t*)(w + l.ws);
            a.wsstride = stride;
        }
        if (codes && (KS % 16 || (uintptr_t)x_scales % 16)) {
            prepare = true;
            q.pad[1] = {a.xs, rows, KS, (uint8_t*)(w + l.xs)};
            a.xs = (const uint8_t*)(w + l.xs);
            a.xsstride = stride;
        }
    }
    if (prepare && (e = qlin::launch_mx4_prepare(q, &plan, st)) != hipSuccess) return device_status(e, what);
    e = qlin::launch_mx4_matmul(a, c, &plan, st);
    if (e == hipSuccess)
        qlin::record_path(tiled ? (gather ? "mxfp4_gather_tiled" : "mxfp4_tiled")
                                : (gather ? "mxfp4_gather_stream" : "mxfp4_stream"));
    return device_status(e, what);
}

}  // namespace

extern "C" {

qlin_status qlin_moe_route(const void* logits, qlin_dtype dtype, int64_t T, int64_t E, int64_t k, const float* bias,
                           const char* score, int renormalize, double scale, int64_t groups, int64_t groups_kept,
                           int group_top, float* weights, int32_t* experts, void* stream) {
    int sigmoid = 0;
    qlin_status s = check_score(score, scale, &sigmoid);
    if (s) return s;
    if ((s = check_route(dtype, T, E, k))) return s;
    if (groups < 1 || groups > qlin::kRouteMaxGroups || E % groups)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "groups must divide E and be in [1, %d] (got %lld)",
                    qlin::kRouteMaxGroups, (long long)groups);
    if (groups_kept < 1 || groups_kept > groups)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "groups_kept must be in [1, groups] (got %lld)", (long long)groups_kept);
    if (group_top < 1 || group_top > 2 || group_top > E / groups)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "group_top must be 1 or 2 and at most a group's experts (got %d)",
                    group_top);
    if (k > groups_kept * (E / groups))
        return fail(QLIN_ERR_INVALID_ARGUMENT, "k = %lld experts do not fit the %lld kept groups of %lld",
                    (long long)k, (long long)groups_kept, (long long)(E / groups));
    if (T == 0) return ok();
    if (!logits || !weights || !experts) return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if ((s = check_aligned(logits, elem(dtype), "logits"))) return s;
    if ((s = check_aligned(bias, 4, "bias"))) return s;
    if ((s = check_aligned(weights, 4, "weights"))) return s;
    if ((s = check_aligned(experts, 4, "experts"))) return s;
    return device_status(qlin::launch_moe_route(logits, dtype, T, (int)E, (int)k, bias, sigmoid, renormalize ? 1 : 0,
                                                (float)scale, (int)groups, (int)groups_kept, group_top, weights,
                                                experts, (hipStream_t)stream),
                         "moe_route");
}

qlin_status qlin_moe_route_grad(const void* logits, qlin_dtype dtype, int64_t T, int64_t E, int64_t k,
                                const int32_t* experts, const float* grad_weights, const char* score, int renormalize,
                                double scale, void* grad_logits, void* stream) {
    int sigmoid = 0;
    qlin_status s = check_score(score, scale, &sigmoid);
    if (s) return s;
    if ((s = check_route(dtype, T, E, k))) return s;
    if (T == 0) return ok();
    if (!logits || !experts || !grad_weights || !grad_logits)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if ((s = check_aligned(logits, elem(dtype), "logits"))) return s;
    if ((s = check_aligned(grad_logits, elem(dtype), "grad_logits"))) return s;
    if ((s = check_aligned(grad_weights, 4, "grad_weights"))) return s;
    if ((s = check_aligned(experts, 4, "experts"))) return s;
    return device_status(qlin::launch_moe_route_grad(logits, dtype, T, (int)E, (int)k, experts, grad_weights, sigmoid,
                                                     renormalize ? 1 : 0, (float)scale, grad_logits,
                                                     (hipStream_t)stream),
                         "moe_route_grad");
}

size_t qlin_mxfp4_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N, qlin_dtype x_dtype) {
    if (M == 0 || !product_sizes_ok(M, K, N)) return 0;
    const bool codes = x_dtype == QLIN_U8;
    return layout(qlin::mx4_choose(M, N, K, 1, false, codes), M, M, K, 1, N, codes, false).bytes;
}

qlin_status qlin_mxfp4_matmul(const void* x, qlin_dtype x_dtype, const void* x_scales, const char* activation,
                              int64_t M, int64_t K, const uint32_t* wq, const void* scales, int64_t N, void* workspace,
                              size_t workspace_bytes, void* y, qlin_dtype y_dtype, void* stream) {
    return product(x, x_dtype, x_scales, activation, M, K, wq, scales, 1, N, nullptr, M, false, workspace,
                   workspace_bytes, y, y_dtype, (hipStream_t)stream, "mxfp4_matmul");
}

size_t qlin_gather_mxfp4_matmul_workspace_bytes(int64_t B, int64_t R, int64_t K, int64_t E, int64_t N,
                                                qlin_dtype x_dtype) {
    if (B < 1 || R < 1 || E < 1 || R > qlin::kMx4MaxRows || E > qlin::kMx4MaxExperts || !product_sizes_ok(B, K, N)) return 0;
    const bool codes = x_dtype == QLIN_U8;
    return layout(qlin::mx4_choose(R, N, K, E, true, codes), B, R, K, E, N, codes, true).bytes;
}

qlin_status qlin_gather_mxfp4_matmul(const void* x, qlin_dtype x_dtype, const void* x_scales, const char* activation,
                                     int64_t B, int64_t K, const uint32_t* wq, const void* scales, int64_t E, int64_t N,
                                     const int32_t* experts, int64_t R, void* workspace, size_t workspace_bytes,
                                     void* y, qlin_dtype y_dtype, void* stream) {
    return product(x, x_dtype, x_scales, activation, B, K, wq, scales, E, N, experts, R, true, workspace,
                   workspace_bytes, y, y_dtype, (hipStream_t)stream, "gather_mxfp4_matmul");
}

namespace {

qlin_status check_combine(int dtype, int64_t T, int64_t k, int64_t D) {
    if (!is_float_dtype(dtype)) return fail(QLIN_ERR_INVALID_ARGUMENT, "h must be f32, f16 or bf16");
    if (T < 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "T must be >= 0");
    if (k < 1 || D < 1) return fail(QLIN_ERR_INVALID_ARGUMENT, "k and D must be positive");
    if (k > kMaxIndex || (T && k > kMaxIndex / T) || D > kMaxIndex)
        return fail(QLIN_ERR_UNSUPPORTED, "more than 2^31 - 1 rows or columns are not supported");
    return QLIN_OK;
}

}  // namespace

qlin_status qlin_moe_combine(const void* h, qlin_dtype dtype, int64_t T, int64_t k, int64_t D, const float* weights,
                             const int32_t* experts, void* y, void* stream) {
    qlin_status s = check_combine(dtype, T, k, D);
    if (s) return s;
    if (T == 0) return ok();
    if (!h || !weights || !y) return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if ((s = check_aligned(h, elem(dtype), "h"))) return s;
    if ((s = check_aligned(y, elem(dtype), "y"))) return s;
    if ((s = check_aligned(weights, 4, "weights"))) return s;
    if ((s = check_aligned(experts, 4, "experts"))) return s;
    return device_status(qlin::launch_moe_combine(h, dtype, T, (int)k, D, weights, experts, y, (hipStream_t)stream),
                         "moe_combine");
}

qlin_status qlin_moe_combine_grad(const void* grad_y, const void* h, qlin_dtype dtype, int64_t T, int64_t k, int64_t D,
                                  const float* weights, const int32_t* experts, void* grad_h, float* grad_weights,
                                  void* stream) {
    qlin_status s = check_combine(dtype, T, k, D);
    if (s) return s;
    if (T == 0) return ok();
    if (!grad_y || !h || !weights || !grad_h || !grad_weights)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if ((s = check_aligned(h, elem(dtype), "h"))) return s;
    if ((s = check_aligned(grad_y, elem(dtype), "grad_y"))) return s;
    if ((s = check_aligned(grad_h, elem(dtype), "grad_h"))) return s;
    if ((s = check_aligned(weights, 4, "weights"))) return s;
    if ((s = check_aligned(grad_weights, 4, "grad_weights"))) return s;
    if ((s = check_aligned(experts, 4, "experts"))) return s;
    return device_status(qlin::launch_moe_combine_grad(grad_y, h, dtype, T, (int)k, D, weights, experts, grad_h,
                                                       grad_weights, (hipStream_t)stream),
                         "moe_combine_grad");
}

}  // extern "C"
