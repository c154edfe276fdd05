// kv_api.cpp -- the C ABI of rotary positions and of the 4-bit cache of keys
// and values: argument validation and launches. As everywhere in the library,
// a rejected call launches nothing.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/qlin.h"
#include "api_common.h"
#include "kv_common.h"

using qlin::device_status;
using qlin::fail;
using qlin::is_float_dtype;
using qlin::ok;

namespace {

constexpr int64_t kMaxIndex = (1LL << 31) - 1;

uintptr_t elem(int dtype) { return dtype == QLIN_F32 ? 4 : 2; }

qlin_status check_aligned(const void* p, uintptr_t align, const char* what) {
    if ((uintptr_t)p % align) return fail(QLIN_ERR_INVALID_ARGUMENT, "%s must be %d-byte aligned", what, (int)align);
    return QLIN_OK;
}

// The cache's format and sizes; its pointers are looked at where a call has work.
qlin_status check_cache(const qlin_kv_cache* c, qlin::KvPool* pool) {
    if (!c) return fail(QLIN_ERR_INVALID_ARGUMENT, "cache is NULL");
    if (!c->mode) return fail(QLIN_ERR_INVALID_ARGUMENT, "mode is NULL");
    const int g = c->group_size;
    if (!strcmp(c->mode, "affine")) {
        pool->mode = qlin::AFFINE;
        if (g != 32 && g != 64 && g != 128)
            return fail(QLIN_ERR_INVALID_ARGUMENT, "affine group_size must be 32, 64 or 128 (got %d)", g);
        if (!is_float_dtype(c->dtype)) return fail(QLIN_ERR_INVALID_ARGUMENT, "the cache's dtype must be f32, f16 or bf16");
    } else if (!strcmp(c->mode, "mxfp4")) {
        pool->mode = qlin::MXFP4;
        if (g != 32) return fail(QLIN_ERR_INVALID_ARGUMENT, "mxfp4 takes group_size 32 (got %d)", g);
    } else if (!strcmp(c->mode, "nvfp4")) {
        pool->mode = qlin::NVFP4;
        if (g != 16) return fail(QLIN_ERR_INVALID_ARGUMENT, "nvfp4 takes group_size 16 (got %d)", g);
    } else if (!strcmp(c->mode, "mxfp8")) {
        return fail(QLIN_ERR_UNSUPPORTED, "a cache is held in 4 bits: affine, mxfp4 or nvfp4");
    } else {
        return fail(QLIN_ERR_INVALID_ARGUMENT, "unknown mode \"%s\"", c->mode);
    }
    if (c->bits != 4) return fail(QLIN_ERR_UNSUPPORTED, "a cache is held in 4 bits (got %d)", c->bits);
    if (c->pages < 1 || c->heads < 1 || c->page_size < 1 || c->head_dim < 1)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "the cache's sizes must be positive");
    if (c->page_size % qlin::kKvUnit)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "page_size must be a multiple of %d (got %lld)", qlin::kKvUnit,
                    (long long)c->page_size);
    if (c->head_dim % 32 || c->head_dim % g)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "head_dim must be a multiple of 32 and of group_size (got %lld)",
                    (long long)c->head_dim);
    if (c->heads > qlin::kKvMaxHeads || c->page_size > qlin::kKvMaxPage || c->head_dim > qlin::kKvMaxDim)
        return fail(QLIN_ERR_UNSUPPORTED, "heads above %d, page_size above %d or head_dim above %d are not supported",
                    qlin::kKvMaxHeads, qlin::kKvMaxPage, qlin::kKvMaxDim);
    if (c->pages > kMaxIndex / c->page_size || c->pages * c->page_size > (1LL << 35) / c->heads - 1)
        return fail(QLIN_ERR_UNSUPPORTED, "pages * page_size from 2^31 or pages * heads * page_size from 2^35 on");
    pool->codes[0] = c->k_codes;
    pool->codes[1] = c->v_codes;
    pool->scales[0] = c->k_scales;
    pool->scales[1] = c->v_scales;
    pool->biases[0] = c->k_biases;
    pool->biases[1] = c->v_biases;
    pool->sdt = pool->mode == qlin::AFFINE ? (int)c->dtype : (int)QLIN_U8;
    pool->g = g;
    pool->pages = c->pages;
    pool->heads = (int)c->heads;
    pool->page = (int)c->page_size;
    pool->D = (int)c->head_dim;
    return QLIN_OK;
}

qlin_status check_pool(const qlin::KvPool& p) {
    const bool affine = p.mode == qlin::AFFINE;
    for (int side = 0; side < 2; ++side) {
        if (!p.codes[side] || !p.scales[side] || (affine && !p.biases[side]))
            return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer in the cache");
        if (!affine && p.biases[side]) return fail(QLIN_ERR_INVALID_ARGUMENT, "only affine caches have biases");
        qlin_status s;
        if ((s = check_aligned(p.codes[side], 16, "codes"))) return s;
        if ((s = check_aligned(p.scales[side], 16, "scales")) || (s = check_aligned(p.biases[side], 16, "biases"))) return s;
    }
    return QLIN_OK;
}

// The type of rows that go into or come out of the attention over a cache.
qlin_status check_rows(const qlin::KvPool& p, int dtype, int64_t T, const char* what) {
    if (!is_float_dtype(dtype)) return fail(QLIN_ERR_INVALID_ARGUMENT, "%s must be f32, f16 or bf16", what);
    if (p.mode == qlin::AFFINE && dtype != p.sdt)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "%s must have the type of an affine cache's scales", what);
    if (T < 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "T must be >= 0");
    if (T > kMaxIndex) return fail(QLIN_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens are not supported");
    return QLIN_OK;
}

qlin_status check_volume(int64_t T, const qlin::KvPool& p) {
    if (T > (1LL << 36) / ((int64_t)p.heads * p.D))
        return fail(QLIN_ERR_UNSUPPORTED, "T * heads * head_dim above 2^36: split the rows over several calls");
    return QLIN_OK;
}

// What attention's sizes have to be; with_offsets: sequences of any number of rows.
qlin_status check_attention(const qlin::KvPool& p, int dtype, int64_t T, int64_t q_heads, int64_t B, int64_t width,
                            bool with_offsets, int64_t window) {
    qlin_status s;
    if ((s = check_rows(p, dtype, T, "q"))) return s;
    if (q_heads < 1 || q_heads % p.heads)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "q_heads (%lld) must be a multiple of the cache's heads (%d)",
                    (long long)q_heads, p.heads);
    if (B < 0 || width < 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "negative size");
    if (window < 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "window must be >= 0");
    if (!with_offsets && B != T)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "without offsets every sequence has one row: T (%lld) must be B (%lld)",
                    (long long)T, (long long)B);
    if (B > kMaxIndex - 1 || width > kMaxIndex || q_heads > kMaxIndex || (T && q_heads > kMaxIndex / T))
        return fail(QLIN_ERR_UNSUPPORTED, "B, width or T * q_heads from 2^31 on");
    return QLIN_OK;
}

qlin_status rotary(const void* x, int dtype, int64_t T, int64_t x_stride, int64_t heads, int64_t D, int64_t R,
                   const int32_t* positions, const float* freqs, int interleaved, double scale, void* y,
                   int64_t y_stride, int backward, hipStream_t st) {
    if (!is_float_dtype(dtype)) return fail(QLIN_ERR_INVALID_ARGUMENT, "x must be f32, f16 or bf16");
    if (T < 0 || heads < 1) return fail(QLIN_ERR_INVALID_ARGUMENT, "T must be >= 0 and heads positive");
    if (D < 8 || D % 8) return fail(QLIN_ERR_INVALID_ARGUMENT, "D must be a positive multiple of 8 (got %lld)", (long long)D);
    if (R < 2 || R % 2 || R > D) return fail(QLIN_ERR_INVALID_ARGUMENT, "R must be even and in [2, D] (got %lld)", (long long)R);
    if (!std::isfinite((float)scale)) return fail(QLIN_ERR_INVALID_ARGUMENT, "scale must be finite in fp32");
    if (D > qlin::kRotaryMaxDim || heads > (1 << 20) || T > kMaxIndex)
        return fail(QLIN_ERR_UNSUPPORTED, "D above %d, more than 2^20 heads or 2^31 - 1 tokens are not supported",
                    qlin::kRotaryMaxDim);
    if (x_stride < 0 || x_stride > (1LL << 31) || y_stride > (1LL << 31) || y_stride < heads * D)
        return fail(QLIN_ERR_INVALID_ARGUMENT, "token strides: x_stride >= 0, y_stride >= heads * D, neither above 2^31");
    if (T == 0) return ok();
    if (!x || !y || !positions || !freqs) return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    qlin_status s;
    if ((s = check_aligned(x, elem(dtype), "x")) || (s = check_aligned(y, elem(dtype), "y")) ||
        (s = check_aligned(positions, 4, "positions")) || (s = check_aligned(freqs, 4, "freqs")))
        return s;
    const uintptr_t xb = (uintptr_t)x, yb = (uintptr_t)y, row = heads * D * elem(dtype);
    const uintptr_t xe = xb + (T - 1) * x_stride * elem(dtype) + row, ye = yb + (T - 1) * y_stride * elem(dtype) + row;
    if (!(xb == yb && (x_stride == y_stride || T == 1)) && xb < ye && yb < xe) {
        // parts of the same rows: y's place in the row of x that it starts behind, apart from that row's and the next one's values
        const uintptr_t step = x_stride * elem(dtype), back = (xb > yb ? xb - yb : 0), skip = step ? (back + step - 1) / step * step : 0;
        const uintptr_t place = step ? (yb + skip - xb) % step : 0;
        if (T == 1 || x_stride != y_stride || place < row || place + row > step)
            return fail(QLIN_ERR_INVALID_ARGUMENT, "x and y overlap and are not one and the same");
    }
    const qlin::RotaryArgs a{x, y, T, x_stride, y_stride, (int)heads, (int)D, (int)R, positions, freqs, (float)scale,
                             interleaved != 0, backward};
    return device_status(qlin::launch_rotary(a, dtype, st), "rotary");
}

}  // namespace

extern "C" {

qlin_status qlin_rotary(const void* x, qlin_dtype dtype, int64_t T, int64_t x_stride, int64_t heads, int64_t D,
                        int64_t R, const int32_t* positions, const float* freqs, int interleaved, double scale, void* y,
                        int64_t y_stride, void* stream) {
    return rotary(x, dtype, T, x_stride, heads, D, R, positions, freqs, interleaved, scale, y, y_stride, 0,
                  (hipStream_t)stream);
}

qlin_status qlin_rotary_grad(const void* grad_y, qlin_dtype dtype, int64_t T, int64_t grad_y_stride, int64_t heads,
                             int64_t D, int64_t R, const int32_t* positions, const float* freqs, int interleaved,
                             double scale, void* grad_x, int64_t grad_x_stride, void* stream) {
    return rotary(grad_y, dtype, T, grad_y_stride, heads, D, R, positions, freqs, interleaved, scale, grad_x,
                  grad_x_stride, 1, (hipStream_t)stream);
}

qlin_status qlin_kv_cache_write(const qlin_kv_cache* cache, const void* k, const void* v, qlin_dtype dtype, int64_t T,
                                int64_t k_stride, int64_t v_stride, const int32_t* slots, void* stream) {
    qlin::KvPool p;
    qlin_status s;
    if ((s = check_cache(cache, &p)) || (s = check_rows(p, dtype, T, "k and v")) || (s = check_volume(T, p))) return s;
    if (k_stride < 0 || v_stride < 0 || k_stride > (1LL << 31) || v_stride > (1LL << 31))
        return fail(QLIN_ERR_INVALID_ARGUMENT, "token strides must be in [0, 2^31]");
    if (T == 0) return ok();
    if (!k || !v || !slots) return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if ((s = check_pool(p)) || (s = check_aligned(k, elem(dtype), "k")) || (s = check_aligned(v, elem(dtype), "v")) ||
        (s = check_aligned(slots, 4, "slots")))
        return s;
    return device_status(qlin::launch_kv_write(p, k, v, dtype, T, k_stride, v_stride, slots, (hipStream_t)stream),
                         "kv_cache_write");
}

qlin_status qlin_kv_cache_read(const qlin_kv_cache* cache, const int32_t* slots, int64_t T, void* k, void* v,
                               qlin_dtype dtype, void* stream) {
    qlin::KvPool p;
    qlin_status s;
    if ((s = check_cache(cache, &p))) return s;
    if (!is_float_dtype(dtype)) return fail(QLIN_ERR_INVALID_ARGUMENT, "k and v must be f32, f16 or bf16");
    if (T < 0) return fail(QLIN_ERR_INVALID_ARGUMENT, "T must be >= 0");
    if (T > kMaxIndex) return fail(QLIN_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens are not supported");
    if ((s = check_volume(T, p))) return s;
    if (T == 0) return ok();
    if (!k || !v || !slots) return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if ((s = check_pool(p)) || (s = check_aligned(k, 16, "k")) || (s = check_aligned(v, 16, "v")) ||
        (s = check_aligned(slots, 4, "slots")))
        return s;
    return device_status(qlin::launch_kv_read(p, slots, T, k, v, dtype, (hipStream_t)stream), "kv_cache_read");
}

size_t qlin_kv_cache_attention_workspace_bytes(const qlin_kv_cache* cache, qlin_dtype dtype, int64_t T, int64_t q_heads,
                                               int64_t B, int64_t width, int has_offsets, int64_t window) {
    qlin::KvPool p;
    if (check_cache(cache, &p) || check_attention(p, dtype, T, q_heads, B, width, has_offsets != 0, window)) return 0;
    if (T == 0 || B == 0) return 0;
    return qlin::attend_plan(dtype, T, (int)q_heads, B, width, p, window, !has_offsets).bytes;
}

qlin_status qlin_kv_cache_attention(const qlin_kv_cache* cache, const void* q, qlin_dtype dtype, int64_t T,
                                    int64_t q_stride, int64_t q_heads, const int32_t* table, int64_t B, int64_t width,
                                    const int32_t* lengths, const int32_t* offsets, double scale, int causal,
                                    int64_t window, void* workspace, size_t workspace_bytes, void* out, void* stream) {
    qlin::KvPool p;
    qlin_status s;
    if ((s = check_cache(cache, &p)) || (s = check_attention(p, dtype, T, q_heads, B, width, offsets != nullptr, window)))
        return s;
    if (!std::isfinite((float)(scale * 2))) return fail(QLIN_ERR_INVALID_ARGUMENT, "twice the scale must be finite in fp32");
    if (q_stride < 0 || q_stride > (1LL << 31)) return fail(QLIN_ERR_INVALID_ARGUMENT, "q_stride must be in [0, 2^31]");
    if (T == 0 || B == 0) return ok();
    if (!q || !lengths || !out || (width && !table)) return fail(QLIN_ERR_INVALID_ARGUMENT, "NULL tensor pointer");
    if ((s = check_pool(p)) || (s = check_aligned(q, elem(dtype), "q")) || (s = check_aligned(out, 16, "out")) ||
        (s = check_aligned(table, 4, "table")) || (s = check_aligned(lengths, 4, "lengths")) ||
        (s = check_aligned(offsets, 4, "offsets")))
        return s;
    const uintptr_t qb = (uintptr_t)q, qe = qb + ((T - 1) * q_stride + q_heads * p.D) * elem(dtype);
    const uintptr_t ob = (uintptr_t)out, oe = ob + T * q_heads * p.D * elem(dtype);
    if (qb < oe && ob < qe) return fail(QLIN_ERR_INVALID_ARGUMENT, "out overlaps q");
    const qlin::AttendPlan plan = qlin::attend_plan(dtype, T, (int)q_heads, B, width, p, window, offsets == nullptr);
    if (!plan.fits) return fail(QLIN_ERR_UNSUPPORTED, "more rows than one launch holds: split them over several calls");
    if (plan.bytes) {
        if (!workspace || workspace_bytes < plan.bytes)
            return fail(QLIN_ERR_INVALID_ARGUMENT, "workspace of %zu bytes needed (got %zu)", plan.bytes,
                        workspace ? workspace_bytes : (size_t)0);
        if ((s = check_aligned(workspace, 16, "workspace"))) return s;
    }
    const qlin::AttendArgs a{q, out, T, q_stride, (int)q_heads, table, lengths, offsets, (int)B, (int)width,
                             (float)scale, causal != 0, window};
    static const char* const names[] = {"kv_attention_simple", "kv_attention_rows", "kv_attention_prompt"};
    qlin::record_path(names[plan.path]);
    return device_status(qlin::launch_attend(a, p, dtype, plan, workspace, (hipStream_t)stream), "kv_cache_attention");
}

}  // extern "C"
