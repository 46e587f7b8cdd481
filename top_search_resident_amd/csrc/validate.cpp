// validate.cpp -- status names and the host-side argument checks of the C ABI
// (include/resident_topk.h).  Plain C++ with no HIP dependency: the library
// links it, and the CPU test suite also builds it on its own with the address
// and undefined-behaviour sanitizers.  Every entry point runs the matching
// check before it enqueues anything, so an argument error leaves outputs and
// device state untouched.
#include <stdint.h>

#include "../../include/resident_topk.h"
#include "limits.hpp"

using rt::kMaxD;
using rt::kMaxK;
using rt::kMaxN;
using rt::kMaxQ;

extern "C" {

const char *rt_status_string(rt_status s) {
    switch (s) {
        case RT_OK: return "ok";
        case RT_EINVAL: return "invalid argument";
        case RT_ESTATE: return "invalid state (no corpus resident, or dimension mismatch)";
        case RT_ENOMEM: return "device memory allocation failed";
        case RT_EHIP: return "HIP runtime error";
    }
    return "unknown status";
}

rt_status rt_check_create(int64_t max_n, int32_t max_d, int32_t max_k, int32_t max_q) {
    if (max_n < 1 || max_n > kMaxN) return RT_EINVAL;
    if (max_d < 1 || max_d > kMaxD) return RT_EINVAL;
    if (max_k < 1 || max_k > kMaxK) return RT_EINVAL;
    if (max_q < 1 || max_q > kMaxQ) return RT_EINVAL;
    return RT_OK;
}

rt_status rt_check_upload(int64_t max_n, int32_t max_d, const void *corpus, int64_t n, int32_t d) {
    if (corpus == nullptr) return RT_EINVAL;
    if (n < 1 || n > max_n) return RT_EINVAL;
    if (d < 1 || d > max_d) return RT_EINVAL;
    return RT_OK;
}

rt_status rt_check_search(int32_t max_k, int32_t max_q, int64_t resident_n, const void *queries, int32_t q,
                          int32_t k, const void *out_idx, const void *out_scores) {
    if (queries == nullptr || out_idx == nullptr || out_scores == nullptr) return RT_EINVAL;
    if (q < 1 || q > max_q) return RT_EINVAL;
    if (k < 1 || k > max_k) return RT_EINVAL;
    if (resident_n < 1) return RT_ESTATE;
    if (k > resident_n) return RT_EINVAL;
    return RT_OK;
}

rt_status rt_check_search_metric(int32_t max_k, int32_t max_q, int64_t resident_n, const void *queries,
                                 int32_t q, int32_t k, int32_t metric, const void *out_idx, const void *out_scores) {
    if (metric != RT_METRIC_DOT && metric != RT_METRIC_COSINE) return RT_EINVAL;
    return rt_check_search(max_k, max_q, resident_n, queries, q, k, out_idx, out_scores);
}

rt_status rt_check_select(int32_t max_k, const void *values, int32_t dtype, int64_t n, int32_t k,
                          const void *out_idx, const void *out_values) {
    if (values == nullptr || out_idx == nullptr || out_values == nullptr) return RT_EINVAL;
    if (dtype != RT_DTYPE_INT32 && dtype != RT_DTYPE_FLOAT32) return RT_EINVAL;
    if ((reinterpret_cast<uintptr_t>(values) & 3u) != 0) return RT_EINVAL;
    if (n < 1 || n > kMaxN) return RT_EINVAL;
    if (k < 1 || k > max_k || k > n) return RT_EINVAL;
    return RT_OK;
}

static bool float_type(int32_t dtype) {
    return dtype == RT_DTYPE_FLOAT32 || dtype == RT_DTYPE_BFLOAT16 || dtype == RT_DTYPE_FLOAT16;
}

static bool misaligned(const void *p, int32_t dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == RT_DTYPE_FLOAT32 ? 3u : 1u)) != 0;
}

static bool bad_ld(int64_t ld, int64_t row) { return ld < row || ld > rt::kMaxLd; }

rt_status rt_check_quantize_rows_int8(const void *x, int32_t dtype, int64_t m, int32_t k, int64_t ldx,
                                      const void *q, int64_t ldq, const void *scale) {
    if (!float_type(dtype)) return RT_EINVAL;
    if (m < 0 || m > kMaxN || k < 1 || k > rt::kMaxRowK) return RT_EINVAL;
    if (bad_ld(ldx, k) || bad_ld(ldq, k)) return RT_EINVAL;
    if (m == 0) return RT_OK;  // an empty tensor's address may be null
    if (x == nullptr || q == nullptr || scale == nullptr) return RT_EINVAL;
    if (misaligned(x, dtype) || misaligned(scale, RT_DTYPE_FLOAT32)) return RT_EINVAL;
    return RT_OK;
}

rt_status rt_check_matmul_int8(const void *a, int64_t lda, const void *a_scale, const void *b, int64_t ldb,
                               const void *b_scale, const void *bias, const void *out, int32_t out_dtype,
                               int64_t ldo, int64_t m, int64_t n, int32_t k) {
    if (!float_type(out_dtype)) return RT_EINVAL;
    if (m < 0 || m > kMaxN || n < 1 || n > kMaxN || k < 1 || k > rt::kMaxRowK) return RT_EINVAL;
    if (m * n > rt::kMaxProduct) return RT_EINVAL;
    if (bad_ld(lda, k) || bad_ld(ldb, k) || bad_ld(ldo, n)) return RT_EINVAL;
    if (m == 0) return RT_OK;
    if (a == nullptr || a_scale == nullptr || b == nullptr || b_scale == nullptr || out == nullptr) return RT_EINVAL;
    if (misaligned(a_scale, RT_DTYPE_FLOAT32) || misaligned(b_scale, RT_DTYPE_FLOAT32) ||
        misaligned(bias, RT_DTYPE_FLOAT32) || misaligned(out, out_dtype))
        return RT_EINVAL;
    return RT_OK;
}

int64_t rt_linear_int8_workspace(int64_t m, int64_t n, int32_t k) {
    if (m < 0 || m > kMaxN || n < 1 || n > kMaxN || k < 1 || k > rt::kMaxRowK) return -1;
    if (m == 0 || rt::int8_few(m, n, k)) return 0;
    return m * rt::int8_padded(k) + (4 * m + 15) / 16 * 16;
}

rt_status rt_check_sample_rows(const void *logits, int32_t dtype, int64_t r, int64_t v, int64_t ld, const void *u,
                               const rt_sample_settings *settings, const void *out_token, const void *out_prob,
                               const void *workspace, int64_t workspace_bytes) {
    if (!float_type(dtype)) return RT_EINVAL;
    if (r < 0 || r > kMaxN || v < 1 || v > kMaxN || bad_ld(ld, v)) return RT_EINVAL;
    if (settings == nullptr) return RT_EINVAL;
    if (r == 0) return RT_OK;
    if (logits == nullptr || u == nullptr || out_token == nullptr) return RT_EINVAL;
    if (misaligned(logits, dtype) || misaligned(u, RT_DTYPE_FLOAT32) || misaligned(out_token, RT_DTYPE_FLOAT32) ||
        misaligned(out_prob, RT_DTYPE_FLOAT32) || misaligned(settings->temperatures, RT_DTYPE_FLOAT32) ||
        misaligned(settings->top_ks, RT_DTYPE_FLOAT32) || misaligned(settings->top_ps, RT_DTYPE_FLOAT32) ||
        misaligned(settings->min_ps, RT_DTYPE_FLOAT32))
        return RT_EINVAL;
    const int64_t need = rt_sample_rows_workspace(r, v);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return RT_EINVAL;
    if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return RT_EINVAL;
    return RT_OK;
}

int64_t rt_sample_rows_workspace(int64_t r, int64_t v) {
    if (r < 0 || r > kMaxN || v < 1 || v > kMaxN) return -1;
    return rt::sample_workspace(r, v);
}

}  // extern "C"
