// Argument checks that the operators' entry points share.
#pragma once

#include <hip/hip_runtime.h>

#include "moe_host.h"
#include "moe_w4a16.h"

namespace moe {

constexpr int kMaxExperts = 4096, kMaxTopk = 64, kMaxRows = 1 << 30, kMaxDim = 1 << 20;
constexpr int64_t kMaxLd = 1 << 21;   // values from row to row: a tile's rows lie within 2 GiB of its first

inline bool type_ok(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F16 || t == MOE_DTYPE_F32; }
inline int type_size(int t) { return t == MOE_DTYPE_F32 ? 4 : 2; }

inline moe_status_t check_matrix(const char* name, const void* p, int64_t ld, int64_t width) {
  if (!p || !aligned(p, 16)) return fail(MOE_ERR_INVALID_ARG, "%s NULL or not 16-byte aligned", name);
  if (ld < width || ld % 8 || ld > kMaxLd)
    return fail(MOE_ERR_INVALID_ARG, "%s: %lld values from row to row; a multiple of 8 in %lld..%lld is needed", name,
                (long long)ld, (long long)width, (long long)kMaxLd);
  return MOE_OK;
}

inline moe_status_t check_router(const void* logits, int dtype, int64_t ld, int T, int E, int topk, int score) {
  if (!type_ok(dtype)) return fail(MOE_ERR_INVALID_ARG, "dtype = %d", dtype);
  if (E < 1 || E > kMaxExperts) return fail(MOE_ERR_INVALID_ARG, "E = %d outside 1..%d", E, kMaxExperts);
  if (T < 0 || T > kMaxRows / kMaxTopk)
    return fail(MOE_ERR_INVALID_ARG, "T = %d outside 0..%d", T, kMaxRows / kMaxTopk);
  if (topk < 1 || topk > E || topk > kMaxTopk)
    return fail(MOE_ERR_INVALID_ARG, "topk = %d outside 1..min(E, %d)", topk, kMaxTopk);
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return fail(MOE_ERR_INVALID_ARG, "score = %d", score);
  if (T > 0 && (!logits || !aligned(logits, type_size(dtype))))
    return fail(MOE_ERR_INVALID_ARG, "logits NULL or misaligned");
  if (ld < E) return fail(MOE_ERR_INVALID_ARG, "logits: %lld values from row to row, E = %d", (long long)ld, E);
  return MOE_OK;
}

inline moe_status_t check_groups(int dtype, const int32_t* offsets, int E, int M, int N, int K, int out_dtype, int unit) {
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
    return fail(MOE_ERR_INVALID_ARG, "dtype = %d: BF16 or FP16 operands", dtype);
  if (!type_ok(out_dtype)) return fail(MOE_ERR_INVALID_ARG, "out_dtype = %d", out_dtype);
  if (E < 1 || E > kMaxExperts) return fail(MOE_ERR_INVALID_ARG, "E = %d outside 1..%d", E, kMaxExperts);
  if (M < 0 || M > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "M = %d outside 0..2^30", M);
  if (N < 8 || N % 8 || N > kMaxDim || K < unit || K % unit || K > kMaxDim)
    return fail(MOE_ERR_INVALID_ARG, "N = %d, K = %d: multiples of 8 and %d up to 2^20", N, K, unit);
  if (!offsets || !aligned(offsets, 4)) return fail(MOE_ERR_INVALID_ARG, "offsets NULL or misaligned");
  return MOE_OK;
}

inline moe_status_t launched(hipError_t e, const char* what) { return e == hipSuccess ? ok() : hip_fail(e, what); }

inline int scale_cols(int K) { return (K / 32 + 15) / 16 * 16; }

inline moe_status_t check_mx(const char* name, const uint8_t* q, const uint8_t* scales) {
  if (!q || !scales || !aligned(q, 16) || !aligned(scales, 16))
    return fail(MOE_ERR_INVALID_ARG, "%s: codes or scales NULL or not 16-byte aligned", name);
  return MOE_OK;
}

inline moe_status_t check_mx_rows(int dtype, int64_t rows, int K, const void* x, int64_t ld, const uint8_t* q,
                           const uint8_t* scales) {
  if (!type_ok(dtype)) return fail(MOE_ERR_INVALID_ARG, "dtype = %d", dtype);
  if (K < 32 || K % 32 || K > kMaxDim) return fail(MOE_ERR_INVALID_ARG, "K = %d: a multiple of 32 up to 2^20", K);
  if (rows < 0 || rows > (int64_t)1 << 40 || (rows > 0 && K > ((int64_t)1 << 42) / rows))
    return fail(MOE_ERR_INVALID_ARG, "rows = %lld", (long long)rows);
  if (rows == 0) return MOE_OK;
  if (!x || !aligned(x, 16) || ld < K || ld % 8)
    return fail(MOE_ERR_INVALID_ARG, "values NULL or not 16-byte aligned, or rows not a multiple of 8 values apart");
  return check_mx("rows", q, scales);
}

}  // namespace moe
