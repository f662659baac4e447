// C ABI of the operators around the expert layer: router top-k, grouped
// products over ragged rows with their gradients, MXFP4 quantisation and
// product. Arguments are validated here before anything is enqueued.
#include <hip/hip_runtime.h>

#include "moe_ops_check.h"
#include "moe_ragged.h"

using namespace moe;

extern "C" {

moe_status_t moe_router_topk(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t topk,
                             int32_t score, const float* bias, int32_t renorm, float scale, int32_t* topk_ids,
                             float* topk_w, moe_stream_t stream) {
  moe_status_t st = check_router(logits, dtype, ld, T, E, topk, score);
  if (st != MOE_OK) return st;
  if (T == 0) return ok();
  if (!topk_ids || !topk_w || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(bias, 4))
    return fail(MOE_ERR_INVALID_ARG, "topk_ids / topk_w NULL or misaligned, or bias misaligned");
  RouterParams p{};
  p.logits = logits, p.ld = ld, p.T = T, p.E = E, p.topk = topk;
  p.sigmoid = score == MOE_SCORE_SIGMOID, p.renorm = renorm != 0;
  p.bias = bias, p.scale = scale, p.ids = topk_ids, p.w = topk_w;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("router_topk", s, [&] { return launch_router_topk(p, dtype, s); }), "router launch");
}

moe_status_t moe_router_topk_grad(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t topk,
                                  int32_t score, int32_t renorm, float scale, const int32_t* topk_ids,
                                  const float* d_topk_w, void* d_logits, int64_t d_ld, moe_stream_t stream) {
  moe_status_t st = check_router(logits, dtype, ld, T, E, topk, score);
  if (st != MOE_OK) return st;
  if (d_ld < E) return fail(MOE_ERR_INVALID_ARG, "d_logits: %lld values from row to row, E = %d", (long long)d_ld, E);
  if (T == 0) return ok();
  if (!topk_ids || !d_topk_w || !d_logits || !aligned(topk_ids, 4) || !aligned(d_topk_w, 4) ||
      !aligned(d_logits, type_size(dtype)))
    return fail(MOE_ERR_INVALID_ARG, "topk_ids / d_topk_w / d_logits NULL or misaligned");
  RouterParams p{};
  p.logits = logits, p.ld = ld, p.T = T, p.E = E, p.topk = topk;
  p.sigmoid = score == MOE_SCORE_SIGMOID, p.renorm = renorm != 0;
  p.scale = scale, p.ids = const_cast<int32_t*>(topk_ids), p.dw = d_topk_w, p.dlogits = d_logits, p.d_ld = d_ld;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("router_topk_grad", s, [&] { return launch_router_topk_grad(p, dtype, s); }),
                  "router gradient launch");
}

moe_status_t moe_grouped_gemm(const void* a, int64_t a_ld, const void* w, int64_t w_stride, int64_t w_ld,
                              int32_t dtype, const int32_t* offsets, int32_t E, int32_t M, int32_t N, int32_t K,
                              void* out, int64_t out_ld, int32_t out_dtype, moe_stream_t stream) {
  moe_status_t st = check_groups(dtype, offsets, E, M, N, K, out_dtype, 8);
  if (st != MOE_OK) return st;
  if (M == 0) return ok();
  if ((st = check_matrix("a", a, a_ld, K)) != MOE_OK || (st = check_matrix("w", w, w_ld, K)) != MOE_OK ||
      (st = check_matrix("out", out, out_ld, N)) != MOE_OK)
    return st;
  if (w_stride % 8 || w_stride < 0) return fail(MOE_ERR_INVALID_ARG, "w: experts not a multiple of 8 values apart");
  RaggedParams p{};
  p.p = w, p.p_stride = w_stride * 2, p.p_ld = w_ld * 2;
  p.q = a, p.q_ld = a_ld * 2;
  p.offsets = offsets, p.E = E, p.M = M, p.I = N, p.C = K;
  p.out = out, p.out_ld = out_ld, p.out_type = out_dtype;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("grouped_gemm", s, [&] { return launch_ragged_gemm(p, WAY_FWD, dtype, s); }),
                  "grouped GEMM launch");
}

moe_status_t moe_grouped_gemm_dgrad(const void* dy, int64_t dy_ld, const void* w, int64_t w_stride, int64_t w_ld,
                                    int32_t dtype, const int32_t* offsets, int32_t E, int32_t M, int32_t N, int32_t K,
                                    void* da, int64_t da_ld, int32_t out_dtype, moe_stream_t stream) {
  moe_status_t st = check_groups(dtype, offsets, E, M, N, K, out_dtype, 8);
  if (st != MOE_OK) return st;
  if (M == 0) return ok();
  if ((st = check_matrix("dy", dy, dy_ld, N)) != MOE_OK || (st = check_matrix("w", w, w_ld, K)) != MOE_OK ||
      (st = check_matrix("da", da, da_ld, K)) != MOE_OK)
    return st;
  if (w_stride % 8 || w_stride < 0) return fail(MOE_ERR_INVALID_ARG, "w: experts not a multiple of 8 values apart");
  RaggedParams p{};
  p.p = w, p.p_stride = w_stride * 2, p.p_ld = w_ld * 2;
  p.q = dy, p.q_ld = dy_ld * 2;
  p.offsets = offsets, p.E = E, p.M = M, p.I = K, p.C = N;
  p.out = da, p.out_ld = da_ld, p.out_type = out_dtype;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("grouped_gemm_dgrad", s, [&] { return launch_ragged_gemm(p, WAY_DGRAD, dtype, s); }),
                  "grouped GEMM input gradient launch");
}

moe_status_t moe_grouped_gemm_wgrad(const void* dy, int64_t dy_ld, const void* a, int64_t a_ld, int32_t dtype,
                                    const int32_t* offsets, int32_t E, int32_t M, int32_t N, int32_t K, void* dw,
                                    int64_t dw_stride, int64_t dw_ld, int32_t out_dtype, moe_stream_t stream) {
  moe_status_t st = check_groups(dtype, offsets, E, M, N, K, out_dtype, 8);
  if (st != MOE_OK) return st;
  if (M > 0 &&
      ((st = check_matrix("dy", dy, dy_ld, N)) != MOE_OK || (st = check_matrix("a", a, a_ld, K)) != MOE_OK))
    return st;
  if ((st = check_matrix("dw", dw, dw_ld, K)) != MOE_OK) return st;
  if (dw_stride % 8 || dw_stride < (int64_t)(N - 1) * dw_ld + K)
    return fail(MOE_ERR_INVALID_ARG, "dw: experts overlap, or are not a multiple of 8 values apart");
  RaggedParams p{};
  p.p = a, p.p_ld = a_ld * 2;
  p.q = dy, p.q_ld = dy_ld * 2;
  p.offsets = offsets, p.E = E, p.M = M, p.I = K, p.J = N;
  p.out = dw, p.out_ld = dw_ld, p.out_stride = dw_stride, p.out_type = out_dtype;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("grouped_gemm_wgrad", s, [&] { return launch_ragged_gemm(p, WAY_WGRAD, dtype, s); }),
                  "grouped GEMM weight gradient launch");
}

int32_t moe_mx_scale_cols(int32_t K) {
  if (K < 32 || K % 32 || K > kMaxDim) {
    fail(MOE_ERR_INVALID_ARG, "K = %d: a multiple of 32 up to 2^20", K);
    return 0;
  }
  return scale_cols(K);
}

moe_status_t moe_mx_quant(const void* x, int32_t dtype, int64_t ld, int64_t rows, int32_t K, uint8_t* q,
                          uint8_t* scales, moe_stream_t stream) {
  moe_status_t st = check_mx_rows(dtype, rows, K, x, ld, q, scales);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  const hipStream_t s = (hipStream_t)stream;
  return launched(
      run("mx_quant", s, [&] { return launch_mx_quant(x, dtype, rows, K, ld, q, scales, scale_cols(K), s); }),
      "MXFP4 quantisation launch");
}

moe_status_t moe_mx_dequant(const uint8_t* q, const uint8_t* scales, int64_t rows, int32_t K, void* out, int32_t dtype,
                            int64_t ld, moe_stream_t stream) {
  moe_status_t st = check_mx_rows(dtype, rows, K, out, ld, q, scales);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  const hipStream_t s = (hipStream_t)stream;
  return launched(
      run("mx_dequant", s, [&] { return launch_mx_dequant(q, scales, rows, K, scale_cols(K), out, dtype, ld, s); }),
      "MXFP4 dequantisation launch");
}

moe_status_t moe_mx_grouped_gemm(const uint8_t* aq, const uint8_t* a_scales, const uint8_t* wq,
                                 const uint8_t* w_scales, const int32_t* offsets, int32_t E, int32_t M, int32_t N,
                                 int32_t K, void* out, int64_t out_ld, int32_t out_dtype, moe_stream_t stream) {
  moe_status_t st = check_groups(MOE_DTYPE_BF16, offsets, E, M, N, K, out_dtype, 32);
  if (st != MOE_OK) return st;
  if (M == 0) return ok();
  if ((st = check_mx("a", aq, a_scales)) != MOE_OK || (st = check_mx("w", wq, w_scales)) != MOE_OK ||
      (st = check_matrix("out", out, out_ld, N)) != MOE_OK)
    return st;
  RaggedParams p{};
  p.p = wq, p.p_ld = K / 2, p.p_stride = (int64_t)N * (K / 2);
  p.q = aq, p.q_ld = K / 2;
  p.s_ld = scale_cols(K), p.ps = w_scales, p.ps_stride = (int64_t)N * p.s_ld, p.qs = a_scales;
  p.offsets = offsets, p.E = E, p.M = M, p.I = N, p.C = K;
  p.out = out, p.out_ld = out_ld, p.out_type = out_dtype;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("mx_grouped_gemm", s, [&] { return launch_ragged_gemm(p, WAY_MX, 0, s); }),
                  "MXFP4 grouped GEMM launch");
}

}  // extern "C"
