// C ABI of the operators of a training step around the experts' products:
// balance loss of the router, a token's sum of rows, rows in 8 bits, SwiGLU
// with such a checkpoint, and their gradients, and the experts' product with an
// epilogue. Arguments are validated here
// before anything is enqueued.
#include <hip/hip_runtime.h>

#include "moe_ops_check.h"
#include "moe_ragged.h"
#include "moe_step.h"

using namespace moe;

namespace {

constexpr int kMaxSequences = 1 << 20;
constexpr int64_t kMaxCounts = (int64_t)1 << 30;   // S * E

moe_status_t check_balance(const void* logits, int dtype, int64_t ld, int T, int E, int topk, int score,
                           const int32_t* offsets, int S) {
  moe_status_t st = check_router(logits, dtype, ld, T, E, topk, score);
  if (st != MOE_OK) return st;
  if (S < 1 || S > kMaxSequences || (int64_t)S * E > kMaxCounts)
    return fail(MOE_ERR_INVALID_ARG, "S = %d outside 1..2^20, or S * E past 2^30", S);
  if (!offsets && S != 1) return fail(MOE_ERR_INVALID_ARG, "offsets NULL with S = %d sequences", S);
  if (!aligned(offsets, 4)) return fail(MOE_ERR_INVALID_ARG, "offsets misaligned");
  return MOE_OK;
}

moe_status_t check_combine(int dtype, int R, int H, int T, int topk, const int32_t* slots, const float* w) {
  if (!type_ok(dtype)) return fail(MOE_ERR_INVALID_ARG, "dtype = %d", dtype);
  if (H < 8 || H % 8 || H > kMaxDim) return fail(MOE_ERR_INVALID_ARG, "H = %d: a multiple of 8 up to 2^20", H);
  if (T < 0 || T > kMaxRows / kMaxTopk)
    return fail(MOE_ERR_INVALID_ARG, "T = %d outside 0..%d", T, kMaxRows / kMaxTopk);
  if (topk < 1 || topk > kMaxTopk) return fail(MOE_ERR_INVALID_ARG, "topk = %d outside 1..%d", topk, kMaxTopk);
  if (R < 0 || R > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "R = %d outside 0..2^30", R);
  if (T > 0 && (!slots || !aligned(slots, 4) || !aligned(w, 4)))
    return fail(MOE_ERR_INVALID_ARG, "slots NULL or misaligned, or weights misaligned");
  return MOE_OK;
}

moe_status_t check_live(const int32_t* offsets, int E) {
  if (!offsets) return MOE_OK;
  if (E < 1 || E > kMaxExperts) return fail(MOE_ERR_INVALID_ARG, "E = %d outside 1..%d", E, kMaxExperts);
  if (!aligned(offsets, 4)) return fail(MOE_ERR_INVALID_ARG, "offsets misaligned");
  return MOE_OK;
}

int mx8_cols(int K) { return ((K + 31) / 32 + 15) / 16 * 16; }

moe_status_t check_mx8_rows(int dtype, int64_t rows, int K) {
  if (!type_ok(dtype)) return fail(MOE_ERR_INVALID_ARG, "dtype = %d", dtype);
  if (K < 8 || K % 8 || K > kMaxDim) return fail(MOE_ERR_INVALID_ARG, "K = %d: a multiple of 8 up to 2^20", K);
  if (rows < 0 || rows > (int64_t)1 << 40 || (rows > 0 && K > ((int64_t)1 << 42) / rows))
    return fail(MOE_ERR_INVALID_ARG, "rows = %lld", (long long)rows);
  return MOE_OK;
}

moe_status_t check_swiglu(int dtype, int rows, int I, const int32_t* offsets, int E) {
  if (!type_ok(dtype)) return fail(MOE_ERR_INVALID_ARG, "dtype = %d", dtype);
  if (I < 8 || I % 8 || I > kMaxDim / 2) return fail(MOE_ERR_INVALID_ARG, "I = %d: a multiple of 8 up to 2^19", I);
  if (rows < 0 || rows > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "rows = %d outside 0..2^30", rows);
  return check_live(offsets, E);
}

}  // namespace

extern "C" {

int64_t moe_router_balance_bytes(int32_t T, int32_t E, int32_t S) {
  if (T < 0 || T > kMaxRows / kMaxTopk || E < 1 || E > kMaxExperts || S < 1 || S > kMaxSequences ||
      (int64_t)S * E > kMaxCounts) {
    fail(MOE_ERR_INVALID_ARG, "T = %d, E = %d, S = %d outside the balance loss's range", T, E, S);
    return -1;
  }
  return (int64_t)balance_ws_bytes(T, E, S);
}

moe_status_t moe_router_balance(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                                const int32_t* topk_ids, int32_t topk, int32_t score, const int32_t* offsets,
                                int32_t S, float* loss, int32_t* counts, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
  moe_status_t st = check_balance(logits, dtype, ld, T, E, topk, score, offsets, S);
  if (st != MOE_OK) return st;
  if ((T > 0 && !topk_ids) || !loss || !counts || !aligned(topk_ids, 4) || !aligned(loss, 4) || !aligned(counts, 4))
    return fail(MOE_ERR_INVALID_ARG, "topk_ids / loss / counts NULL or misaligned");
  const size_t need = balance_ws_bytes(T, E, S);
  if (need > 0 && (!ws || !aligned(ws, 16)))
    return fail(MOE_ERR_INVALID_ARG, "workspace NULL or not 16-byte aligned");
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  BalanceParams p{};
  p.logits = logits, p.ld = ld, p.T = T, p.E = E, p.topk = topk, p.sigmoid = score == MOE_SCORE_SIGMOID;
  p.ids = topk_ids, p.offsets = offsets, p.S = S, p.counts = counts, p.loss = loss, p.ws = ws;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("router_balance", s, [&] { return launch_balance(p, dtype, s); }), "balance loss launch");
}

moe_status_t moe_router_balance_grad(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                                     int32_t topk, int32_t score, const int32_t* offsets, int32_t S,
                                     const int32_t* counts, const float* d_loss, const void* add, int64_t add_ld,
                                     void* d_logits, int64_t d_ld, moe_stream_t stream) {
  moe_status_t st = check_balance(logits, dtype, ld, T, E, topk, score, offsets, S);
  if (st != MOE_OK) return st;
  if (d_ld < E) return fail(MOE_ERR_INVALID_ARG, "d_logits: %lld values from row to row, E = %d", (long long)d_ld, E);
  if (add && add_ld < E) return fail(MOE_ERR_INVALID_ARG, "add: %lld values from row to row, E = %d", (long long)add_ld, E);
  if (T == 0) return ok();
  if (!counts || !d_loss || !d_logits || !aligned(counts, 4) || !aligned(d_loss, 4) ||
      !aligned(d_logits, type_size(dtype)) || !aligned(add, type_size(dtype)))
    return fail(MOE_ERR_INVALID_ARG, "counts / d_loss / d_logits NULL or misaligned, or add misaligned");
  BalanceParams p{};
  p.logits = logits, p.ld = ld, p.T = T, p.E = E, p.topk = topk, p.sigmoid = score == MOE_SCORE_SIGMOID;
  p.offsets = offsets, p.S = S, p.counts_in = counts, p.d_loss = d_loss;
  p.add = add, p.add_ld = add_ld, p.d_logits = d_logits, p.d_ld = d_ld;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("router_balance_grad", s, [&] { return launch_balance_grad(p, dtype, s); }),
                  "balance gradient launch");
}

moe_status_t moe_combine(const void* y, int32_t dtype, int64_t y_ld, int32_t R, int32_t H, const int32_t* slots,
                         int32_t T, int32_t topk, const float* w, void* out, int64_t out_ld, int32_t out_dtype,
                         moe_stream_t stream) {
  moe_status_t st = check_combine(dtype, R, H, T, topk, slots, w);
  if (st != MOE_OK) return st;
  if (!type_ok(out_dtype)) return fail(MOE_ERR_INVALID_ARG, "out_dtype = %d", out_dtype);
  if (T == 0) return ok();
  if ((R > 0 && (st = check_matrix("y", y, y_ld, H)) != MOE_OK) ||
      (st = check_matrix("out", out, out_ld, H)) != MOE_OK)
    return st;
  CombineParams p{};
  p.y = y, p.y_ld = y_ld, p.R = R, p.H = H, p.T = T, p.topk = topk, p.slots = slots, p.w = w;
  p.out = out, p.out_ld = out_ld;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("combine", s, [&] { return launch_combine_out(p, dtype, out_dtype, s); }), "combine launch");
}

moe_status_t moe_combine_grad(const void* d_out, int32_t dtype, int64_t d_ld, int32_t T, int32_t H,
                              const int32_t* slots, int32_t topk, const float* w, const void* y, int64_t y_ld,
                              const int32_t* row_src, const int32_t* offsets, int32_t E, void* d_y, int64_t dy_ld,
                              int32_t R, float* d_w, moe_stream_t stream) {
  moe_status_t st = check_combine(dtype, R, H, T, topk, slots, w);
  if (st != MOE_OK || (st = check_live(offsets, E)) != MOE_OK) return st;
  if (!row_src && offsets) return fail(MOE_ERR_INVALID_ARG, "offsets without row_src");
  if (!aligned(row_src, 4) || !aligned(d_w, 4)) return fail(MOE_ERR_INVALID_ARG, "row_src or d_w misaligned");
  if (d_w && !y && R > 0) return fail(MOE_ERR_INVALID_ARG, "d_w without y");
  if (T > 0 && (st = check_matrix("d_out", d_out, d_ld, H)) != MOE_OK) return st;
  if (R > 0 && ((st = check_matrix("d_y", d_y, dy_ld, H)) != MOE_OK ||
                (y && (st = check_matrix("y", y, y_ld, H)) != MOE_OK)))
    return st;
  if (T == 0 && R == 0) return ok();
  CombineParams p{};
  p.y = d_w ? y : nullptr, p.y_ld = y_ld, p.R = R, p.H = H, p.T = T, p.topk = topk, p.slots = slots, p.w = w;
  p.d_out = d_out, p.d_ld = d_ld, p.row_src = row_src, p.offsets = offsets, p.E = E;
  p.d_y = d_y, p.dy_ld = dy_ld, p.d_w = d_w;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("combine_grad", s, [&] { return launch_combine_grad(p, dtype, s); }),
                  "combine gradient launch");
}

int32_t moe_mx8_scale_cols(int32_t K) {
  if (K < 8 || K % 8 || K > kMaxDim) {
    fail(MOE_ERR_INVALID_ARG, "K = %d: a multiple of 8 up to 2^20", K);
    return 0;
  }
  return mx8_cols(K);
}

moe_status_t moe_mx8_quant(const void* x, int32_t dtype, int64_t ld, int64_t rows, int32_t K, int8_t* q,
                           uint8_t* scales, moe_stream_t stream) {
  moe_status_t st = check_mx8_rows(dtype, rows, K);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  if ((st = check_matrix("x", x, ld, K)) != MOE_OK || (st = check_mx("rows", (const uint8_t*)q, scales)) != MOE_OK)
    return st;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("mx8_quant", s, [&] { return launch_mx8_quant(x, dtype, rows, K, ld, q, scales, mx8_cols(K), s); }),
                  "8-bit quantisation launch");
}

moe_status_t moe_mx8_dequant(const int8_t* q, const uint8_t* scales, int64_t rows, int32_t K, const int32_t* row_src,
                             int32_t topk, const int32_t* offsets, int32_t E, void* out, int32_t dtype, int64_t ld,
                             int64_t out_rows, moe_stream_t stream) {
  moe_status_t st = check_mx8_rows(dtype, rows, K);
  if (st != MOE_OK || (st = check_mx8_rows(dtype, out_rows, K)) != MOE_OK || (st = check_live(offsets, E)) != MOE_OK)
    return st;
  if (row_src) {
    if (!aligned(row_src, 4)) return fail(MOE_ERR_INVALID_ARG, "row_src misaligned");
    if (topk < 1) return fail(MOE_ERR_INVALID_ARG, "topk = %d: at least 1", topk);
    if (rows > kMaxRows || out_rows > kMaxRows)
      return fail(MOE_ERR_INVALID_ARG, "rows = %lld and %lld: up to 2^30 with row_src", (long long)rows,
                  (long long)out_rows);
  } else if (rows != out_rows) {
    return fail(MOE_ERR_INVALID_ARG, "out_rows = %lld, rows = %lld without row_src", (long long)out_rows,
                (long long)rows);
  }
  if (out_rows == 0) return ok();
  if ((rows > 0 && (st = check_mx("rows", (const uint8_t*)q, scales)) != MOE_OK) ||
      (st = check_matrix("out", out, ld, K)) != MOE_OK)
    return st;
  Mx8Rows p{};
  p.q = q, p.scales = scales, p.rows = rows, p.K = K, p.s_ld = mx8_cols(K);
  p.row_src = row_src, p.topk = topk, p.live = LiveRows{offsets, E}, p.out_rows = out_rows, p.out = out, p.ld = ld;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("mx8_dequant", s, [&] { return launch_mx8_dequant(p, dtype, s); }),
                  "8-bit dequantisation launch");
}

moe_status_t moe_swiglu_save(const void* h, int32_t dtype, int64_t h_ld, int32_t rows, int32_t inter,
                             const int32_t* offsets, int32_t E, void* a, int64_t a_ld, int8_t* q, uint8_t* scales,
                             moe_stream_t stream) {
  moe_status_t st = check_swiglu(dtype, rows, inter, offsets, E);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  if ((st = check_matrix("h", h, h_ld, 2 * (int64_t)inter)) != MOE_OK ||
      (st = check_matrix("a", a, a_ld, inter)) != MOE_OK ||
      (st = check_mx("h", (const uint8_t*)q, scales)) != MOE_OK)
    return st;
  SwigluParams p{};
  p.h = h, p.h_ld = h_ld, p.rows = rows, p.I = inter, p.s_ld = mx8_cols(inter), p.live = LiveRows{offsets, E};
  p.q = q, p.scales = scales, p.a = a, p.a_ld = a_ld;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("swiglu_save", s, [&] { return launch_swiglu_save(p, dtype, s); }), "SwiGLU launch");
}

moe_status_t moe_swiglu_grad(const void* h, int64_t h_ld, const int8_t* q, const uint8_t* scales, int32_t dtype,
                             int32_t rows, int32_t inter, const void* d_a, int64_t da_ld, const int32_t* offsets,
                             int32_t E, void* d_h, int64_t dh_ld, void* a, int64_t a_ld, moe_stream_t stream) {
  moe_status_t st = check_swiglu(dtype, rows, inter, offsets, E);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  if (h && (q || scales)) return fail(MOE_ERR_INVALID_ARG, "h as values and as a checkpoint");
  if ((h && (st = check_matrix("h", h, h_ld, 2 * (int64_t)inter)) != MOE_OK) ||
      (!h && (st = check_mx("h", (const uint8_t*)q, scales)) != MOE_OK) ||
      (st = check_matrix("d_a", d_a, da_ld, inter)) != MOE_OK ||
      (st = check_matrix("d_h", d_h, dh_ld, 2 * (int64_t)inter)) != MOE_OK ||
      (a && (st = check_matrix("a", a, a_ld, inter)) != MOE_OK))
    return st;
  SwigluParams p{};
  p.h = h, p.h_ld = h_ld, p.rows = rows, p.I = inter, p.s_ld = mx8_cols(inter), p.live = LiveRows{offsets, E};
  p.q_in = q, p.scales_in = scales, p.d_a = d_a, p.da_ld = da_ld, p.d_h = d_h, p.dh_ld = dh_ld, p.a = a, p.a_ld = a_ld;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("swiglu_grad", s, [&] { return launch_swiglu_grad(p, dtype, s); }), "SwiGLU gradient launch");
}

moe_status_t moe_grouped_linear(const void* a, int64_t a_ld, const void* w, int64_t w_stride, int64_t w_ld,
                                int32_t dtype, const int32_t* offsets, int32_t E, int32_t M, int32_t N, int32_t K,
                                const void* bias, int32_t bias_dtype, int64_t bias_ld, int32_t act,
                                const void* residual, int64_t res_ld, void* out, int64_t out_ld, int32_t out_dtype,
                                moe_stream_t stream) {
  moe_status_t st = check_groups(dtype, offsets, E, M, N, K, out_dtype, 8);
  if (st != MOE_OK) return st;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return fail(MOE_ERR_INVALID_ARG, "act = %d", act);
  const bool glu = act == MOE_ACT_SWIGLU;
  if (glu && N % 16) return fail(MOE_ERR_INVALID_ARG, "N = %d: a multiple of 16 for gate | up weights", N);
  if (bias) {
    if (!type_ok(bias_dtype)) return fail(MOE_ERR_INVALID_ARG, "bias_dtype = %d", bias_dtype);
    if ((st = check_matrix("bias", bias, bias_ld, N)) != MOE_OK) return st;
  }
  if (M == 0) return ok();
  const int I = glu ? N / 2 : N;
  if ((st = check_matrix("a", a, a_ld, K)) != MOE_OK || (st = check_matrix("w", w, w_ld, K)) != MOE_OK ||
      (st = check_matrix("out", out, out_ld, I)) != MOE_OK ||
      (residual && (st = check_matrix("residual", residual, res_ld, I)) != MOE_OK))
    return st;
  if (w_stride % 8 || w_stride < 0) return fail(MOE_ERR_INVALID_ARG, "w: experts not a multiple of 8 values apart");
  RaggedParams p{};
  p.p = w, p.p_stride = w_stride * 2, p.p_ld = w_ld * 2;
  p.q = a, p.q_ld = a_ld * 2;
  p.offsets = offsets, p.E = E, p.M = M, p.I = I, p.C = K;
  p.out = out, p.out_ld = out_ld, p.out_type = out_dtype;
  p.epi.bias = bias, p.epi.bias_ld = bias_ld, p.epi.bias_type = bias_dtype;
  p.epi.swiglu = glu, p.epi.res = residual, p.epi.res_ld = res_ld;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("grouped_linear", s, [&] { return launch_ragged_linear(p, dtype, s); }),
                  "grouped linear launch");
}

int64_t moe_grouped_bias_grad_bytes(int32_t E, int32_t M, int32_t N) {
  if (E < 1 || E > kMaxExperts || M < 0 || M > kMaxRows || N < 8 || N % 8 || N > kMaxDim) {
    fail(MOE_ERR_INVALID_ARG, "E = %d, M = %d, N = %d outside the bias gradient's range", E, M, N);
    return -1;
  }
  return (int64_t)bias_grad_ws_bytes(E, M, N);
}

moe_status_t moe_grouped_bias_grad(const void* dy, int64_t dy_ld, int32_t dtype, const int32_t* offsets, int32_t E,
                                   int32_t M, int32_t N, void* db, int64_t db_ld, int32_t out_dtype, void* ws,
                                   size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = check_groups(dtype, offsets, E, M, N, 8, out_dtype, 8);
  if (st != MOE_OK) return st;
  if ((M > 0 && (st = check_matrix("dy", dy, dy_ld, N)) != MOE_OK) ||
      (st = check_matrix("db", db, db_ld, N)) != MOE_OK)
    return st;
  const size_t need = bias_grad_ws_bytes(E, M, N);
  if (need > 0 && (!ws || !aligned(ws, 16)))
    return fail(MOE_ERR_INVALID_ARG, "workspace NULL or not 16-byte aligned");
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  BiasGradParams p{};
  p.dy = dy, p.ld = dy_ld, p.offsets = offsets, p.E = E, p.M = M, p.N = N, p.db = db, p.db_ld = db_ld, p.ws = ws;
  const hipStream_t s = (hipStream_t)stream;
  return launched(run("grouped_bias_grad", s, [&] { return launch_bias_grad(p, dtype, out_dtype, s); }),
                  "bias gradient launch");
}

}  // extern "C"
