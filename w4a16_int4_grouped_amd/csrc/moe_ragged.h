// Grouped products over ragged groups of rows: parameters and launchers of
// the kernels behind moe_grouped_gemm, its two gradients and
// moe_mx_grouped_gemm.
//
// All four are one product per expert, out[j][i] = sum_c Q(j, c) P(i, c),
// written with i along the output's rows:
//   forward    j token row, i = n, c = k: Q = a, P = w[e]       (both contiguous along c)
//   dgrad      j token row, i = k, c = n: Q = dy, P = w[e]^T    (P contiguous along i)
//   wgrad      j = n, i = k, c = token row: Q = dy^T, P = a^T   (both contiguous along the output's axes)
//   MX         as forward, on FP4 codes with a scale per 32 of c
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

enum RaggedWay : int { WAY_FWD = 0, WAY_DGRAD = 1, WAY_WGRAD = 2, WAY_MX = 3 };
enum RaggedType : int { TYPE_BF16 = 0, TYPE_F16 = 1, TYPE_F32 = 2 };   // moe_dtype_t

struct RaggedParams {
  const void* p;          // weights (wgrad: a)
  const void* q;          // token rows (a; dgrad and wgrad: dy)
  const uint8_t* ps;      // MX scales of the weights [E][I][s_ld]
  const uint8_t* qs;      //   and of the token rows [M][s_ld]
  int64_t p_stride, ps_stride;   // bytes from expert to expert
  int64_t p_ld, q_ld, s_ld;      // bytes from row to row
  const int32_t* offsets;        // device [E + 1]
  int E, M;
  int I;                  // output columns
  int J;                  // wgrad: output rows of an expert
  int C;                  // contraction length (values; wgrad: the group's rows)
  void* out;
  int64_t out_ld, out_stride;    // elements; wgrad: from expert to expert
  int out_type;
  int stream_out;         // set by the launcher: the output passes the caches by
};

// type: of both operands (bf16 / f16), ignored for WAY_MX.
hipError_t launch_ragged_gemm(const RaggedParams& p, int way, int type, hipStream_t s);

// e2m1 codes (low nibble first) and E8M0 scale bytes of `rows` rows of K
// values, and back. x_ld / out_ld in elements; codes [rows][K/2], scales
// [rows][s_ld].
hipError_t launch_mx_quant(const void* x, int type, int64_t rows, int K, int64_t x_ld, uint8_t* q, uint8_t* scales,
                           int s_ld, hipStream_t s);
hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* scales, int64_t rows, int K, int s_ld, void* out,
                             int type, int64_t out_ld, hipStream_t s);

struct RouterParams {
  const void* logits;     // [T][ld]
  int64_t ld;
  int T, E, topk;
  int sigmoid, renorm;
  const float* bias;      // [E] or NULL
  float scale;
  int32_t* ids;           // [T][topk]
  float* w;               // [T][topk]
  const float* dw;        // gradient of w
  void* dlogits;          // [T][d_ld]
  int64_t d_ld;
};
hipError_t launch_router_topk(const RouterParams& p, int type, hipStream_t s);
hipError_t launch_router_topk_grad(const RouterParams& p, int type, hipStream_t s);

}  // namespace moe
