// Operators of a training step around the experts' products: parameters and
// launchers of the kernels behind moe_router_balance, moe_combine,
// moe_mx8_quant, moe_swiglu_save, their gradients and ways back, and
// moe_grouped_bias_grad.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// ---- balance loss of the router ----

struct BalanceParams {
  const void* logits;       // [T][ld]
  int64_t ld;
  int T, E, topk, sigmoid;
  const int32_t* ids;       // [T][topk]
  const int32_t* offsets;   // [S + 1] rows of the sequences, or NULL: one of all rows
  int S;
  int32_t* counts;          // [S][E]
  float* loss;              // [S]
  void* ws;
  // gradient
  const int32_t* counts_in;
  const float* d_loss;      // [S]
  const void* add;          // [T][add_ld] or NULL
  void* d_logits;           // [T][d_ld]
  int64_t add_ld, d_ld;
};
size_t balance_ws_bytes(int T, int E, int S);
hipError_t launch_balance(const BalanceParams& p, int type, hipStream_t s);
hipError_t launch_balance_grad(const BalanceParams& p, int type, hipStream_t s);

// ---- a token's rows ----

struct CombineParams {
  const void* y;            // [R][y_ld]
  int64_t y_ld;
  int R, H, T, topk;
  const int32_t* slots;     // [T][topk]
  const float* w;           // [T][topk] or NULL
  void* out;                // [T][out_ld]
  int64_t out_ld;
  // gradient
  const void* d_out;        // [T][d_ld]
  int64_t d_ld;
  const int32_t* row_src;   // [R] or NULL
  const int32_t* offsets;   // [E + 1] or NULL
  int E;
  void* d_y;                // [R][dy_ld]
  int64_t dy_ld;
  float* d_w;               // [T][topk] or NULL
};
hipError_t launch_combine_out(const CombineParams& p, int type, int out_type, hipStream_t s);
hipError_t launch_combine_grad(const CombineParams& p, int type, hipStream_t s);

// ---- 8-bit rows ----

// Rows of a call: those in [offsets[0], offsets[E]), all where offsets is NULL.
struct LiveRows {
  const int32_t* offsets;
  int E;
};

hipError_t launch_mx8_quant(const void* x, int type, int64_t rows, int K, int64_t ld, int8_t* q, uint8_t* scales,
                            int s_ld, hipStream_t s);

struct Mx8Rows {
  const int8_t* q;          // [rows][K]
  const uint8_t* scales;    // [rows][s_ld]
  int64_t rows;
  int K, s_ld;
  const int32_t* row_src;   // [out_rows] or NULL: out_rows = rows
  int topk;
  LiveRows live;
  int64_t out_rows;
  void* out;                // [out_rows][ld]
  int64_t ld;
};
hipError_t launch_mx8_dequant(const Mx8Rows& p, int type, hipStream_t s);

struct SwigluParams {
  const void* h;            // [rows][h_ld], gate | up
  int64_t h_ld;
  int rows, I, s_ld;
  LiveRows live;
  int8_t* q;                // [rows][2][I]
  uint8_t* scales;          // [rows][2][s_ld]
  void* a;                  // [rows][a_ld] or (gradient) NULL
  int64_t a_ld;
  // gradient: of h, or where h is NULL of the values of q
  const int8_t* q_in;
  const uint8_t* scales_in;
  const void* d_a;          // [rows][da_ld]
  int64_t da_ld;
  void* d_h;                // [rows][dh_ld]
  int64_t dh_ld;
};
hipError_t launch_swiglu_save(const SwigluParams& p, int type, hipStream_t s);
hipError_t launch_swiglu_grad(const SwigluParams& p, int type, hipStream_t s);

// ---- gradient of the experts' biases ----

struct BiasGradParams {
  const void* dy;           // [M][ld]
  int64_t ld;
  const int32_t* offsets;
  int E, M, N;
  void* db;                 // [E][db_ld]
  int64_t db_ld;
  void* ws;                 // of bias_grad_ws_bytes
};
size_t bias_grad_ws_bytes(int E, int M, int N);
hipError_t launch_bias_grad(const BiasGradParams& p, int type, int out_type, hipStream_t s);

}  // namespace moe
