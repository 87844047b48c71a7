// hcgr_block.h -- what the C ABI of the block operators (hcgr_block_api.hip)
// hands to their kernels (hcgr_block.hip,
// hcgr_layer_norm.hip, hcgr_linear.hip, hcgr_mx.hip). Not installed.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace hcgr {

// Forward of the norms: hcgr_block_norm (residual = false: R is x with row
// pitch ld_R, one stream, used as it is) and hcgr_block_residual.
struct NormArgs {
  const void *R, *y, *inj, *w_post, *w_pre;  // y, inj, w_post, w_pre: NULL when absent
  int64_t ld_R, ld_y, ld_inj, M;
  int hs, hc;
  float eps, rho;
  void *R2, *x;  // x: NULL when absent
  int8_t* q;     // NULL when absent
  int64_t ld_q;
  float *q_scale, *rr_post, *rr_pre;  // rr_*: column of each norm, NULL when not wanted
  int rr_ld;                          // floats from one token's r to the next
  int nt = 0;                         // set by the launch: outputs with the streaming policy
  int64_t m_first = 0;                // likewise: the launch's first row
};

// Backward of both. For hcgr_block_norm_bwd: residual = false, R = x, w_pre =
// w, dx = dxn, dR = the gradient of x (NULL: not wanted).
struct NormBwdArgs {
  const void *R, *y, *inj, *w_post, *w_pre, *dR2, *dx;
  int64_t ld_R, ld_y, ld_inj, ld_dinj, M;
  int hs, hc;
  float rho;
  const float *rr_post, *rr_pre;
  int rr_ld;
  void *dR, *dy, *dinj;
  float *dw_post, *dw_pre;
  void* ws;
};

int launch_norm(const NormArgs& a, int dtype, bool residual, void* stream);
int launch_norm_bwd(const NormBwdArgs& a, int dtype, bool residual, void* stream);
// Rows -> int8 rows and a scale each: launch_norm without the norm.
int launch_quantize(const NormArgs& a, int dtype, void* stream);
// configure_*: raise the dynamic-LDS limits of the kernels that a handle of this
// type (and width) may launch, on the current device. Each costs some 50 ns,
// the first of a source's kernels in a process the load of its code (1 to 3 ms).
int configure_block_kernels(int dtype);
// The workspace of every norm's backward pass: two floats a row, then up to
// norm_bwd_groups(M) pairs of partial sums [2][HS] of the weight gradients.
size_t norm_bwd_workspace(int hs, int64_t M);
size_t norm_bwd_row_floats(int64_t M);
int64_t norm_bwd_groups(int64_t M);
// dw0, dw1 [hs] (NULL: not wanted) from `groups` pairs, in a fixed order.
int launch_weight_sums(const float* part, int hs, int64_t groups, float* dw0, float* dw1, hipStream_t st);

// hcgr_block_layer_norm
struct LayerNormArgs {
  const void *x, *w, *b;  // w, b: NULL when absent
  int64_t ld_x, M;
  int hs;
  float eps;
  void* xn;           // NULL when absent
  uint8_t *q, *q_scale;  // NULL when absent
  int64_t ld_q, ld_qs;
  float* stats;       // NULL when not wanted
  int nt = 0;         // set by the launch: outputs with the streaming policy
  int64_t m_first = 0;  // likewise: the launch's first row
};
// hcgr_block_layer_norm_bwd; rows, part: the two parts of the workspace
struct LayerNormBwdArgs {
  const void *x, *w, *dxn;
  int64_t ld_x, M;
  int hs;
  const float* stats;
  void* dx;         // NULL: not wanted
  float *dw, *db;   // likewise
  float *rows, *part;
};
int launch_layer_norm(const LayerNormArgs& a, int dtype, void* stream);
int launch_layer_norm_bwd(const LayerNormBwdArgs& a, int dtype, void* stream);
int configure_layer_norm_kernels(int hs, int dtype);

struct LinearArgs {
  const int8_t *q, *w;
  const float *q_scale, *w_scale;
  const void* bias;  // NULL when absent
  void* out;
  int64_t ld_q, ld_w, ld_out, M;
  int n, k;
};
int launch_linear(const LinearArgs& a, int dtype, void* stream);
int configure_linear_kernels(int dtype);

// Rows to microscaled 4 bits, and back.
template <typename X, typename Q>
struct MxRows {
  X* x;
  Q *q, *q_scale;
  int64_t ld_x, ld_q, ld_qs, M;
  int k;
};
using MxRowsToArgs = MxRows<const void, uint8_t>;
using MxRowsFromArgs = MxRows<void, const uint8_t>;
struct MxLinearArgs {
  const uint8_t *q, *w, *q_scale, *w_scale;
  const void* bias;  // NULL when absent
  void* out;
  int64_t ld_q, ld_w, ld_qs, ld_ws, ld_out, M;
  int n, k;
};
int launch_mx_quantize(const MxRowsToArgs& a, int dtype, void* stream);
int launch_mx_dequantize(const MxRowsFromArgs& a, int dtype, void* stream);
int launch_mx_linear(const MxLinearArgs& a, int dtype, void* stream);
int configure_mx_kernels(int dtype);

}  // namespace hcgr
