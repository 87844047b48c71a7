// hcgr_block.h -- what the C ABI of the block operators (hcgr_block_api.hip)
// hands to their kernels (hcgr_block.hip, hcgr_linear.hip). Not installed.
#pragma once

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
int configure_block_kernels();
size_t norm_bwd_workspace(int hs, int64_t M);

struct LinearArgs {
  const int8_t *q, *w;
  const float *q_scale, *w_scale;
  const void* bias;  // NULL when absent
  void* out;
  int64_t ld_q, ld_w, ld_out, M;
  int n, k;
};
int launch_linear(const LinearArgs& a, int dtype, void* stream);
int configure_linear_kernels();

}  // namespace hcgr
