// hcgr_linear.hip -- the 8-bit linear layer (hcgr_linear_forward):
//   out[m, n] = (sum_k q[m, k]*w[n, k]) * q_scale[m] * w_scale[n] + bias[n]
// on v_mfma_i32_16x16x64_i8. Weight rows are the first (row) operand and
// tokens the second (column) operand, so a lane ends with four neighbouring
// output channels of one token.
#include <hip/hip_runtime.h>

#include "hcgr_block.h"
#include "hcgr_device.h"

namespace hcgr {
namespace {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4_t mfma_i8(uint4 a, uint4 b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0,
                                               0, 0);
}

// Keeps the first n of 16 bytes (n <= 0: none, n >= 16: all).
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n) {
  auto word = [&](uint32_t x, int k) { return k >= 4 ? x : k <= 0 ? 0u : x & ((1u << (8 * k)) - 1u); };
  return make_uint4(word(v.x, n), word(v.y, n - 4), word(v.z, n - 8), word(v.w, n - 12));
}

// Output element types: 0 bf16, 1 fp16, 2 fp32.
template <int DT>
__device__ __forceinline__ float bias_at(const void* bias, int n) {
  if constexpr (DT == 0) return bf1(reinterpret_cast<const uint16_t*>(bias)[n]);
  else if constexpr (DT == 1) return (float)reinterpret_cast<const _Float16*>(bias)[n];
  else return reinterpret_cast<const float*>(bias)[n];
}
template <int DT>
__device__ __forceinline__ void store1(void* out, int64_t i, float v) {
  if constexpr (DT == 0) reinterpret_cast<uint16_t*>(out)[i] = to_bf(v);
  else if constexpr (DT == 1) reinterpret_cast<_Float16*>(out)[i] = (_Float16)v;
  else reinterpret_cast<float*>(out)[i] = v;
}

// ---------------------------------------------------------------------------
// linear_direct: a workgroup of four waves owns 64 output channels (16 a
// wave) of 64 tokens; operands go straight from memory into MFMA registers.
// ---------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(256) void linear_direct(LinearArgs a) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int r16 = lane % 16, kq = lane / 16;
  const int n0 = (int)blockIdx.x * 64 + wave * 16;
  const int64_t m0 = (int64_t)blockIdx.y * 64;
  if (n0 >= a.n) return;
  const int k16 = (a.k + 15) / 16 * 16;
  const int nr = min(16, a.n - n0), mr = (int)min((int64_t)64, a.M - m0);
  // ranges over the tile's own rows: rows past the last are never in range
  const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * a.ld_w, (uint32_t)((nr - 1) * a.ld_w + k16));
  const rsrc_t rq = make_rsrc(a.q + m0 * a.ld_q, (uint32_t)((mr - 1) * a.ld_q + k16));
  constexpr uint32_t kOut = 0x7ffffff0u;  // past every range (at most 64 rows of 2^22 bytes)
  i32x4_t acc[4] = {};
  for (int k0 = 0; k0 < a.k; k0 += 64) {
    const int k = k0 + kq * 16;
    const uint4 w = bld16(rw, k < a.k && r16 < nr ? (uint32_t)(r16 * a.ld_w) + (uint32_t)k : kOut);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = t * 16 + r16;
      uint4 x = bld16(rq, k < a.k && r < mr ? (uint32_t)(r * a.ld_q) + (uint32_t)k : kOut);
      x = keep_bytes(x, a.k - k);  // a row's bytes past K count as zero
      acc[t] = mfma_i8(w, x, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t m = m0 + t * 16 + r16;
    if (m >= a.M) continue;
    const float qs = a.q_scale[m];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + kq * 4 + i;
      if (n >= a.n) continue;
      float v = (float)acc[t][i] * (qs * a.w_scale[n]);
      if (a.bias) v += bias_at<DT>(a.bias, n);
      store1<DT>(a.out, m * a.ld_out + n, v);
    }
  }
}

}  // namespace

int configure_linear_kernels() { return (int)hipSuccess; }

int launch_linear(const LinearArgs& args, int dtype, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const unsigned gx = (unsigned)((args.n + 63) / 64);
  // the grid's second dimension holds 65535 tiles: larger M in several launches
  constexpr int64_t kRows = (int64_t)65535 * 64;
  const size_t b = dtype == 2 ? 4 : 2;
  for (int64_t m0 = 0; m0 < args.M; m0 += kRows) {
    LinearArgs a = args;
    a.M = args.M - m0 < kRows ? args.M - m0 : kRows;
    a.q += m0 * a.ld_q;
    a.q_scale += m0;
    a.out = reinterpret_cast<uint8_t*>(a.out) + (size_t)(m0 * a.ld_out) * b;
    const dim3 g(gx, (unsigned)((a.M + 63) / 64)), blk(256);
    if (dtype == 0) hipLaunchKernelGGL(linear_direct<0>, g, blk, 0, st, a);
    else if (dtype == 1) hipLaunchKernelGGL(linear_direct<1>, g, blk, 0, st, a);
    else hipLaunchKernelGGL(linear_direct<2>, g, blk, 0, st, a);
    const int e = (int)hipGetLastError();
    if (e != (int)hipSuccess) return e;
  }
  return (int)hipSuccess;
}

}  // namespace hcgr
