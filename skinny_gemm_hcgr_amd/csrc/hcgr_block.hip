// hcgr_block.hip -- the norms around a block (hcgr_block_norm,
// hcgr_block_residual), their gradients, and the row quantizer. The
// mathematics stands in include/hcgr.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "hcgr_block.h"
#include "hcgr_device.h"

namespace hcgr {
namespace {

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------- element types ----
struct Bf16 { using S = uint16_t; };
struct Fp16 { using S = _Float16; };
struct Fp32 { using S = float; };

__device__ __forceinline__ float up(uint16_t v) { return bf1(v); }
__device__ __forceinline__ float up(_Float16 v) { return (float)v; }
__device__ __forceinline__ float up(float v) { return v; }
template <typename T> __device__ __forceinline__ typename T::S down(float v);
template <> __device__ __forceinline__ uint16_t down<Bf16>(float v) { return to_bf(v); }
template <> __device__ __forceinline__ _Float16 down<Fp16>(float v) { return (_Float16)v; }
template <> __device__ __forceinline__ float down<Fp32>(float v) { return v; }

// 16 bytes of a row: V = vec<T>() values. n says how many of them the row
// still has (<= 0: none, they read as zero and are not stored). AL: every row
// starts on 16 bytes and has a whole number of such pieces; otherwise a piece
// may start at any element (gfx950 loads and stores 16 bytes at any alignment)
// and a row's last piece is moved one element at a time.
template <typename T>
constexpr int vec() { return 16 / (int)sizeof(typename T::S); }

template <typename T, bool AL>
__device__ __forceinline__ uint4 load_raw(const typename T::S* p, int n) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if constexpr (AL) {
    if (n > 0) u = ld16(p);
  } else {
    if (n >= vec<T>()) {
      __builtin_memcpy(&u, p, 16);
    } else {
      typename T::S s[vec<T>()] = {};
      for (int i = 0; i < vec<T>(); ++i)
        if (i < n) s[i] = p[i];
      __builtin_memcpy(&u, s, 16);
    }
  }
  return u;
}
template <typename T>
__device__ __forceinline__ void unpack(uint4 u, float (&f)[vec<T>()]) {
  typename T::S s[vec<T>()];
  __builtin_memcpy(s, &u, 16);
#pragma unroll
  for (int i = 0; i < vec<T>(); ++i) f[i] = up(s[i]);
}
template <typename T, bool AL>
__device__ __forceinline__ void load(const typename T::S* p, int n, float (&f)[vec<T>()]) {
  unpack<T>(load_raw<T, AL>(p, n), f);
}
template <typename T, bool AL>
__device__ __forceinline__ void store(typename T::S* p, int n, const float (&f)[vec<T>()]) {
  typename T::S s[vec<T>()];
#pragma unroll
  for (int i = 0; i < vec<T>(); ++i) s[i] = down<T>(f[i]);
  if (AL ? n > 0 : n >= vec<T>()) {
    uint4 u;
    __builtin_memcpy(&u, s, 16);
    if constexpr (AL) st16(p, u);
    else __builtin_memcpy(p, &u, 16);
  } else if constexpr (!AL) {
    for (int i = 0; i < vec<T>(); ++i)
      if (i < n) p[i] = s[i];
  }
}

// ------------------------------------------------------------ reductions --
// Over the 64 lanes of a wave, the result in each of them: lanes 1, 2, 4 and 8
// apart meet through DPP, the rows of 16 through the lane swaps of gfx950.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <typename F>
__device__ __forceinline__ uint32_t wave_all(uint32_t v, F f) {
  v = f(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
  v = f(v, dpp<0x141>(v));  // row_half_mirror
  v = f(v, dpp<0x140>(v));  // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return f(b[0], b[1]);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_all(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  return wave_all(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
// Sum of N values over the workgroup, the same bits in every thread. `red`
// holds N floats a wave; the caller does not reuse it before a barrier.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  const int nw = (int)blockDim.x / 64, w = (int)threadIdx.x / 64;
  if (nw == 1) return;
  if (threadIdx.x % 64 == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[w * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.0f;
    for (int k = 0; k < nw; ++k) s += red[k * N + i];
    v[i] = s;
  }
}
__device__ __forceinline__ uint32_t group_umax(uint32_t v, uint32_t* red) {
  v = wave_umax(v);
  const int nw = (int)blockDim.x / 64;
  if (nw == 1) return v;
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  v = 0;
  for (int k = 0; k < nw; ++k) v = max(v, red[k]);
  return v;
}

__device__ __forceinline__ float rrms_of(float sum, int hs, float eps) {
  return 1.0f / sqrtf(sum / (float)hs + eps);
}
// 2*sigmoid(inj/HC), and its derivative in inj: an even function, from e =
// exp(-|inj|/HC) as 2*e/(1 + e)^2/HC. (iw*(1 - iw/2)/HC, from a gate iw that is
// rounded near 2, loses all its digits towards inj/HC = 17.)
__device__ __forceinline__ float gate(float inj, int hc) { return 2.0f / (1.0f + expf(-inj / (float)hc)); }
__device__ __forceinline__ float gate_slope(float inj, int hc) {
  const float e = expf(-fabsf(inj) / (float)hc), r = 1.0f / (1.0f + e);
  return 2.0f / (float)hc * e * r * r;
}

// ---------------------------------------------------------- quantization --
// Magnitudes are compared as their bit patterns (an infinity or a NaN is
// above every number), so a row's maximum says whether the row is finite.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
struct Quant {
  float scale, pre, step, inv;  // q = round(v * pre / step), inv = 1/step (within a step of its own)
};
// Brings a row's values up by pre where it is not 1 (few rows are so small).
template <int V>
__device__ __forceinline__ void lift(float (&v)[V], const Quant& z) {
  if (z.pre == 1.0f) return;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] *= z.pre;
}
// Rows whose largest value is below 2^-60 are brought up by 2^100 first (exact),
// so that the reciprocal does not overflow and no remainder below underflows.
__device__ __forceinline__ Quant quant_of(uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits);
  Quant z;
  z.pre = amax < 0x1p-60f ? 0x1p100f : 1.0f;
  const bool finite = amax_bits < 0x7f800000u;
  z.scale = finite ? amax / 127.0f : __uint_as_float(0x7fc00000u);
  z.step = z.pre == 1.0f ? z.scale : amax * z.pre / 127.0f;
  z.inv = finite && amax > 0.0f ? __builtin_amdgcn_rcpf(z.step) : 0.0f;
  return z;
}
// v/step rounded to the nearest, ties to even. The product with a reciprocal
// alone is off by a few steps of its own, which turns ties (37.5 in a row whose
// largest value is 1905: 2.5); its remainder puts it right: within 2^-44 of the
// quotient before its one rounding. (Norm + quantized product of 8192 x 2560 to
// 64: 30.1 -> 30.7 us; 32.7 with a divided reciprocal.)
__device__ __forceinline__ int quant1(float v, const Quant& z) {  // v: lifted
  // z.inv = 0 (an all-zero row, or one that is not finite) gives 0: what is NaN
  // there the comparison sends to 0
  const float t = v * z.inv, r = rintf(fmaf(fmaf(-t, z.step, v), z.inv, t));
  return fabsf(r) <= 127.0f ? (int)r : 0;
}
// n of V quantized values (rows of q start on 16 bytes and V divides the
// column, so whole pieces are aligned).
template <int V, bool AL>
__device__ __forceinline__ void store_q(int8_t* p, int n, const float (&v)[V], const Quant& z) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V; i += 4)
    w[i / 4] = (uint32_t)(quant1(v[i], z) & 255) | (uint32_t)(quant1(v[i + 1], z) & 255) << 8 |
               (uint32_t)(quant1(v[i + 2], z) & 255) << 16 | (uint32_t)(quant1(v[i + 3], z) & 255) << 24;
  if (AL ? n > 0 : n >= V) {
    if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else if constexpr (!AL) {
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

constexpr int kMaxHc = 8;

// ---------------------------------------------------------------------------
// norm_loop: the forward pass for any width, alignment and stream count. One
// workgroup a row at a time; threads walk the row V values at a time. The row
// is read again (from the caches) in each of up to three passes: the sum of
// y^2, then R2 and the sum of u^2, then the output. RES: hcgr_block_residual;
// otherwise one stream that is used as it is (hcgr_block_norm, and without
// NORM the quantizer).
// ---------------------------------------------------------------------------
template <typename T, bool AL, bool RES, bool NORM>
__global__ __launch_bounds__(1024) void norm_loop(NormArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  __shared__ float red[2][16];
  __shared__ uint32_t redq[16];
  const int hs = a.hs, hc = RES ? a.hc : 1, step = (int)blockDim.x * V;
  const S* wpost = reinterpret_cast<const S*>(a.w_post);
  const S* wpre = reinterpret_cast<const S*>(a.w_pre);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const S* R = reinterpret_cast<const S*>(a.R) + m * a.ld_R;
    const S* y = RES ? reinterpret_cast<const S*>(a.y) + m * a.ld_y : nullptr;
    S* R2 = RES ? reinterpret_cast<S*>(a.R2) + m * a.ld_R : nullptr;
    float iw[kMaxHc];
    float ry = 1.0f;
    if constexpr (RES) {
      for (int s = 0; s < hc; ++s)
        iw[s] = a.inj ? gate(up(reinterpret_cast<const S*>(a.inj)[m * a.ld_inj + s]), hc) : 1.0f;
      if (wpost) {
        float ss[1] = {0.0f};
        for (int c = (int)threadIdx.x * V; c < hs; c += step) {
          float f[V];
          load<T, AL>(y + c, hs - c, f);
#pragma unroll
          for (int i = 0; i < V; ++i) ss[0] += f[i] * f[i];
        }
        group_sum(ss, red[0]);
        ry = rrms_of(ss[0], hs, a.eps);
        if (a.rr_post && threadIdx.x == 0) a.rr_post[m * a.rr_ld] = ry;
      }
    }
    // u of V channels at c; with WRITE also R2
    auto form = [&](int c, float (&u)[V], bool write) {
      if constexpr (!RES) {
        load<T, AL>(R + c, hs - c, u);
      } else {
        float z[V];
        load<T, AL>(y + c, hs - c, z);
        if (wpost) {
          float w[V];
          load<T, AL>(wpost + c, hs - c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) z[i] = z[i] * ry * (1.0f + w[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = 0.0f;
        for (int s = 0; s < hc; ++s) {
          float r[V];
          load<T, AL>(R + (int64_t)s * hs + c, hs - c, r);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            r[i] = fmaf(iw[s], z[i], a.rho * r[i]);
            u[i] += r[i];
          }
          if (write) store<T, AL>(R2 + (int64_t)s * hs + c, hs - c, r);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] /= (float)hc;
      }
    };
    float ss[1] = {0.0f};
    uint32_t am = 0;
    for (int c = (int)threadIdx.x * V; c < hs; c += step) {
      float u[V];
      form(c, u, true);
      if (NORM && wpre) {
        float w[V];
        if (a.q) load<T, AL>(wpre + c, hs - c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ss[0] += u[i] * u[i];
          if (a.q) am = max(am, mag(u[i] * (1.0f + w[i])));
        }
      } else if (!NORM) {
#pragma unroll
        for (int i = 0; i < V; ++i) am = max(am, mag(u[i]));
      }
    }
    if (!NORM || wpre) {
      float ru = 1.0f;
      if constexpr (NORM) {
        group_sum(ss, red[1]);
        ru = rrms_of(ss[0], hs, a.eps);
        if (a.rr_pre && threadIdx.x == 0) a.rr_pre[m * a.rr_ld] = ru;
      }
      Quant z{};
      if (a.q) {
        am = group_umax(am, redq);
        // the largest |u(1 + w)| times r is the largest norm; a value that is
        // not finite stays so
        z = quant_of(mag(__uint_as_float(am) * ru));
        if (threadIdx.x == 0) a.q_scale[m] = z.scale;
      }
      for (int c = (int)threadIdx.x * V; c < hs; c += step) {
        float u[V];
        form(c, u, false);
        if constexpr (NORM) {
          float w[V];
          load<T, AL>(wpre + c, hs - c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) u[i] = u[i] * (1.0f + w[i]) * ru;
          if (a.x) store<T, AL>(reinterpret_cast<S*>(a.x) + m * hs + c, hs - c, u);
        }
        if (a.q) {
          lift(u, z);
          store_q<V, AL>(a.q + m * a.ld_q + c, hs - c, u, z);
        }
      }
    }
    __syncthreads();  // the next row reuses the reduction arrays
  }
}

// ---------------------------------------------------------------------------
// The backward pass for any width, alignment and stream count, in three
// kernels. With h = u*ru, e = dx*(1 + w_pre) and B_s = sum_c dR2[s]*z, every
// row sum that the formulas need comes from one pass over the row:
//   m_pre = mean(e*h) = ru*A/HS,              A = sum e*u
//   sum_c du*z = ru*(C - m_pre*ru*D),         C = sum e*z, D = sum u*z
//   diw[s] = sum_c d[s]*z = B_s + (sum_c du*z)/HC
//   m_post = mean(dz*(1 + w_post)*y*ry) = sum_s iw[s]*diw[s]/HS,
// since z = y*ry*(1 + w_post). norm_bwd_rows forms them (one workgroup a row)
// and writes dinj, m_pre and m_post; norm_bwd_cols then needs nothing across
// the row: each thread keeps V columns, walks its group's rows, writes dR and
// dy and sums the weight gradients of its columns; norm_bwd_sum adds the
// groups' sums in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kRowGroups = 768;  // partial sums of the weight gradients
constexpr int kColThreads = 256;

// Workspace: m_pre and m_post of each row, then [groups][2][HS] partial sums.
__host__ __device__ inline int64_t bwd_groups(int64_t M) { return M < kRowGroups ? M : kRowGroups; }
__host__ __device__ inline int64_t bwd_row_floats(int64_t M) { return (2 * M + 3) / 4 * 4; }

template <typename T, bool AL, bool RES>
struct BwdRow {
  using S = typename T::S;
  static constexpr int V = vec<T>();
  const NormBwdArgs& a;
  int64_t m;
  const S *R, *y, *dR2, *dx, *wpost, *wpre;
  float ry, ru, iw[kMaxHc];
  int hc;
  __device__ __forceinline__ BwdRow(const NormBwdArgs& a_, int64_t m_) : a(a_), m(m_) {
    hc = RES ? a.hc : 1;
    R = reinterpret_cast<const S*>(a.R) + m * a.ld_R;
    y = RES ? reinterpret_cast<const S*>(a.y) + m * a.ld_y : nullptr;
    dR2 = RES && a.dR2 ? reinterpret_cast<const S*>(a.dR2) + m * a.ld_R : nullptr;
    dx = a.dx ? reinterpret_cast<const S*>(a.dx) + m * a.hs : nullptr;
    wpost = RES ? reinterpret_cast<const S*>(a.w_post) : nullptr;
    wpre = reinterpret_cast<const S*>(a.w_pre);
    ry = wpost ? a.rr_post[m * a.rr_ld] : 1.0f;
    ru = wpre ? a.rr_pre[m * a.rr_ld] : 1.0f;
    for (int s = 0; s < hc; ++s)
      iw[s] = RES && a.inj ? gate(up(reinterpret_cast<const S*>(a.inj)[m * a.ld_inj + s]), hc) : 1.0f;
  }
  // z = y*ry*(1 + w_post) (h = y*ry, g = 1 + w_post); RES only
  __device__ __forceinline__ void form_z(int c, float (&h)[V], float (&g)[V], float (&z)[V]) const {
    load<T, AL>(y + c, a.hs - c, h);
    if (wpost) load<T, AL>(wpost + c, a.hs - c, g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] *= ry;
      g[i] = wpost ? 1.0f + g[i] : 1.0f;
      z[i] = h[i] * g[i];
    }
  }
  __device__ __forceinline__ void form_u(int c, const float (&z)[V], float (&u)[V]) const {
    if constexpr (!RES) {
      load<T, AL>(R + c, a.hs - c, u);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = 0.0f;
      for (int s = 0; s < hc; ++s) {
        float r[V];
        load<T, AL>(R + (int64_t)s * a.hs + c, a.hs - c, r);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] += fmaf(iw[s], z[i], a.rho * r[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] /= (float)hc;
    }
  }
  // e = dx*(1 + w_pre)
  __device__ __forceinline__ void form_e(int c, float (&d)[V], float (&e)[V]) const {
    float w[V];
    load<T, AL>(dx + c, a.hs - c, d);
    load<T, AL>(wpre + c, a.hs - c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = d[i] * (1.0f + w[i]);
  }
};

template <typename T, bool AL, bool RES>
__global__ __launch_bounds__(1024) void norm_bwd_rows(NormBwdArgs a) {
  constexpr int V = vec<T>();
  __shared__ float red[16 * (kMaxHc + 3)];
  float* rows = reinterpret_cast<float*>(a.ws);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const BwdRow<T, AL, RES> row(a, m);
    float sums[kMaxHc + 3] = {};  // B_s, A, C, D
    for (int c = (int)threadIdx.x * V; c < a.hs; c += (int)blockDim.x * V) {
      float h[V], g[V], z[V] = {}, u[V], d[V], e[V];
      if constexpr (RES) row.form_z(c, h, g, z);
      if (row.dx) {
        row.form_u(c, z, u);
        row.form_e(c, d, e);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sums[kMaxHc] += e[i] * u[i];
          sums[kMaxHc + 1] += e[i] * z[i];
          sums[kMaxHc + 2] += u[i] * z[i];
        }
      }
      if (RES && row.dR2)
        for (int s = 0; s < row.hc; ++s) {
          load<T, AL>(row.dR2 + (int64_t)s * a.hs + c, a.hs - c, d);
#pragma unroll
          for (int i = 0; i < V; ++i) sums[s] += d[i] * z[i];
        }
    }
    group_sum(sums, red);
    if (threadIdx.x == 0) {
      const float m_pre = row.ru * sums[kMaxHc] / (float)a.hs;
      float m_post = 0.0f;
      if constexpr (RES) {
        const float duz = row.ru * (sums[kMaxHc + 1] - m_pre * row.ru * sums[kMaxHc + 2]) / (float)row.hc;
        for (int s = 0; s < row.hc; ++s) {
          const float diw = sums[s] + (row.dx ? duz : 0.0f);
          m_post += row.iw[s] * diw;
          if (a.dinj) {
            const float inj = up(reinterpret_cast<const typename T::S*>(a.inj)[m * a.ld_inj + s]);
            reinterpret_cast<typename T::S*>(a.dinj)[m * a.ld_dinj + s] = down<T>(diw * gate_slope(inj, row.hc));
          }
        }
      }
      rows[2 * m] = m_pre;
      rows[2 * m + 1] = m_post / (float)a.hs;
    }
    __syncthreads();  // the next row reuses red
  }
}

template <typename T, bool AL, bool RES>
__global__ __launch_bounds__(kColThreads) void norm_bwd_cols(NormBwdArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  const int c = ((int)blockIdx.x * kColThreads + (int)threadIdx.x) * V;
  if (c >= a.hs) return;
  const float* rows = reinterpret_cast<const float*>(a.ws);
  float apost[V] = {}, apre[V] = {};
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    const BwdRow<T, AL, RES> row(a, m);
    const float m_pre = rows[2 * m], m_post = rows[2 * m + 1];
    float h[V], g[V], z[V] = {}, u[V], dx[V], e[V], du[V] = {};
    if constexpr (RES) row.form_z(c, h, g, z);
    if (row.dx) {
      row.form_u(c, z, u);
      row.form_e(c, dx, e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float hu = u[i] * row.ru;
        du[i] = row.ru * (e[i] - hu * m_pre);
        apre[i] += dx[i] * hu;
      }
    }
    if constexpr (!RES) {
      if (a.dR) store<T, AL>(reinterpret_cast<S*>(a.dR) + m * a.hs + c, a.hs - c, du);
    } else {
      float dz[V] = {};
      for (int s = 0; s < row.hc; ++s) {
        float d[V] = {};
        if (row.dR2) load<T, AL>(row.dR2 + (int64_t)s * a.hs + c, a.hs - c, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          d[i] += du[i] / (float)row.hc;
          dz[i] = fmaf(row.iw[s], d[i], dz[i]);
          d[i] *= a.rho;
        }
        store<T, AL>(reinterpret_cast<S*>(a.dR) + m * a.ld_R + (int64_t)s * a.hs + c, a.hs - c, d);
      }
      if (row.wpost) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          apost[i] += dz[i] * h[i];
          dz[i] = row.ry * (dz[i] * g[i] - h[i] * m_post);
        }
      }
      store<T, AL>(reinterpret_cast<S*>(a.dy) + m * a.hs + c, a.hs - c, dz);
    }
  }
  float* part = reinterpret_cast<float*>(a.ws) + bwd_row_floats(a.M) + (int64_t)blockIdx.y * 2 * a.hs;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (a.dw_post && c + i < a.hs) part[c + i] = apost[i];
    if (a.dw_pre && c + i < a.hs) part[a.hs + c + i] = apre[i];
  }
}

__global__ __launch_bounds__(1024) void norm_bwd_sum(NormBwdArgs a, int groups) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int c = (int)blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? a.dw_pre : a.dw_post;
  if (!out) return;
  const float* part = reinterpret_cast<const float*>(a.ws) + bwd_row_floats(a.M) + (int64_t)blockIdx.y * a.hs;
  float s = 0.0f;
  if (c < a.hs) {
#pragma unroll 8
    for (int g = w; g < groups; g += 32) s += part[(int64_t)g * 2 * a.hs + c];
  }
  red[w][lane] = s;
  __syncthreads();
  s = red[lane][w];  // wave w/2 holds column w of the 32 partial sums in lanes (w % 2)*32 ..
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0 && (int)blockIdx.x * 32 + w < a.hs) out[(int)blockIdx.x * 32 + w] = s;
}

// Rows as buffer ranges: one 32-bit offset a piece serves every tensor and
// stream (the stream's offset is scalar), a piece past the row reads as zero
// and is not stored, and so does every piece of an absent tensor.
template <typename S>
__device__ __forceinline__ rsrc_t row_of(const void* base, int64_t off, uint32_t bytes) {
  return base ? make_rsrc(reinterpret_cast<const S*>(base) + off, bytes) : make_rsrc(nullptr, 0u);
}
template <typename S>
__device__ __forceinline__ i32x4_t words_of(const void* base, int64_t off, uint32_t bytes) {
  return range_words(reinterpret_cast<const S*>(base) + (base ? off : 0), base ? bytes : 0u);
}
__device__ __forceinline__ uint32_t piece_at(int j, uint32_t row) {
  const uint32_t at = (threadIdx.x + (uint32_t)j * blockDim.x) * 16u;
  return at < row ? at : 0x7ffffff0u;
}
// A token's row of one or several streams. AL: as above; otherwise the row
// starts at any element and its pieces go by pointers.
template <typename T, bool AL>
struct Row {
  using S = typename T::S;
  rsrc_t r;
  S* p;
  int hs;
  __device__ __forceinline__ Row(const void* base, int64_t off, int streams, int hs_) {
    hs = hs_;
    if constexpr (AL) r = row_of<S>(base, off, (uint32_t)(streams * hs * (int)sizeof(S)));
    else p = base ? const_cast<S*>(reinterpret_cast<const S*>(base)) + off : nullptr;
  }
  // piece j of this thread in stream s
  __device__ __forceinline__ uint4 get(int j, int s = 0) const {
    if constexpr (AL) {
      const uint32_t row = (uint32_t)hs * sizeof(S);
      return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)piece_at(j, row), (int)(s * row), 0));
    } else {
      const int c = ((int)threadIdx.x + j * (int)blockDim.x) * vec<T>();
      return p ? load_raw<T, false>(p + (int64_t)s * hs + c, hs - c) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void put(int j, int s, const float (&f)[vec<T>()], int nt) const;
};
// nt: the streaming policy, for outputs too large for the caches to keep until
// they are read. The stream's offset goes into the vector offset here: after a
// 16-byte buffer store whose scalar offset is a register, the compiler lets
// the next instruction overwrite the stored registers, and on MI355X such
// stores have written the new values (with a constant scalar offset it keeps
// them apart).
template <typename T, bool AL>
__device__ __forceinline__ void Row<T, AL>::put(int j, int s, const float (&f)[vec<T>()], int nt) const {
  if constexpr (AL) {
    typename T::S v[vec<T>()];
#pragma unroll
    for (int i = 0; i < vec<T>(); ++i) v[i] = down<T>(f[i]);
    u32x4_t u;
    __builtin_memcpy(&u, v, 16);
    const uint32_t row = (uint32_t)hs * sizeof(S), at = piece_at(j, row) + s * row;
    if (nt) __builtin_amdgcn_raw_buffer_store_b128(u, r, (int)at, 0, kNonTemporal);
    else __builtin_amdgcn_raw_buffer_store_b128(u, r, (int)at, 0, 0);
  } else {
    const int c = ((int)threadIdx.x + j * (int)blockDim.x) * vec<T>();
    store<T, false>(p + (int64_t)s * hs + c, hs - c, f);
  }
}

// ---------------------------------------------------------------------------
// norm_row: the forward pass of rows that fit the registers of a workgroup
// (NCH 16-byte pieces of every tensor a thread): each value is read once.
// Every load of a row is issued before the first reduction. Rows of at most
// 64 * NCH pieces take one wave, four rows a workgroup, without barriers;
// wider rows take the whole workgroup.
// ---------------------------------------------------------------------------
template <typename T, int HC, int NCH, bool AL, bool RES, bool NORM>
__global__ __launch_bounds__(1024) void norm_row(NormArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  __shared__ float red[2][16];
  __shared__ uint32_t redq[16];
  const int hs = a.hs;
  const int64_t m = a.m_first + (int64_t)blockIdx.x * blockDim.y + __builtin_amdgcn_readfirstlane((int)threadIdx.y);
  if (m >= a.M) return;  // blockDim.y > 1 only without barriers
  const bool wpre = a.w_pre != nullptr, wpost = RES && a.w_post != nullptr;
  const Row<T, AL> rR(a.R, m * a.ld_R, HC, hs), rY(a.y, m * a.ld_y, 1, hs), rG(a.w_post, 0, 1, hs), rW(a.w_pre, 0, 1, hs);
  uint4 rr[NCH][HC], yr[NCH], gr[NCH], wr[NCH];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    if constexpr (RES) yr[j] = rY.get(j);
#pragma unroll
    for (int s = 0; s < HC; ++s) rr[j][s] = rR.get(j, s);
    if (wpost) gr[j] = rG.get(j);
    if (NORM && wpre) wr[j] = rW.get(j);
  }
  float u[NCH][V];
  if constexpr (RES) {
    float iw[HC];
#pragma unroll
    for (int s = 0; s < HC; ++s)
      iw[s] = a.inj ? gate(up(reinterpret_cast<const S*>(a.inj)[m * a.ld_inj + s]), HC) : 1.0f;
    float ry = 1.0f;
    if (wpost) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float f[V];
        unpack<T>(yr[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) ss[0] += f[i] * f[i];
      }
      group_sum(ss, red[0]);
      ry = rrms_of(ss[0], hs, a.eps);
      if (a.rr_post && threadIdx.x == 0) a.rr_post[m * a.rr_ld] = ry;
    }
    const Row<T, AL> r2(a.R2, m * a.ld_R, HC, hs);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float z[V], w[V];
      unpack<T>(yr[j], z);
      if (wpost) {
        unpack<T>(gr[j], w);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] * ry * (1.0f + w[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] = 0.0f;
#pragma unroll
      for (int s = 0; s < HC; ++s) {
        float r[V];
        unpack<T>(rr[j][s], r);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          r[i] = fmaf(iw[s], z[i], a.rho * r[i]);
          u[j][i] += r[i];
        }
        r2.put(j, s, r, a.nt);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] *= 1.0f / (float)HC;
    }
    if (!wpre) return;
  } else {
#pragma unroll
    for (int j = 0; j < NCH; ++j) unpack<T>(rr[j][0], u[j]);
  }
  float ru = 1.0f;
  if constexpr (NORM) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float w[V];
      unpack<T>(wr[j], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss[0] += u[j][i] * u[j][i];
        u[j][i] *= 1.0f + w[i];
      }
    }
    group_sum(ss, red[1]);
    ru = rrms_of(ss[0], hs, a.eps);
    if (a.rr_pre && threadIdx.x == 0) a.rr_pre[m * a.rr_ld] = ru;
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) u[j][i] *= ru;
  if (NORM && a.x) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) Row<T, AL>(a.x, m * hs, 1, hs).put(j, 0, u[j], a.nt);
  }
  if (a.q) {
    uint32_t am = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) am = max(am, mag(u[j][i]));
    const Quant z = quant_of(group_umax(am, redq));
    if (threadIdx.x == 0) a.q_scale[m] = z.scale;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = ((int)threadIdx.x + j * (int)blockDim.x) * V;
      lift(u[j], z);
      store_q<V, AL>(a.q + m * a.ld_q + c, hs - c, u[j], z);
    }
  }
}

// ---------------------------------------------------------------------------
// norm_bwd_row: the backward pass of rows that fit the registers of a
// workgroup, in one pass over the data. A workgroup walks every G-th row,
// keeps the weights and the sums of its columns' weight gradients in
// registers, and gets all row sums from one reduction (see above norm_bwd_rows).
// One-wave rows: four rows at a time, the four waves' sums meet in LDS. Up to
// 512 threads the next row's pieces come to LDS behind this row's products and
// stores, each wave's into a place of its own (no barrier). At M = 8192, HC =
// 4, HS = 2560, bf16, the call takes 156 us with norm_bwd_sum (4.0 TB/s; 5.2
// TB/s, what a copy reaches, would take 121): 194 us with the loads of a row
// waiting for the row before, 169 with the next row ahead, 162 with three
// workgroups a CU (128 registers) in place of two, 158 by streaming stores, 156
// with the gates formed before the next row's loads (the compiler's wait for the
// logits took those in). fp16 takes 148. What bounds it: 128 registers do not
// hold four streams in 16 bits; 3 are spilled, and a reload waits for every load
// in flight, the next row's among them, before the reduction.
// ---------------------------------------------------------------------------
constexpr int bwd_loads(int hc) { return hc ? 2 * hc + 2 : 2; }  // hc = 0: the norm alone
// Dynamic LDS of norm_bwd_row: the waves' places, and room for the sums of
// one-wave rows (three waves' two gradients).
inline size_t bwd_lds(int hc, int nch, int waves, int v, bool ahead, bool one_wave) {
  const size_t ring = ahead ? (size_t)waves * bwd_loads(hc) * nch * 1024 : 0;
  const size_t sums = one_wave ? (size_t)3 * 2 * 64 * nch * v * 4 : 0;
  return ring > sums ? ring : sums;
}

template <typename T, int HC, int NCH, int THREADS, bool AL, bool RES>
__global__ __launch_bounds__(THREADS, AL && THREADS <= 512 && NCH == 1 && HC <= 4 ? 4 : 1) void norm_bwd_row(NormBwdArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>(), N = RES ? HC + 3 : 1;
  constexpr bool AHEAD = AL && THREADS <= 512 && NCH == 1;
  constexpr int L = bwd_loads(RES ? HC : 0) * NCH;  // a wave's loads a row, 1 KB each
  __shared__ float red[2][16 * N];
  // The slopes of a row's gates, each for the thread that forms it and writes its
  // dinj: the row's threads 0 .. HC - 1, in wave 0 or, of one-wave rows, in wave y.
  // (Kept in registers until then they spill: 4 streams in bf16 3 -> 11 registers.)
  __shared__ float slopes[4][HC];
  extern __shared__ __attribute__((aligned(16))) uint8_t ring[];  // [waves][L KB]; at the end the sums of one-wave rows
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.y * blockDim.x + threadIdx.x) / 64), lane = (int)threadIdx.x % 64;
  const uint8_t* mine = ring + wave * (L * 1024) + lane * 16;
  const uint32_t mine0 = (uint32_t)(uintptr_t)(lds_u8_t*)ring + (uint32_t)(wave * (L * 1024));
  const int hs = a.hs;
  const bool wpre = a.w_pre != nullptr, wpost = RES && a.w_post != nullptr;
  const uint32_t row = (uint32_t)hs * sizeof(S);  // bytes of a stream
  float apost[NCH][V] = {}, apre[NCH][V] = {};
  uint4 gr[NCH], wr[NCH];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    gr[j] = Row<T, AL>(a.w_post, 0, 1, hs).get(j);
    wr[j] = Row<T, AL>(a.w_pre, 0, 1, hs).get(j);
  }
  int flip = 0;
  const int64_t stride = (int64_t)gridDim.x * blockDim.y;
  uint4 rr[NCH][HC], dr[NCH][HC], yr[NCH], xr[NCH];
  // Row m's pieces to LDS (AHEAD) or registers. An absent tensor, and a row
  // past the last, is an empty range, which reads as zero.
  auto fetch = [&](int64_t m) {
    const bool in = m < a.M;
    const void* R = in && wpre ? a.R : nullptr;
    if constexpr (AHEAD) {
      const i32x4_t rR = words_of<S>(R, m * a.ld_R, HC * row), rX = words_of<S>(in ? a.dx : nullptr, m * hs, row);
      const i32x4_t rD = words_of<S>(RES && in ? a.dR2 : nullptr, m * a.ld_R, HC * row);
      const i32x4_t rY = words_of<S>(RES && in ? a.y : nullptr, m * a.ld_y, row);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t at = piece_at(j, row), to = mine0 + (uint32_t)(j * (L / NCH) * 1024);
        load_lds(rX, at, to);
#pragma unroll
        for (int s = 0; s < HC; ++s) load_lds(rR, at + s * row, to + (1 + s) * 1024);
        if constexpr (RES) {
          load_lds(rY, at, to + (1 + HC) * 1024);
#pragma unroll
          for (int s = 0; s < HC; ++s) load_lds(rD, at + s * row, to + (2 + HC + s) * 1024);
        }
      }
    } else {
      const Row<T, AL> rR(R, m * a.ld_R, HC, hs), rX(in ? a.dx : nullptr, m * hs, 1, hs);
      const Row<T, AL> rD(RES && in ? a.dR2 : nullptr, m * a.ld_R, HC, hs), rY(RES && in ? a.y : nullptr, m * a.ld_y, 1, hs);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        xr[j] = rX.get(j);
        yr[j] = rY.get(j);
#pragma unroll
        for (int s = 0; s < HC; ++s) rr[j][s] = rR.get(j, s);
#pragma unroll
        for (int s = 0; s < HC; ++s) dr[j][s] = rD.get(j, s);
      }
    }
  };
  // the row's scalars, asked for one row ahead too
  struct Scalars {
    float ry, ru;
    S inj[HC];
  };
  auto scalars = [&](int64_t m) {
    Scalars z;
    m = m < a.M ? m : a.M - 1;
    z.ry = wpost ? a.rr_post[m * a.rr_ld] : 1.0f;
    z.ru = wpre ? a.rr_pre[m * a.rr_ld] : 1.0f;
    if (RES && a.inj) {
#pragma unroll
      for (int s = 0; s < HC; ++s) z.inj[s] = reinterpret_cast<const S*>(a.inj)[m * a.ld_inj + s];
    }
    return z;
  };
  const int64_t m0 = (int64_t)blockIdx.x * blockDim.y + __builtin_amdgcn_readfirstlane((int)threadIdx.y);
  Scalars sc = scalars(m0);
  if constexpr (AHEAD) fetch(m0);
  for (int64_t m = m0; m < a.M; m += stride) {
    const Scalars now = sc;
    const float ry = now.ry, ru = now.ru;
    float iw[HC], iwm = 0.0f;
    auto gates = [&]() {
#pragma unroll
      for (int s = 0; s < HC; ++s) {
        iw[s] = RES && a.inj ? gate(up(now.inj[s]), HC) : 1.0f;
        iwm += iw[s] * (1.0f / (float)HC);
      }
      if (RES && a.dinj && threadIdx.x < HC) {
        float inj = up(now.inj[0]);
#pragma unroll
        for (int s = 1; s < HC; ++s) inj = (int)threadIdx.x == s ? up(now.inj[s]) : inj;
        slopes[wave][threadIdx.x] = gate_slope(inj, HC);
      }
    };
    if constexpr (AHEAD) {
      gates();  // before the next row's loads, which the wait for the logits would take in
      // the loads are older than the row before's HC + 1 stores a piece, which
      // may still be on their way (the norm's one store is optional)
      if (RES && m != m0) landed<(HC + 1) * NCH>();
      else landed<0>();
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint8_t* from = mine + j * (L / NCH) * 1024;
        xr[j] = ld16(from);
#pragma unroll
        for (int s = 0; s < HC; ++s) rr[j][s] = ld16(from + (1 + s) * 1024);
        if constexpr (RES) {
          yr[j] = ld16(from + (1 + HC) * 1024);
#pragma unroll
          for (int s = 0; s < HC; ++s) dr[j][s] = ld16(from + (2 + HC + s) * 1024);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's place is read
      fetch(m + stride);
    } else {
      fetch(m);
      gates();
    }
    sc = scalars(m + stride);
    // u, and the row sums B_s, A, C, D
    float u[NCH][V], sums[N] = {};
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float z[V], g[V];
      if constexpr (RES) {
        unpack<T>(yr[j], z);
        unpack<T>(gr[j], g);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] * ry * (1.0f + g[i]);
#pragma unroll
        for (int s = 0; s < HC; ++s) {
          float d[V];
          unpack<T>(dr[j][s], d);
#pragma unroll
          for (int i = 0; i < V; ++i) sums[s] += d[i] * z[i];
        }
      }
      if (wpre) {
        float w[V], e[V];
        unpack<T>(rr[j][0], u[j]);
        if constexpr (RES) {
#pragma unroll
          for (int s = 1; s < HC; ++s) {
            float r[V];
            unpack<T>(rr[j][s], r);
#pragma unroll
            for (int i = 0; i < V; ++i) u[j][i] += r[i];
          }
#pragma unroll
          for (int i = 0; i < V; ++i) u[j][i] = fmaf(iwm, z[i], u[j][i] * (a.rho / (float)HC));
        }
        unpack<T>(xr[j], e);
        unpack<T>(wr[j], w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          e[i] *= 1.0f + w[i];
          sums[N == 1 ? 0 : HC] += e[i] * u[j][i];
          if constexpr (RES) {
            sums[HC + 1] += e[i] * z[i];
            sums[HC + 2] += u[j][i] * z[i];
          }
        }
      }
    }
    group_sum(sums, red[flip]);
    flip ^= 1;  // the next row's sums go where no thread still reads
    const float m_pre = wpre ? ru * sums[N == 1 ? 0 : HC] / (float)hs : 0.0f;
    float m_post = 0.0f;
    if constexpr (RES) {
      const float duz = wpre ? ru * (sums[HC + 1] - m_pre * ru * sums[HC + 2]) / (float)HC : 0.0f;
#pragma unroll
      for (int s = 0; s < HC; ++s) {
        const float diw = sums[s] + duz;
        m_post += iw[s] * diw;
        if (a.dinj && (int)threadIdx.x == s)
          reinterpret_cast<S*>(a.dinj)[m * a.ld_dinj + s] = down<T>(diw * slopes[wave][s]);
      }
      m_post /= (float)hs;
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float du[V] = {};
      if (wpre) {
        float dx[V], w[V];
        unpack<T>(xr[j], dx);
        unpack<T>(wr[j], w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float hu = u[j][i] * ru;
          du[i] = ru * (dx[i] * (1.0f + w[i]) - hu * m_pre);
          apre[j][i] += dx[i] * hu;
        }
      }
      if constexpr (!RES) {
        if (a.dR) Row<T, AL>(a.dR, m * hs, 1, hs).put(j, 0, du, 1);
      } else {
        float dz[V] = {};
#pragma unroll
        for (int s = 0; s < HC; ++s) {
          float d[V];
          unpack<T>(dr[j][s], d);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            d[i] = fmaf(du[i], 1.0f / (float)HC, d[i]);
            dz[i] = fmaf(iw[s], d[i], dz[i]);
            d[i] *= a.rho;
          }
          Row<T, AL>(a.dR, m * a.ld_R, HC, hs).put(j, s, d, 1);
        }
        if (wpost) {
          float h[V], g[V];
          unpack<T>(yr[j], h);
          unpack<T>(gr[j], g);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            h[i] *= ry;
            apost[j][i] += dz[i] * h[i];
            dz[i] = ry * (dz[i] * (1.0f + g[i]) - h[i] * m_post);
          }
        }
        Row<T, AL>(a.dy, m * hs, 1, hs).put(j, 0, dz, 1);
      }
    }
  }
  if constexpr (AHEAD) landed<0>();  // no load into this workgroup's LDS outlives it
  if (!a.dw_post && !a.dw_pre) return;
  if (blockDim.y > 1) {  // four waves, blockDim.x = 64
    float(*wred)[2][64 * NCH * V] = reinterpret_cast<float(*)[2][64 * NCH * V]>(ring);
    __syncthreads();  // every wave's place is read
    const int w = (int)threadIdx.y, t = (int)threadIdx.x;
    if (w > 0) {
#pragma unroll
      for (int j = 0; j < NCH; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          wred[w - 1][0][(j * V + i) * 64 + t] = apost[j][i];
          wred[w - 1][1][(j * V + i) * 64 + t] = apre[j][i];
        }
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          apost[j][i] += wred[k][0][(j * V + i) * 64 + t];
          apre[j][i] += wred[k][1][(j * V + i) * 64 + t];
        }
  }
  float* part = reinterpret_cast<float*>(a.ws) + bwd_row_floats(a.M) + (int64_t)blockIdx.x * 2 * hs;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c = ((int)threadIdx.x + j * (int)blockDim.x) * V;
    if (c >= hs) continue;
    if constexpr (AL) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        if (a.dw_post)
          *reinterpret_cast<float4*>(part + c + i) = make_float4(apost[j][i], apost[j][i + 1], apost[j][i + 2], apost[j][i + 3]);
        if (a.dw_pre)
          *reinterpret_cast<float4*>(part + hs + c + i) = make_float4(apre[j][i], apre[j][i + 1], apre[j][i + 2], apre[j][i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (c + i >= hs) break;
        if (a.dw_post) part[c + i] = apost[j][i];
        if (a.dw_pre) part[hs + c + i] = apre[j][i];
      }
    }
  }
}

// ---------------------------------------------------------------- launches --
constexpr int64_t kMaxGrid = 1 << 20;
// Threads of a launch in one dimension: HIP takes fewer than 2^32.
constexpr int64_t kMaxThreads = (int64_t)1 << 31;

bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool ld16_ok(int64_t ld, int b) { return ld * b % 16 == 0; }

// Whether every row of the call starts on 16 bytes and HS is whole pieces.
bool aligned(const NormArgs& a, int b) {
  return ld16_ok(a.hs, b) && al16(a.R) && ld16_ok(a.ld_R, b) && al16(a.y) && ld16_ok(a.ld_y, b) && al16(a.w_post) &&
         al16(a.w_pre) && al16(a.R2) && al16(a.x);
}
bool aligned(const NormBwdArgs& a, int b) {
  return ld16_ok(a.hs, b) && al16(a.R) && ld16_ok(a.ld_R, b) && al16(a.y) && ld16_ok(a.ld_y, b) && al16(a.w_post) &&
         al16(a.w_pre) && al16(a.dR2) && al16(a.dx) && al16(a.dR) && al16(a.dy);
}

// Whether outputs of that many rows of HS values a token outgrow the L2s (8 x 4
// MB). Measured with the streaming policy on one MI355X (HS = 2560, bf16):
// residual M = 16384 HC = 4 148 -> 142 us, but the residual of 333 tokens, whose
// outputs stay in the caches, 3.7 -> 4.0 us. (The backward kernels always use
// it: a choice at run time costs registers that they do not have.)
bool streamed(int64_t M, int hs, int rows, size_t b) {
  return (double)M * hs * rows * (double)b > 32.0 * 1024 * 1024;
}

int loop_threads(int64_t pieces) {
  const int64_t t = cdiv64(pieces, 64) * 64;
  return (int)(t < 1024 ? t : 1024);
}

template <typename T, bool AL>
int forward_loop(const NormArgs& a, bool residual, bool norm, hipStream_t st) {
  const dim3 grid((unsigned)(a.M < kMaxGrid ? a.M : kMaxGrid)), blk((unsigned)loop_threads(cdiv64(a.hs, vec<T>())));
  if (!norm) hipLaunchKernelGGL((norm_loop<T, AL, false, false>), grid, blk, 0, st, a);
  else if (residual) hipLaunchKernelGGL((norm_loop<T, AL, true, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((norm_loop<T, AL, false, true>), grid, blk, 0, st, a);
  return (int)hipGetLastError();
}

template <typename T, int NCH, bool AL>
int forward_row(NormArgs a, bool residual, bool norm, hipStream_t st) {
  a.nt = streamed(a.M, a.hs, residual ? a.hc + 1 : 1, sizeof(typename T::S));
  const int64_t pieces = cdiv64(a.hs, vec<T>());
  const int nw = (int)cdiv64(pieces, 64 * NCH);
  const dim3 blk((unsigned)nw * 64, nw == 1 ? 4 : 1);
  const int64_t rows = kMaxThreads / blk.x * blk.y;  // of a launch; longer calls take several
  for (; a.m_first < a.M; a.m_first += rows) {
    const dim3 grid((unsigned)cdiv64(std::min(rows, a.M - a.m_first), blk.y));
    if (!norm) hipLaunchKernelGGL((norm_row<T, 1, NCH, AL, false, false>), grid, blk, 0, st, a);
    else if (!residual) hipLaunchKernelGGL((norm_row<T, 1, NCH, AL, false, true>), grid, blk, 0, st, a);
    else if (a.hc == 1) hipLaunchKernelGGL((norm_row<T, 1, NCH, AL, true, true>), grid, blk, 0, st, a);
    else if (a.hc == 2) hipLaunchKernelGGL((norm_row<T, 2, NCH, AL, true, true>), grid, blk, 0, st, a);
    else if (a.hc == 4) hipLaunchKernelGGL((norm_row<T, 4, NCH, AL, true, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((norm_row<T, 8, NCH, AL, true, true>), grid, blk, 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
  }
  return (int)hipSuccess;
}

template <typename T>
int forward_of(const NormArgs& a, bool residual, bool norm, hipStream_t st) {
  const bool al = aligned(a, (int)sizeof(typename T::S));
  const int64_t pieces = cdiv64(a.hs, vec<T>());
  if (pieces <= 1024) return al ? forward_row<T, 1, true>(a, residual, norm, st) : forward_row<T, 1, false>(a, residual, norm, st);
  if (pieces <= 2048 && al) return forward_row<T, 2, true>(a, residual, norm, st);
  return al ? forward_loop<T, true>(a, residual, norm, st) : forward_loop<T, false>(a, residual, norm, st);
}

int sum_groups(const NormBwdArgs& a, int64_t groups, hipStream_t st) {
  if (a.dw_post || a.dw_pre)
    hipLaunchKernelGGL(norm_bwd_sum, dim3((unsigned)cdiv64(a.hs, 32), 2), dim3(1024), 0, st, a, (int)groups);
  return (int)hipGetLastError();
}

template <typename T, bool AL, bool RES>
int backward_loop(const NormBwdArgs& a, hipStream_t st) {
  const int64_t groups = bwd_groups(a.M), pieces = cdiv64(a.hs, vec<T>());
  hipLaunchKernelGGL((norm_bwd_rows<T, AL, RES>), dim3((unsigned)(a.M < kMaxGrid ? a.M : kMaxGrid)),
                     dim3((unsigned)loop_threads(pieces)), 0, st, a);
  hipLaunchKernelGGL((norm_bwd_cols<T, AL, RES>), dim3((unsigned)cdiv64(pieces, kColThreads), (unsigned)groups),
                     dim3(kColThreads), 0, st, a);
  return sum_groups(a, groups, st);
}

template <typename T, int NCH, int THREADS, bool AL>
int backward_row(const NormBwdArgs& a, bool residual, hipStream_t st) {
  const int64_t pieces = cdiv64(a.hs, vec<T>());
  const int nw = (int)cdiv64(pieces, 64 * NCH);
  const dim3 blk((unsigned)nw * 64, nw == 1 ? 4 : 1);
  const int64_t rows = cdiv64(a.M, blk.y);
  int64_t groups = bwd_groups(rows);
  // One stream: a row is little work next to its share of the partial sums, so
  // up to four rows a workgroup before the chip has more than one a CU (M =
  // 1500, HS = 2560: 15.8 -> 14.1 us; four streams, M = 1000: 29.9 -> 31.6 us).
  if (!residual || a.hc == 1) groups = std::min(groups, std::max<int64_t>(256, rows / 4));
  const dim3 grid((unsigned)groups);
  const size_t lds = bwd_lds(residual ? a.hc : 0, NCH, (int)(blk.x * blk.y / 64), vec<T>(), AL && THREADS <= 512 && NCH == 1, nw == 1);
  if constexpr (THREADS == 512) {
    if (residual && a.hc == 8) hipLaunchKernelGGL((norm_bwd_row<T, 8, NCH, THREADS, AL, true>), grid, blk, lds, st, a);
  }
  if constexpr (NCH == 1 || THREADS == 1024) {
    if (!residual) hipLaunchKernelGGL((norm_bwd_row<T, 1, NCH, THREADS, AL, false>), grid, blk, lds, st, a);
  }
  if constexpr (NCH == 1) {
    if (residual && a.hc == 1) hipLaunchKernelGGL((norm_bwd_row<T, 1, NCH, THREADS, AL, true>), grid, blk, lds, st, a);
    else if (residual && a.hc == 2) hipLaunchKernelGGL((norm_bwd_row<T, 2, NCH, THREADS, AL, true>), grid, blk, lds, st, a);
    else if (residual && a.hc == 4) hipLaunchKernelGGL((norm_bwd_row<T, 4, NCH, THREADS, AL, true>), grid, blk, lds, st, a);
  }
  return sum_groups(a, groups, st);
}

template <typename T>
hipError_t raise_lds() {
  const void* f[] = {(const void*)norm_bwd_row<T, 4, 1, 512, true, true>, (const void*)norm_bwd_row<T, 8, 1, 512, true, true>};
  for (const void* k : f) {
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, 152 * 1024);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
int backward_of(const NormBwdArgs& a, bool residual, hipStream_t st) {
  const int64_t pieces = cdiv64(a.hs, vec<T>());
  const bool al = aligned(a, (int)sizeof(typename T::S));
  if (pieces <= 512) return al ? backward_row<T, 1, 512, true>(a, residual, st) : backward_row<T, 1, 512, false>(a, residual, st);
  if (pieces <= 1024 && residual && a.hc == 8)
    // eight streams do not fit the 128 registers of 1024 threads: 512 threads
    // with two pieces each, 179 us instead of 358 at M = 1000, HS = 8192 (bf16)
    return al ? backward_row<T, 2, 512, true>(a, residual, st) : backward_row<T, 2, 512, false>(a, residual, st);
  if (pieces <= 1024) return al ? backward_row<T, 1, 1024, true>(a, residual, st) : backward_row<T, 1, 1024, false>(a, residual, st);
  if (pieces <= 2048 && !residual)
    return al ? backward_row<T, 2, 1024, true>(a, residual, st) : backward_row<T, 2, 1024, false>(a, residual, st);
  if (!al) return residual ? backward_loop<T, false, true>(a, st) : backward_loop<T, false, false>(a, st);
  return residual ? backward_loop<T, true, true>(a, st) : backward_loop<T, true, false>(a, st);
}

int dispatch(const NormArgs& a, int dtype, bool residual, bool norm, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? forward_of<Bf16>(a, residual, norm, st)
         : dtype == 1 ? forward_of<Fp16>(a, residual, norm, st)
                      : forward_of<Fp32>(a, residual, norm, st);
}

}  // namespace

int launch_norm(const NormArgs& a, int dtype, bool residual, void* stream) {
  return dispatch(a, dtype, residual, true, stream);
}
int launch_quantize(const NormArgs& a, int dtype, void* stream) { return dispatch(a, dtype, false, false, stream); }

int launch_norm_bwd(const NormBwdArgs& a, int dtype, bool residual, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? backward_of<Bf16>(a, residual, st)
         : dtype == 1 ? backward_of<Fp16>(a, residual, st)
                      : backward_of<Fp32>(a, residual, st);
}

// Raises the dynamic-LDS limit of the backward kernels on the current device.
int configure_block_kernels() {
  for (const hipError_t e : {raise_lds<Bf16>(), raise_lds<Fp16>(), raise_lds<Fp32>()})
    if (e != hipSuccess) return (int)e;
  return (int)hipSuccess;
}

size_t norm_bwd_workspace(int hs, int64_t M) {
  if (M == 0) return 0;
  return (size_t)(bwd_row_floats(M) + bwd_groups(M) * 2 * hs) * sizeof(float);
}

}  // namespace hcgr
