// hcgr_block.hip -- the norms around a block (hcgr_block_norm,
// hcgr_block_residual), their gradients, and the row quantizer. The
// mathematics stands in include/hcgr.h.
#include <hip/hip_runtime.h>

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

// V values of a row: V = 1, or as many as 16 bytes hold.
template <typename T, int V>
__device__ __forceinline__ void load(const typename T::S* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = up(*p);
  } else {
    union { uint4 u; typename T::S s[V]; } x;
    x.u = ld16(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = up(x.s[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store(typename T::S* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = down<T>(f[0]);
  } else {
    union { uint4 u; typename T::S s[V]; } x;
#pragma unroll
    for (int i = 0; i < V; ++i) x.s[i] = down<T>(f[i]);
    st16(p, x.u);
  }
}

// ------------------------------------------------------------ reductions --
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
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
// 2*sigmoid(inj/HC), and its derivative in inj
__device__ __forceinline__ float gate(float inj, int hc) { return 2.0f / (1.0f + expf(-inj / (float)hc)); }
__device__ __forceinline__ float gate_slope(float iw, int hc) { return iw * (1.0f - 0.5f * iw) / (float)hc; }

// ---------------------------------------------------------- quantization --
// Magnitudes are compared as their bit patterns (an infinity or a NaN is
// above every number), so a row's maximum says whether the row is finite.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
struct Quant {
  float scale, pre, inv;  // q = round(v * pre * inv)
};
// For rows whose largest value is below 2^-100, 127/amax would overflow: such
// values are brought up by 2^100 first (exact).
__device__ __forceinline__ Quant quant_of(uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits);
  Quant z;
  z.pre = amax < 0x1p-100f ? 0x1p100f : 1.0f;
  const bool finite = amax_bits < 0x7f800000u;
  z.scale = finite ? amax / 127.0f : __uint_as_float(0x7fc00000u);
  z.inv = finite && amax > 0.0f ? 127.0f / (amax * z.pre) : 0.0f;
  return z;
}
__device__ __forceinline__ int quant1(float v, const Quant& z) {
  // z.inv = 0 (an all-zero row, or one that is not finite) gives 0: the
  // product may be NaN there, which the comparison sends to 0
  const float t = rintf(v * z.pre * z.inv);
  return fabsf(t) <= 127.0f ? (int)t : 0;
}
template <int V>
__device__ __forceinline__ void store_q(int8_t* p, const float (&v)[V], const Quant& z) {
  if constexpr (V == 1) {
    *p = (int8_t)quant1(v[0], z);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V; i += 4)
      w[i / 4] = (uint32_t)(quant1(v[i], z) & 255) | (uint32_t)(quant1(v[i + 1], z) & 255) << 8 |
                 (uint32_t)(quant1(v[i + 2], z) & 255) << 16 | (uint32_t)(quant1(v[i + 3], z) & 255) << 24;
    if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
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
template <typename T, int V, bool RES, bool NORM>
__global__ __launch_bounds__(1024) void norm_loop(NormArgs a) {
  using S = typename T::S;
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
          load<T, V>(y + c, f);
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
        load<T, V>(R + c, u);
      } else {
        float z[V];
        load<T, V>(y + c, z);
        if (wpost) {
          float w[V];
          load<T, V>(wpost + c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) z[i] = z[i] * ry * (1.0f + w[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = 0.0f;
        for (int s = 0; s < hc; ++s) {
          float r[V];
          load<T, V>(R + (int64_t)s * hs + c, r);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            r[i] = fmaf(iw[s], z[i], a.rho * r[i]);
            u[i] += r[i];
          }
          if (write) store<T, V>(R2 + (int64_t)s * hs + c, r);
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
        if (a.q) load<T, V>(wpre + c, w);
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
          load<T, V>(wpre + c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) u[i] = u[i] * (1.0f + w[i]) * ru;
          if (a.x) store<T, V>(reinterpret_cast<S*>(a.x) + m * hs + c, u);
        }
        if (a.q) store_q<V>(a.q + m * a.ld_q + c, u, z);
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
constexpr int kRowGroups = 512;  // partial sums of the weight gradients
constexpr int kColThreads = 256;

// Workspace: m_pre and m_post of each row, then [groups][2][HS] partial sums.
__host__ __device__ inline int64_t bwd_groups(int64_t M) { return M < kRowGroups ? M : kRowGroups; }
__host__ __device__ inline int64_t bwd_row_floats(int64_t M) { return (2 * M + 3) / 4 * 4; }

template <typename T, int V, bool RES>
struct BwdRow {
  using S = typename T::S;
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
    load<T, V>(y + c, h);
    if (wpost) load<T, V>(wpost + c, g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] *= ry;
      g[i] = wpost ? 1.0f + g[i] : 1.0f;
      z[i] = h[i] * g[i];
    }
  }
  __device__ __forceinline__ void form_u(int c, const float (&z)[V], float (&u)[V]) const {
    if constexpr (!RES) {
      load<T, V>(R + c, u);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = 0.0f;
      for (int s = 0; s < hc; ++s) {
        float r[V];
        load<T, V>(R + (int64_t)s * a.hs + c, r);
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
    load<T, V>(dx + c, d);
    load<T, V>(wpre + c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = d[i] * (1.0f + w[i]);
  }
};

template <typename T, int V, bool RES>
__global__ __launch_bounds__(1024) void norm_bwd_rows(NormBwdArgs a) {
  __shared__ float red[16 * (kMaxHc + 3)];
  float* rows = reinterpret_cast<float*>(a.ws);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const BwdRow<T, V, RES> row(a, m);
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
          load<T, V>(row.dR2 + (int64_t)s * a.hs + c, d);
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
          if (a.dinj)
            reinterpret_cast<typename T::S*>(a.dinj)[m * a.ld_dinj + s] = down<T>(diw * gate_slope(row.iw[s], row.hc));
        }
      }
      rows[2 * m] = m_pre;
      rows[2 * m + 1] = m_post / (float)a.hs;
    }
    __syncthreads();  // the next row reuses red
  }
}

template <typename T, int V, bool RES>
__global__ __launch_bounds__(kColThreads) void norm_bwd_cols(NormBwdArgs a) {
  using S = typename T::S;
  const int c = ((int)blockIdx.x * kColThreads + (int)threadIdx.x) * V;
  if (c >= a.hs) return;
  const float* rows = reinterpret_cast<const float*>(a.ws);
  float apost[V] = {}, apre[V] = {};
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    const BwdRow<T, V, RES> row(a, m);
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
      if (a.dR) store<T, V>(reinterpret_cast<S*>(a.dR) + m * a.hs + c, du);
    } else {
      float dz[V] = {};
      for (int s = 0; s < row.hc; ++s) {
        float d[V] = {};
        if (row.dR2) load<T, V>(row.dR2 + (int64_t)s * a.hs + c, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          d[i] += du[i] / (float)row.hc;
          dz[i] = fmaf(row.iw[s], d[i], dz[i]);
          d[i] *= a.rho;
        }
        store<T, V>(reinterpret_cast<S*>(a.dR) + m * a.ld_R + (int64_t)s * a.hs + c, d);
      }
      if (row.wpost) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          apost[i] += dz[i] * h[i];
          dz[i] = row.ry * (dz[i] * g[i] - h[i] * m_post);
        }
      }
      store<T, V>(reinterpret_cast<S*>(a.dy) + m * a.hs + c, dz);
    }
  }
  float* part = reinterpret_cast<float*>(a.ws) + bwd_row_floats(a.M) + (int64_t)blockIdx.y * 2 * a.hs;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (a.dw_post) part[c + i] = apost[i];
    if (a.dw_pre) part[a.hs + c + i] = apre[i];
  }
}

__global__ __launch_bounds__(256) void norm_bwd_sum(NormBwdArgs a, int groups) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const int c = (int)blockIdx.x * 64 + lane;
  float* out = blockIdx.y ? a.dw_pre : a.dw_post;
  if (!out) return;
  const float* part = reinterpret_cast<const float*>(a.ws) + bwd_row_floats(a.M) + (int64_t)blockIdx.y * a.hs;
  float s = 0.0f;
  if (c < a.hs)
    for (int g = w; g < groups; g += 4) s += part[(int64_t)g * 2 * a.hs + c];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < a.hs) out[c] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
}

// ---------------------------------------------------------------- launches --
constexpr int64_t kMaxGrid = 1 << 20;

template <typename T>
constexpr int vec() { return 16 / (int)sizeof(typename T::S); }

bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool ld16_ok(int64_t ld, int b) { return ld * b % 16 == 0; }

// Whether every row of the call starts on 16 bytes and HS is whole pieces.
bool vec_ok(const NormArgs& a, int b) {
  return ld16_ok(a.hs, b) && al16(a.R) && ld16_ok(a.ld_R, b) && al16(a.y) && ld16_ok(a.ld_y, b) && al16(a.w_post) &&
         al16(a.w_pre) && al16(a.R2) && al16(a.x);
}
bool vec_ok(const NormBwdArgs& a, int b) {
  return ld16_ok(a.hs, b) && al16(a.R) && ld16_ok(a.ld_R, b) && al16(a.y) && ld16_ok(a.ld_y, b) && al16(a.w_post) &&
         al16(a.w_pre) && al16(a.dR2) && al16(a.dx) && al16(a.dR) && al16(a.dy);
}

int loop_threads(int hs, int v) {
  const int64_t t = cdiv64(cdiv64(hs, v), 64) * 64;
  return (int)(t < 1024 ? t : 1024);
}

template <typename T, int V>
int norm_forward(const NormArgs& a, bool residual, bool norm, hipStream_t st) {
  const dim3 grid((unsigned)(a.M < kMaxGrid ? a.M : kMaxGrid)), blk((unsigned)loop_threads(a.hs, V));
  if (!norm) hipLaunchKernelGGL((norm_loop<T, V, false, false>), grid, blk, 0, st, a);
  else if (residual) hipLaunchKernelGGL((norm_loop<T, V, true, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((norm_loop<T, V, false, true>), grid, blk, 0, st, a);
  return (int)hipGetLastError();
}

template <typename T, int V, bool RES>
int norm_backward(const NormBwdArgs& a, hipStream_t st) {
  const int64_t groups = bwd_groups(a.M);
  hipLaunchKernelGGL((norm_bwd_rows<T, V, RES>), dim3((unsigned)(a.M < kMaxGrid ? a.M : kMaxGrid)),
                     dim3((unsigned)loop_threads(a.hs, V)), 0, st, a);
  hipLaunchKernelGGL((norm_bwd_cols<T, V, RES>),
                     dim3((unsigned)cdiv64(a.hs, kColThreads * V), (unsigned)groups), dim3(kColThreads), 0, st, a);
  if (a.dw_post || a.dw_pre)
    hipLaunchKernelGGL(norm_bwd_sum, dim3((unsigned)cdiv64(a.hs, 64), 2), dim3(256), 0, st, a, (int)groups);
  return (int)hipGetLastError();
}

template <typename T>
int forward_of(const NormArgs& a, bool residual, bool norm, hipStream_t st) {
  return vec_ok(a, (int)sizeof(typename T::S)) ? norm_forward<T, vec<T>()>(a, residual, norm, st)
                                               : norm_forward<T, 1>(a, residual, norm, st);
}
template <typename T>
int backward_of(const NormBwdArgs& a, bool residual, hipStream_t st) {
  if (vec_ok(a, (int)sizeof(typename T::S)))
    return residual ? norm_backward<T, vec<T>(), true>(a, st) : norm_backward<T, vec<T>(), false>(a, st);
  return residual ? norm_backward<T, 1, true>(a, st) : norm_backward<T, 1, false>(a, st);
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

size_t norm_bwd_workspace(int hs, int64_t M) {
  if (M == 0) return 0;
  return (size_t)(bwd_row_floats(M) + bwd_groups(M) * 2 * hs) * sizeof(float);
}

}  // namespace hcgr
