// hcgr_layer_norm.hip -- the layer norm and its gradients
// (hcgr_block_layer_norm, hcgr_block_layer_norm_bwd). The mathematics stands
// in include/hcgr.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "hcgr_block.h"
#include "hcgr_device.h"
#include "hcgr_mx.h"
#include "hcgr_rows.h"

namespace hcgr {
namespace {

// ---------------------------------------------------------------------------
// The statistics of a row whose values lie in the registers of several waves,
// with one exchange between them and without cancellation: each wave takes its
// own mean a (rounded) and the sums S1, S2 of x - a and (x - a)^2. With A the
// first wave's a and n values of each wave,
//   mean = A + D,  D = sum_w (n (a - A) + S1) / HS
//   var  = sum_w (S2 + 2 c S1 + n c^2) / HS,  c = a - mean = (a - A) - D,
// and a value's distance from the mean is (x - a) + c: the mean is never
// rounded to one number where it is large next to the deviations.
//
// A row gives the same bits whatever batch it stands in: how its sums are cut
// and joined is a function of its width alone. Where few rows take more waves
// than many do (whole_row), they add up what one wave would, in its order.
// ---------------------------------------------------------------------------
struct Spread {
  float mean, rstd, c;  // c: what a value's distance from its wave's mean lacks
};
__device__ __forceinline__ float rstd_of(float var, float eps) {
  return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);  // (NaN stays NaN)
}
// Values a wave holds when it takes pieces t + j*threads, t its 64 threads.
template <int V>
__device__ __forceinline__ int values_of_wave(int wave, int threads, int nch, int hs) {
  int n = 0;
  for (int j = 0; j < nch; ++j) n += min(max(hs - (j * threads + wave * 64) * V, 0), 64 * V);
  return n;
}
// A lane's N sums over its pieces of the whole row, of which each wave has one
// piece a lane: in the order of the pieces, as one wave that holds all of them
// adds. `red`: 64*N floats a wave.
template <int N>
__device__ __forceinline__ void whole_row(float (&v)[N], float* red) {
  const int nw = (int)blockDim.x / 64, w = (int)threadIdx.x / 64, lane = (int)threadIdx.x % 64;
  if (nw == 1) return;
#pragma unroll
  for (int i = 0; i < N; ++i) red[(w * N + i) * 64 + lane] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = red[i * 64 + lane];
  for (int k = 1; k < nw; ++k) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += red[(k * N + i) * 64 + lane];
  }
}
// The statistics of a row from the sums over all of it.
__device__ __forceinline__ Spread spread_of_row(float a, float s1, float s2, int hs, float eps) {
  const float d = s1 / (float)hs;
  return {a + d, rstd_of(fmaf(-d, d, s2 / (float)hs), eps), -d};
}
// And from those of its waves. `red`: three floats a wave.
template <int V>
__device__ __forceinline__ Spread spread_of(float a, float s1, float s2, int nch, int hs, float eps, float* red) {
  const int nw = (int)blockDim.x / 64, w = (int)threadIdx.x / 64;
  if (nw == 1) return spread_of_row(a, s1, s2, hs, eps);
  Spread z;
  if (threadIdx.x % 64 == 0) {
    red[w * 3] = a;
    red[w * 3 + 1] = s1;
    red[w * 3 + 2] = s2;
  }
  __syncthreads();
  const float A = red[0];
  float d = 0.0f;
  for (int k = 0; k < nw; ++k)
    d += fmaf((float)values_of_wave<V>(k, (int)blockDim.x, nch, hs), red[k * 3] - A, red[k * 3 + 1]);
  d /= (float)hs;
  float var = 0.0f;
  for (int k = 0; k < nw; ++k) {
    const float c = (red[k * 3] - A) - d;
    var += red[k * 3 + 2] + c * fmaf((float)values_of_wave<V>(k, (int)blockDim.x, nch, hs), c, 2.0f * red[k * 3 + 1]);
  }
  z.mean = A + d;
  z.rstd = rstd_of(var / (float)hs, eps);
  z.c = (a - A) - d;
  return z;
}

// V normed values, from their distances to the mean (add/r short of it), n of
// which the row still has; zero past the row.
template <int V, bool AL>
__device__ __forceinline__ void affine(float (&d)[V], float add, float r, bool has_w, const float (&w)[V],
                                       const float (&b)[V], int n) {
  if (has_w) {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = fmaf(fmaf(d[i], r, add), w[i], b[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = fmaf(d[i], r, add) + b[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = (AL ? n > 0 : i < n) ? d[i] : 0.0f;
}

// ---------------------------------------------------------------------------
// layer_norm_row: rows that fit the registers of a workgroup (NCH 16-byte
// pieces a thread): each value is read once. Rows of at most 64 * NCH pieces
// take one wave, four rows a workgroup, without barriers. With one piece a
// thread the waves (up to kWholeWaves) sum as one wave would.
// ---------------------------------------------------------------------------
constexpr int kWholeWaves = 5;
template <typename T, int NCH, bool AL>
__global__ __launch_bounds__(1024) void layer_norm_row(LayerNormArgs a) {
  constexpr int V = vec<T>();
  __shared__ float red[NCH == 1 ? kWholeWaves * 64 * 3 : 16 * 3];
  const int hs = a.hs, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
  const int64_t m = a.m_first + (int64_t)blockIdx.x * blockDim.y + __builtin_amdgcn_readfirstlane((int)threadIdx.y);
  if (m >= a.M) return;  // blockDim.y > 1 only without barriers
  const Row<T, AL> rx(a.x, m * a.ld_x, 1, hs), rw(a.w, 0, 1, hs), rb(a.b, 0, 1, hs);
  uint4 xr[NCH], wr[NCH], br[NCH];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    xr[j] = rx.get(j);
    wr[j] = rw.get(j);
    br[j] = rb.get(j);
  }
  // From three pieces a thread on, whose rows one wave or several may hold: sums
  // of each piece, then of the pieces in turn. Otherwise in one go (1000 fp16
  // channels, 1024 rows: 3.2 us for 3.3).
  constexpr bool APART = NCH >= 3;
  float d[NCH][V], s[1] = {};
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    unpack<T>(xr[j], d[j]);
    float p = APART ? 0.0f : s[0];
#pragma unroll
    for (int i = 0; i < V; ++i) p += d[j][i];
    s[0] = APART && j > 0 ? s[0] + p : p;
  }
  if constexpr (NCH == 1) whole_row(s, red);
  const int values = NCH == 1 ? hs : values_of_wave<V>(wave, (int)blockDim.x, NCH, hs);
  const float mine = wave_sum(s[0]) / (float)values;
  float dev[2] = {};
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int n = hs - ((int)threadIdx.x + j * (int)blockDim.x) * V;
    float p1 = APART ? 0.0f : dev[0], p2 = APART ? 0.0f : dev[1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      d[j][i] = (AL ? n > 0 : i < n) ? d[j][i] - mine : 0.0f;
      p1 += d[j][i];
      p2 = fmaf(d[j][i], d[j][i], p2);
    }
    dev[0] = APART && j > 0 ? dev[0] + p1 : p1;
    dev[1] = APART && j > 0 ? dev[1] + p2 : p2;
  }
  if constexpr (NCH == 1) whole_row(dev, red + kWholeWaves * 64);
  const float s1 = wave_sum(dev[0]), s2 = wave_sum(dev[1]);
  const Spread z = NCH == 1 ? spread_of_row(mine, s1, s2, hs, a.eps) : spread_of<V>(mine, s1, s2, NCH, hs, a.eps, red);
  if (a.stats && threadIdx.x == 0) {
    a.stats[2 * m] = z.mean;
    a.stats[2 * m + 1] = z.rstd;
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c = ((int)threadIdx.x + j * (int)blockDim.x) * V;
    float w[V], b[V];
    unpack<T>(wr[j], w);
    unpack<T>(br[j], b);
    affine<V, AL>(d[j], z.c * z.rstd, z.rstd, a.w != nullptr, w, b, hs - c);
    if (a.xn) Row<T, AL>(a.xn, m * hs, 1, hs).put(j, 0, d[j], a.nt);
    if (a.q) mx_store<V>(a.q + m * a.ld_q, a.q_scale + m * a.ld_qs, c, (hs + 31) / 32, d[j]);
  }
}

// ---------------------------------------------------------------------------
// layer_norm_loop: any width. One workgroup a row at a time walks it three
// times (from the caches): the mean, the deviations, the output.
// ---------------------------------------------------------------------------
template <typename T, bool AL>
__global__ __launch_bounds__(1024) void layer_norm_loop(LayerNormArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  __shared__ float red[3][16 * 2];
  const int hs = a.hs, step = (int)blockDim.x * V;
  // whole blocks of 32 values, so that the lanes of a block stay together
  const int end = (hs + 31) / 32 * 32;
  const S *w = reinterpret_cast<const S*>(a.w), *b = reinterpret_cast<const S*>(a.b);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const S* x = reinterpret_cast<const S*>(a.x) + m * a.ld_x;
    float s[1] = {0.0f};
    for (int c = (int)threadIdx.x * V; c < hs; c += step) {
      float f[V];
      load<T, AL>(x + c, hs - c, f);
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] += f[i];
    }
    group_sum(s, red[0]);
    const float mean = s[0] / (float)hs;
    float dev[2] = {};
    for (int c = (int)threadIdx.x * V; c < hs; c += step) {
      float f[V];
      load<T, AL>(x + c, hs - c, f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = c + i < hs ? f[i] - mean : 0.0f;
        dev[0] += d;
        dev[1] += d * d;
      }
    }
    group_sum(dev, red[1]);
    const float d = dev[0] / (float)hs, rstd = rstd_of(fmaf(-d, d, dev[1] / (float)hs), a.eps);
    if (a.stats && threadIdx.x == 0) {
      a.stats[2 * m] = mean + d;
      a.stats[2 * m + 1] = rstd;
    }
    for (int c = (int)threadIdx.x * V; c < end; c += step) {
      float f[V], g[V] = {}, h[V] = {};
      load<T, AL>(x + c, hs - c, f);
      if (w) load<T, AL>(w + c, hs - c, g);
      if (b) load<T, AL>(b + c, hs - c, h);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] -= mean;
      affine<V, false>(f, -d * rstd, rstd, w != nullptr, g, h, hs - c);
      if (a.xn) store<T, AL>(reinterpret_cast<S*>(a.xn) + m * hs + c, hs - c, f);
      if (a.q) mx_store<V>(a.q + m * a.ld_q, a.q_scale + m * a.ld_qs, c, end / 32, f);
    }
    __syncthreads();  // the next row reuses the reduction arrays
  }
}

// ---------------------------------------------------------------------------
// The backward pass. With h = (x - mean)*r and e = dx*w a row needs the two
// sums P = sum e and Q = sum e*h:
//   dv = r*(e - P/HS - h*Q/HS),   dw += dx*h,   db += dx.
// layer_norm_bwd_row: rows that fit the registers of a team of waves, in one
// pass over the data. A workgroup's teams walk the rows together, each keeps
// its columns' sums for dw and db in registers; the teams' sums meet in LDS at
// the end, and norm_bwd_sum adds the workgroups' sums in a fixed order. A team of
// one wave needs no barrier. AL: the next row's pieces come to LDS behind this
// row's products and stores, each wave's into a place of its own. Bound by
// memory where there are rows enough: 29.3 us for 8192 rows of 2560 bf16
// channels (4.3 TB/s of x, dxn and dx; 9.3 us are spent before the first row is
// there and in the sums of dw and db), 55.4 us for 16384 (4.5 TB/s). Rows off 16
// bytes pay for it (2563 channels: 145 us): each of a thread's loads stands behind
// a branch of its own for the row's end, and no row is loaded ahead.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void hide(uint4& v) { asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }
// Waves of a workgroup, one workgroup a CU: as many as the registers of a wave
// allow (dw and db take 2*NCH*V of them).
template <typename T, int NCH>
constexpr int bwd_waves() { return vec<T>() == 8 ? (NCH <= 2 ? 16 : 8) : (NCH <= 4 ? 16 : 12); }
// The statistics lie behind a pointer to constant memory, so that the compiler
// reads them with scalar loads: a vector load would wait for the direct loads
// that are in flight.
typedef const __attribute__((address_space(4))) float const_f32_t;

template <typename T, int NCH, bool AL>
__global__ __launch_bounds__((64 * bwd_waves<T, NCH>())) void layer_norm_bwd_row(LayerNormBwdArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>(), L = 2 * NCH;
  __shared__ float red[2][bwd_waves<T, NCH>() * 2];
  // w [NCH][threads of a team] (in registers it would make others spill), then
  // [waves][L KB]; at the end the teams' sums
  extern __shared__ __attribute__((aligned(16))) uint8_t shared[];
  uint4* const wl = reinterpret_cast<uint4*>(shared);
  uint8_t* const ring = shared + NCH * blockDim.x * 16;
  const int team = __builtin_amdgcn_readfirstlane((int)threadIdx.y), teams = (int)blockDim.y;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.y * blockDim.x + threadIdx.x) / 64);
  const uint8_t* mine = ring + wave * (L * 1024) + (int)threadIdx.x % 64 * 16;
  const uint32_t mine0 = (uint32_t)(uintptr_t)(lds_u8_t*)ring + (uint32_t)(wave * (L * 1024));
  const int hs = a.hs;
  const uint32_t row = (uint32_t)hs * sizeof(S);
  uint4 xr[NCH], dr[NCH];
  if (team == 0) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) wl[j * blockDim.x + threadIdx.x] = Row<T, AL>(a.w, 0, 1, hs).get(j);
  }
  __syncthreads();
  float dw[NCH][V] = {}, db[NCH][V] = {};
  // Row m's pieces to LDS (AL) or registers; a row past the last reads as zero.
  auto fetch = [&](int64_t m) {
    const bool in = m < a.M;
    if constexpr (AL) {
      const i32x4_t rx = words_of<S>(in ? a.x : nullptr, m * a.ld_x, row), rd = words_of<S>(in ? a.dxn : nullptr, m * hs, row);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        load_lds(rx, piece_at(j, row), mine0 + (uint32_t)(2 * j * 1024));
        load_lds(rd, piece_at(j, row), mine0 + (uint32_t)((2 * j + 1) * 1024));
      }
    } else {
      const Row<T, AL> rx(in ? a.x : nullptr, m * a.ld_x, 1, hs), rd(in ? a.dxn : nullptr, m * hs, 1, hs);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        xr[j] = rx.get(j);
        dr[j] = rd.get(j);
      }
    }
  };
  const_f32_t* stats = (const_f32_t*)(uintptr_t)a.stats;
  const int64_t stride = (int64_t)gridDim.x * teams;
  int64_t m = (int64_t)blockIdx.x * teams + team;
  if constexpr (AL) fetch(m);
  // every team takes as many turns (they share barriers)
  const int64_t turns = (a.M - (int64_t)blockIdx.x * teams + stride - 1) / stride;
  for (int64_t t = 0; t < turns; ++t, m += stride) {
    const int64_t ms = m < a.M ? m : a.M - 1;
    const float mean = stats[2 * ms], r = stats[2 * ms + 1];
    if constexpr (AL) {
      // this row's loads are older than the NCH stores of the row before
      if (a.dx && t > 0) landed<NCH>();
      else landed<0>();
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        xr[j] = ld16(mine + 2 * j * 1024);
        dr[j] = ld16(mine + (2 * j + 1) * 1024);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's place is read
      fetch(m + stride);
    } else {
      fetch(m);
    }
    float sums[2] = {};
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float x[V], d[V], w[V];
      unpack<T>(xr[j], x);
      unpack<T>(dr[j], d);
      unpack<T>(wl[j * blockDim.x + threadIdx.x], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float h = (x[i] - mean) * r, e = a.w ? d[i] * w[i] : d[i];
        sums[0] += e;
        sums[1] += e * h;
        dw[j][i] += d[i] * h;
        db[j][i] += d[i];
      }
      __builtin_amdgcn_sched_barrier(0);  // (one piece's values at a time)
    }
    group_sum(sums, red[t & 1] + team * (int)(blockDim.x / 64) * 2);
    // (h and e are formed again from the pieces: kept, 40 of each spill)
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      hide(xr[j]);
      hide(dr[j]);
    }
    if (a.dx && m < a.M) {
      const float P = sums[0] / (float)hs, Q = sums[1] / (float)hs;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float x[V], d[V], w[V];
        unpack<T>(xr[j], x);
        unpack<T>(dr[j], d);
        unpack<T>(wl[j * blockDim.x + threadIdx.x], w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float h = (x[i] - mean) * r, e = a.w ? d[i] * w[i] : d[i];
          d[i] = r * (e - P - h * Q);
        }
        Row<T, AL>(a.dx, m * hs, 1, hs).put(j, 0, d, 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if constexpr (AL) landed<0>();  // no load into this workgroup's LDS outlives it
  if (!a.dw && !a.db) return;
  // The teams' sums meet in LDS: half of the teams that are left hand theirs over.
  const int tx = (int)threadIdx.x, nx = (int)blockDim.x;
  f32x4_t* place = reinterpret_cast<f32x4_t*>(ring);  // [teams/2][2][NCH*V/4][nx]
  auto four = [](float (&v)[NCH][V], int k) { return reinterpret_cast<f32x4_t*>(&v[0][0]) + k; };
  for (int left = teams; left > 1; left = (left + 1) / 2) {
    const int half = (left + 1) / 2;
    __syncthreads();
    if (team >= half && team < left) {
#pragma unroll
      for (int k = 0; k < NCH * V / 4; ++k) {
        place[(((team - half) * 2) * (NCH * V / 4) + k) * nx + tx] = *four(dw, k);
        place[(((team - half) * 2 + 1) * (NCH * V / 4) + k) * nx + tx] = *four(db, k);
      }
    }
    __syncthreads();
    if (team + half < left) {
#pragma unroll
      for (int k = 0; k < NCH * V / 4; ++k) {
        *four(dw, k) += place[((team * 2) * (NCH * V / 4) + k) * nx + tx];
        *four(db, k) += place[((team * 2 + 1) * (NCH * V / 4) + k) * nx + tx];
      }
    }
  }
  if (team > 0) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * hs;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c = (tx + j * nx) * V;
    if (c >= hs) continue;
    if constexpr (AL) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        *reinterpret_cast<f32x4_t*>(part + c + i) = *four(dw, (j * V + i) / 4);
        *reinterpret_cast<f32x4_t*>(part + hs + c + i) = *four(db, (j * V + i) / 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < hs) {
          part[c + i] = dw[j][i];
          part[hs + c + i] = db[j][i];
        }
    }
  }
}

// ---------------------------------------------------------------------------
// The backward pass for any width: layer_norm_bwd_rows forms P/HS and Q/HS of
// each row, layer_norm_bwd_cols needs nothing across the row: each thread
// keeps V columns and walks its group's rows.
// ---------------------------------------------------------------------------
template <typename T, bool AL>
__global__ __launch_bounds__(1024) void layer_norm_bwd_rows(LayerNormBwdArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  __shared__ float red[16 * 2];
  const S* w = reinterpret_cast<const S*>(a.w);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const S *x = reinterpret_cast<const S*>(a.x) + m * a.ld_x, *dxn = reinterpret_cast<const S*>(a.dxn) + m * a.hs;
    const float mean = a.stats[2 * m], r = a.stats[2 * m + 1];
    float sums[2] = {};
    for (int c = (int)threadIdx.x * V; c < a.hs; c += (int)blockDim.x * V) {
      float f[V], e[V], g[V];
      load<T, AL>(x + c, a.hs - c, f);
      load<T, AL>(dxn + c, a.hs - c, e);
      if (w) load<T, AL>(w + c, a.hs - c, g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (w) e[i] *= g[i];
        sums[0] += e[i];
        sums[1] += e[i] * ((f[i] - mean) * r);
      }
    }
    group_sum(sums, red);
    if (threadIdx.x == 0) {
      a.rows[2 * m] = sums[0] / (float)a.hs;
      a.rows[2 * m + 1] = sums[1] / (float)a.hs;
    }
    __syncthreads();  // the next row reuses red
  }
}

constexpr int kBwdColThreads = 256;
template <typename T, bool AL>
__global__ __launch_bounds__(kBwdColThreads) void layer_norm_bwd_cols(LayerNormBwdArgs a) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  const int c = ((int)blockIdx.x * kBwdColThreads + (int)threadIdx.x) * V;
  if (c >= a.hs) return;
  float w[V], dw[V] = {}, db[V] = {};
  if (a.w) load<T, AL>(reinterpret_cast<const S*>(a.w) + c, a.hs - c, w);
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    const float mean = a.stats[2 * m], r = a.stats[2 * m + 1], P = a.rows[2 * m], Q = a.rows[2 * m + 1];
    float x[V], d[V];
    load<T, AL>(reinterpret_cast<const S*>(a.x) + m * a.ld_x + c, a.hs - c, x);
    load<T, AL>(reinterpret_cast<const S*>(a.dxn) + m * a.hs + c, a.hs - c, d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float h = (x[i] - mean) * r;
      dw[i] += d[i] * h;
      db[i] += d[i];
      d[i] = r * ((a.w ? d[i] * w[i] : d[i]) - P - h * Q);
    }
    if (a.dx) store<T, AL>(reinterpret_cast<S*>(a.dx) + m * a.hs + c, a.hs - c, d);
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * a.hs;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i < a.hs) {
      part[c + i] = dw[i];
      part[a.hs + c + i] = db[i];
    }
}

// ---------------------------------------------------------------- launches --
bool aligned(const LayerNormArgs& a, int b) {
  return ld16_ok(a.hs, b) && al16(a.x) && ld16_ok(a.ld_x, b) && al16(a.w) && al16(a.b) && al16(a.xn);
}
bool aligned(const LayerNormBwdArgs& a, int b) {
  return ld16_ok(a.hs, b) && al16(a.x) && ld16_ok(a.ld_x, b) && al16(a.w) && al16(a.dxn) && al16(a.dx);
}

template <typename T, int NCH, bool AL>
int forward_row(LayerNormArgs a, hipStream_t st) {
  a.nt = streamed(a.M, a.hs, 1, sizeof(typename T::S));
  const int nw = (int)cdiv64(cdiv64(a.hs, vec<T>()), 64 * NCH);
  const dim3 blk((unsigned)nw * 64, nw == 1 ? 4 : 1);
  const int64_t rows = kMaxThreads / blk.x * blk.y;  // of a launch; longer calls take several
  for (; a.m_first < a.M; a.m_first += rows) {
    const dim3 grid((unsigned)cdiv64(std::min(rows, a.M - a.m_first), blk.y));
    hipLaunchKernelGGL((layer_norm_row<T, NCH, AL>), grid, blk, 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
  }
  return (int)hipSuccess;
}
template <typename T, bool AL>
int forward_loop(const LayerNormArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)std::min(a.M, kMaxGrid)), blk((unsigned)loop_threads(cdiv64(a.hs, vec<T>())));
  hipLaunchKernelGGL((layer_norm_loop<T, AL>), grid, blk, 0, st, a);
  return (int)hipGetLastError();
}
// A row by as few waves as its registers allow, so that the reductions and the
// statistics are not repeated wave by wave (16384 rows of 2560 bf16 channels by
// one wave 27 us, 6.2 TB/s, by five 43 us; 512 rows of 8192 channels by four
// 6.0 us, by eight 8.0). Few rows of 129 to 320 pieces leave CUs idle and go by
// one piece a thread, with the same bits (one row of 2560 channels 3.0 us, by one
// wave 3.4; 512 rows 3.9 and 4.0, 1024 rows 5.3 and 4.5; off 16 bytes one row of
// 2555 3.7 and 5.0, 1024 rows 5.8 and 6.2). Rows of 321 to 640 pieces go by two a
// thread, which serves few and many (4096 channels by one, two, four pieces: one
// row 3.1, 3.2, 3.6 us, 512 rows 4.5, 4.2, 4.8, 16384 rows 68, 50, 49; 5120 by five:
// one row 3.9 for 3.5, 16384 rows 62 for 67).
template <typename T, bool AL>
int forward_al(const LayerNormArgs& a, hipStream_t st) {
  const int64_t pieces = cdiv64(a.hs, vec<T>());
  if (pieces > 2048) return forward_loop<T, AL>(a, st);
  if (pieces <= 64 || (a.M < 640 && pieces > 128 && pieces <= 64 * kWholeWaves)) return forward_row<T, 1, AL>(a, st);
  if (pieces <= 128) return forward_row<T, 2, AL>(a, st);
  if (pieces <= 192) return forward_row<T, 3, AL>(a, st);
  if (pieces <= 256) return forward_row<T, 4, AL>(a, st);
  if (pieces <= 320) return forward_row<T, 5, AL>(a, st);
  if (pieces <= 640) return forward_row<T, 2, AL>(a, st);
  return forward_row<T, 4, AL>(a, st);
}
template <typename T>
int forward_of(const LayerNormArgs& a, hipStream_t st) {
  return aligned(a, (int)sizeof(typename T::S)) ? forward_al<T, true>(a, st) : forward_al<T, false>(a, st);
}

constexpr size_t kBwdLds = 152 * 1024;  // dynamic, of a workgroup's 160 KB
// Workspace: as of the other norms' backward passes (launch_weight_sums).
template <typename T, int NCH, bool AL>
int backward_row(LayerNormBwdArgs a, hipStream_t st) {
  const int nw = (int)cdiv64(cdiv64(a.hs, vec<T>()), 64 * NCH);
  // w, and each team's place for the next row, fit the LDS that raise_lds asks for
  const size_t w_lds = (size_t)NCH * nw * 1024, team_lds = 2 * w_lds;
  const int most = std::max(1, std::min(bwd_waves<T, NCH>() / nw, (int)((kBwdLds - w_lds) / team_lds)));
  // the rows go to all CUs first (one row, 2560 channels: 13.3 -> 7.3 us)
  const int teams = (int)cdiv64(a.M, 256 * cdiv64(a.M, 256 * most));
  const dim3 blk((unsigned)nw * 64, (unsigned)teams);
  const int64_t groups = std::min<int64_t>(cdiv64(a.M, teams), 256);
  const size_t ring = AL ? teams * team_lds : 0;
  const size_t sums = (size_t)(teams / 2) * 2 * NCH * vec<T>() * nw * 64 * 4;
  hipLaunchKernelGGL((layer_norm_bwd_row<T, NCH, AL>), dim3((unsigned)groups), blk,
                     w_lds + std::max(ring, sums), st, a);
  return launch_weight_sums(a.part, a.hs, groups, a.dw, a.db, st);
}
template <typename T, bool AL>
int backward_loop(const LayerNormBwdArgs& a, hipStream_t st) {
  const int64_t groups = norm_bwd_groups(a.M), pieces = cdiv64(a.hs, vec<T>());
  hipLaunchKernelGGL((layer_norm_bwd_rows<T, AL>), dim3((unsigned)std::min(a.M, kMaxGrid)),
                     dim3((unsigned)loop_threads(pieces)), 0, st, a);
  hipLaunchKernelGGL((layer_norm_bwd_cols<T, AL>), dim3((unsigned)cdiv64(pieces, kBwdColThreads), (unsigned)groups),
                     dim3(kBwdColThreads), 0, st, a);
  return launch_weight_sums(a.part, a.hs, groups, a.dw, a.db, st);
}
// Pieces a thread of layer_norm_bwd_row for a row of that many; 0: the kernels
// for any width.
int bwd_pieces(int64_t pieces) {
  if (pieces <= 64) return 1;
  if (pieces <= 128) return 2;
  // five where they leave fewer threads idle than four (2560 channels: 320 or
  // 640 pieces)
  if (pieces <= 2048) return cdiv64(pieces, 320) * 320 < cdiv64(pieces, 256) * 256 ? 5 : 4;
  return 0;
}
template <typename T, bool AL>
int backward_al(const LayerNormBwdArgs& a, hipStream_t st) {
  switch (bwd_pieces(cdiv64(a.hs, vec<T>()))) {
    case 1: return backward_row<T, 1, AL>(a, st);
    case 2: return backward_row<T, 2, AL>(a, st);
    case 4: return backward_row<T, 4, AL>(a, st);
    case 5: return backward_row<T, 5, AL>(a, st);
    default: return backward_loop<T, AL>(a, st);
  }
}
template <typename T>
int backward_of(const LayerNormBwdArgs& a, hipStream_t st) {
  return aligned(a, (int)sizeof(typename T::S)) ? backward_al<T, true>(a, st) : backward_al<T, false>(a, st);
}

template <typename T, int NCH>
int raise_lds() {
  for (const void* k : {(const void*)layer_norm_bwd_row<T, NCH, true>, (const void*)layer_norm_bwd_row<T, NCH, false>}) {
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kBwdLds);
    if (e != hipSuccess) return (int)e;
  }
  return (int)hipSuccess;
}
// (One piece a thread takes at most 33 KB.)
template <typename T>
int configure_of(int hs) {
  switch (bwd_pieces(cdiv64(hs, vec<T>()))) {
    case 2: return raise_lds<T, 2>();
    case 4: return raise_lds<T, 4>();
    case 5: return raise_lds<T, 5>();
    default: return (int)hipSuccess;
  }
}

}  // namespace

int launch_layer_norm(const LayerNormArgs& a, int dtype, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? forward_of<Bf16>(a, st) : dtype == 1 ? forward_of<Fp16>(a, st) : forward_of<Fp32>(a, st);
}
int launch_layer_norm_bwd(const LayerNormBwdArgs& a, int dtype, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? backward_of<Bf16>(a, st) : dtype == 1 ? backward_of<Fp16>(a, st) : backward_of<Fp32>(a, st);
}
int configure_layer_norm_kernels(int hs, int dtype) {
  return dtype == 0 ? configure_of<Bf16>(hs) : dtype == 1 ? configure_of<Fp16>(hs) : configure_of<Fp32>(hs);
}

}  // namespace hcgr
