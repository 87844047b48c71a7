// hcgr_linear.hip -- the 8-bit linear layer (hcgr_linear_forward):
//   out[m, n] = (sum_k q[m, k]*w[n, k]) * q_scale[m] * w_scale[n] + bias[n]
// on v_mfma_i32_16x16x64_i8 and v_mfma_i32_32x32x32_i8. Weight rows are the
// first (row) operand and tokens the second (column) operand, so a lane ends
// with four neighbouring output channels of one token. Sums are exact; one
// conversion to float, the product with w_scale and a fused multiply-add with
// q_scale and bias follow. (The scales' product, formed first, would leave the
// range of 32 bits where the result does not: below 2^-126 it loses bits, above
// 2^128 a zero sum gives NaN. A sum is 0 or at least 1, so its product with any
// normal w_scale below 2^97 stays inside.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "hcgr_block.h"
#include "hcgr_device.h"

namespace hcgr {
namespace {

__device__ __forceinline__ i32x4_t mfma_i8(uint4 a, uint4 b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0,
                                               0, 0);
}

// Keeps the first n of 16 bytes (n <= 0: none, n >= 16: all).
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n) {
  auto word = [&](uint32_t x, int k) { return k >= 4 ? x : k <= 0 ? 0u : x & ((1u << (8 * k)) - 1u); };
  return make_uint4(word(v.x, n), word(v.y, n - 4), word(v.z, n - 8), word(v.w, n - 12));
}

// An offset past every range (at most 256 rows of 2^22 bytes), also with a
// row's bytes added.
constexpr uint32_t kOut = 0x7ffffff0u;

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

// Four output channels n .. n+3 of token m from their sums. VEC: the row's
// pieces of four values are aligned and whole; otherwise those below `end`, at
// any alignment. NT: with the streaming policy, for outputs that outgrow the
// L2s: the workgroups of a round write them at the same time (8192x10240x2560:
// 245 -> 230 us).
template <int DT, bool VEC, bool NT = false>
__device__ __forceinline__ void store4(const LinearArgs& a, int64_t m, int n, float qs, const float (&ws)[4],
                                       const float (&bias)[4], const int (&acc)[4], int end) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fmaf((float)acc[i] * ws[i], qs, bias[i]);
  const int64_t at = m * a.ld_out + n;
  if (VEC || n + 4 <= end) {
    typedef uint32_t words_t __attribute__((ext_vector_type(DT == 2 ? 4 : 2)));
    words_t w;
    if constexpr (DT == 0) {
      w = words_t{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
    } else if constexpr (DT == 1) {
      typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
      w = __builtin_bit_cast(words_t, f16x4_t{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]});
    } else {
      w = __builtin_bit_cast(words_t, f32x4_t{v[0], v[1], v[2], v[3]});
    }
    uint8_t* to = reinterpret_cast<uint8_t*>(a.out) + at * (DT == 2 ? 4 : 2);
    if constexpr (!VEC) __builtin_memcpy(to, &w, sizeof w);  // gfx950 stores at any alignment
    else if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<words_t*>(to));
    else *reinterpret_cast<words_t*>(to) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < end) store1<DT>(a.out, at + i, v[i]);
  }
}
// Scales and bias of channels n .. n+3 (zero past N).
template <int DT>
__device__ __forceinline__ void channel4(const LinearArgs& a, int n, float (&ws)[4], float (&bias)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = n + i < a.n;
    ws[i] = in ? a.w_scale[n + i] : 0.0f;
    bias[i] = in && a.bias ? bias_at<DT>(a.bias, n + i) : 0.0f;
  }
}

template <int N>
using ic = std::integral_constant<int, N>;
// f(ic<0>), f(ic<1>), .. f(ic<N - 1>)
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) { (f(ic<I>{}), ...); }
template <int N, typename F>
__device__ __forceinline__ void each(F f) { each_of(f, std::make_integer_sequence<int, N>{}); }

// ---------------------------------------------------------------------------
// linear_split: 16*MT tokens and `rows` (up to 16*NT) output channels a
// workgroup, whose waves share K in units of 128 bytes. For few tokens the
// product streams the weights once and is bound by their bytes, and by the
// tokens, which every workgroup reads whole. Each wave runs a ring of D units
// of its own in LDS, without barriers, 1 KB a direct load, 8 rows of 8 pieces
// (a row's line by neighbouring lanes: fragments loaded straight into
// registers ask for 16 bytes of 16 lines at a time, which took the address
// units four times as long), place p of row r holding piece p ^ (r/2 % 8), so
// that 16 lanes reading one piece of 16 rows meet every bank once. The waves'
// sums meet in LDS.
// ---------------------------------------------------------------------------
template <int DT, int MT, int NT, int D>
__global__ __launch_bounds__(512) void linear_split(LinearArgs a, int rows, int tiles_m, int vec) {
  extern __shared__ uint8_t lds[];
  constexpr int L = 2 * (NT + MT), UB = L * 1024;  // a unit's loads and bytes
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
  const int nw = (int)blockDim.x / 64, r16 = lane % 16, kq = lane / 16;
  // Workgroups b, b + 8, b + 16, .. share an XCD: those of one XCD take the
  // tokens of the same channels one after the other, so that the weights come
  // from memory once.
  const int tiles = tiles_m * ((a.n + rows - 1) / rows), per = (tiles + 7) / 8;
  const int tile = (int)blockIdx.x % 8 * per + (int)blockIdx.x / 8;
  if ((int)blockIdx.x / 8 >= per || tile >= tiles) return;  // the whole workgroup
  const int n0 = tile / tiles_m * rows;
  const int64_t m0 = (int64_t)(tile % tiles_m) * (16 * MT);
  const int k16 = (a.k + 15) / 16 * 16, units = (a.k + 127) / 128;
  const int nr = min(rows, a.n - n0), mr = (int)min((int64_t)(16 * MT), a.M - m0);
  // rows past the last are past the range (a pitch is at least k16)
  const i32x4_t rw = range_words(a.w + (int64_t)n0 * a.ld_w, (uint32_t)((nr - 1) * a.ld_w + k16));
  const i32x4_t rq = range_words(a.q + m0 * a.ld_q, (uint32_t)((mr - 1) * a.ld_q + k16));
  uint8_t* ring = lds + wave * (D * UB);
  const uint32_t ring0 = (uint32_t)(uintptr_t)(lds_u8_t*)lds + (uint32_t)(wave * (D * UB));
  // load i of a matrix fills rows 8*i .. 8*i + 7; the piece's place depends on i's parity
  const int lr = lane / 8;
  const uint32_t piece[2] = {(uint32_t)((lane % 8) ^ (lr / 2)) * 16u, (uint32_t)((lane % 8) ^ (4 + lr / 2)) * 16u};
  uint32_t woff[2 * NT], qoff[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) woff[i] = (uint32_t)((8 * i + lr) * a.ld_w) + piece[i % 2];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) qoff[i] = (uint32_t)((8 * i + lr) * a.ld_q) + piece[i % 2];
  auto issue = [&](int u, int slot) {  // unit u of K; past the last, or past the row's last piece: zeros
    const uint32_t k = (uint32_t)u * 128u, buf = ring0 + (uint32_t)(slot * UB);
    const bool in[2] = {(int)(k + piece[0]) < k16, (int)(k + piece[1]) < k16};
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) load_lds(rw, in[i % 2] ? woff[i] + k : kOut, buf + i * 1024);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) load_lds(rq, in[i % 2] ? qoff[i] + k : kOut, buf + NT * 2048 + i * 1024);
  };
#pragma unroll
  for (int i = 0; i < D; ++i) issue(wave + i * nw, i);
  const uint32_t at = (uint32_t)(r16 * 128), key = (uint32_t)(r16 / 2 % 8);
  i32x4_t acc[NT][MT] = {};
  int slot = 0;
  for (int u = wave; u < units; u += nw) {
    landed<(D - 1) * L>();
    const uint8_t* buf = ring + slot * UB;
    uint4 w[NT][2], x[MT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t o = at + (((uint32_t)(h * 4 + kq) ^ key) * 16u);
#pragma unroll
      for (int t = 0; t < NT; ++t) w[t][h] = ld16(buf + t * 2048 + o);
#pragma unroll
      for (int t = 0; t < MT; ++t) x[t][h] = ld16(buf + (NT + t) * 2048 + o);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read
    issue(u + D * nw, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = u * 128 + h * 64 + kq * 16;
      if (a.k % 16 && k + 16 > a.k) {  // bytes past K count as zero
#pragma unroll
        for (int c = 0; c < NT; ++c) w[c][h] = keep_bytes(w[c][h], a.k - k);
      }
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[c][t] = mfma_i8(w[c][h], x[t][h], acc[c][t]);
    }
  }
  landed<0>();
  __syncthreads();  // the rings make room for the sums: [waves][MT][NT][64 lanes][4]
  int32_t* part = reinterpret_cast<int32_t*>(lds);
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int c = 0; c < NT; ++c)
      *reinterpret_cast<i32x4_t*>(part + (((wave * MT + t) * NT + c) * 64 + lane) * 4) = acc[c][t];
  __syncthreads();
  // thread -> four neighbouring channels of a token, in the products' layout
  for (int i = threadIdx.x; i < 64 * MT * NT; i += blockDim.x) {
    const int c = i / 64 % NT * 16 + i % 64 / 16 * 4, r = i / (64 * NT) * 16 + i % 16;
    if (c >= nr || r >= mr) continue;
    i32x4_t sum = *reinterpret_cast<const i32x4_t*>(part + i * 4);
    for (int v = 1; v < nw; ++v) sum += *reinterpret_cast<const i32x4_t*>(part + (v * MT * NT * 64 + i) * 4);
    const int four[4] = {sum[0], sum[1], sum[2], sum[3]};
    float ws[4], bias[4];
    channel4<DT>(a, n0 + c, ws, bias);
    if (vec) store4<DT, true>(a, m0 + r, n0 + c, a.q_scale[m0 + r], ws, bias, four, a.n);
    else store4<DT, false>(a, m0 + r, n0 + c, a.q_scale[m0 + r], ws, bias, four, n0 + nr);
  }
}

// ---------------------------------------------------------------------------
// linear_tile: TM tokens x TN channels a tile, 4 waves as 2 x 2, each
// (TM/2) x (TN/2) on v_mfma_i32_32x32x32_i8. K passes through a ring of NB
// LDS buffers in stages of 64 bytes a row, written by direct loads: 1 KB an
// instruction, 16 rows of 4 pieces, place p of row r holding the row's piece
// p ^ (r/4 % 4), so that 16 lanes reading one piece of 16 rows meet every bank
// once. A stage's fragments are read into registers while the products of the
// stage before run, so its buffer is free one stage later and NB - 1 stages
// of loads stay in flight. Workgroups are persistent: the loads run ahead
// into the next tile, so that its first stages arrive behind this one's
// epilogue. Past the last tile they are out of range and bring zeros. A tile's
// scales come the same way. The epilogue turns the sums around in the one free
// ring buffer, so that stores are whole 128-byte lines; without a bias nothing
// in it waits for memory. A bias is loaded there and waited for, with all that
// is in flight (8192x10240x2560: 216 us without, 218 with).
// ---------------------------------------------------------------------------
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));
template <int TM, int TN>
constexpr int stage_bytes() { return (TM + TN) * 64; }
constexpr int kTables = 4096;  // [tile parity][w_scale, q_scale][256 floats]
constexpr int kRing = 4;
template <int TM, int TN>
constexpr int tile_lds() { return kRing * stage_bytes<TM, TN>() + kTables; }

template <int DT, int TM, int TN, bool VEC, bool NT>
__global__ __launch_bounds__(256, TM * TN >= 256 * 256 ? 1 : 2) void linear_tile(LinearArgs a, int tiles_m, int tiles_n) {
  extern __shared__ uint8_t lds[];
  constexpr int FM = TM / 64, FN = TN / 64, SB = stage_bytes<TM, TN>(), NB = kRing;
  constexpr int LW = TN / 64, LQ = TM / 64, L = LW + LQ;  // a wave's loads a stage
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
  const int wm = wave % 2, wn = wave / 2;
  // Workgroups b, b + 8, b + 16, .. share an XCD and take neighbouring tiles,
  // eight rows of tiles at a time, so that they meet in that XCD's L2.
  const int tiles = tiles_m * tiles_n, per = (tiles + 7) / 8;
  const int first = (int)blockIdx.x / 8, stride = (int)gridDim.x / 8;
  auto place = [&](int j, int64_t& m0, int& n0) {  // the workgroup's tile j; false past the last
    const int local = first + j * stride, tile = (int)(blockIdx.x % 8) * per + local;
    if (local >= per || tile >= tiles) return false;
    const int band = tile / (8 * tiles_n), in = tile % (8 * tiles_n), high = min(8, tiles_m - band * 8);
    m0 = (int64_t)(band * 8 + in % high) * TM;
    n0 = in / high * TN;
    return true;
  };
  const int k16 = (a.k + 15) / 16 * 16, stages = max((a.k + 127) / 128 * 2, NB);
  // (an even count, the last may be empty; not below NB, so that the loads run
  // ahead by less than two tiles and two sets of scales suffice)
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8_t*)lds;

  // Loads: instruction i = wave + 4*j fills rows 16*i .. 16*i + 15. Rows past
  // the matrix are past the range (a pitch is at least k16).
  const int lrow = wave * 16 + lane / 4, lpiece = ((lane % 4) ^ (lane / 16)) * 16;
  uint32_t woff[LW], qoff[LQ];
#pragma unroll
  for (int j = 0; j < LW; ++j) woff[j] = (uint32_t)((lrow + 64 * j) * a.ld_w) + (uint32_t)lpiece;
#pragma unroll
  for (int j = 0; j < LQ; ++j) qoff[j] = (uint32_t)((lrow + 64 * j) * a.ld_q) + (uint32_t)lpiece;
  const int8_t *wbase = a.w, *qbase = a.q;
  uint32_t wbytes = 0, qbytes = 0;
  int lt = 0, ls = 0;  // the next stage to load: of the workgroup's tile lt, stage ls
  auto aim = [&]() {
    int64_t m0 = 0;
    int n0 = 0;
    const bool in = place(lt, m0, n0);
    const int nr = min(TN, a.n - n0), mr = (int)min((int64_t)TM, a.M - m0);
    wbase = a.w + (int64_t)n0 * a.ld_w;
    qbase = a.q + m0 * a.ld_q;
    wbytes = in ? (uint32_t)((nr - 1) * a.ld_w + k16) : 0u;
    qbytes = in ? (uint32_t)((mr - 1) * a.ld_q + k16) : 0u;
  };
  struct Loads {  // one stage's loads
    i32x4_t rw, rq;
    uint32_t buf, k;
    bool in_row;
  };
  auto loads_into = [&](int slot) {
    Loads z;
    z.rw = range_words(wbase, wbytes);
    z.rq = range_words(qbase, qbytes);
    z.buf = lds0 + (uint32_t)(slot * SB + wave * 1024);
    z.k = (uint32_t)ls * 64u;
    z.in_row = (int)z.k + lpiece < k16;  // bytes past the row's last piece read as zero
    return z;
  };
  auto load_one = [&](const Loads& z, auto I) {  // the i-th of a stage's L loads
    constexpr int i = decltype(I)::value;
    if constexpr (i < LW) load_lds(z.rw, z.in_row ? woff[i] + z.k : kOut, z.buf + i * 4096);
    else load_lds(z.rq, z.in_row ? qoff[i - LW] + z.k : kOut, z.buf + TN * 64 + (i - LW) * 4096);
  };
  auto loaded = [&]() {  // on to the next stage; after a tile's first stage, its scales
    if (ls == 0) {
      int64_t m0 = 0;
      int n0 = 0;
      const bool in = place(lt, m0, n0);
      const uint32_t at = (uint32_t)(wave * 64 + lane) * 4u, to = lds0 + NB * SB + (lt & 1) * 2048 + wave * 256;
      load_lds4(range_words(a.w_scale + n0, in ? (uint32_t)min(TN, a.n - n0) * 4u : 0u), at, to);
      load_lds4(range_words(a.q_scale + m0, in ? (uint32_t)min((int64_t)TM, a.M - m0) * 4u : 0u), at, to + 1024);
    }
    if (++ls == stages) {
      ls = 0;
      ++lt;
      aim();
    }
  };
  auto issue = [&](int slot) {
    const Loads z = loads_into(slot);
    each<L>([&](auto I) { load_one(z, I); });
    loaded();
  };

  // fragments: lane -> row lane % 32, 16 bytes at 32*step + 16*(lane/32)
  uint4 fa[2][2][FN], fb[2][2][FM];  // [stage parity][step][fragment]
  const uint32_t frow = (uint32_t)(lane % 32) * 64u;
  constexpr int R = 2 * (FN + FM);  // a wave's reads a stage
  uint32_t fat[2];
#pragma unroll
  for (int st = 0; st < 2; ++st) fat[st] = frow + (uint32_t)(((st * 2 + lane / 32) ^ (lane / 4 % 4)) * 16);
  auto read_one = [&](int slot, auto P, auto I) {  // the i-th of them
    constexpr int p = decltype(P)::value, st = decltype(I)::value / (FN + FM), f = decltype(I)::value % (FN + FM);
    const uint8_t* buf = lds + slot * SB + fat[st];
    if constexpr (f < FN) fa[p][st][f] = ld16(buf + (wn * FN + f) * 2048);
    else fb[p][st][f - FN] = ld16(buf + TN * 64 + (wm * FM + f - FN) * 2048);
  };
  i32x16_t acc[FN][FM];
  const int tail = a.k % 16 ? a.k / 64 : -1;  // the stage whose last piece holds bytes past K
  int cur = 0;  // slot of the stage whose products come next
  auto step = [&](int s, auto P, auto ZERO, auto LAST) {
    constexpr int p = decltype(P)::value;
    // Every wave has read stage s (into registers), and stage s + 1 has
    // landed: NB - 2 younger stages may be in flight (a store of an epilogue
    // among them only lengthens the wait).
    landed<(NB - 2) * L>();
    lds_sync();
    if (s == tail) {  // bytes past K count as zero
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int f = 0; f < FN; ++f) fa[p][st][f] = keep_bytes(fa[p][st][f], a.k - s * 64 - st * 32 - lane / 32 * 16);
    }
    // Stage s's slot takes the stage NB further on, and the next stage's
    // fragments come in: these reads and loads are spread over the products,
    // which would otherwise wait while a wave issues them.
    const Loads z = loads_into(cur);
    const int next = cur + 1 == NB ? 0 : cur + 1;
    constexpr int NM = 2 * FN * FM, NO = decltype(LAST)::value ? 0 : R + L;
    __builtin_amdgcn_sched_barrier(0);
    each<NM>([&](auto T) {
      constexpr int t = decltype(T)::value, st = t / (FN * FM), f = t / FM % FN, g = t % FM;
      acc[f][g] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
          __builtin_bit_cast(i32x4_t, fa[p][st][f]), __builtin_bit_cast(i32x4_t, fb[p][st][g]),
          decltype(ZERO)::value && st == 0 ? i32x16_t{} : acc[f][g], 0, 0, 0);
      constexpr int o0 = t * NO / NM, o1 = (t + 1) * NO / NM;
      each<o1 - o0>([&](auto O) {
        constexpr int o = o0 + decltype(O)::value;
        if constexpr (o < R) read_one(next, ic<1 - p>{}, ic<o>{});
        else load_one(z, ic<o - R>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (!decltype(LAST)::value) {
      cur = next;
      loaded();
    }
  };

  aim();
  for (int i = 0; i < NB; ++i) issue(i);
  landed<(NB - 1) * L>();
  lds_sync();
  each<R>([&](auto I) { read_one(0, ic<0>{}, I); });
  int64_t m0 = 0;
  int n0 = 0;
  for (int j = 0; place(j, m0, n0); ++j) {
    step(0, ic<0>{}, ic<1>{}, ic<0>{});
    for (int s = 1; s + 1 < stages; s += 2) {
      step(s, ic<1>{}, ic<0>{}, ic<0>{});
      step(s + 1, ic<0>{}, ic<0>{}, ic<0>{});
    }
    step(stages - 1, ic<1>{}, ic<0>{}, ic<1>{});
    // Sums: lane -> token lane % 32, channels 8*(i/4) + 4*(lane/32) + i % 4.
    // Through the wave's quarter of slot `cur`, which every wave has read:
    // ROWS tokens x COLS channels a pass, a row's 16-byte places xored with
    // the row.
    constexpr int COLS = TN / 2 < 64 ? TN / 2 : 64, ROWS = SB / 4 / (COLS * 4), P = COLS / 4;
    uint8_t* turn = lds + cur * SB + wave * (SB / 4);
    const float* table = reinterpret_cast<const float*>(lds + NB * SB + (j & 1) * 2048);
#pragma unroll
    for (int h = 0; h < TN / 2 / COLS; ++h) {
      const int nl = wn * (TN / 2) + h * COLS + lane % P * 4, n = n0 + nl;
      float ws[4], bias[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ws[i] = table[nl + i];
        bias[i] = a.bias && n + i < a.n ? bias_at<DT>(a.bias, n + i) : 0.0f;
      }
#pragma unroll
      for (int g = 0; g < FM; ++g)
#pragma unroll
        for (int part = 0; part < 32 / ROWS; ++part) {
          if (lane % 32 / ROWS == part) {
#pragma unroll
            for (int f = 0; f < COLS / 32; ++f)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const i32x16_t& c = acc[h * (COLS / 32) + f][g];
                const int place16 = (f * 8 + q * 2 + lane / 32) ^ (lane % P);
                *reinterpret_cast<i32x4_t*>(turn + (lane % ROWS) * (COLS * 4) + place16 * 16) =
                    i32x4_t{c[q * 4], c[q * 4 + 1], c[q * 4 + 2], c[q * 4 + 3]};
              }
          }
          wave_sync();  // lanes read what others wrote
#pragma unroll
          for (int k = 0; k < ROWS * P / 64; ++k) {
            const int row = k * (64 / P) + lane / P;
            const i32x4_t c = *reinterpret_cast<const i32x4_t*>(turn + row * (COLS * 4) + ((lane % P) ^ (row % P)) * 16);
            const int ml = wm * (TM / 2) + g * 32 + part * ROWS + row;
            const int v[4] = {c[0], c[1], c[2], c[3]};
            if (m0 + ml < a.M && n < a.n) store4<DT, VEC, NT>(a, m0 + ml, n, table[256 + ml], ws, bias, v, a.n);
          }
          wave_sync();  // and the next part writes where they read
        }
    }
    lds_sync();  // every wave is done with the slot
    issue(cur);
    cur = cur + 1 == NB ? 0 : cur + 1;
    each<R>([&](auto I) { read_one(cur, ic<0>{}, I); });
  }
  landed<0>();  // no load into this workgroup's LDS outlives it
}

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether a row of out is whole, aligned pieces of four values.
template <int DT>
bool pieces_of_four(const LinearArgs& a) {
  return a.n % 4 == 0 && a.ld_out % 4 == 0 && (uintptr_t)a.out % (DT == 2 ? 16 : 8) == 0;
}

template <int DT, int MT, int NT, int D>
int launch_split(const LinearArgs& a, int rows, int nw, hipStream_t st) {
  const int tm = (int)cdiv64(a.M, 16 * MT);
  const dim3 g((unsigned)(cdiv64(cdiv64(a.n, rows) * tm, 8) * 8)), blk((unsigned)nw * 64);
  hipLaunchKernelGGL((linear_split<DT, MT, NT, D>), g, blk, (size_t)nw * D * (MT + NT) * 2048, st, a, rows, tm,
                     rows % 4 == 0 && pieces_of_four<DT>(a));
  return (int)hipGetLastError();
}

// Up to 16*MT tokens: as many channels a workgroup (at most 16) as fill the
// 256 CUs in whole rounds; the rings of the workgroups that share a CU fill
// its LDS: one of eight waves, or two or three of four.
template <int DT, int MT>
int run_skinny(const LinearArgs& a, hipStream_t st) {
  const int rounds = (int)cdiv64(a.n, 256 * 16), rows = (int)cdiv64(a.n, 256 * rounds);
  constexpr int kFew = MT == 1 ? 5 : 3, kMany = MT == 1 ? 3 : 2;
  if (rounds == 1) return launch_split<DT, MT, 1, kFew>(a, rows, 8, st);
  if (rounds == 2) return launch_split<DT, MT, 1, kFew>(a, rows, 4, st);
  return launch_split<DT, MT, 1, kMany>(a, rows, 4, st);
}

template <int DT, int TM, int TN, bool VEC, bool NT>
int launch_tile(const LinearArgs& a, hipStream_t st) {
  const int tm = (int)cdiv64(a.M, TM), tn = (int)cdiv64(a.n, TN);
  // persistent workgroups: as many as the 256 CUs hold at once
  constexpr int kHeld = TM * TN >= 256 * 256 ? 256 : 512;
  const int64_t tiles = cdiv64((int64_t)tm * tn, 8) * 8;
  hipLaunchKernelGGL((linear_tile<DT, TM, TN, VEC, NT>), dim3((unsigned)std::min<int64_t>(tiles, kHeld)), dim3(256),
                     (tile_lds<TM, TN>()), st, a, tm, tn);
  return (int)hipGetLastError();
}
template <int DT, int TM, int TN>
int run_tile(const LinearArgs& a, hipStream_t st) {
  if (!pieces_of_four<DT>(a)) return launch_tile<DT, TM, TN, false, false>(a, st);
  const bool nt = (double)a.M * a.n * (DT == 2 ? 4 : 2) > 32.0 * 1024 * 1024;  // more than the L2s hold
  return nt ? launch_tile<DT, TM, TN, true, true>(a, st) : launch_tile<DT, TM, TN, true, false>(a, st);
}

// The kernel is the one that a model of its time, in microseconds, puts first:
// a start, then rounds of workgroups over the 256 CUs, each with a part of its
// own and one for each unit of 128 bytes of K; the kernels for few tokens are
// also bound by the weights' bytes at 5.2 TB/s. The constants are fitted on
// one MI355X to N x K = 1024 x 1024 .. 10240 x 2560 and 2560 x 10240, M = 1 ..
// 2048 (mostly within a quarter of the measured times). Measured, split 32x32 /
// split 64x64 / tile 128 / tile 256: 2560x10240 at M = 64: 10.9 / 20 / 47 /
// 101 us, M = 384: 33 / 21 / 51 / 107, M = 1024: - / 74 / 51 / 113; 10240x2560
// at M = 384: 37 / 33 / 21 / 39, M = 3000: - / 179 / 116 / 92.
template <int DT>
int run(const LinearArgs& a, hipStream_t st) {
  const double u = (double)cdiv64(a.k, 128);
  auto rounds = [&](int tm, int tn) { return (double)cdiv64(cdiv64(a.M, tm) * cdiv64(a.n, tn), 256); };
  const double stream = 3.0 + (double)a.n * a.k / 5.2e6;
  // (more than one tile of tokens: part of the weights comes from memory again)
  const double t32 = std::max(1.8 + rounds(32, 32) * (1.2 + 0.08 * u), a.M <= 32 ? stream : 1.5 * stream);
  if (a.M <= 32 && std::max(3.8, stream - 0.1) <= t32) return a.M <= 16 ? run_skinny<DT, 1>(a, st) : run_skinny<DT, 2>(a, st);
  const double t64 = rounds(64, 64) * (4.6 + 0.19 * u), t128 = 1.0 + rounds(128, 128) * (4.4 + 0.55 * u);
  const double t256 = rounds(256, 256) * (14.0 + 1.25 * u), best = std::min({t32, t64, t128, t256});
  if (best == t32) return launch_split<DT, 2, 2, 2>(a, 32, 4, st);
  if (best == t64) return launch_split<DT, 4, 4, 2>(a, 64, 4, st);
  return best == t128 ? run_tile<DT, 128, 128>(a, st) : run_tile<DT, 256, 256>(a, st);
}

template <int DT>
int raise_lds() {
  const void* f[] = {
      (const void*)linear_tile<DT, 256, 256, true, true>,  (const void*)linear_tile<DT, 256, 256, true, false>,
      (const void*)linear_tile<DT, 256, 256, false, false>, (const void*)linear_tile<DT, 128, 128, true, true>,
      (const void*)linear_tile<DT, 128, 128, true, false>, (const void*)linear_tile<DT, 128, 128, false, false>,
      (const void*)linear_split<DT, 1, 1, 5>,              (const void*)linear_split<DT, 1, 1, 3>,
      (const void*)linear_split<DT, 2, 1, 3>,              (const void*)linear_split<DT, 2, 1, 2>,
      (const void*)linear_split<DT, 2, 2, 2>,              (const void*)linear_split<DT, 4, 4, 2>};
  for (const void* k : f) {
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != hipSuccess) return (int)e;
  }
  return (int)hipSuccess;
}

}  // namespace

// Raises the dynamic-LDS limit of the kernels on the current device.
int configure_linear_kernels() {
  for (int e : {raise_lds<0>(), raise_lds<1>(), raise_lds<2>()})
    if (e != (int)hipSuccess) return e;
  return (int)hipSuccess;
}

int launch_linear(const LinearArgs& args, int dtype, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  // tile counts stay in 32 bits: larger M in several launches
  constexpr int64_t kRows = (int64_t)1 << 20;
  const size_t b = dtype == 2 ? 4 : 2;
  for (int64_t m0 = 0; m0 < args.M; m0 += kRows) {
    LinearArgs a = args;
    a.M = args.M - m0 < kRows ? args.M - m0 : kRows;
    a.q += m0 * a.ld_q;
    a.q_scale += m0;
    a.out = reinterpret_cast<uint8_t*>(a.out) + (size_t)(m0 * a.ld_out) * b;
    const int e = dtype == 0 ? run<0>(a, st) : dtype == 1 ? run<1>(a, st) : run<2>(a, st);
    if (e != (int)hipSuccess) return e;
  }
  return (int)hipSuccess;
}

}  // namespace hcgr
