// hcgr_mx.hip -- the linear layer in microscaled 4-bit floating point: its
// quantizer and the way back (hcgr_linear_quantize_mx,
// hcgr_linear_dequantize_mx) and its product (hcgr_linear_forward_mx):
//   out[m, n] = sum_k q[m, k] s[m, k/32] w[n, k] t[n, k/32] + bias[n]
// on v_mfma_scale_f32_16x16x128_f8f6f4 and _32x32x64_, which take 32 E2M1
// values and one E8M0 scale a lane and operand. Weight rows are the first (row)
// operand and tokens the second (column) operand, so a lane ends with four
// neighbouring output channels of one token. Products and scales are exact;
// sums are held in 32 bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "hcgr_block.h"
#include "hcgr_device.h"
#include "hcgr_mx.h"
#include "hcgr_products.h"
#include "hcgr_rows.h"

namespace hcgr {
namespace {

// ------------------------------------------------------------- quantizer --
// n / d for n < 2^31, as (n * mul) >> shift: mul = ceil(2^shift / d) < 2^32
// with shift = 31 + ceil(log2 d) is off by less than 2^-31 of a d-th.
struct Divide {
  uint32_t mul;
  int shift;
};
Divide divide_by(uint32_t d) {
  int up = 0;
  while (((uint32_t)1 << up) < d) ++up;
  return {(uint32_t)((((uint64_t)1 << (31 + up)) + d - 1) / d), 31 + up};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, Divide d) { return (uint32_t)((uint64_t)n * d.mul >> d.shift); }

// mx_quantize, mx_dequantize: the rows' 16-byte pieces of float values (V of
// them: half a dword of codes to a dword) one after the other, kPieces a
// thread, all of them asked for before the first is used. A block's 32/V lanes
// are neighbours; a row's pieces are whole blocks, so they stay together. Bound by
// memory, or by the launch: 10240 x 2560 in bf16 11.8 us and back 11.5, 32 x 10240
// 2.5 us, each kernel again and again over three sets of rows (157 MB, which the
// Infinity Cache holds). Four pieces a thread 12.5, 11.5 and 2.95 us, one 12.2, 11.9
// and 2.4. In turn, over 354 MB and behind the 52 MB that the way back has just
// written, the quantizer takes 15.4 us (4.3 TB/s) and the way back 11.3.
constexpr int kPieces = 2;
template <typename T, bool AL>
__global__ __launch_bounds__(256) void mx_quantize(MxRowsToArgs a, int blocks, Divide per_row, uint32_t pieces) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  const uint32_t i0 = (uint32_t)blockIdx.x * (256 * kPieces) + threadIdx.x;
  uint4 x[kPieces];
  uint32_t row[kPieces];
  int c[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const uint32_t i = i0 + u * 256;
    row[u] = quotient(i, per_row);
    c[u] = (int)(i - row[u] * (uint32_t)(blocks * (32 / V))) * V;
    x[u] = make_uint4(0, 0, 0, 0);
    if (i < pieces) x[u] = load_raw<T, AL>(reinterpret_cast<const S*>(a.x) + (int64_t)row[u] * a.ld_x + c[u], a.k - c[u]);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    if (i0 + u * 256 >= pieces) return;
    float f[V];
    unpack<T>(x[u], f);
    mx_store<V>(a.q + (int64_t)row[u] * a.ld_q, a.q_scale + (int64_t)row[u] * a.ld_qs, c[u], blocks, f);
  }
}

// V values of a block from their codes.
template <int V>
__device__ __forceinline__ void mx_values(uint32_t w, uint32_t byte, float (&v)[V]) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const float s = byte == 255u ? __uint_as_float(0x7fc00000u) : mx_scale(byte);
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  if constexpr (V == 8) {
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    v[4] = c[0] * s; v[5] = c[1] * s; v[6] = d[0] * s; v[7] = d[1] * s;
  }
}
template <typename T, bool AL>
__global__ __launch_bounds__(256) void mx_dequantize(MxRowsFromArgs a, int blocks, Divide per_row, uint32_t pieces) {
  using S = typename T::S;
  constexpr int V = vec<T>();
  const uint32_t i0 = (uint32_t)blockIdx.x * (256 * kPieces) + threadIdx.x;
  uint32_t w[kPieces], byte[kPieces], row[kPieces];
  int c[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const uint32_t i = i0 + u * 256;
    row[u] = quotient(i, per_row);
    c[u] = (int)(i - row[u] * (uint32_t)(blocks * (32 / V))) * V;
    w[u] = byte[u] = 0;
    if (i < pieces) {
      const uint8_t* q = a.q + (int64_t)row[u] * a.ld_q + c[u] / 2;
      w[u] = V == 8 ? *reinterpret_cast<const uint32_t*>(q) : *reinterpret_cast<const uint16_t*>(q);
      byte[u] = a.q_scale[(int64_t)row[u] * a.ld_qs + c[u] / 32];
    }
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    if (i0 + u * 256 >= pieces) return;
    float f[V];
    mx_values<V>(w[u], byte[u], f);
    store<T, AL>(reinterpret_cast<S*>(a.x) + (int64_t)row[u] * a.ld_x + c[u], a.k - c[u], f);
  }
}

// --------------------------------------------------------------- products --
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
// 4-bit operands use the first four of eight registers; the format code is 4.
// SA, SB: the byte of the scale registers that a lane's block takes.
__device__ __forceinline__ i32x8_t codes_of(uint4 v) {
  return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}
template <int SA, int SB>
__device__ __forceinline__ f32x4_t mfma_mx16(uint4 a, uint4 b, f32x4_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes_of(a), codes_of(b), c, 4, 4, SA, (int)sa, SB, (int)sb);
}
template <int SA, int SB>
__device__ __forceinline__ f32x16_t mfma_mx32(uint4 a, uint4 b, f32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(codes_of(a), codes_of(b), c, 4, 4, SA, (int)sa, SB, (int)sb);
}

// The same number, hidden from the compiler, which would form what depends on
// it ahead of the loop and keep it in registers that the products need (117 of
// them spilled, with reloads between the products that wait for the loads).
__device__ __forceinline__ int hidden(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Two values in 16 bits.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  if constexpr (DT == 0) return pack_bf2(lo, hi);
  else return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)lo, (_Float16)hi});
}
// 64 channels' bias to LDS, a value in each 32-bit word (zero past `bytes`): asked
// for ahead of the products, as its latency would stand behind them (1024 x 10240 x
// 2560: 2.4 us; by way of LDS 0.6).
template <int DT>
__device__ __forceinline__ void load_bias(const void* bias, int n0, int channels, int lane, uint32_t lds) {
  constexpr int B = DT == 2 ? 4 : 2;
  const i32x4_t r = range_words(reinterpret_cast<const uint8_t*>(bias) + (int64_t)n0 * B, (uint32_t)(max(channels, 0) * B));
  if constexpr (DT == 2) load_lds4(r, (uint32_t)(lane * B), lds);
  else load_lds2(r, (uint32_t)(lane * B), lds);
}
// Four of them.
template <int DT>
__device__ __forceinline__ void bias4(const uint8_t* at, float (&bias)[4]) {
  const uint4 u = ld16(at);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == 0) bias[i] = bf1((uint16_t)w[i]);
    else if constexpr (DT == 1) bias[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w[i]);
    else bias[i] = __uint_as_float(w[i]);
  }
}

// ---------------------------------------------------------------------------
// mx_split: 16*MT tokens and 16*NT output channels a workgroup, whose waves share
// K in units of 128 bytes a row (256 values). For few tokens the product
// streams the weights once and is bound by their bytes, and by the tokens, which
// every workgroup reads whole: a start of 3.3 us, then 5 to 7 TB/s (one token: 10240
// x 2560 5.7 us, 8192 x 8192 9.0). Each wave runs a ring of D units of its own in
// LDS, without barriers, 1 KB a direct load (rings of three, four and six units are
// no faster than two: 6.1, 6.3 and 6.5 us for 5.7; 64 x 64 tiles have room for one,
// 2560 x 10240 at M = 512 26 us, 28 with two units of 64 bytes a row); place p of row r holds the
// row's piece p ^ key(r), so that 16 lanes reading one piece of 16 rows meet every
// bank once. The scales come first, kSplitScales 16-byte pieces
// a row (K = 16384; longer rows take several turns), each row's pieces by
// neighbouring lanes: asked for unit by unit they would be 8 bytes of 16 lines
// at a time. The waves' sums meet in LDS.
// ---------------------------------------------------------------------------
constexpr int kSplitScales = 32;
__host__ __device__ inline int split_pitch(int blocks) {  // an odd number of pieces: rows spread over the banks
  const int p = (blocks + 15) / 16;
  return ((p < kSplitScales ? p : kSplitScales) | 1) * 16;
}
// LDS of one matrix's scales: whole loads of 1 KB.
__host__ __device__ inline int split_table(int rows, int pitch) { return (rows * pitch + 1023) / 1024 * 1024; }

template <int DT, int MT, int NT, int D>
__global__ __launch_bounds__(512) void mx_split(MxLinearArgs a, int tiles_m, int vec) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int rows = 16 * NT;
  constexpr int H = 2;                            // steps of 128 values a unit
  constexpr int RL = 8;                           // rows a load fills, of 8 pieces
  constexpr int FL = 16 / RL;                     // loads a fragment of 16 rows
  constexpr int L = FL * (NT + MT), UB = L * 1024;  // a unit's loads and bytes
  static_assert(D * UB >= MT * NT * 1024 && rows <= 64, "the rings make room for the sums; a load of bias");
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
  const int blocks = (a.k + 31) / 32, bytes = blocks * 16, units = (blocks + 4 * H - 1) / (4 * H);
  const int pieces = (blocks + 15) / 16;  // of a row's scales
  const int nr = min(rows, a.n - n0), mr = (int)min((int64_t)(16 * MT), a.M - m0);
  // rows past the last are past the range (a pitch is at least `bytes`)
  const i32x4_t rw = range_words(a.w + (int64_t)n0 * a.ld_w, (uint32_t)((nr - 1) * a.ld_w + bytes));
  const i32x4_t rq = range_words(a.q + m0 * a.ld_q, (uint32_t)((mr - 1) * a.ld_q + bytes));
  const i32x4_t rws = range_words(a.w_scale + (int64_t)n0 * a.ld_ws, (uint32_t)((nr - 1) * a.ld_ws + pieces * 16));
  const i32x4_t rqs = range_words(a.q_scale + m0 * a.ld_qs, (uint32_t)((mr - 1) * a.ld_qs + pieces * 16));
  const int pitch = split_pitch(blocks), wtable = split_table(16 * NT, pitch), table = wtable + split_table(16 * MT, pitch);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8_t*)lds;
  uint8_t* ring = lds + table + wave * (D * UB);
  const uint32_t ring0 = lds0 + (uint32_t)(table + wave * (D * UB));
  const int bias_at = table + nw * (D * UB);
  if (a.bias && wave == 0) load_bias<DT>(a.bias, n0, nr, lane, lds0 + (uint32_t)bias_at);
  // load i of a fragment fills its rows RL*i .. RL*i + RL - 1
  const int lr = lane / 8, lp = lane % 8;
  auto key = [](int r) { return r / 2 % 8; };
  uint32_t piece[FL], woff[FL * NT], qoff[FL * MT];
#pragma unroll
  for (int i = 0; i < FL; ++i) piece[i] = (uint32_t)(lp ^ key(RL * i + lr)) * 16u;
#pragma unroll
  for (int i = 0; i < FL * NT; ++i) woff[i] = (uint32_t)((RL * i + lr) * a.ld_w) + piece[i % FL];
#pragma unroll
  for (int i = 0; i < FL * MT; ++i) qoff[i] = (uint32_t)((RL * i + lr) * a.ld_q) + piece[i % FL];
  auto issue = [&](int u, int slot) {  // unit u of K; past the last, or past the row's last block: zeros
    const uint32_t k = (uint32_t)u * (64 * H), buf = ring0 + (uint32_t)(slot * UB);
    bool in[FL];
#pragma unroll
    for (int i = 0; i < FL; ++i) in[i] = (int)(k + piece[i]) < bytes;
#pragma unroll
    for (int i = 0; i < FL * NT; ++i) load_lds(rw, in[i % FL] ? woff[i] + k : kOut, buf + i * 1024);
#pragma unroll
    for (int i = 0; i < FL * MT; ++i) load_lds(rq, in[i % FL] ? qoff[i] + k : kOut, buf + (FL * NT + i) * 1024);
  };
  const uint32_t at = (uint32_t)(r16 * (64 * H));
  f32x4_t acc[NT][MT] = {};
  constexpr int kPass = kSplitScales * 16 / (4 * H);  // units that a turn's scales serve
  for (int u0 = 0; u0 < units; u0 += kPass) {
    const int u1 = min(u0 + kPass, units);
    if (u0) __syncthreads();  // the table and the rings are read
    const int ppr = pitch / 16, first = u0 / kPass * kSplitScales;
    auto scales = [&](i32x4_t r, int nrows, int64_t ld, uint32_t to) {
      for (int i = wave; i * 64 < nrows * ppr; i += nw) {
        const int row = (i * 64 + lane) / ppr, p = (i * 64 + lane) % ppr;
        const bool in = row < nrows && p < kSplitScales && first + p < pieces;
        load_lds(r, in ? (uint32_t)(row * ld + (first + p) * 16) : kOut, to + (uint32_t)(i * 1024));
      }
    };
    scales(rws, 16 * NT, a.ld_ws, lds0);
    scales(rqs, 16 * MT, a.ld_qs, lds0 + (uint32_t)wtable);
#pragma unroll
    for (int i = 0; i < D; ++i) issue(u0 + wave + i * nw < u1 ? u0 + wave + i * nw : units, i);
    landed<D * L>();
    lds_sync();
    int slot = 0;
    for (int u = u0 + wave; u < u1; u += nw) {
      landed<(D - 1) * L>();
      const uint8_t* buf = ring + slot * UB;
      uint4 w[NT][H], x[MT][H];
      uint32_t ws[NT][H], xs[MT][H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint32_t o = at + (uint32_t)(((h * 4 + kq) ^ key(r16)) * 16);
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t][h] = ld16(buf + t * (FL * 1024) + o);
#pragma unroll
        for (int t = 0; t < MT; ++t) x[t][h] = ld16(buf + (NT + t) * (FL * 1024) + o);
        const uint8_t* sc = lds + r16 * pitch + (u - u0) * (4 * H) + h * 4;
        const uint8_t* xc = sc + wtable;
#pragma unroll
        for (int t = 0; t < NT; ++t) ws[t][h] = *reinterpret_cast<const uint32_t*>(sc + t * 16 * pitch);
#pragma unroll
        for (int t = 0; t < MT; ++t) xs[t][h] = *reinterpret_cast<const uint32_t*>(xc + t * 16 * pitch);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read
      const int next = u + D * nw;
      issue(next < u1 ? next : units, slot);
      slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int block = u * (4 * H) + h * 4 + kq;
#pragma unroll
        for (int t = 0; t < NT; ++t) ws[t][h] >>= 8 * kq;
#pragma unroll
        for (int t = 0; t < MT; ++t) xs[t][h] >>= 8 * kq;
        if (u + 1 == units) {  // scale bytes past the last block do not count
#pragma unroll
          for (int t = 0; t < NT; ++t) ws[t][h] = block < blocks ? ws[t][h] : 0u;
#pragma unroll
          for (int t = 0; t < MT; ++t) xs[t][h] = block < blocks ? xs[t][h] : 0u;
        }
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[c][t] = mfma_mx16<0, 0>(w[c][h], x[t][h], acc[c][t], ws[c][h], xs[t][h]);
      }
    }
    landed<0>();
  }
  __syncthreads();  // the LDS makes room for the sums: [waves][MT][NT][64 lanes][4]
  float* part = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int c = 0; c < NT; ++c)
      *reinterpret_cast<f32x4_t*>(part + (((wave * MT + t) * NT + c) * 64 + lane) * 4) = acc[c][t];
  __syncthreads();
  // thread -> four neighbouring channels of a token, in the products' layout
  for (int i = threadIdx.x; i < 64 * MT * NT; i += blockDim.x) {
    const int c = i / 64 % NT * 16 + i % 64 / 16 * 4, r = i / (64 * NT) * 16 + i % 16;
    if (c >= nr || r >= mr) continue;
    f32x4_t sum = *reinterpret_cast<const f32x4_t*>(part + i * 4);
    for (int v = 1; v < nw; ++v) sum += *reinterpret_cast<const f32x4_t*>(part + (v * MT * NT * 64 + i) * 4);
    float bias[4] = {};
    if (a.bias) bias4<DT>(lds + bias_at + c * 4, bias);
    const float v[4] = {sum[0] + bias[0], sum[1] + bias[1], sum[2] + bias[2], sum[3] + bias[3]};
    if (vec) put4<DT, true, false>(a.out, (m0 + r) * a.ld_out, n0 + c, v, a.n);
    else put4<DT, false, false>(a.out, (m0 + r) * a.ld_out, n0 + c, v, n0 + nr);
  }
}

template <int DT, int MT, int NT, int D>
int launch_split(const MxLinearArgs& a, int nw, hipStream_t st) {
  const int tm = (int)cdiv64(a.M, 16 * MT);
  const dim3 g((unsigned)(cdiv64(cdiv64(a.n, 16 * NT) * tm, 8) * 8)), blk((unsigned)nw * 64);
  const int pitch = split_pitch((a.k + 31) / 32);
  const size_t table = (size_t)(split_table(16 * NT, pitch) + split_table(16 * MT, pitch));
  const size_t lds = table + (size_t)nw * D * (MT + NT) * 2048 + 256;
  hipLaunchKernelGGL((mx_split<DT, MT, NT, D>), g, blk, lds, st, a, tm,
                     pieces_of_four<DT>(a.out, a.ld_out, a.n));
  return (int)hipGetLastError();
}

// ---------------------------------------------------------------------------
// mx_tile: TM tokens x TN channels a tile, NW waves as 2 x NW/2, on
// v_mfma_scale_f32_32x32x64. K passes through two LDS buffers in units of 128
// bytes (256 values, four steps of the products) a row, written by direct loads:
// 1 KB an instruction, 8 rows of 8 pieces, place p of row r holding the row's
// piece p ^ (r/2 % 8), so that 16 lanes reading one piece of 16 rows meet every
// bank once. (Rows of 64 bytes, which would leave room for more buffers, cost the
// load path 31 to 39 clocks a KB in place of 17 to 20.) A step's fragments are
// read into registers while the products of the step before run. Before a unit's
// last step every wave has read all of it and the next unit has landed: one
// barrier, and the buffer takes the unit after the next. The scales come 16 bytes
// a row (two units) at a time, into a buffer that the waves take over into
// registers at once. Workgroups are persistent: the loads run ahead into the next
// tile; past the last tile they are out of range and bring zeros. Measured: 8192 x
// 10240 x 2560 115 us (3.7 PFLOP/s; the matrix cores are busy 42% of the cycles at
// 2.07 GHz, LDS, which the fragments' reads and the loads' writes share, 58%), 8192^3
// 251 us (4.4 PFLOP/s). Outputs that are not whole pieces go to memory from the
// products' layout, 8 bytes a row and lane: 8192 x 10239 x 2560 185 us. Four waves of 128 x 128 take 152 us for the first; eight
// waves of 32 x 64 on a 128 x 128 tile 37 us for 31 at 1024 x 2560 x 10240.
// ---------------------------------------------------------------------------
constexpr int kTurn = 2048;  // a wave's LDS in the epilogue: 16 rows of 128 bytes
template <int TM, int TN, int NW>
constexpr int tile_lds() { return (TM + TN) * (2 * 128 + 16) + NW * kTurn + 3 * TN * 4; }
template <int TM, int TN, int NW>
constexpr int tile_groups() { return 160 * 1024 / tile_lds<TM, TN, NW>(); }  // workgroups a CU

template <int DT, int TM, int TN, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, (tile_groups<TM, TN, NW>() * NW / 4)) void mx_tile(MxLinearArgs a, int tiles_m, int tiles_n) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int FM = TM / 64, FN = TN / (16 * NW), F = FN + FM, UB = (TM + TN) * 128;
  constexpr int LW = TN / (8 * NW), LQ = TM / (8 * NW), L = LW + LQ;  // a wave's loads a unit
  constexpr int B = DT == 2 ? 4 : 2, V = 16 / B;                      // bytes of an output, outputs a piece
  constexpr int NS = VEC ? FN * FM * 2 * B / 2 : 0;                   // a wave's stores a tile
  static_assert(TN % (8 * NW) == 0 && TM % (8 * NW) == 0 && TM + TN <= 64 * NW && TN % 64 == 0, "whole loads, at most one of scales and of bias a wave");
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
  const int wm = wave % 2, wn = wave / 2;
  // Workgroups b, b + 8, b + 16, .. share an XCD and take neighbouring tiles,
  // eight rows of tiles at a time, so that they meet in that XCD's L2.
  const int tiles = tiles_m * tiles_n, per = (tiles + 7) / 8;
  const int first = (int)blockIdx.x / 8, stride = (int)gridDim.x / 8;
  auto place = [&](int j, int& m0, int& n0) {  // the workgroup's tile j; false past the last
    const int local = first + j * stride, tile = (int)(blockIdx.x % 8) * per + local;
    if (local >= per || tile >= tiles) return false;
    const int band = tile / (8 * tiles_n), in = tile % (8 * tiles_n), high = min(8, tiles_m - band * 8);
    // (the division runs on the vector unit: the same in every lane)
    const int column = __builtin_amdgcn_readfirstlane(in / high);
    m0 = (band * 8 + in - column * high) * TM;
    n0 = column * TN;
    return true;
  };
  const int blocks = (a.k + 31) / 32, bytes = blocks * 16, scale_bytes = (blocks + 15) / 16 * 16;
  const int units = (blocks + 15) / 16 * 2;  // whole groups of two; the last may bring zeros
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8_t*)lds;

  // Loads: instruction i = wave + NW*j fills rows 8*i .. 8*i + 7. Rows past the
  // matrix are past the range (a pitch is at least `bytes`). Scales: instruction
  // i fills rows 64*i .. 64*i + 63 of the TN + TM.
  const int lpiece = ((lane % 8) ^ (wave % 2 * 4 + lane / 16)) * 16;
  const uint32_t woff = (uint32_t)((wave * 8 + lane / 8) * (int)a.ld_w + lpiece);
  const uint32_t qoff = (uint32_t)((wave * 8 + lane / 8) * (int)a.ld_q + lpiece);
  // Where a tile's loads read: ranges of its rows, and of the scales that this
  // wave fetches. The loads run up to two units ahead, so that of a tile and the
  // next; both stand ready, and a unit has no branch (across which the compiler
  // would move its products).
  constexpr int SW = (TM + TN) / 64;  // loads of scales; the waves past them repeat the first's
  const int sw = wave < SW ? wave : wave - SW;
  const bool ws = sw * 64 < TN;  // whether these are of weights
  const int64_t ld_s = ws ? a.ld_ws : a.ld_qs;
  const int srow = sw * 64 - (ws ? 0 : TN);
  struct Aim {
    const uint8_t *w, *q, *s;
    uint32_t wbytes, qbytes, sbytes;
    int n0, channels;
  };
  auto aim = [&](int j) {
    int m0 = 0, n0 = 0;
    const uint32_t in = place(j, m0, n0) ? ~0u : 0u;
    const int nr = min(TN, a.n - n0), mr = min(TM, (int)a.M - m0);
    Aim z;
    z.w = a.w + (int64_t)n0 * a.ld_w;
    z.q = a.q + (int64_t)m0 * a.ld_q;
    z.s = ws ? a.w_scale + (int64_t)n0 * ld_s : a.q_scale + (int64_t)m0 * ld_s;
    z.n0 = n0;
    z.channels = (int)(in & (uint32_t)nr);
    z.wbytes = in & (uint32_t)((nr - 1) * (int)a.ld_w + bytes);
    z.qbytes = in & (uint32_t)((mr - 1) * (int)a.ld_q + bytes);
    z.sbytes = in & (uint32_t)(((ws ? nr : mr) - 1) * (int)ld_s + scale_bytes);
    return z;
  };
  Aim now = aim(0), next = aim(1);
  int lu = 0, gu = 0;              // the next unit and group to load
  bool ltile = false, gtile = false;  // whether they are of the tile after this one
  auto load_scales = [&]() {
    load_lds(range_words(gtile ? next.s : now.s, gtile ? next.sbytes : now.sbytes),
             (uint32_t)((srow + hidden(lane)) * (int)ld_s + gu * 16), lds0 + (uint32_t)(2 * UB + sw * 1024));
    const bool end = ++gu * 2 == units;
    gu = end ? 0 : gu;
    gtile = gtile || end;
  };
  struct Loads {  // one unit's loads
    i32x4_t rw, rq;
    uint32_t buf, k;
    bool in_row;
  };
  auto loads_into = [&](int slot) {
    Loads z;
    z.rw = range_words(ltile ? next.w : now.w, ltile ? next.wbytes : now.wbytes);
    z.rq = range_words(ltile ? next.q : now.q, ltile ? next.qbytes : now.qbytes);
    z.buf = lds0 + (uint32_t)(slot * UB + wave * 1024);
    z.k = (uint32_t)lu * 128u;
    z.in_row = (int)z.k + lpiece < bytes;  // past the row's last block: zeros
    const bool end = ++lu == units;
    lu = end ? 0 : lu;
    ltile = ltile || end;
    return z;
  };
  auto load_one = [&](const Loads& z, auto I) {  // the i-th of a unit's L loads
    constexpr int i = decltype(I)::value;
    if constexpr (i < LW) load_lds(z.rw, z.in_row ? woff + (z.k + (uint32_t)(8 * NW * i * (int)a.ld_w)) : kOut, z.buf + i * (NW * 1024));
    else load_lds(z.rq, z.in_row ? qoff + (z.k + (uint32_t)(8 * NW * (i - LW) * (int)a.ld_q)) : kOut,
                  z.buf + TN * 128 + (i - LW) * (NW * 1024));
  };

  // fragments: lane -> row lane % 32, block 2*step + lane/32 of the unit's eight
  uint4 frag[2][F], raw[F];  // [step parity][weights, tokens]; a group's scales of the lane's rows as read
  uint32_t scale[F][2];      // and of the lane's blocks: byte `step` of word `unit`
  const uint32_t fat = (uint32_t)(lane % 32 * 128 + ((lane / 32) ^ (lane / 2 % 8)) * 16);  // of step 0; step s: xor 32*s
  auto read_one = [&](int slot, auto ST, auto I) {  // the i-th fragment of a step
    // in the order of their use: the first weights, the tokens, the other weights
    constexpr int st = decltype(ST)::value, i = decltype(I)::value, f = i == 0 ? 0 : i <= FM ? FN + i - 1 : i - FM;
    const uint8_t* buf = lds + slot * UB + (fat ^ (st * 32));
    if constexpr (f < FN) frag[st % 2][f] = ld16(buf + (wn * FN + f) * 4096);
    else frag[st % 2][f] = ld16(buf + TN * 128 + (wm * FM + f - FN) * 4096);
  };
  auto read_scales = [&](auto I) {
    constexpr int f = decltype(I)::value;
    const uint8_t* sc = lds + 2 * UB + hidden(lane) % 32 * 16;
    raw[f] = ld16(sc + (f < FN ? wn * FN + f : TN / 32 + wm * FM + f - FN) * 512);
  };
  // Of the 16 blocks that start at `block` a lane takes every second: bytes h and
  // 2 + h of each word, h = lane / 32.
  auto take_scales = [&](int block) {
    auto keep = [&](int i) {  // bytes past the last block do not count
      const int n = min(max(blocks - block - i * 4, 0), 4);
      return n == 4 ? ~0u : (1u << (8 * n)) - 1u;
    };
    const uint32_t pick = 0x06040200u + (uint32_t)(hidden(lane) / 32) * 0x01010101u;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      scale[f][0] = __builtin_amdgcn_perm(raw[f].y & keep(1), raw[f].x & keep(0), pick);
      scale[f][1] = __builtin_amdgcn_perm(raw[f].w & keep(3), raw[f].z & keep(2), pick);
    }
  };
  f32x16_t acc[FN][FM];
  // Unit u, the POS-th of its group, in buffer POS. Its first step's fragments
  // are in registers, and in POS 0 its group's scales. FIRST: of its tile.
  auto unit = [&](int u, auto POS, auto FIRST) {
    constexpr int pos = decltype(POS)::value, NM = FN * FM;
    if constexpr (pos == 0) take_scales(u * 8);
    auto products = [&](auto ST, auto after) {  // a step's products, after(t) behind the t-th
      constexpr int st = decltype(ST)::value;
      asm volatile("" ::: "memory");  // no step's reads before the step
      __builtin_amdgcn_sched_barrier(0);
      each<NM>([&](auto T) {
        constexpr int t = decltype(T)::value, f = t / FM, g = t % FM;
        acc[f][g] = mfma_mx32<st, st>(frag[st % 2][f], frag[st % 2][FN + g],
                                      decltype(FIRST)::value && st == 0 ? f32x16_t{} : acc[f][g], scale[f][pos], scale[FN + g][pos]);
        after(T);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    // operations 0 .. N - 1, spread behind products FROM .. FROM + COUNT - 1
    auto spread = [&](auto T, auto FROM, auto COUNT, auto N, auto op) {
      constexpr int t = decltype(T)::value - decltype(FROM)::value, c = decltype(COUNT)::value, n = decltype(N)::value;
      if constexpr (t >= 0 && t < c) each<(t + 1) * n / c - t * n / c>([&](auto O) { op(ic<t * n / c + decltype(O)::value>{}); });
    };
    const int slot = pos;
    products(ic<0>{}, [&](auto T) { spread(T, ic<0>{}, ic<(F < NM ? F : NM)>{}, ic<F>{}, [&](auto O) { read_one(slot, ic<1>{}, O); }); });
    products(ic<1>{}, [&](auto T) { spread(T, ic<0>{}, ic<(F < NM ? F : NM)>{}, ic<F>{}, [&](auto O) { read_one(slot, ic<2>{}, O); }); });
    // The products of the last two steps, numbered through. Behind the one at
    // FREE every wave has read the unit, and its buffer takes the one after the
    // next; behind the one at HERE the next unit has landed. One barrier for both
    // where one workgroup has the CU: 118 us at 8192x10240x2560, 121 with two.
    // Apart they give the loads two steps more where several workgroups share the
    // CU and the load path: 36 -> 31 us at 1024x2560x10240.
    constexpr bool APART = tile_groups<TM, TN, NW>() > 1;
    constexpr int FREE = APART ? NM / 2 - 1 : NM - 1, HERE = APART ? NM + NM / 2 - 1 : NM - 1;
    Loads z;
    auto behind = [&](auto T) {
      constexpr int t = decltype(T)::value;
      spread(T, ic<0>{}, ic<(F < FREE + 1 ? F : FREE > 1 ? FREE : 1)>{}, ic<F>{}, [&](auto O) { read_one(slot, ic<3>{}, O); });
      spread(T, ic<FREE + 1>{}, ic<NM>{}, ic<L>{}, [&](auto O) { load_one(z, O); });
      if constexpr (t == HERE) {
        // Younger than the next unit are, apart, the L loads since FREE (all of
        // them are issued by here), and behind a tile's second unit an epilogue's
        // stores. (Loads and stores of a wave are counted off in the order of
        // their issue.)
        static_assert(!APART || FREE + NM <= HERE, "all loads issued");
        landed<(APART ? L + (pos == 0 ? 1 : 0) : 0) + (decltype(FIRST)::value ? NS : 0)>();
      }
      if constexpr (t == FREE || t == HERE) lds_sync();
      if constexpr (t == FREE) {
        if constexpr (pos == 0) load_scales();  // the buffer's group is in registers
        z = loads_into(slot);
      }
      spread(T, ic<HERE + 1>{}, ic<2 * NM - HERE - 1>{}, ic<F + (pos == 1 ? F : 0)>{}, [&](auto O) {
        constexpr int o = decltype(O)::value;
        if constexpr (o < F) read_one(1 - slot, ic<0>{}, O);
        else read_scales(ic<o - F>{});
      });
    };
    products(ic<2>{}, behind);
    products(ic<3>{}, [&](auto T) { behind(ic<NM + decltype(T)::value>{}); });
  };

  // A tile's bias comes with the tile before, in three places in turn: it is
  // read at the tile's end, when a wave that is ahead asks for that of the tile
  // after the next.
  constexpr int kBias = 2 * UB + (TM + TN) * 16 + NW * kTurn;
  auto bias_of = [&](const Aim& z, int j) {
    if (a.bias && wave * 64 < TN)
      load_bias<DT>(a.bias, z.n0 + wave * 64, min(z.channels - wave * 64, 64), lane,
                    lds0 + (uint32_t)(kBias + j % 3 * (TN * 4) + wave * 256));
  };
  bias_of(now, 0);
  load_scales();
  each<2>([&](auto S) {
    const Loads z = loads_into(decltype(S)::value);
    each<L>([&](auto I) { load_one(z, I); });
  });
  landed<0>();  // (both units: the first tile's first wait allows for stores)
  lds_sync();
  each<F>([&](auto I) { read_one(0, ic<0>{}, I); });
  each<F>([&](auto I) { read_scales(I); });
  int m0 = 0, n0 = 0;
  for (int j = 0; place(j, m0, n0); ++j) {
    const int el = hidden(lane), col = wn * (32 * FN), mr = min(TM, (int)a.M - m0), nr = min(TN, a.n - n0);
    bias_of(next, j + 1);
    unit(0, ic<0>{}, ic<1>{});
    unit(1, ic<1>{}, ic<0>{});
    for (int u = 2; u < units; u += 2) {
      unit(u, ic<0>{}, ic<0>{});
      unit(u + 1, ic<1>{}, ic<0>{});
    }
    // Sums: lane -> token lane % 32, channels 8*(i/4) + 4*(lane/32) + i % 4. The
    // bias joins the whole sum: at the start of the accumulators each of K/64
    // additions would round at its size (and 8192 x 10240 x 2560 take 112.4 us for
    // 113.7).
    if (a.bias) {
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float bias[4];
          bias4<DT>(lds + kBias + j % 3 * (TN * 4) + (col + f * 32 + q * 8 + el / 32 * 4) * 4, bias);
#pragma unroll
          for (int g = 0; g < FM; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[f][g][q * 4 + i] += bias[i];
        }
    }
    if constexpr (VEC) {
      // Rounded, and through the wave's 2 KB of LDS, so that a store is whole
      // 128-byte lines: 16 tokens x CH channels a pass, place p of row r holding
      // piece p ^ (r % 8). Always NS stores: what lies outside goes past the range.
      // Streamed, they leave no lines that the kernel's end has to write back (1024 x
      // 10240 x 2560 with the quantizer that reads it next 30.0 -> 28.3 us, 512 x
      // 10240 x 2560 21.3 -> 20.6, 512 x 2560 x 2560 14.1 -> 14.4).
      constexpr int FP = FN * 32 * B <= 128 ? FN : 128 / (32 * B), CH = FP * 32, P = CH / V;  // P: pieces a row
      static_assert(CH * B <= 128 && FN % FP == 0 && NS == FN / FP * FM * 2 * (16 * P / 64), "stores");
      uint8_t* turn = lds + 2 * UB + (TM + TN) * 16 + wave * kTurn;
      const rsrc_t out = make_rsrc(reinterpret_cast<uint8_t*>(a.out) + ((int64_t)m0 * a.ld_out + n0) * B,
                                   (uint32_t)(((mr - 1) * (int)a.ld_out + nr) * B));
#pragma unroll
      for (int f0 = 0; f0 < FN; f0 += FP)
#pragma unroll
        for (int g = 0; g < FM; ++g)
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const int r16 = el % 16;
            if (el % 32 / 16 == part) {
#pragma unroll
              for (int f = 0; f < FP; ++f)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  auto value = [&](int i) { return acc[f0 + f][g][q * 4 + i]; };
                  const int at = (f * 32 + q * 8 + el / 32 * 4) * B;  // the byte in the row
                  uint8_t* to = turn + r16 * 128 + ((at / 16) ^ (r16 % 8)) * 16 + at % 16;
                  if constexpr (DT == 2) *reinterpret_cast<f32x4_t*>(to) = f32x4_t{value(0), value(1), value(2), value(3)};
                  else *reinterpret_cast<uint2*>(to) = make_uint2(pack2<DT>(value(0), value(1)), pack2<DT>(value(2), value(3)));
                }
            }
            wave_sync();  // lanes read what others wrote
#pragma unroll
            for (int k = 0; k < 16 * P / 64; ++k) {
              const int r = k * (64 / P) + el / P, p = el % P;
              const u32x4_t w = *reinterpret_cast<const u32x4_t*>(turn + r * 128 + (p ^ (r % 8)) * 16);
              const int m = wm * (TM / 2) + g * 32 + part * 16 + r, n = col + f0 * 32 + p * V;
              const uint32_t to = m < mr && n < nr ? (uint32_t)((m * (int)a.ld_out + n) * B) : kOut;
              __builtin_amdgcn_raw_buffer_store_b128(w, out, (int)to, 0, kNonTemporal);
            }
            wave_sync();  // and the next part writes where they read
          }
    } else {
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int g = 0; g < FM; ++g)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& c = acc[f][g];
            const int m = wm * (TM / 2) + el % 32 + g * 32, n = n0 + col + f * 32 + q * 8 + el / 32 * 4;
            const float v[4] = {c[q * 4], c[q * 4 + 1], c[q * 4 + 2], c[q * 4 + 3]};
            if (m < mr && n < a.n) put4<DT, false, false>(a.out, (int64_t)(m0 + m) * a.ld_out, n, v, a.n);
            __builtin_amdgcn_sched_barrier(0);  // (not all addresses at once)
          }
    }
    now = next;
    next = aim(j + 2);
    ltile = gtile = units == 2;  // (of so short a tile all is loaded already)
  }
  landed<0>();  // no load into this workgroup's LDS outlives it
}

// Whether rows of out are whole 16-byte pieces, and a tile of them a 32-bit range.
template <int DT>
bool whole_pieces(const MxLinearArgs& a) {
  constexpr int V = DT == 2 ? 4 : 8;
  return a.n % V == 0 && a.ld_out % V == 0 && al16(a.out) && a.ld_out <= (1 << 20);
}

template <int DT, int TM, int TN, int NW, bool VEC>
int launch_tile(const MxLinearArgs& a, hipStream_t st) {
  const int tm = (int)cdiv64(a.M, TM), tn = (int)cdiv64(a.n, TN);
  // persistent workgroups: as many as the 256 CUs hold at once
  const int64_t tiles = cdiv64((int64_t)tm * tn, 8) * 8, held = 256 * tile_groups<TM, TN, NW>();
  hipLaunchKernelGGL((mx_tile<DT, TM, TN, NW, VEC>), dim3((unsigned)std::min(tiles, held)), dim3(64 * NW),
                     (tile_lds<TM, TN, NW>()), st, a, tm, tn);
  return (int)hipGetLastError();
}
template <int DT, int TM, int TN, int NW>
int run_tile(const MxLinearArgs& a, hipStream_t st) {
  return whole_pieces<DT>(a) ? launch_tile<DT, TM, TN, NW, true>(a, st) : launch_tile<DT, TM, TN, NW, false>(a, st);
}

// The kernel is the one that a model of its time, in microseconds, puts first: a
// start and a part for each unit of 128 bytes of K with up to 256 tiles (one a
// CU), and what every further 256 tiles add. The constants are fitted on one MI355X
// to eleven N x K from 400 x 800 to 8192 x 8192 and 16384 x 512 at M = 1 .. 4096:
// the kernel taken is within 1% of the fastest on average, 16% at worst. Measured,
// split 32x32 / split 64x64 / tile 128 / tile 192 / tile 256: 2560x10240 at M = 64:
// 8.3 / 16 / 28 / - / 57 us, M = 300: 24 / 15 / 28 / 53 / 59, M = 2048: - / - / 47 /
// 53 / 61; 10240x2560 at M = 64: 7.5 / 8.6 / 11 / - / 20, M = 300: 22 / 17 / 12 / 17 /
// 20, M = 1024: - / 40 / 24 / 20.4 / 22, M = 4096: - / - / 73 / 67 / 63.
struct Cost {
  int tm, tn;  // tokens and channels a tile
  double start, unit, more, more_unit;
  double of(const MxLinearArgs& a) const {
    const double u = (double)cdiv64(a.k, 256), turns = (double)cdiv64(cdiv64(a.M, tm) * cdiv64(a.n, tn), 256);
    return start + unit * u + (turns - 1) * (more + more_unit * u);
  }
};
constexpr Cost kCosts[] = {{16, 16, 3.2, 0.096, 0.2, 0.037},  {32, 16, 3.25, 0.098, 0.26, 0.06}, {32, 32, 3.33, 0.124, 0.4, 0.119},
                           {64, 32, 4.0, 0.204, 0.65, 0.234}, {64, 64, 5.0, 0.268, 0.51, 0.269}, {128, 128, 4.7, 0.637, 1.3, 0.54},
                           {192, 256, 6.0, 1.185, 5.5, 1.4},  {256, 256, 7.1, 1.36, 7.5, 1.72}};

// Waves of a split kernel's workgroup: two where several workgroups share a CU
// (10240x2560, M = 64: 7.5 us, 9.4 with four), eight where one wave in four would
// walk ten units or more (2560x10240, M = 1: 6.2 us, 6.5 with four). Of 64x64 tiles
// from 512 on: 320 tiles of 10240x2560 take four waves 10.6 us and two 11.2, 512 of
// 8192x20000, whose scales leave room for one workgroup a CU, 71 and 98; two waves
// are the faster ones from 257 tiles on where K is between (2560x5120, M = 512: 15.8
// us for 18.0; 8192x8192, M = 256: 22.3 for 24.6).
inline int split_waves(int64_t tiles, int most, int k, int few) { return tiles > most ? 2 : k > 32 * 256 ? few : 4; }

template <int DT>
int run(const MxLinearArgs& a, hipStream_t st) {
  int best = 0;
  for (int i = 1; i < (int)(sizeof kCosts / sizeof *kCosts); ++i)
    if (kCosts[i].of(a) < kCosts[best].of(a)) best = i;
  const Cost& c = kCosts[best];
  const int64_t tiles = cdiv64(a.M, c.tm) * cdiv64(a.n, c.tn);
  switch (best) {
    case 0: return launch_split<DT, 1, 1, 2>(a, split_waves(tiles, 256, a.k, 8), st);
    case 1: return launch_split<DT, 2, 1, 2>(a, split_waves(tiles, 256, a.k, 4), st);
    case 2: return launch_split<DT, 2, 2, 2>(a, split_waves(tiles, 256, a.k, 4), st);
    case 3: return launch_split<DT, 4, 2, 2>(a, split_waves(tiles, 256, a.k, 4), st);
    case 4: return launch_split<DT, 4, 4, 1>(a, split_waves(tiles, 512, a.k, 4), st);
    case 5: return run_tile<DT, 128, 128, 4>(a, st);
    case 6: return run_tile<DT, 192, 256, 8>(a, st);
    default: return run_tile<DT, 256, 256, 8>(a, st);
  }
}

template <int DT>
hipError_t raise_lds() {
  const void* f[] = {
      (const void*)mx_tile<DT, 256, 256, 8, true>, (const void*)mx_tile<DT, 256, 256, 8, false>,
      (const void*)mx_tile<DT, 192, 256, 8, true>, (const void*)mx_tile<DT, 192, 256, 8, false>,
      (const void*)mx_tile<DT, 128, 128, 4, true>, (const void*)mx_tile<DT, 128, 128, 4, false>,
      (const void*)mx_split<DT, 1, 1, 2>,       (const void*)mx_split<DT, 2, 1, 2>,
      (const void*)mx_split<DT, 2, 2, 2>,       (const void*)mx_split<DT, 4, 2, 2>,
      (const void*)mx_split<DT, 4, 4, 1>};
  for (const void* k : f) {
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, bool AL>
void launch_rows(const MxRowsToArgs& a, dim3 g, int blocks, Divide d, uint32_t pieces, hipStream_t st) {
  hipLaunchKernelGGL((mx_quantize<T, AL>), g, dim3(256), 0, st, a, blocks, d, pieces);
}
template <typename T, bool AL>
void launch_rows(const MxRowsFromArgs& a, dim3 g, int blocks, Divide d, uint32_t pieces, hipStream_t st) {
  hipLaunchKernelGGL((mx_dequantize<T, AL>), g, dim3(256), 0, st, a, blocks, d, pieces);
}
template <typename T, typename A>
int rows_of(A a, hipStream_t st) {
  constexpr int b = (int)sizeof(typename T::S), V = vec<T>();
  const bool al = ld16_ok(a.k, b) && al16(a.x) && ld16_ok(a.ld_x, b);
  const int blocks = (a.k + 31) / 32, per_row = blocks * (32 / V);
  const Divide d = divide_by((uint32_t)per_row);
  // piece numbers stay below 2^31: more rows in several launches
  const int64_t most = ((int64_t)1 << 30) / per_row;
  auto* x = reinterpret_cast<std::conditional_t<std::is_const_v<std::remove_pointer_t<decltype(a.x)>>, const typename T::S*,
                                                typename T::S*>>(a.x);
  for (int64_t left = a.M; left > 0; left -= most) {
    const uint32_t pieces = (uint32_t)(std::min(left, most) * per_row);
    const dim3 g((unsigned)cdiv64(pieces, 256 * kPieces));
    a.x = x;
    if (al) launch_rows<T, true>(a, g, blocks, d, pieces, st);
    else launch_rows<T, false>(a, g, blocks, d, pieces, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    x += most * a.ld_x;
    a.q += most * a.ld_q;
    a.q_scale += most * a.ld_qs;
  }
  return (int)hipSuccess;
}
template <typename A>
int rows_of(const A& a, int dtype, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == 0 ? rows_of<Bf16>(a, st) : dtype == 1 ? rows_of<Fp16>(a, st) : rows_of<Fp32>(a, st);
}

}  // namespace

int launch_mx_quantize(const MxRowsToArgs& a, int dtype, void* stream) { return rows_of(a, dtype, stream); }
int launch_mx_dequantize(const MxRowsFromArgs& a, int dtype, void* stream) { return rows_of(a, dtype, stream); }

int launch_mx_linear(const MxLinearArgs& args, int dtype, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  // tile counts stay in 32 bits: larger M in several launches
  constexpr int64_t kRows = (int64_t)1 << 20;
  const size_t b = dtype == 2 ? 4 : 2;
  for (int64_t m0 = 0; m0 < args.M; m0 += kRows) {
    MxLinearArgs a = args;
    a.M = std::min(args.M - m0, kRows);
    a.q += m0 * a.ld_q;
    a.q_scale += m0 * a.ld_qs;
    a.out = reinterpret_cast<uint8_t*>(a.out) + (size_t)(m0 * a.ld_out) * b;
    const int e = dtype == 0 ? run<0>(a, st) : dtype == 1 ? run<1>(a, st) : run<2>(a, st);
    if (e != (int)hipSuccess) return e;
  }
  return (int)hipSuccess;
}

int configure_mx_kernels(int dtype) {
  return (int)(dtype == 0 ? raise_lds<0>() : dtype == 1 ? raise_lds<1>() : raise_lds<2>());
}

}  // namespace hcgr
