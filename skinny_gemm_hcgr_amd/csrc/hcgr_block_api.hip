// hcgr_block_api.hip -- C ABI of the block operators (declarations and
// contract in include/hcgr.h). Host code only: checks and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <new>

#include "../../include/hcgr.h"
#include "hcgr_block.h"
#include "hcgr_host.h"

struct hcgr_block_op {
  hcgr_block_config cfg;
  int device;
};
struct hcgr_linear_op {
  hcgr_linear_config cfg;
  int device;
};

namespace {

using namespace hcgr_host;

size_t elem(int dtype) { return dtype == HCGR_FP32 ? 4 : 2; }

// Bytes from the first to past the last element of M rows.
uint64_t span(int64_t M, int64_t ld, int64_t cols, size_t b) {
  return ((uint64_t)(M - 1) * (uint64_t)ld + (uint64_t)cols) * b;
}

hcgr_status check_dtype(int dtype) {
  if (dtype != HCGR_BF16 && dtype != HCGR_FP16 && dtype != HCGR_FP32)
    return fail(HCGR_ERR_INVALID_ARGUMENT, "unknown dtype %d", dtype);
  return HCGR_OK;
}

hcgr_status check_block(const hcgr_block_config* c) {
  if (!c) return fail(HCGR_ERR_INVALID_ARGUMENT, "config is NULL");
  if (c->hc < 1 || c->hs < 1)
    return fail(HCGR_ERR_INVALID_ARGUMENT, "hc and hs must be positive (hc=%d hs=%d)", c->hc, c->hs);
  const hcgr_status st = check_dtype(c->dtype);
  if (st != HCGR_OK) return st;
  if (!std::isfinite(c->eps) || c->eps < 0.0f)
    return fail(HCGR_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (!std::isfinite(c->res_scale)) return fail(HCGR_ERR_INVALID_ARGUMENT, "res_scale must be finite");
  if (c->hc != 1 && c->hc != 2 && c->hc != 4 && c->hc != 8)
    return fail(HCGR_ERR_UNSUPPORTED, "hc=%d: the kernels support hc = 1, 2, 4 or 8", c->hc);
  if (c->hs > 65536) return fail(HCGR_ERR_UNSUPPORTED, "hs=%d: the kernels support widths up to 65536", c->hs);
  return HCGR_OK;
}

hcgr_status check_linear(const hcgr_linear_config* c) {
  if (!c) return fail(HCGR_ERR_INVALID_ARGUMENT, "config is NULL");
  if (c->n < 1 || c->k < 1)
    return fail(HCGR_ERR_INVALID_ARGUMENT, "n and k must be positive (n=%d k=%d)", c->n, c->k);
  const hcgr_status st = check_dtype(c->dtype);
  if (st != HCGR_OK) return st;
  if (c->k > HCGR_LINEAR_MAX_K)
    return fail(HCGR_ERR_UNSUPPORTED, "k=%d: 32-bit sums are exact up to k = %d", c->k, HCGR_LINEAR_MAX_K);
  if (c->n > HCGR_LINEAR_MAX_N) return fail(HCGR_ERR_UNSUPPORTED, "n=%d exceeds %d", c->n, HCGR_LINEAR_MAX_N);
  return HCGR_OK;
}

hcgr_status check_m(int64_t M) {
  if (M < 0) return fail(HCGR_ERR_INVALID_ARGUMENT, "M=%lld is negative", (long long)M);
  if (M > (int64_t)1 << 31) return fail(HCGR_ERR_UNSUPPORTED, "M=%lld exceeds 2^31", (long long)M);
  return HCGR_OK;
}

hcgr_status check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols) return fail(HCGR_ERR_INVALID_ARGUMENT, "%s=%lld < %lld", name, (long long)ld, (long long)cols);
  if (ld > (int64_t)1 << 31) return fail(HCGR_ERR_UNSUPPORTED, "%s=%lld exceeds 2^31", name, (long long)ld);
  return HCGR_OK;
}

// An int8 matrix: 16-byte aligned rows of at least `cols` bytes.
hcgr_status check_int8(const void* p, int64_t ld, int64_t cols, const char* name, const char* ld_name) {
  const PtrCheck c{p, name, 16};
  hcgr_status st = check_ptrs(&c, 1);
  if (st != HCGR_OK) return st;
  if ((st = check_ld(ld, cols, ld_name)) != HCGR_OK) return st;
  if (ld % 16) return fail(HCGR_ERR_INVALID_ARGUMENT, "%s=%lld is not a multiple of 16", ld_name, (long long)ld);
  return HCGR_OK;
}

hcgr_status check_aligned(const void* p, const char* name, size_t align) {
  if ((uintptr_t)p % align) return fail(HCGR_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", name, align);
  return HCGR_OK;
}

hcgr_status check_ws(const void* ws, size_t bytes, size_t need, int64_t M) {
  if (bytes < need)
    return fail(HCGR_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed for M=%lld", bytes, need,
                (long long)M);
  const PtrCheck c{ws, "workspace", 16};
  return check_ptrs(&c, 1);
}

hcgr_status norm_checks(const hcgr_block_config* c, const void* x, int64_t ld_x, const void* w, int64_t M,
                        const void* xn, const int8_t* q, int64_t ld_q, const float* q_scale, const float* rrms) {
  hcgr_status st = check_m(M);
  if (st != HCGR_OK || M == 0) return st;
  const size_t b = elem(c->dtype);
  const int64_t hs = c->hs;
  const PtrCheck need[] = {{x, "x", b}, {w, "w", b}};
  if ((st = check_ptrs(need, 2)) != HCGR_OK) return st;
  if ((st = check_ld(ld_x, hs, "ld_x")) != HCGR_OK) return st;
  if (!xn && !q) return fail(HCGR_ERR_INVALID_ARGUMENT, "neither xn nor q is given");
  if ((q != nullptr) != (q_scale != nullptr))
    return fail(HCGR_ERR_INVALID_ARGUMENT, "q and q_scale are given together or not at all");
  if ((st = check_aligned(xn, "xn", b)) != HCGR_OK) return st;
  if ((st = check_aligned(q_scale, "q_scale", 4)) != HCGR_OK) return st;
  if ((st = check_aligned(rrms, "rrms", 4)) != HCGR_OK) return st;
  if (q && (st = check_int8(q, ld_q, hs, "q", "ld_q")) != HCGR_OK) return st;
  const uint64_t m = (uint64_t)M;
  const Range ins[] = {range_of(x, span(M, ld_x, hs, b), "x"), range_of(w, (uint64_t)hs * b, "w")};
  const Range outs[] = {range_of(xn, xn ? m * (uint64_t)hs * b : 0, "xn"),
                        range_of(q, q ? span(M, ld_q, hs, 1) : 0, "q"),
                        range_of(q_scale, q_scale ? m * 4 : 0, "q_scale"), range_of(rrms, rrms ? m * 4 : 0, "rrms")};
  return check_overlaps(outs, 4, ins, 2);
}

hcgr_status norm_bwd_checks(const hcgr_block_config* c, const void* x, int64_t ld_x, const void* w,
                            const float* rrms, const void* dxn, int64_t M, const void* dx, const float* dw,
                            const void* ws, size_t ws_bytes) {
  hcgr_status st = check_m(M);
  if (st != HCGR_OK || M == 0) return st;
  const size_t b = elem(c->dtype);
  const int64_t hs = c->hs;
  const PtrCheck need[] = {{x, "x", b}, {w, "w", b}, {rrms, "rrms", 4}, {dxn, "dxn", b}};
  if ((st = check_ptrs(need, 4)) != HCGR_OK) return st;
  if ((st = check_ld(ld_x, hs, "ld_x")) != HCGR_OK) return st;
  if (!dx && !dw) return fail(HCGR_ERR_INVALID_ARGUMENT, "neither dx nor dw is given");
  if ((st = check_aligned(dx, "dx", b)) != HCGR_OK) return st;
  if ((st = check_aligned(dw, "dw", 4)) != HCGR_OK) return st;
  const size_t wneed = hcgr::norm_bwd_workspace(c->hs, M);
  if ((st = check_ws(ws, ws_bytes, wneed, M)) != HCGR_OK) return st;
  const uint64_t m = (uint64_t)M;
  const Range ins[] = {range_of(x, span(M, ld_x, hs, b), "x"), range_of(w, (uint64_t)hs * b, "w"),
                       range_of(rrms, m * 4, "rrms"), range_of(dxn, m * (uint64_t)hs * b, "dxn")};
  const Range outs[] = {range_of(dx, dx ? m * (uint64_t)hs * b : 0, "dx"),
                        range_of(dw, dw ? (uint64_t)hs * 4 : 0, "dw"), range_of(ws, wneed, "workspace")};
  return check_overlaps(outs, 3, ins, 4);
}

hcgr_status residual_checks(const hcgr_block_config* c, const void* R, const void* y, int64_t ld_y,
                            const void* inj, int64_t ld_inj, const void* w_post, const void* w_pre, int64_t M,
                            const void* R2, const void* x, const int8_t* q, int64_t ld_q, const float* q_scale,
                            const float* rrms) {
  hcgr_status st = check_m(M);
  if (st != HCGR_OK || M == 0) return st;
  const size_t b = elem(c->dtype);
  const int64_t hs = c->hs, hc = c->hc;
  const PtrCheck need[] = {{R, "R", b}, {y, "y", b}, {R2, "R2", b}};
  if ((st = check_ptrs(need, 3)) != HCGR_OK) return st;
  if ((st = check_aligned(inj, "inj", b)) != HCGR_OK) return st;
  if ((st = check_aligned(w_post, "w_post", b)) != HCGR_OK) return st;
  if ((st = check_aligned(w_pre, "w_pre", b)) != HCGR_OK) return st;
  if ((st = check_aligned(x, "x", b)) != HCGR_OK) return st;
  if ((st = check_aligned(q_scale, "q_scale", 4)) != HCGR_OK) return st;
  if ((st = check_aligned(rrms, "rrms", 4)) != HCGR_OK) return st;
  if ((st = check_ld(ld_y, hs, "ld_y")) != HCGR_OK) return st;
  if (inj && (st = check_ld(ld_inj, hc, "ld_inj")) != HCGR_OK) return st;
  if (w_pre && !x && !q) return fail(HCGR_ERR_INVALID_ARGUMENT, "w_pre is given, but neither x nor q");
  if (!w_pre && (x || q)) return fail(HCGR_ERR_INVALID_ARGUMENT, "x and q need w_pre");
  if ((q != nullptr) != (q_scale != nullptr))
    return fail(HCGR_ERR_INVALID_ARGUMENT, "q and q_scale are given together or not at all");
  if (q && (st = check_int8(q, ld_q, hs, "q", "ld_q")) != HCGR_OK) return st;
  const uint64_t m = (uint64_t)M, k = (uint64_t)hc * (uint64_t)hs;
  const Range ins[] = {range_of(R, m * k * b, "R"), range_of(y, span(M, ld_y, hs, b), "y"),
                       range_of(inj, inj ? span(M, ld_inj, hc, b) : 0, "inj"),
                       range_of(w_post, w_post ? (uint64_t)hs * b : 0, "w_post"),
                       range_of(w_pre, w_pre ? (uint64_t)hs * b : 0, "w_pre")};
  const Range outs[] = {range_of(R2, m * k * b, "R2"), range_of(x, x ? m * (uint64_t)hs * b : 0, "x"),
                        range_of(q, q ? span(M, ld_q, hs, 1) : 0, "q"),
                        range_of(q_scale, q_scale ? m * 4 : 0, "q_scale"), range_of(rrms, rrms ? m * 8 : 0, "rrms")};
  return check_overlaps(outs, 5, ins, 5);
}

hcgr_status residual_bwd_checks(const hcgr_block_config* c, const void* R, const void* y, int64_t ld_y,
                                const void* inj, int64_t ld_inj, const void* w_post, const void* w_pre,
                                const float* rrms, const void* dR2, const void* dx, int64_t M, const void* dR,
                                const void* dy, const void* dinj, int64_t ld_dinj, const float* dw_post,
                                const float* dw_pre, const void* ws, size_t ws_bytes) {
  hcgr_status st = check_m(M);
  if (st != HCGR_OK || M == 0) return st;
  const size_t b = elem(c->dtype);
  const int64_t hs = c->hs, hc = c->hc;
  const PtrCheck need[] = {{R, "R", b}, {y, "y", b}, {dR, "dR", b}, {dy, "dy", b}};
  if ((st = check_ptrs(need, 4)) != HCGR_OK) return st;
  const PtrCheck opt[] = {{inj, "inj", b},   {w_post, "w_post", b}, {w_pre, "w_pre", b},     {rrms, "rrms", 4},
                          {dR2, "dR2", b},   {dx, "dx", b},         {dinj, "dinj", b},       {dw_post, "dw_post", 4},
                          {dw_pre, "dw_pre", 4}};
  for (const PtrCheck& p : opt)
    if ((st = check_aligned(p.p, p.name, p.align)) != HCGR_OK) return st;
  if ((st = check_ld(ld_y, hs, "ld_y")) != HCGR_OK) return st;
  if (inj && (st = check_ld(ld_inj, hc, "ld_inj")) != HCGR_OK) return st;
  if (dinj && (st = check_ld(ld_dinj, hc, "ld_dinj")) != HCGR_OK) return st;
  if (!dR2 && !dx) return fail(HCGR_ERR_INVALID_ARGUMENT, "neither dR2 nor dx is given");
  if ((w_pre != nullptr) != (dx != nullptr))
    return fail(HCGR_ERR_INVALID_ARGUMENT, "dx is given exactly when w_pre is");
  if ((w_pre != nullptr) != (dw_pre != nullptr))
    return fail(HCGR_ERR_INVALID_ARGUMENT, "dw_pre is given exactly when w_pre is");
  if ((w_post != nullptr) != (dw_post != nullptr))
    return fail(HCGR_ERR_INVALID_ARGUMENT, "dw_post is given exactly when w_post is");
  if ((inj != nullptr) != (dinj != nullptr))
    return fail(HCGR_ERR_INVALID_ARGUMENT, "dinj is given exactly when inj is");
  if ((w_post || w_pre) && !rrms) return fail(HCGR_ERR_INVALID_ARGUMENT, "rrms is NULL");
  const size_t wneed = hcgr::norm_bwd_workspace(c->hs, M);
  if ((st = check_ws(ws, ws_bytes, wneed, M)) != HCGR_OK) return st;
  const uint64_t m = (uint64_t)M, k = (uint64_t)hc * (uint64_t)hs, row = (uint64_t)hs * b;
  const Range ins[] = {range_of(R, m * k * b, "R"),
                       range_of(y, span(M, ld_y, hs, b), "y"),
                       range_of(inj, inj ? span(M, ld_inj, hc, b) : 0, "inj"),
                       range_of(w_post, w_post ? row : 0, "w_post"),
                       range_of(w_pre, w_pre ? row : 0, "w_pre"),
                       range_of(rrms, rrms ? m * 8 : 0, "rrms"),
                       range_of(dR2, dR2 ? m * k * b : 0, "dR2"),
                       range_of(dx, dx ? m * row : 0, "dx")};
  const Range outs[] = {range_of(dR, m * k * b, "dR"),
                        range_of(dy, m * row, "dy"),
                        range_of(dinj, dinj ? span(M, ld_dinj, hc, b) : 0, "dinj"),
                        range_of(dw_post, dw_post ? (uint64_t)hs * 4 : 0, "dw_post"),
                        range_of(dw_pre, dw_pre ? (uint64_t)hs * 4 : 0, "dw_pre"),
                        range_of(ws, wneed, "workspace")};
  return check_overlaps(outs, 6, ins, 8);
}

hcgr_status quantize_checks(const hcgr_linear_config* c, const void* x, int64_t ld_x, int64_t M, const int8_t* q,
                            int64_t ld_q, const float* q_scale) {
  hcgr_status st = check_m(M);
  if (st != HCGR_OK || M == 0) return st;
  const size_t b = elem(c->dtype);
  const PtrCheck need[] = {{x, "x", b}, {q_scale, "q_scale", 4}};
  if ((st = check_ptrs(need, 2)) != HCGR_OK) return st;
  if ((st = check_ld(ld_x, c->k, "ld_x")) != HCGR_OK) return st;
  if ((st = check_int8(q, ld_q, c->k, "q", "ld_q")) != HCGR_OK) return st;
  const Range ins[] = {range_of(x, span(M, ld_x, c->k, b), "x")};
  const Range outs[] = {range_of(q, span(M, ld_q, c->k, 1), "q"), range_of(q_scale, (uint64_t)M * 4, "q_scale")};
  return check_overlaps(outs, 2, ins, 1);
}

hcgr_status linear_checks(const hcgr_linear_config* c, const int8_t* q, int64_t ld_q, const float* q_scale,
                          const int8_t* w, int64_t ld_w, const float* w_scale, const void* bias, int64_t M,
                          const void* out, int64_t ld_out) {
  hcgr_status st = check_m(M);
  if (st != HCGR_OK || M == 0) return st;
  const size_t b = elem(c->dtype);
  const PtrCheck need[] = {{q_scale, "q_scale", 4}, {w_scale, "w_scale", 4}, {out, "out", b}};
  if ((st = check_ptrs(need, 3)) != HCGR_OK) return st;
  if ((st = check_aligned(bias, "bias", b)) != HCGR_OK) return st;
  if ((st = check_int8(q, ld_q, c->k, "q", "ld_q")) != HCGR_OK) return st;
  if ((st = check_int8(w, ld_w, c->k, "w", "ld_w")) != HCGR_OK) return st;
  if (ld_q > HCGR_LINEAR_MAX_LD || ld_w > HCGR_LINEAR_MAX_LD)
    return fail(HCGR_ERR_UNSUPPORTED, "ld_q=%lld, ld_w=%lld: at most %d", (long long)ld_q, (long long)ld_w,
                HCGR_LINEAR_MAX_LD);
  if ((st = check_ld(ld_out, c->n, "ld_out")) != HCGR_OK) return st;
  const int64_t kr = ((int64_t)c->k + 15) / 16 * 16;  // bytes read of a row
  const Range ins[] = {range_of(q, span(M, ld_q, kr, 1), "q"),
                       range_of(w, span(c->n, ld_w, kr, 1), "w"),
                       range_of(q_scale, (uint64_t)M * 4, "q_scale"),
                       range_of(w_scale, (uint64_t)c->n * 4, "w_scale"),
                       range_of(bias, bias ? (uint64_t)c->n * b : 0, "bias")};
  const Range outs[] = {range_of(out, span(M, ld_out, c->n, b), "out")};
  return check_overlaps(outs, 1, ins, 5);
}

// Runs `launch` (which enqueues on `stream` and returns a hipError_t) with
// the handle's device current.
template <typename F>
hcgr_status on_device(int device, void* stream, F launch) {
  int cur = -1;
  const hcgr_status st = enter_device(device, stream, &cur);
  if (st != HCGR_OK) return st;
  const int le = launch();
  restore_device(device, cur);
  if (le != (int)hipSuccess)
    return fail(HCGR_ERR_HIP, "kernel launch failed: %s", hipGetErrorString((hipError_t)le));
  return ok();
}

// Sets the kernels' attributes on `device`.
hcgr_status configure(int device, int (*set)()) {
  int cur = -1;
  hipError_t e = hipGetDevice(&cur);
  if (e != hipSuccess) return fail(HCGR_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (cur != device && (e = hipSetDevice(device)) != hipSuccess)
    return fail(HCGR_ERR_HIP, "hipSetDevice: %s", hipGetErrorString(e));
  const int ke = set();
  restore_device(device, cur);
  if (ke != (int)hipSuccess)
    return fail(HCGR_ERR_HIP, "kernel attribute set-up failed: %s", hipGetErrorString((hipError_t)ke));
  return HCGR_OK;
}

}  // namespace

extern "C" {

hcgr_status hcgr_block_create(const hcgr_block_config* cfg, int device, hcgr_block_handle* out) {
  if (!out) return fail(HCGR_ERR_INVALID_ARGUMENT, "out is NULL");
  *out = nullptr;
  hcgr_status st = check_block(cfg);
  if (st != HCGR_OK) return st;
  if ((st = check_device(device)) != HCGR_OK) return st;
  if ((st = configure(device, hcgr::configure_block_kernels)) != HCGR_OK) return st;
  hcgr_block_op* op = new (std::nothrow) hcgr_block_op;
  if (!op) return fail(HCGR_ERR_INVALID_ARGUMENT, "out of host memory");
  op->cfg = *cfg;
  op->device = device;
  *out = op;
  return ok();
}

void hcgr_block_destroy(hcgr_block_handle h) { delete h; }

hcgr_status hcgr_block_workspace_size_for(const hcgr_block_config* cfg, int64_t M, size_t* bytes) {
  hcgr_status st = check_block(cfg);
  if (st != HCGR_OK) return st;
  if (!bytes) return fail(HCGR_ERR_INVALID_ARGUMENT, "bytes is NULL");
  if ((st = check_m(M)) != HCGR_OK) return st;
  *bytes = hcgr::norm_bwd_workspace(cfg->hs, M);
  return ok();
}

hcgr_status hcgr_block_workspace_size(hcgr_block_handle h, int64_t M, size_t* bytes) {
  if (!h) return fail(HCGR_ERR_INVALID_ARGUMENT, "handle is NULL");
  return hcgr_block_workspace_size_for(&h->cfg, M, bytes);
}

hcgr_status hcgr_validate_block_norm(const hcgr_block_config* cfg, const void* x, int64_t ld_x, const void* w,
                                     int64_t M, const void* xn, const int8_t* q, int64_t ld_q,
                                     const float* q_scale, const float* rrms) {
  hcgr_status st = check_block(cfg);
  if (st == HCGR_OK) st = norm_checks(cfg, x, ld_x, w, M, xn, q, ld_q, q_scale, rrms);
  return st == HCGR_OK ? ok() : st;
}

hcgr_status hcgr_block_norm(hcgr_block_handle h, const void* x, int64_t ld_x, const void* w, int64_t M, void* xn,
                            int8_t* q, int64_t ld_q, float* q_scale, float* rrms, void* stream) {
  if (!h) return fail(HCGR_ERR_INVALID_ARGUMENT, "handle is NULL");
  const hcgr_block_config& c = h->cfg;
  const hcgr_status st = norm_checks(&c, x, ld_x, w, M, xn, q, ld_q, q_scale, rrms);
  if (st != HCGR_OK) return st;
  if (M == 0) return ok();
  hcgr::NormArgs a{};
  a.R = x; a.w_pre = w; a.ld_R = ld_x; a.M = M; a.hs = c.hs; a.hc = 1; a.eps = c.eps; a.rho = 1.0f;
  a.x = xn; a.q = q; a.ld_q = ld_q; a.q_scale = q_scale; a.rr_pre = rrms; a.rr_ld = 1;
  return on_device(h->device, stream, [&] { return hcgr::launch_norm(a, c.dtype, false, stream); });
}

hcgr_status hcgr_validate_block_norm_bwd(const hcgr_block_config* cfg, const void* x, int64_t ld_x, const void* w,
                                         const float* rrms, const void* dxn, int64_t M, const void* dx,
                                         const float* dw, const void* workspace, size_t workspace_bytes) {
  hcgr_status st = check_block(cfg);
  if (st == HCGR_OK) st = norm_bwd_checks(cfg, x, ld_x, w, rrms, dxn, M, dx, dw, workspace, workspace_bytes);
  return st == HCGR_OK ? ok() : st;
}

hcgr_status hcgr_block_norm_bwd(hcgr_block_handle h, const void* x, int64_t ld_x, const void* w, const float* rrms,
                                const void* dxn, int64_t M, void* dx, float* dw, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!h) return fail(HCGR_ERR_INVALID_ARGUMENT, "handle is NULL");
  const hcgr_block_config& c = h->cfg;
  const hcgr_status st = norm_bwd_checks(&c, x, ld_x, w, rrms, dxn, M, dx, dw, workspace, workspace_bytes);
  if (st != HCGR_OK) return st;
  if (M == 0) return ok();
  hcgr::NormBwdArgs a{};
  a.R = x; a.w_pre = w; a.dx = dxn; a.ld_R = ld_x; a.M = M; a.hs = c.hs; a.hc = 1; a.rho = 1.0f;
  a.rr_pre = rrms; a.rr_ld = 1; a.dR = dx; a.dw_pre = dw; a.ws = workspace;
  return on_device(h->device, stream, [&] { return hcgr::launch_norm_bwd(a, c.dtype, false, stream); });
}

hcgr_status hcgr_validate_block_residual(const hcgr_block_config* cfg, const void* R, const void* y, int64_t ld_y,
                                         const void* inj, int64_t ld_inj, const void* w_post, const void* w_pre,
                                         int64_t M, const void* R2, const void* x, const int8_t* q, int64_t ld_q,
                                         const float* q_scale, const float* rrms) {
  hcgr_status st = check_block(cfg);
  if (st == HCGR_OK)
    st = residual_checks(cfg, R, y, ld_y, inj, ld_inj, w_post, w_pre, M, R2, x, q, ld_q, q_scale, rrms);
  return st == HCGR_OK ? ok() : st;
}

hcgr_status hcgr_block_residual(hcgr_block_handle h, const void* R, const void* y, int64_t ld_y, const void* inj,
                                int64_t ld_inj, const void* w_post, const void* w_pre, int64_t M, void* R2, void* x,
                                int8_t* q, int64_t ld_q, float* q_scale, float* rrms, void* stream) {
  if (!h) return fail(HCGR_ERR_INVALID_ARGUMENT, "handle is NULL");
  const hcgr_block_config& c = h->cfg;
  const hcgr_status st =
      residual_checks(&c, R, y, ld_y, inj, ld_inj, w_post, w_pre, M, R2, x, q, ld_q, q_scale, rrms);
  if (st != HCGR_OK) return st;
  if (M == 0) return ok();
  hcgr::NormArgs a{};
  a.R = R; a.y = y; a.inj = inj; a.w_post = w_post; a.w_pre = w_pre;
  a.ld_R = (int64_t)c.hc * c.hs; a.ld_y = ld_y; a.ld_inj = ld_inj; a.M = M;
  a.hs = c.hs; a.hc = c.hc; a.eps = c.eps; a.rho = c.res_scale;
  a.R2 = R2; a.x = x; a.q = q; a.ld_q = ld_q; a.q_scale = q_scale; a.rr_ld = 2;
  if (rrms) {
    a.rr_post = rrms;
    a.rr_pre = rrms + 1;
  }
  return on_device(h->device, stream, [&] { return hcgr::launch_norm(a, c.dtype, true, stream); });
}

hcgr_status hcgr_validate_block_residual_bwd(const hcgr_block_config* cfg, const void* R, const void* y,
                                             int64_t ld_y, const void* inj, int64_t ld_inj, const void* w_post,
                                             const void* w_pre, const float* rrms, const void* dR2, const void* dx,
                                             int64_t M, const void* dR, const void* dy, const void* dinj,
                                             int64_t ld_dinj, const float* dw_post, const float* dw_pre,
                                             const void* workspace, size_t workspace_bytes) {
  hcgr_status st = check_block(cfg);
  if (st == HCGR_OK)
    st = residual_bwd_checks(cfg, R, y, ld_y, inj, ld_inj, w_post, w_pre, rrms, dR2, dx, M, dR, dy, dinj, ld_dinj,
                             dw_post, dw_pre, workspace, workspace_bytes);
  return st == HCGR_OK ? ok() : st;
}

hcgr_status hcgr_block_residual_bwd(hcgr_block_handle h, const void* R, const void* y, int64_t ld_y,
                                    const void* inj, int64_t ld_inj, const void* w_post, const void* w_pre,
                                    const float* rrms, const void* dR2, const void* dx, int64_t M, void* dR,
                                    void* dy, void* dinj, int64_t ld_dinj, float* dw_post, float* dw_pre,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!h) return fail(HCGR_ERR_INVALID_ARGUMENT, "handle is NULL");
  const hcgr_block_config& c = h->cfg;
  const hcgr_status st = residual_bwd_checks(&c, R, y, ld_y, inj, ld_inj, w_post, w_pre, rrms, dR2, dx, M, dR, dy,
                                             dinj, ld_dinj, dw_post, dw_pre, workspace, workspace_bytes);
  if (st != HCGR_OK) return st;
  if (M == 0) return ok();
  hcgr::NormBwdArgs a{};
  a.R = R; a.y = y; a.inj = inj; a.w_post = w_post; a.w_pre = w_pre; a.dR2 = dR2; a.dx = dx;
  a.ld_R = (int64_t)c.hc * c.hs; a.ld_y = ld_y; a.ld_inj = ld_inj; a.ld_dinj = ld_dinj; a.M = M;
  a.hs = c.hs; a.hc = c.hc; a.rho = c.res_scale;
  a.rr_ld = 2;
  if (rrms) {
    a.rr_post = rrms;
    a.rr_pre = rrms + 1;
  }
  a.dR = dR; a.dy = dy; a.dinj = dinj; a.dw_post = dw_post; a.dw_pre = dw_pre; a.ws = workspace;
  return on_device(h->device, stream, [&] { return hcgr::launch_norm_bwd(a, c.dtype, true, stream); });
}

hcgr_status hcgr_linear_create(const hcgr_linear_config* cfg, int device, hcgr_linear_handle* out) {
  if (!out) return fail(HCGR_ERR_INVALID_ARGUMENT, "out is NULL");
  *out = nullptr;
  hcgr_status st = check_linear(cfg);
  if (st != HCGR_OK) return st;
  if ((st = check_device(device)) != HCGR_OK) return st;
  if ((st = configure(device, hcgr::configure_linear_kernels)) != HCGR_OK) return st;
  hcgr_linear_op* op = new (std::nothrow) hcgr_linear_op;
  if (!op) return fail(HCGR_ERR_INVALID_ARGUMENT, "out of host memory");
  op->cfg = *cfg;
  op->device = device;
  *out = op;
  return ok();
}

void hcgr_linear_destroy(hcgr_linear_handle h) { delete h; }

hcgr_status hcgr_validate_linear_quantize(const hcgr_linear_config* cfg, const void* x, int64_t ld_x, int64_t M,
                                          const int8_t* q, int64_t ld_q, const float* q_scale) {
  hcgr_status st = check_linear(cfg);
  if (st == HCGR_OK) st = quantize_checks(cfg, x, ld_x, M, q, ld_q, q_scale);
  return st == HCGR_OK ? ok() : st;
}

hcgr_status hcgr_linear_quantize(hcgr_linear_handle h, const void* x, int64_t ld_x, int64_t M, int8_t* q,
                                 int64_t ld_q, float* q_scale, void* stream) {
  if (!h) return fail(HCGR_ERR_INVALID_ARGUMENT, "handle is NULL");
  const hcgr_linear_config& c = h->cfg;
  const hcgr_status st = quantize_checks(&c, x, ld_x, M, q, ld_q, q_scale);
  if (st != HCGR_OK) return st;
  if (M == 0) return ok();
  hcgr::NormArgs a{};
  a.R = x; a.ld_R = ld_x; a.M = M; a.hs = c.k; a.hc = 1; a.q = q; a.ld_q = ld_q; a.q_scale = q_scale;
  return on_device(h->device, stream, [&] { return hcgr::launch_quantize(a, c.dtype, stream); });
}

hcgr_status hcgr_validate_linear_forward(const hcgr_linear_config* cfg, const int8_t* q, int64_t ld_q,
                                         const float* q_scale, const int8_t* w, int64_t ld_w, const float* w_scale,
                                         const void* bias, int64_t M, const void* out, int64_t ld_out) {
  hcgr_status st = check_linear(cfg);
  if (st == HCGR_OK) st = linear_checks(cfg, q, ld_q, q_scale, w, ld_w, w_scale, bias, M, out, ld_out);
  return st == HCGR_OK ? ok() : st;
}

hcgr_status hcgr_linear_forward(hcgr_linear_handle h, const int8_t* q, int64_t ld_q, const float* q_scale,
                                const int8_t* w, int64_t ld_w, const float* w_scale, const void* bias, int64_t M,
                                void* out, int64_t ld_out, void* stream) {
  if (!h) return fail(HCGR_ERR_INVALID_ARGUMENT, "handle is NULL");
  const hcgr_linear_config& c = h->cfg;
  const hcgr_status st = linear_checks(&c, q, ld_q, q_scale, w, ld_w, w_scale, bias, M, out, ld_out);
  if (st != HCGR_OK) return st;
  if (M == 0) return ok();
  hcgr::LinearArgs a{};
  a.q = q; a.w = w; a.q_scale = q_scale; a.w_scale = w_scale; a.bias = bias; a.out = out;
  a.ld_q = ld_q; a.ld_w = ld_w; a.ld_out = ld_out; a.M = M; a.n = c.n; a.k = c.k;
  return on_device(h->device, stream, [&] { return hcgr::launch_linear(a, c.dtype, stream); });
}

}  // extern "C"
