// extern "C" entry points of the operators around the FFN: dropout, residual
// addition with RMS norm, 4-bit products. Argument checks and launch order;
// declared and documented in include/twell.h.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/twell.h"
#include "twell_internal.hpp"

using twell::align256;

namespace {

// Every grid of these shapes stays under the 2^32 threads that a launch holds in a
// dimension (the norm's forward, of up to 1024 threads a row, by a second one).
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxN = int64_t(1) << 24;
constexpr int64_t kMaxK = int64_t(1) << 24;
constexpr int64_t kMaxQ4Rows = int64_t(1) << 18;

bool float_type(int32_t t) { return t == TWELL_BF16 || t == TWELL_F32; }

int hip_status(hipError_t e) { return e == hipSuccess ? TWELL_OK : TWELL_E_HIP; }

bool make_dropout(double p, uint64_t seed, uint64_t offset, twell::Dropout* out) {
  if (!(p >= 0.0 && p < 1.0)) return false;
  const double t = floor(p * 65536.0 + 0.5);
  if (t > 65535.0) return false;
  out->seed_lo = uint32_t(seed);
  out->seed_hi = uint32_t(seed >> 32);
  out->off_lo = uint32_t(offset);
  out->off_hi = uint32_t(offset >> 32);
  out->threshold = uint32_t(t);
  out->scale = float(65536.0 / (65536.0 - t));
  return true;
}

int check_rows(int64_t M, int64_t d, int64_t max_d) {
  if (M < 0 || d <= 0) return TWELL_E_INVALID_ARG;
  if (M > kMaxRows || d > max_d) return TWELL_E_UNSUPPORTED;
  return TWELL_OK;
}

bool q4_ok(const twell_q4* w) { return w && w->codes && w->scales; }

twell::Q4Weight q4_weight(const twell_q4* w) { return {w->codes, w->scales, w->zeros}; }

int check_q4(int64_t M, int64_t N, int64_t K, int32_t group) {
  if (M < 0 || N <= 0 || K <= 0) return TWELL_E_INVALID_ARG;
  if (M > kMaxQ4Rows || N > kMaxN || K > kMaxK || M * N > (int64_t(1) << 33)) return TWELL_E_UNSUPPORTED;
  if (group != 32 && group != 64 && group != 128) return TWELL_E_UNSUPPORTED;
  return TWELL_OK;
}

bool q4_x_type(int32_t t) { return t == TWELL_BF16 || t == TWELL_F32 || t == TWELL_E4M3; }

int check_q4_x(const void* x, int32_t x_type, const float* x_scale) {
  if (!q4_x_type(x_type)) return TWELL_E_UNSUPPORTED;
  if (!x || (x_type == TWELL_E4M3) != (x_scale != nullptr)) return TWELL_E_INVALID_ARG;
  return TWELL_OK;
}

twell::Q4X q4_x(int32_t t) {
  return t == TWELL_BF16 ? twell::Q4X::bf16 : t == TWELL_F32 ? twell::Q4X::f32 : twell::Q4X::e4m3;
}

twell::Q4Y q4_y(int32_t t) { return t == TWELL_F32 ? twell::Q4Y::f32 : twell::Q4Y::bf16; }

int check_ws(void* ws, size_t bytes, size_t need) {
  if (need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < need)) return TWELL_E_WORKSPACE;
  return TWELL_OK;
}

// One product (Wu null) or the gated pair, arguments checked.
int q4(const void* x, int32_t x_type, const float* x_scale, const twell_q4* W, const twell_q4* Wu, int64_t M,
       int64_t N, int64_t K, int32_t group, void* y, twell::Q4Y y_type, void* workspace, void* stream) {
  const twell::Q4Args a{x,      x_scale, q4_weight(W), Wu ? q4_weight(Wu) : twell::Q4Weight{}, Wu != nullptr, int(M),
                        int(N), int(K),  group,        y,                                      y_type};
  return hip_status(twell::launch_q4(a, q4_x(x_type), workspace, static_cast<hipStream_t>(stream)));
}

// The FFN's hidden matrix: three bf16 planes.
size_t hidden_bytes(int64_t M, int64_t F) { return align256(size_t(twell::q4_rows(M)) * size_t(twell::q4_pad(F)) * 6); }

}  // namespace

extern "C" {

int twell_dropout(const void* x, int32_t x_type, const void* residual, int64_t M, int64_t d, double p, uint64_t seed,
                  uint64_t offset, void* y, int32_t y_type, void* stream) {
  twell::DropoutArgs a;
  int st = check_rows(M, d, kMaxK);
  if (st != TWELL_OK) return st;
  if (!float_type(x_type) || !float_type(y_type)) return TWELL_E_UNSUPPORTED;
  if (!make_dropout(p, seed, offset, &a.drop)) return TWELL_E_INVALID_ARG;
  if (M == 0) return TWELL_OK;
  if (M * ((d + 7) / 8) > (int64_t(1) << 33)) return TWELL_E_UNSUPPORTED;
  if (!x || !y) return TWELL_E_INVALID_ARG;
  a.x = x;
  a.residual = residual;
  a.M = M;
  a.d = int(d);
  a.y = y;
  return hip_status(
      twell::launch_dropout(a, x_type == TWELL_F32, y_type == TWELL_F32, static_cast<hipStream_t>(stream)));
}

int twell_add_rmsnorm(const void* x, int32_t x_type, const void* residual, const void* weight, int32_t w_type,
                      int64_t M, int64_t d, double eps, double p, uint64_t seed, uint64_t offset, void* h,
                      int32_t h_type, void* out, int32_t out_type, float* out_scale, float* rstd, void* stream) {
  twell::NormArgs a;
  int st = check_rows(M, d, twell::kNormMaxD);
  if (st != TWELL_OK) return st;
  if (!float_type(x_type) || !float_type(w_type) || !float_type(h_type)) return TWELL_E_UNSUPPORTED;
  if (out_type != TWELL_BF16 && out_type != TWELL_E4M3) return TWELL_E_UNSUPPORTED;
  if (!(eps >= 0.0) || isinf(eps)) return TWELL_E_INVALID_ARG;
  if (!make_dropout(p, seed, offset, &a.drop)) return TWELL_E_INVALID_ARG;
  if (M == 0) return TWELL_OK;
  if (!x || !weight || !out || (out_type == TWELL_E4M3) != (out_scale != nullptr)) return TWELL_E_INVALID_ARG;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.w_f32 = w_type == TWELL_F32;
  a.M = M;
  a.d = int(d);
  a.eps = float(eps);
  a.h = h;
  a.out = out;
  a.out_scale = out_scale;
  a.rstd = rstd;
  return hip_status(twell::launch_add_rmsnorm(a, x_type == TWELL_F32, h_type == TWELL_F32, out_type == TWELL_E4M3,
                                              static_cast<hipStream_t>(stream)));
}

size_t twell_rmsnorm_workspace_bytes(int64_t M, int64_t d) {
  if (check_rows(M, d, twell::kNormMaxD) != TWELL_OK || M == 0) return 0;
  return align256(size_t(twell::norm_backward_groups(M, d)) * size_t(d) * 4);
}

int twell_add_rmsnorm_backward(const void* dout, int32_t g_type, const void* dh, const void* h, int32_t h_type,
                               const void* weight, int32_t w_type, const float* rstd, int64_t M, int64_t d, double p,
                               uint64_t seed, uint64_t offset, void* dres, void* dx, int32_t dx_type, float* dweight,
                               void* workspace, size_t ws_bytes, void* stream) {
  twell::NormBackwardArgs a;
  int st = check_rows(M, d, twell::kNormMaxD);
  if (st != TWELL_OK) return st;
  if (!float_type(g_type) || !float_type(h_type) || !float_type(w_type) || !float_type(dx_type))
    return TWELL_E_UNSUPPORTED;
  if (!make_dropout(p, seed, offset, &a.drop)) return TWELL_E_INVALID_ARG;
  if (!weight || !dweight) return TWELL_E_INVALID_ARG;
  if (M > 0) {
    if (!dout || !h || !rstd || (!dres && !dx)) return TWELL_E_INVALID_ARG;
    if ((st = check_ws(workspace, ws_bytes, twell_rmsnorm_workspace_bytes(M, d))) != TWELL_OK) return st;
  }
  a.dout = dout;
  a.dh = dh;
  a.h = h;
  a.weight = weight;
  a.w_f32 = w_type == TWELL_F32;
  a.rstd = rstd;
  a.M = M;
  a.d = int(d);
  a.dres = dres;
  a.dx = dx;
  a.part = static_cast<float*>(workspace);
  return hip_status(twell::launch_add_rmsnorm_backward(a, g_type == TWELL_F32, h_type == TWELL_F32,
                                                       dx_type == TWELL_F32, dweight,
                                                       static_cast<hipStream_t>(stream)));
}

int twell_q4_quantize(const uint16_t* W, int64_t N, int64_t K, int32_t group, uint8_t* codes, uint16_t* scales,
                      void* stream) {
  const int st = check_q4(0, N, K, group);
  if (st != TWELL_OK) return st;
  if (N * ((K + group - 1) / group) * (group / 8) > (int64_t(1) << 31)) return TWELL_E_UNSUPPORTED;
  if (!W || !codes || !scales) return TWELL_E_INVALID_ARG;
  return hip_status(
      twell::launch_q4_quantize(W, int(N), int(K), group, codes, scales, static_cast<hipStream_t>(stream)));
}

size_t twell_q4_workspace_bytes(int32_t x_type, int64_t M, int64_t N, int64_t K, int32_t gated) {
  if (check_q4(M, N, K, 32) != TWELL_OK || M == 0 || !q4_x_type(x_type)) return 0;
  return twell::q4_workspace_bytes(q4_x(x_type), gated != 0, M, N, K);
}

int twell_q4_matmul(const void* x, int32_t x_type, const float* x_scale, const twell_q4* W, int64_t M, int64_t N,
                    int64_t K, int32_t group, void* y, int32_t y_type, void* workspace, size_t ws_bytes,
                    void* stream) {
  int st = check_q4(M, N, K, group);
  if (st != TWELL_OK) return st;
  if (!float_type(y_type)) return TWELL_E_UNSUPPORTED;
  if (M == 0) return TWELL_OK;
  if ((st = check_q4_x(x, x_type, x_scale)) != TWELL_OK) return st;
  if (!q4_ok(W) || !y) return TWELL_E_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, twell_q4_workspace_bytes(x_type, M, N, K, 0))) != TWELL_OK) return st;
  return q4(x, x_type, x_scale, W, nullptr, M, N, K, group, y, q4_y(y_type), workspace, stream);
}

int twell_q4_gateup(const void* x, int32_t x_type, const float* x_scale, const twell_q4* Wg, const twell_q4* Wu,
                    int64_t M, int64_t F, int64_t d, int32_t group, void* h, int32_t h_type, void* workspace,
                    size_t ws_bytes, void* stream) {
  int st = check_q4(M, F, d, group);
  if (st != TWELL_OK) return st;
  if (!float_type(h_type)) return TWELL_E_UNSUPPORTED;
  if (M == 0) return TWELL_OK;
  if ((st = check_q4_x(x, x_type, x_scale)) != TWELL_OK) return st;
  if (!q4_ok(Wg) || !q4_ok(Wu) || !h) return TWELL_E_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, twell_q4_workspace_bytes(x_type, M, F, d, 1))) != TWELL_OK) return st;
  return q4(x, x_type, x_scale, Wg, Wu, M, F, d, group, h, q4_y(h_type), workspace, stream);
}

size_t twell_ffn_q4_workspace_bytes(int32_t x_type, int64_t M, int64_t d, int64_t F) {
  if (check_q4(M, F, d, 32) != TWELL_OK || check_q4(M, d, F, 32) != TWELL_OK || M == 0 || !q4_x_type(x_type)) return 0;
  return hidden_bytes(M, F) + std::max(twell::q4_workspace_bytes(q4_x(x_type), true, M, F, d),
                                       twell::q4_workspace_bytes(twell::Q4X::planes, false, M, d, F));
}

int twell_ffn_forward_q4(const void* x, int32_t x_type, const float* x_scale, const twell_q4* Wg, const twell_q4* Wu,
                         const twell_q4* Wd, int64_t M, int64_t d, int64_t F, int32_t group, float* y, void* workspace,
                         size_t ws_bytes, void* stream) {
  int st = check_q4(M, F, d, group);
  if (st == TWELL_OK) st = check_q4(M, d, F, group);
  if (st != TWELL_OK) return st;
  if (M == 0) return TWELL_OK;
  if ((st = check_q4_x(x, x_type, x_scale)) != TWELL_OK) return st;
  if (!q4_ok(Wg) || !q4_ok(Wu) || !q4_ok(Wd) || !y) return TWELL_E_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, twell_ffn_q4_workspace_bytes(x_type, M, d, F))) != TWELL_OK) return st;
  void* rest = static_cast<uint8_t*>(workspace) + hidden_bytes(M, F);
  st = q4(x, x_type, x_scale, Wg, Wu, M, F, d, group, workspace, twell::Q4Y::planes, rest, stream);
  if (st != TWELL_OK) return st;
  const twell::Q4Args down{workspace, nullptr, q4_weight(Wd), {}, false, int(M), int(d), int(F), group, y,
                           twell::Q4Y::f32};
  return hip_status(twell::launch_q4(down, twell::Q4X::planes, rest, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
