// extern "C" entry points of the operators around the FFN: dropout, residual
// addition with RMS or layer norm, 4-bit products and the adapters beside them,
// the gradients' norm and the optimizer's step. Argument checks and launch
// order; declared and documented in include/twell.h.
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

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
constexpr int64_t kMaxLoraN = int64_t(1) << 22;
constexpr int64_t kMaxElements = int64_t(1) << 34;  // of a tensor of a step

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

int check_lora(int64_t M, int64_t K, int64_t R) {
  if (M < 0 || K <= 0 || R <= 0) return TWELL_E_INVALID_ARG;
  if (M > kMaxQ4Rows || K > kMaxK || R > twell::kLoraMaxRank) return TWELL_E_UNSUPPORTED;
  return TWELL_OK;
}

int check_grads(const twell_grad* grads, int64_t count) {
  if (count < 0 || (count > 0 && !grads)) return TWELL_E_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (grads[i].n < 0 || (grads[i].n > 0 && !grads[i].g)) return TWELL_E_INVALID_ARG;
    if (grads[i].n > kMaxElements || !float_type(grads[i].g_type)) return TWELL_E_UNSUPPORTED;
  }
  return TWELL_OK;
}

int64_t chunks_of(int64_t n, int chunk) { return (n + chunk - 1) / chunk; }

bool not_negative(double v) { return v >= 0.0 && !isinf(v); }

// The largest fp32 at or below v >= 0.
float round_down(double v) {
  const float f = float(v);
  return double(f) > v ? nextafterf(f, 0.f) : f;
}

// Below a half both coefficients to nearest: beta rounded down would be up to 2^-23 of itself off, and what the two of
// them leave is at most 2^-24 of 1 - beta.
twell::Decay decay_of(double beta) {
  if (beta < 0.5) return {float(beta), FLT_TRUE_MIN, float(1.0 - beta)};
  const float b = round_down(beta), c = round_down(1.0 - beta);
  return {b, std::max(float((1.0 - b) - c), FLT_TRUE_MIN), c};
}

// ------------------------------------------------ places that overlap
// Bytes that a call reads or writes; tensor: whose they are.
struct Span {
  uintptr_t from, to;
  int64_t tensor;
};
Span span(const void* p, double bytes, int64_t tensor = 0) {  // (double: past any address, not past the range)
  const uintptr_t from = reinterpret_cast<uintptr_t>(p);
  return {from, from + uintptr_t(std::min(bytes, 0x1p62)), tensor};
}
bool overlap(const Span& a, const Span& b) { return a.from < b.to && b.from < a.to; }

// Whether what a tensor of the step writes is written or read by another one, or in part by itself: of two workgroups
// that meet in a place either may come first. An old value or gradient may lie exactly where the same tensor
// writes, as a thread reads its elements before it writes them. Returns TWELL_OK, TWELL_E_INVALID_ARG, or
// TWELL_E_WORKSPACE where there is no memory to sort them.
int check_places(const twell_adamw_tensor* tensors, int64_t count, bool e4m3, const float* grad_scale) {
  constexpr int kMost = 6;  // places that a tensor writes
  Span few[32 * kMost];
  Span* written = count <= 32 ? few : static_cast<Span*>(malloc(size_t(count) * kMost * sizeof(Span)));
  if (written == nullptr) return TWELL_E_WORKSPACE;
  const double state = e4m3 ? 1.0 : 4.0;
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    const twell_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const double size = double(t.n);
    written[n++] = span(t.p_out, 4.0 * size, i);
    written[n++] = span(t.m_out, state * size, i);
    written[n++] = span(t.v_out, state * size, i);
    if (t.copy) written[n++] = span(t.copy, 2.0 * size, i);
    if (!e4m3) continue;
    const double scales = 4.0 * double(chunks_of(t.n, twell::kStateBlock));
    written[n++] = span(t.m_scale_out, scales, i);
    written[n++] = span(t.v_scale_out, scales, i);
  }
  std::sort(written, written + n, [](const Span& a, const Span& b) { return a.from < b.from; });
  bool meet = false;
  for (int64_t k = 1; k < n; ++k) meet = meet || overlap(written[k - 1], written[k]);
  // The written ones are apart from here on, so one that a place meets is the last that begins before its end, or that
  // place is not exactly one of them.
  auto reads = [&](const void* p, double bytes, int64_t tensor) {
    const Span r = span(p, bytes, tensor);
    const Span* w = std::lower_bound(written, written + n, r.to, [](const Span& a, uintptr_t to) { return a.from < to; });
    if (w == written || !overlap(*--w, r)) return;
    meet = meet || w->from != r.from || w->to != r.to || w->tensor != tensor;
  };
  for (int64_t i = 0; i < count && !meet; ++i) {
    const twell_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const double size = double(t.n), scales = 4.0 * double(chunks_of(t.n, twell::kStateBlock));
    reads(t.g, (t.g_type == TWELL_F32 ? 4.0 : 2.0) * size, i);
    if (t.p != t.p_out) reads(t.p, 4.0 * size, i);
    if (t.m != t.m_out) reads(t.m, state * size, i);
    if (t.v != t.v_out) reads(t.v, state * size, i);
    if (e4m3 && t.m_scale != t.m_scale_out) reads(t.m_scale, scales, i);
    if (e4m3 && t.v_scale != t.v_scale_out) reads(t.v_scale, scales, i);
  }
  if (grad_scale != nullptr && !meet) reads(grad_scale, 4.0, -1);
  if (written != few) free(written);
  return meet ? TWELL_E_INVALID_ARG : TWELL_OK;
}

// A launch's share of `count` tensors from `i` on: up to kStepTensors of them and 2^24 - 1 chunks, as 256
// threads each stay under the 2^32 of a launch. fill(slot, tensor) writes a slot of the table; `first` gets the
// chunks before each and is past every chunk behind the last. Returns the chunks.
template <class Size, class Fill>
int64_t fill_launch(int64_t* i, int64_t count, int chunk, int32_t* first, Size&& size, Fill&& fill) {
  int64_t chunks = 0;
  int slot = 0;
  for (; slot < twell::kStepTensors && *i < count; ++slot, ++*i) {
    const int64_t more = chunks_of(size(*i), chunk);
    if (chunks + more >= (int64_t(1) << 24)) break;
    first[slot] = int32_t(chunks);
    fill(slot, *i);
    chunks += more;
  }
  for (; slot < twell::kStepTensors; ++slot) first[slot] = INT32_MAX;
  return chunks;
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

int twell_add_layernorm(const void* x, int32_t x_type, const void* residual, const void* weight, const void* bias,
                        int32_t w_type, int64_t M, int64_t d, double eps, double p, uint64_t seed, uint64_t offset,
                        void* h, int32_t h_type, void* out, int32_t out_type, float* out_scale, float* mean,
                        float* rstd, void* stream) {
  twell::LayerNormArgs a;
  int st = check_rows(M, d, twell::kNormMaxD);
  if (st != TWELL_OK) return st;
  if (!float_type(x_type) || !float_type(w_type) || !float_type(h_type)) return TWELL_E_UNSUPPORTED;
  if (out_type != TWELL_BF16 && out_type != TWELL_E4M3) return TWELL_E_UNSUPPORTED;
  if (!not_negative(eps)) return TWELL_E_INVALID_ARG;
  if (!make_dropout(p, seed, offset, &a.drop)) return TWELL_E_INVALID_ARG;
  if (M == 0) return TWELL_OK;
  if (!x || !weight || !out || (out_type == TWELL_E4M3) != (out_scale != nullptr)) return TWELL_E_INVALID_ARG;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.w_f32 = w_type == TWELL_F32;
  a.bias = bias;
  a.M = M;
  a.d = int(d);
  a.eps = float(eps);
  a.h = h;
  a.out = out;
  a.out_scale = out_scale;
  a.mean = mean;
  a.rstd = rstd;
  return hip_status(twell::launch_add_layernorm(a, x_type == TWELL_F32, h_type == TWELL_F32, out_type == TWELL_E4M3,
                                                static_cast<hipStream_t>(stream)));
}

size_t twell_layernorm_workspace_bytes(int64_t M, int64_t d) {
  if (check_rows(M, d, twell::kNormMaxD) != TWELL_OK || M == 0) return 0;
  return align256(size_t(twell::layernorm_backward_groups(M, d)) * size_t(d) * 8);
}

int twell_add_layernorm_backward(const void* dout, int32_t g_type, const void* dh, const void* h, int32_t h_type,
                                 const void* weight, int32_t w_type, const float* mean, const float* rstd, int64_t M,
                                 int64_t d, double p, uint64_t seed, uint64_t offset, void* dres, void* dx,
                                 int32_t dx_type, float* dweight, float* dbias, void* workspace, size_t ws_bytes,
                                 void* stream) {
  twell::LayerNormBackwardArgs a;
  int st = check_rows(M, d, twell::kNormMaxD);
  if (st != TWELL_OK) return st;
  if (!float_type(g_type) || !float_type(h_type) || !float_type(w_type) || !float_type(dx_type))
    return TWELL_E_UNSUPPORTED;
  if (!make_dropout(p, seed, offset, &a.drop)) return TWELL_E_INVALID_ARG;
  if (!weight || !dweight) return TWELL_E_INVALID_ARG;
  if (M > 0) {
    if (!dout || !h || !mean || !rstd || (!dres && !dx)) return TWELL_E_INVALID_ARG;
    if ((st = check_ws(workspace, ws_bytes, twell_layernorm_workspace_bytes(M, d))) != TWELL_OK) return st;
  }
  a.dout = dout;
  a.dh = dh;
  a.h = h;
  a.weight = weight;
  a.w_f32 = w_type == TWELL_F32;
  a.mean = mean;
  a.rstd = rstd;
  a.M = M;
  a.d = int(d);
  a.dres = dres;
  a.dx = dx;
  a.part = static_cast<float*>(workspace);
  return hip_status(twell::launch_add_layernorm_backward(a, g_type == TWELL_F32, h_type == TWELL_F32,
                                                         dx_type == TWELL_F32, dweight, dbias,
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

int twell_lora(const void* x, int32_t x_type, const float* x_scale, const int32_t* index, const uint16_t* A,
               const uint16_t* B, const float* scaling, int64_t adapters, int64_t M, int64_t N, int64_t K, int64_t R,
               const void* base, void* y, int32_t y_type, void* stream) {
  const int st = check_lora(M, K, R);
  if (st != TWELL_OK) return st;
  if (N <= 0 || adapters < 0) return TWELL_E_INVALID_ARG;
  if (N > kMaxLoraN || M * N > (int64_t(1) << 33) || adapters > INT32_MAX || !float_type(y_type))
    return TWELL_E_UNSUPPORTED;
  if (M == 0) return TWELL_OK;
  if (const int bad = check_q4_x(x, x_type, x_scale); bad != TWELL_OK) return bad;
  if (!index || !base || !y || (adapters > 0 && (!A || !B))) return TWELL_E_INVALID_ARG;
  // A workgroup writes its part of y while others read all of x and their own rows of base.
  const auto bytes = [](int32_t t) { return t == TWELL_F32 ? 4.0 : t == TWELL_BF16 ? 2.0 : 1.0; };
  const double m = double(M), n = double(adapters);
  const Span out = span(y, m * double(N) * bytes(y_type));
  if ((y != base && overlap(out, span(base, m * double(N) * bytes(y_type)))) ||
      overlap(out, span(x, m * double(K) * bytes(x_type))) || overlap(out, span(index, 4.0 * m)) ||
      (x_scale && overlap(out, span(x_scale, 4.0 * m))) ||
      (adapters > 0 && (overlap(out, span(A, 2.0 * n * double(R) * double(K))) ||
                        overlap(out, span(B, 2.0 * n * double(N) * double(R))) ||
                        (scaling && overlap(out, span(scaling, 4.0 * n))))))
    return TWELL_E_INVALID_ARG;
  twell::LoraArgs a;
  a.x = x;
  a.x_scale = x_scale;
  a.index = index;
  a.A = A;
  a.B = B;
  a.scaling = scaling;
  a.n = int(adapters);
  a.M = int(M);
  a.N = int(N);
  a.K = int(K);
  a.R = int(R);
  a.base = base;
  a.y = y;
  const twell::LoraX t = x_type == TWELL_BF16  ? twell::LoraX::bf16
                         : x_type == TWELL_F32 ? twell::LoraX::f32
                                               : twell::LoraX::e4m3;
  return hip_status(twell::launch_lora(a, t, y_type == TWELL_F32, static_cast<hipStream_t>(stream)));
}

size_t twell_grad_norm_workspace_bytes(const twell_grad* grads, int64_t count) {
  if (check_grads(grads, count) != TWELL_OK) return 0;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) chunks += chunks_of(grads[i].n, twell::kNormChunk);
  return align256(size_t(chunks) * 8);
}

int twell_grad_norm(const twell_grad* grads, int64_t count, double max_norm, float* out, void* workspace,
                    size_t ws_bytes, void* stream) {
  int st = check_grads(grads, count);
  if (st != TWELL_OK) return st;
  if (!(max_norm > 0.0) || !out) return TWELL_E_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, twell_grad_norm_workspace_bytes(grads, count))) != TWELL_OK) return st;
  double* part = static_cast<double*>(workspace);
  int64_t done = 0;
  for (int64_t i = 0; i < count;) {
    twell::GradNormArgs a = {};
    a.part = part + done;
    const int64_t chunks = fill_launch(
        &i, count, twell::kNormChunk, a.first, [&](int64_t k) { return grads[k].n; },
        [&](int slot, int64_t k) { a.tensor[slot] = {grads[k].g, grads[k].n, grads[k].g_type == TWELL_F32}; });
    if (chunks > 0) {
      const hipError_t e = twell::launch_grad_norm(a, chunks, static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return TWELL_E_HIP;
    }
    done += chunks;
  }
  return hip_status(twell::launch_grad_norm_join(part, done, max_norm, out, static_cast<hipStream_t>(stream)));
}

int twell_adamw(const twell_adamw_tensor* tensors, int64_t count, int32_t state_type, int64_t step, double lr,
                double beta1, double beta2, double eps, const float* grad_scale, uint64_t seed, uint64_t offset,
                void* stream) {
  if (count < 0 || (count > 0 && !tensors) || step < 1) return TWELL_E_INVALID_ARG;
  if (!not_negative(lr) || !not_negative(eps) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
    return TWELL_E_INVALID_ARG;
  if (state_type != TWELL_F32 && state_type != TWELL_E4M3) return TWELL_E_UNSUPPORTED;
  const bool e4m3 = state_type == TWELL_E4M3;
  int64_t elements = 0;
  for (int64_t i = 0; i < count; ++i) {
    const twell_adamw_tensor& t = tensors[i];
    if (t.n < 0 || !not_negative(t.weight_decay)) return TWELL_E_INVALID_ARG;
    if (t.n > kMaxElements || !float_type(t.g_type)) return TWELL_E_UNSUPPORTED;
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || !t.p_out || !t.m_out || !t.v_out) return TWELL_E_INVALID_ARG;
    if (e4m3 != (t.m_scale != nullptr) || e4m3 != (t.v_scale != nullptr) || e4m3 != (t.m_scale_out != nullptr) ||
        e4m3 != (t.v_scale_out != nullptr))
      return TWELL_E_INVALID_ARG;
    elements += t.n;
  }
  if (const int bad = check_places(tensors, count, e4m3, grad_scale); bad != TWELL_OK) return bad;
  twell::AdamwArgs a = {};
  make_dropout(0.0, seed, offset, &a.random);
  a.grad_scale = grad_scale;
  a.mean = decay_of(beta1);
  a.square = decay_of(beta2);
  a.rate = float(lr / (1.0 - pow(beta1, double(step))));
  a.root = float(1.0 / sqrt(1.0 - pow(beta2, double(step))));
  a.eps = float(eps);
  a.stream = elements * 8 >= (int64_t(32) << 20);
  for (int64_t i = 0; i < count;) {
    a.number = int32_t(i);
    const int64_t chunks = fill_launch(
        &i, count, twell::kStepChunk, a.first, [&](int64_t k) { return tensors[k].n; },
        [&](int slot, int64_t k) {
          const twell_adamw_tensor& t = tensors[k];
          a.tensor[slot] = {t.g,           t.p,           t.m,    t.v, t.m_scale,                  t.v_scale,
                            t.p_out,       t.m_out,       t.v_out, t.m_scale_out, t.v_scale_out, t.copy,
                            t.n, float(lr * t.weight_decay), t.g_type == TWELL_F32};
        });
    if (chunks > 0) {
      const hipError_t e = twell::launch_adamw(a, chunks, e4m3, static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return TWELL_E_HIP;
    }
  }
  return TWELL_OK;
}

}  // extern "C"
