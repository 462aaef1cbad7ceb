// The optimizer's step over many tensors in one launch, and the norm of all
// gradients, for gfx950.
//
//   g' = scale g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// (Loshchilov, Hutter, "Decoupled weight decay regularization", 2019.) p is fp32;
// a bf16 copy of the new p, which the layer's calls read, is written along.
//
// States in 8 bits: m and sqrt(v) (whose range is half of v's on a logarithmic
// scale) in e4m3 with one scale for each 256 elements, the block's largest value
// becoming 448. Rounded to nearest, b2 = 0.999 could never move a value whose
// neighbours are 6 to 12% away, so values are rounded up with the probability of their
// place between their neighbours: 8 bits of dropout's generator for each state, from
// the counter (element / 8, tensor, offset). Only what is kept is rounded: this step's
// update uses the unrounded fp32 m and v. A root that is not zero stays at least
// the smallest step, 2^-9 of the scale, as a zero under a non-zero m would
// divide by eps alone.
//
// Bound by HBM: 28 bytes an element with fp32 states and gradients (30 with the copy),
// 16.1 with 8-bit states (18.1). A thread takes 8 consecutive elements, so one
// evaluation of the generator serves it and 32 lanes hold a block of the states.
// Measured: 50.3 M elements with the copy 275 us with fp32 states (5.5 TB/s), 51.3 M 164 us with 8-bit ones
// (5.6 TB/s), the norm of 50.3 M fp32 gradients 33 us and 3 for its join (5.6 TB/s of reads); a copy of 512 MiB
// reaches 5.4 TB/s. Twice 4 elements a thread, so that a wave's accesses are runs, took the same 275 us; outputs
// of 32 MB and more that are not stored past the L2 took 1% longer.
#include <algorithm>

#include "block_device.hpp"

namespace twell {
namespace {

constexpr int kStepThreads = kStepChunk / 8;
constexpr float kStateFloor = 0x1p-100f;  // least largest value of a block, as in the norm's rows

// The tensor that chunk `at` belongs to: the last whose first chunk is at or before it. A
// tensor without chunks has its successor's first and is never the last.
__device__ __forceinline__ int tensor_of(const int32_t* first, int at) {
  const int lane = threadIdx.x & 63;
  const bool before = lane < kStepTensors && first[lane & (kStepTensors - 1)] <= at;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(before)) - 1);
}

// 8 elements of a tensor of n from `at` on; those past the end are zero or not stored.
template <class T>
__device__ __forceinline__ void load_at(const T* p, int64_t at, int left, Raw8<T>& r) {
  load_block(p + at, 0, left, r);
}

__device__ __forceinline__ void load_gradient(const void* g, bool f32, int64_t at, int left, float* v) {
  if (f32) {
    Raw8<float> r;
    load_at(static_cast<const float*>(g), at, left, r);
    unpack8(r, v);
  } else {
    Raw8<uint16_t> r;
    load_at(static_cast<const uint16_t*>(g), at, left, r);
    unpack8(r, v);
  }
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int left, float* v) {
  const u32x2_t w = load_bytes(p, left);
  unpack_e4m3(w[0], v);
  unpack_e4m3(w[1], v + 4);
}

// Largest of |v| over the 32 lanes of a block, NaN if one is.
__device__ __forceinline__ float block_max(const float* v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = (fabsf(v[i]) > m || v[i] != v[i]) ? fabsf(v[i]) : m;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float o = __shfl_xor(m, off, 64);
    m = (o > m || o != o) ? o : m;
  }
  return m;
}

// x (at most 448 and a rounding) to its e4m3 neighbour below, or above where
// u, between 0 and 1, reaches one minus its place between them.
__device__ __forceinline__ float to_neighbour(float x, float u) {
  const float a = fabsf(x);
  const uint32_t e = max(__float_as_uint(a) & 0x7F800000u, 121u << 23);  // below 2^-6 the step stays 2^-9
  const float ulp = __uint_as_float(e - (3u << 23)), inv = __uint_as_float((257u << 23) - e);
  return copysignf(floorf(fmaf(a, inv, u)) * ulp, x);
}

// New codes and scale of a block's state. bits: 8 random ones an element.
__device__ __forceinline__ void store_codes(uint8_t* codes, float* scale, int left, const float* v, const uint32_t* bits,
                                            float least, bool stream) {
  const float amax = block_max(v);
  const float top = amax < kStateFloor ? kStateFloor : amax;
  const float inv = 448.f / top;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = to_neighbour(v[i] * inv, fmaf(static_cast<float>(bits[i]), 0x1p-8f, 0x1p-9f));
    if (least > 0.f) q[i] = v[i] > 0.f && q[i] < least ? least : q[i];  // the root's, which has no sign
  }
  if ((threadIdx.x & 31) == 0 && left > 0) *scale = top / 448.f;
  store_block(codes, 0, left, q, stream);
}

template <bool kE4m3>
__global__ __launch_bounds__(kStepThreads) void adamw_kernel(const AdamwArgs a) {
  const float scale = a.grad_scale != nullptr ? *a.grad_scale : 1.f;
  // What a norm that is not finite leaves (max / inf, max / NaN): the step is skipped.
  if (!(fabsf(scale) <= 3.402823466e38f) || scale == 0.f) return;
  const int t = tensor_of(a.first, blockIdx.x);
  const StepTensor& w = a.tensor[t];
  const int64_t at = static_cast<int64_t>(static_cast<int>(blockIdx.x) - a.first[t]) * kStepChunk + 8 * threadIdx.x;
  const int left = static_cast<int>(min(w.n - at, static_cast<int64_t>(8)));
  // Lanes past the end hold zeros and take part in the block's reductions.
  float g[8], p[8], m[8], v[8];
  Raw8<float> rp, rm, rv;
  float ms = 0.f, vs = 0.f;
  const bool any = left > 0;
  load_gradient(w.g, w.g_f32, at, left, g);
  load_at(w.p, at, left, rp);
  if constexpr (kE4m3) {
    load_codes(static_cast<const uint8_t*>(w.m) + at, left, m);
    load_codes(static_cast<const uint8_t*>(w.v) + at, left, v);
    if (any) {
      ms = w.m_scale[at / kStateBlock];
      vs = w.v_scale[at / kStateBlock];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] *= ms;
      v[i] *= vs;
      v[i] *= v[i];
    }
  } else {
    load_at(static_cast<const float*>(w.m), at, left, rm);
    load_at(static_cast<const float*>(w.v), at, left, rv);
    unpack8(rm, m);
    unpack8(rv, v);
  }
  unpack8(rp, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] *= scale;
    m[i] = fmaf(a.mean.b, m[i], fmaf(a.mean.rest, m[i], a.mean.c * g[i]));
    v[i] = fmaf(a.square.b, v[i], fmaf(a.square.rest, v[i], a.square.c * g[i] * g[i]));
    const float root = sqrtf(v[i]);
    p[i] -= fmaf(w.decay, p[i], a.rate * m[i] / fmaf(root, a.root, a.eps));
    if constexpr (kE4m3) v[i] = root;
  }
  if constexpr (kE4m3) {
    const u32x4_t r = philox(static_cast<uint32_t>(at / 8), static_cast<uint32_t>(a.number + t), a.random);
    uint32_t mb[8], vb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t half = (i & 1) ? r[i / 2] >> 16 : r[i / 2] & 0xFFFFu;
      mb[i] = half & 255u;
      vb[i] = half >> 8;
    }
    // Every lane of a block has read its scale before one writes the new one: the
    // value to write comes out of a reduction over all of them.
    const int64_t block = any ? at / kStateBlock : 0;
    store_codes(static_cast<uint8_t*>(w.m_out) + at, w.m_scale_out + block, left, m, mb, 0.f, a.stream);
    store_codes(static_cast<uint8_t*>(w.v_out) + at, w.v_scale_out + block, left, v, vb, 0x1p-9f, a.stream);
  } else {
    store_block(static_cast<float*>(w.m_out) + at, 0, left, m, a.stream);
    store_block(static_cast<float*>(w.v_out) + at, 0, left, v, a.stream);
  }
  store_block(w.p_out + at, 0, left, p, a.stream);
  if (w.copy != nullptr) store_block(w.copy + at, 0, left, p, a.stream);
}

// Sum over the waves of a workgroup of up to 1024 threads, in wave order, on every thread.
__device__ __forceinline__ double workgroup_sum(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (unsigned i = 1; i < blockDim.x / 64; ++i) v += red[i];
  return v;
}

// A chunk's sum of squares in fp64, so that no finite gradient leaves the range and many
// elements lose nothing: two conversions and multiply-adds an element are a tenth of what
// the time of loading it allows.
__global__ __launch_bounds__(256) void grad_norm_kernel(const GradNormArgs a) {
  __shared__ double red[4];
  const int t = tensor_of(a.first, blockIdx.x);
  const NormTensor& w = a.tensor[t];
  const int64_t at = static_cast<int64_t>(static_cast<int>(blockIdx.x) - a.first[t]) * kNormChunk + 8 * threadIdx.x;
  constexpr int kTimes = kNormChunk / 2048;
  float g[kTimes][8];
#pragma unroll
  for (int k = 0; k < kTimes; ++k) {
    const int64_t here = at + 2048 * k;
    load_gradient(w.g, w.g_f32, here, static_cast<int>(min(w.n - here, static_cast<int64_t>(8))), g[k]);
  }
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kTimes; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(g[k][i]), static_cast<double>(g[k][i]), sum);
  sum = workgroup_sum(sum, red);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
}

// The chunks' sums in a fixed order; the norm, and what gradients are multiplied by to keep it at most max_norm.
__global__ __launch_bounds__(1024) void grad_norm_join_kernel(const double* part, int64_t chunks, double max_norm,
                                                              float* out) {
  __shared__ double red[16];
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < chunks; i += 1024) sum += part[i];
  const double norm = sqrt(workgroup_sum(sum, red));
  if (threadIdx.x == 0) {
    out[0] = static_cast<float>(norm);
    out[1] = static_cast<float>(norm <= max_norm && !isinf(norm) ? 1.0 : max_norm / norm);
  }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, int64_t chunks, bool e4m3, hipStream_t s) {
  if (e4m3) {
    adamw_kernel<true><<<static_cast<unsigned>(chunks), kStepThreads, 0, s>>>(a);
  } else {
    adamw_kernel<false><<<static_cast<unsigned>(chunks), kStepThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_grad_norm(const GradNormArgs& a, int64_t chunks, hipStream_t s) {
  grad_norm_kernel<<<static_cast<unsigned>(chunks), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_norm_join(const double* part, int64_t chunks, double max_norm, float* out, hipStream_t s) {
  grad_norm_join_kernel<<<1, 1024, 0, s>>>(part, chunks, max_norm, out);
  return hipGetLastError();
}

}  // namespace twell
