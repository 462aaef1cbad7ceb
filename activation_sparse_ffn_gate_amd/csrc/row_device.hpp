// What the norms share (residual.hip, layernorm.hip): who holds a row, reductions
// over its threads, and the join of the backward's partial weight gradients.
#pragma once

#include <algorithm>

#include "block_device.hpp"

namespace twell {
namespace {

constexpr int kThreads = 256;     // of a workgroup with a row a wave, and of dropout
constexpr int kMaxThreads = 1024;  // of a workgroup with one row
// Least max|out| an e4m3 row is scaled by: keeps the scale of a zero row and
// its inverse finite and normal.
constexpr float kAmaxFloor = 0x1p-100f;
constexpr int kBackwardGroups = 512;
// Workgroups of the forward in the grid's first dimension, where 1024 threads
// each stay under the 2^32 that a dimension holds; the second counts these.
constexpr int64_t kGridX = int64_t(1) << 21;

// Sum (or maximum) over the threads of a row from each wave's: the wave itself
// (kWaveRow), or the workgroup, whose waves exchange through `red` in wave order.
template <bool kWaveRow, class Op>
__device__ __forceinline__ float across_waves(float v, float* red, Op op) {
  if constexpr (!kWaveRow) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    lds_barrier();
    v = red[0];
    for (unsigned i = 1; i < blockDim.x / 64; ++i) v = op(v, red[i]);
  }
  return v;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) { return (b > a || b != b) ? b : a; }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v = max_nan(v, __shfl_xor(v, off, 64));
  return v;
}

// Sums over n partial rows of `width` columns, in a fixed order: 16 columns a
// workgroup, 64 threads a column taking every 64th row, then a tree over them. The
// first d columns are dw, the others (a layer norm's) db where it is asked for. What it
// waits for is the loads' latency, so a thread's (at most kBackwardGroups / 64) are
// all requested at once.
__global__ __launch_bounds__(1024) void dweight_kernel(const float* part, int n, int width, int d, float* dw,
                                                       float* db) {
  __shared__ float s[64][17];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + tx;
  float v[kBackwardGroups / 64];
#pragma unroll
  for (int i = 0; i < kBackwardGroups / 64; ++i) {
    const int r = ty + 64 * i;
    v[i] = c < width && r < n ? part[static_cast<int64_t>(r) * width + c] : 0.f;
  }
#pragma unroll
  for (int i = 1; i < kBackwardGroups / 64; ++i) v[0] += v[i];
  s[ty][tx] = v[0];
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (ty < o) s[ty][tx] += s[ty + o][tx];
    __syncthreads();
  }
  if (ty != 0 || c >= width) return;
  if (c < d) {
    dw[c] = s[0][tx];
  } else if (db != nullptr) {
    db[c - d] = s[0][tx];
  }
}

// Calls f with a pointer of the element type: fp32 or bf16.
template <class Fn>
void by_type(bool f32, Fn&& f) {
  if (f32) {
    f(static_cast<float*>(nullptr));
  } else {
    f(static_cast<uint16_t*>(nullptr));
  }
}

template <bool kWaveRow, int kBlocks>
struct RowShape {
  static constexpr bool wave_row = kWaveRow;
  static constexpr int blocks = kBlocks;
};

// Who holds a row of d columns: a wave up to 512, else a workgroup of just
// enough waves with 8 columns a thread; with 16 above 8192, and where `two`
// says so above 2048 (then at least 4 waves). A row of 2048 columns a wave with
// 32 a thread measured worse: 16.0 us forward and 23.7 backward for 4096 rows,
// against 15.5 and 21.2. 16 a thread in the forward, against 8: fp32 to e4m3 of 8192
// rows of 8192 106 us (117), of 5120 70 (78), of 4096 56 (56), 16384 rows of
// 2560 74 (72); bf16 to bf16 93 (92), 59 (59), 48 (47), 58 (58), of 2056 24 (26).
// The backward of 777 rows of 2560 22 us (13).
template <class Fn>
void by_shape(int d, bool two, Fn&& f) {
  const int nb = (d + 7) / 8;
  if (nb <= 64) {
    f(RowShape<true, 1>{}, kThreads);
  } else if (nb <= (two ? 256 : kMaxThreads)) {
    f(RowShape<false, 1>{}, (nb + 63) / 64 * 64);
  } else {
    f(RowShape<false, 2>{}, std::max((nb + 127) / 128 * 64, 256));
  }
}

// Outputs of this many bytes and more are stored past the L2 (32 MB on the
// device): 4096 x 2048 forward 15.5 -> 14.6 us, dropout of 4096 x 8192 25.5 ->
// 23.3 us. Smaller ones stay for the kernel that reads them next.
constexpr int64_t kStreamBytes = int64_t(32) << 20;

}  // namespace
}  // namespace twell
