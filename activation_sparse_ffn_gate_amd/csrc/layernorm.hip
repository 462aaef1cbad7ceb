// Residual addition with dropout and layer norm in one pass over the row, and its
// backward, for gfx950: the sibling of residual.hip's norm for models whose block
// subtracts the mean and adds a bias.
//
//   s = residual + keep x / (1 - p)
//   mean = sum s / d,  rstd = 1 / sqrt(sum (s - mean)^2 / d + eps),  out = (s - mean) rstd w + b
//   g = dout w,  xh = (h - mean) rstd,  c1 = mean(g),  c2 = mean(g xh)
//   dres = rstd (g - c1 - xh c2) + dh,  dx = keep dres / (1 - p)
//   dw = sum over rows of dout xh,  db = sum over rows of dout
//
// Bound by HBM as the other norm is, with the same split: a row stays in registers
// between its statistics and its output, so every input byte is read once. The
// variance is never a difference of large sums: a wave takes the mean of its own
// columns and the squares around that, and the waves of a row are joined by
//   mean = sum n_i mean_i / d,  S = sum S_i + n_i (mean_i - mean)^2
// (Chan, Golub, LeVeque, "Updating formulae and a pairwise algorithm for computing
// sample variances", 1979), which needs one exchange through LDS where a mean and
// then the squares around it would need two.
#include "row_device.hpp"

namespace twell {
namespace {

// Columns that a wave of a row holds: blocks of 8 at lane + 64 wave + i threads.
template <int kBlocks>
__device__ __forceinline__ int wave_columns(int wave, int threads, int d) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) n += min(max(d - 8 * (64 * wave + i * threads), 0), 512);
  return n;
}

template <bool kF32>
__device__ __forceinline__ void load_weight(const void* w, int b, int d, float* v) {
  using T = std::conditional_t<kF32, float, uint16_t>;
  Raw8<T> r;
  load_block(static_cast<const T*>(w), b, d, r);
  unpack8(r, v);
}
__device__ __forceinline__ void load_weight(const void* w, bool f32, int b, int d, float* v) {
  if (f32) {
    load_weight<true>(w, b, d, v);
  } else {
    load_weight<false>(w, b, d, v);
  }
}

struct RowStats {
  float mean, squares;  // of the row's values: their mean, the sum of squares around it
};

// Statistics of the row's s * before, the deviations from the mean times `after`;
// columns past d take no part.
template <bool kWaveRow, int kBlocks>
__device__ __forceinline__ RowStats row_stats(const float (&s)[kBlocks][8], int t, int tpr, int d, float before,
                                              float after, float (*red)[kMaxThreads / 64]) {
  const int wave = kWaveRow ? 0 : threadIdx.x >> 6;
  const float n = static_cast<float>(wave_columns<kBlocks>(wave, tpr, d));
  const float inv_n = n > 0.f ? 1.f / n : 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(s[i][j], before, sum);
  float mean = wave_sum(sum) * inv_n;
  // What the deviations from the rounded mean sum to corrects it: the mean of equal values is
  // that value, and their squares zero.
  float rest = 0.f, squares = 0.f;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) rest += j < d - 8 * (t + i * tpr) ? fmaf(s[i][j], before, -mean) : 0.f;
  mean += wave_sum(rest) * inv_n;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = j < d - 8 * (t + i * tpr) ? fmaf(s[i][j], before, -mean) * after : 0.f;
      squares = fmaf(c, c, squares);
    }
  squares = wave_sum(squares);
  if constexpr (kWaveRow) return {mean, squares};
  if ((threadIdx.x & 63) == 0) {
    red[0][wave] = mean;
    red[1][wave] = squares;
  }
  lds_barrier();
  const int waves = tpr / 64;
  const float first = red[0][0];
  float off = 0.f;  // from the first wave's mean
  for (int i = 1; i < waves; ++i) off = fmaf(static_cast<float>(wave_columns<kBlocks>(i, tpr, d)), red[0][i] - first, off);
  const float all = first + off / static_cast<float>(d);
  float total = 0.f;
  for (int i = 0; i < waves; ++i) {
    const float c = (red[0][i] - all) * after;
    total += fmaf(static_cast<float>(wave_columns<kBlocks>(i, tpr, d)) * c, c, red[1][i]);
  }
  return {all, total};
}

template <class TX, class TH, class TO, bool kWaveRow, int kBlocks>
__global__ __launch_bounds__(kWaveRow ? kThreads : kMaxThreads) void add_layernorm_kernel(LayerNormArgs a) {
  constexpr int kRows = kWaveRow ? kThreads / 64 : 1;
  __shared__ float red[5][kMaxThreads / 64];
  const int kTpr = kWaveRow ? 64 : blockDim.x;  // threads of a row
  const int t = kWaveRow ? threadIdx.x & 63 : threadIdx.x;
  const int64_t group = blockIdx.x + blockIdx.y * kGridX;
  const int64_t row = group * kRows + (kWaveRow ? threadIdx.x >> 6 : 0);
  if (row >= a.M) return;  // whole waves, and no barrier follows; or the workgroup
  const int d = a.d;
  const TX* x = static_cast<const TX*>(a.x) + row * d;
  Raw8<TX> rx[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) load_block(x, t + i * kTpr, d, rx[i]);
  Raw8<TH> rr[kBlocks];
  if (a.residual != nullptr) {
    const TH* r = static_cast<const TH*>(a.residual) + row * d;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) load_block(r, t + i * kTpr, d, rr[i]);
  }
  float s[kBlocks][8];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    unpack8(rx[i], s[i]);
    if (a.drop.threshold != 0) drop8(s[i], t + i * kTpr, static_cast<uint32_t>(row), a.drop);
    if (a.residual != nullptr) {
      float v[8];
      unpack8(rr[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += v[j];
    }
  }
  if (a.h != nullptr) {
    TH* h = static_cast<TH*>(a.h) + row * d;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) store_block(h, t + i * kTpr, d, s[i], a.stream);
  }
  float before = 1.f, after = 1.f;
  const float inv_d = 1.f / static_cast<float>(d);
  RowStats st = row_stats<kWaveRow, kBlocks>(s, t, kTpr, d, 1.f, 1.f, red);
  float var = fmaf(st.squares, inv_d, a.eps);
  // Squares leave fp32's range long before s does: such a row is summed again with a
  // power of two, large values (whose sum may have passed the range too, so not
  // finite as well) before the mean is taken, small deviations after.
  if (!(var <= 0x1p120f && var >= 0x1p-100f)) {  // the same for the row's threads
    if (var < 1.f) {
      after = 0x1p100f;
    } else {
      before = 0x1p-100f;
    }
    st = row_stats<kWaveRow, kBlocks>(s, t, kTpr, d, before, after, red + 2);
    var = fmaf(st.squares, inv_d, a.eps * (before * after) * (before * after));
  }
  float r = 1.f / sqrtf(var), rstd = r * before * after;  // r: of before * after * s
  // Large equal values, whose deviations are zero: eps, which 2^-200 takes out of the range, is their variance.
  if (before != 1.f && var == 0.f) r = rstd = 1.f / sqrtf(a.eps);
  if (t == 0) {
    if (a.rstd != nullptr) a.rstd[row] = rstd;
    if (a.mean != nullptr) a.mean[row] = st.mean / before;
  }

  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const int b = t + i * kTpr;
    float w[8], add[8];
    load_weight(a.weight, a.w_f32, b, d, w);
    if (a.bias != nullptr) {
      load_weight(a.bias, a.w_f32, b, d, add);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) add[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[i][j] = fmaf(fmaf(s[i][j], before, -st.mean) * after * r, w[j], add[j]);
      if constexpr (sizeof(TO) == 1) amax = max_nan(amax, fabsf(s[i][j]));
    }
  }
  if constexpr (sizeof(TO) == 1) {
    // Columns past d hold zeros (their weight and bias are) and cannot raise the maximum, unless mean * after * r leaves
    // the range (rows of large equal values) and its product with their weight is NaN: those rows, the same for
    // their threads, are looked at again without them.
    if (!(fabsf(st.mean * after * r) <= 3.402823466e38f)) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = j < d - 8 * (t + i * kTpr) ? max_nan(amax, fabsf(s[i][j])) : amax;
    }
    amax = across_waves<kWaveRow>(wave_max(amax), red[4], max_nan);
    amax = max_nan(kAmaxFloor, amax);
    const float q = 448.f / amax;
    if (t == 0) a.out_scale[row] = amax / 448.f;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * q;
  }
  TO* out = static_cast<TO*>(a.out) + row * d;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) store_block(out, t + i * kTpr, d, s[i], a.stream);
}

// Sums of two values over the threads of a row, in wave order.
template <bool kWaveRow>
__device__ __forceinline__ void sum_pair(float& a, float& b, float (*red)[kMaxThreads / 64]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (!kWaveRow) {
    if ((threadIdx.x & 63) == 0) {
      red[0][threadIdx.x >> 6] = a;
      red[1][threadIdx.x >> 6] = b;
    }
    lds_barrier();
    a = red[0][0];
    b = red[1][0];
    for (unsigned i = 1; i < blockDim.x / 64; ++i) {
      a += red[0][i];
      b += red[1][i];
    }
  }
}

// Rows are dealt and dw and db summed as in the other norm's backward: registers
// over a workgroup's rows, its waves in wave order through LDS, one row of partial
// sums a workgroup, added in row order by dweight_kernel: two calls give the same bits.
template <class TG, class TH, class TX, bool kWaveRow, int kBlocks>
__global__ __launch_bounds__(kWaveRow ? kThreads : kMaxThreads) void add_layernorm_backward_kernel(
    LayerNormBackwardArgs a) {
  constexpr int kRows = kWaveRow ? kThreads / 64 : 1;
  constexpr int kLdsFloats = kWaveRow ? 64 * 8 * kBlocks : 1;
  // Two blocks a thread leave no registers to hold the next row's data or the weight.
  constexpr bool kAhead = kBlocks == 1;
  __shared__ float red[2][2][kMaxThreads / 64];
  __shared__ float sums[2][kLdsFloats];
  const int kTpr = kWaveRow ? 64 : blockDim.x;  // threads of a row
  const int t = kWaveRow ? threadIdx.x & 63 : threadIdx.x;
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  float dw[kBlocks][8], db[kBlocks][8];
  float w[kAhead ? kBlocks : 1][8];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    if constexpr (kAhead) load_weight(a.weight, a.w_f32, t + i * kTpr, d, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  int flip = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  Raw8<TG> rg[kBlocks];
  Raw8<TH> rh[kBlocks], rn[kBlocks];
  float next_rstd = 0.f, next_mean = 0.f;
  auto fetch = [&](int64_t row) {
    next_rstd = a.rstd[row];
    next_mean = a.mean[row];
    const TG* dout = static_cast<const TG*>(a.dout) + row * d;
    const TH* h = static_cast<const TH*>(a.h) + row * d;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      load_block(dout, t + i * kTpr, d, rg[i]);
      load_block(h, t + i * kTpr, d, rh[i]);
    }
    if (a.dh != nullptr) {
      const TH* dh = static_cast<const TH*>(a.dh) + row * d;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) load_block(dh, t + i * kTpr, d, rn[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) rn[i] = Raw8<TH>{};
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (kWaveRow ? threadIdx.x >> 6 : 0);
  if (kAhead && row < a.M) fetch(row);
  for (; row < a.M; row += step) {
    if constexpr (!kAhead) fetch(row);
    const float rstd = next_rstd, mean = next_mean;
    // Half of a deviation from a large mean: the whole may pass the range where the row's values do not.
    const float half = fabsf(mean) < 0x1p100f ? 1.f : 0.5f, rstd_2 = fabsf(mean) < 0x1p100f ? rstd : 2.f * rstd;
    float g[kBlocks][8], xh[kBlocks][8], nx[kBlocks][8];
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      unpack8(rg[i], g[i]);
      unpack8(rh[i], xh[i]);
      unpack8(rn[i], nx[i]);
      float wv[8];
      if constexpr (!kAhead) load_weight(a.weight, a.w_f32, t + i * kTpr, d, wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] = fmaf(xh[i][j], half, -half * mean) * rstd_2;
        dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= kAhead ? w[kAhead ? i : 0][j] : wv[j];
        c1 += g[i][j];
        c2 = fmaf(g[i][j], xh[i][j], c2);
      }
    }
    if (kAhead && row + step < a.M) fetch(row + step);
    // Past d, where h and g are zeros, xh may be infinite (rows of large equal values have an rstd of 1 / sqrt(eps)) and
    // its product with g NaN: such a row, the same for its threads, is summed again without those.
    if (!(fabsf(mean * rstd) <= 3.402823466e38f)) {
      c2 = 0.f;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        // The compiler would keep these conditions for all rows, and spill those of the loads (4096 x 2047 39 -> 42 us).
        int n = d - 8 * (t + i * kTpr);
        asm volatile("" : "+v"(n));
#pragma unroll
        for (int j = 0; j < 8; ++j) c2 = j < n ? fmaf(g[i][j], xh[i][j], c2) : c2;
      }
    }
    // red[flip] alternates, so the next row's writes cannot overtake this
    // row's reads with one barrier a row
    sum_pair<kWaveRow>(c1, c2, red[flip]);
    c1 *= inv_d;
    c2 *= inv_d;
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int b = t + i * kTpr;
      float* v = nx[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(rstd, fmaf(-xh[i][j], c2, g[i][j] - c1), v[j]);
      if (a.dres != nullptr) store_block(static_cast<TH*>(a.dres) + row * d, b, d, v, a.stream);
      if (a.dx != nullptr) {
        if (a.drop.threshold != 0) drop8(v, b, static_cast<uint32_t>(row), a.drop);
        store_block(static_cast<TX*>(a.dx) + row * d, b, d, v, a.stream);
      }
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * d;
  if constexpr (kWaveRow) {
    // the four waves add in turn; a block's 8 sums sit at [block][j]
    const int wave = threadIdx.x >> 6;
    for (int k = 0; k < kRows; ++k) {
      if (wave == k) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int at = (i * 8 + j) * 64 + t;
            if (k > 0) {
              dw[i][j] += sums[0][at];
              db[i][j] += sums[1][at];
            }
            sums[0][at] = dw[i][j];
            sums[1][at] = db[i][j];
          }
      }
      __syncthreads();
    }
    if (wave != kRows - 1) return;
  }
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    store_block(part, t + i * kTpr, d, dw[i]);
    store_block(part + d, t + i * kTpr, d, db[i]);
  }
}

}  // namespace

hipError_t launch_add_layernorm(LayerNormArgs a, bool x_f32, bool h_f32, bool out_e4m3, hipStream_t s) {
  a.stream = a.M * a.d * ((a.h ? (h_f32 ? 4 : 2) : 0) + (out_e4m3 ? 1 : 2)) >= kStreamBytes;
  by_shape(a.d, true, [&](auto shape, int threads) {
    constexpr bool kWaveRow = decltype(shape)::wave_row;
    constexpr int kBlocks = decltype(shape)::blocks;
    const int64_t groups = kWaveRow ? (a.M + 3) / 4 : a.M;
    const dim3 grid(static_cast<unsigned>(std::min(groups, kGridX)),
                    static_cast<unsigned>((groups + kGridX - 1) / kGridX));
    by_type(x_f32, [&](auto* x) {
      by_type(h_f32, [&](auto* h) {
        using TX = std::remove_pointer_t<decltype(x)>;
        using TH = std::remove_pointer_t<decltype(h)>;
        if (out_e4m3) {
          add_layernorm_kernel<TX, TH, uint8_t, kWaveRow, kBlocks><<<grid, threads, 0, s>>>(a);
        } else {
          add_layernorm_kernel<TX, TH, uint16_t, kWaveRow, kBlocks><<<grid, threads, 0, s>>>(a);
        }
      });
    });
  });
  return hipGetLastError();
}

// Workgroups of the backward = rows of partial sums, of dw and db: 4 rows of the batch each, one workgroup a CU above 2048
// columns, else between one and two. (Two there, as in the other norm, whose partial rows are half as long: 4096 rows of 4096
// from fp32 42 us against 38, of 8192 78 against 70, 2000 rows of 8192 49 against 40, 16384 of 2560 80 and 80; one
// at 2048: 22 against 21.)
int layernorm_backward_groups(int64_t M, int64_t d) {
  const int64_t rows = d <= 512 ? 4 : 1;
  const int64_t groups = d > 2048 ? 256 : std::min<int64_t>(std::max<int64_t>(M / 4, 256), kBackwardGroups);
  return static_cast<int>(std::min<int64_t>((M + rows - 1) / rows, groups));
}

hipError_t launch_add_layernorm_backward(LayerNormBackwardArgs a, bool g_f32, bool h_f32, bool x_f32, float* dweight,
                                         float* dbias, hipStream_t s) {
  a.stream = a.M * a.d * ((a.dres ? (h_f32 ? 4 : 2) : 0) + (a.dx ? (x_f32 ? 4 : 2) : 0)) >= kStreamBytes;
  const int groups = layernorm_backward_groups(a.M, a.d);
  if (groups > 0) by_shape(a.d, false, [&](auto shape, int threads) {
    constexpr bool kWaveRow = decltype(shape)::wave_row;
    constexpr int kBlocks = decltype(shape)::blocks;
    by_type(g_f32, [&](auto* g) {
      by_type(h_f32, [&](auto* h) {
        by_type(x_f32, [&](auto* x) {
          using TG = std::remove_pointer_t<decltype(g)>;
          using TH = std::remove_pointer_t<decltype(h)>;
          using TX = std::remove_pointer_t<decltype(x)>;
          add_layernorm_backward_kernel<TG, TH, TX, kWaveRow, kBlocks><<<groups, threads, 0, s>>>(a);
        });
      });
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int columns = dbias ? 2 * a.d : a.d;
  dweight_kernel<<<(columns + 15) / 16, 1024, 0, s>>>(a.part, groups, 2 * a.d, a.d, dweight, dbias);
  return hipGetLastError();
}

}  // namespace twell
