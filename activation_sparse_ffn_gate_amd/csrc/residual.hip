// The residual branch around the FFN, for gfx950: dropout, residual addition
// and root-mean-square norm in one pass over the row, and its backward.
//
//   s = residual + keep x / (1 - p)          rstd = 1 / sqrt(mean(s^2) + eps)
//   out = s rstd w                           (bf16, or e4m3 with max|out| / 448 a row)
//   g = dout w,  xh = h rstd,  c = mean(g xh)
//   dres = rstd (g - xh c) + dh,  dx = keep dres / (1 - p),  dw = sum over rows of dout xh
//
// All of it is bound by HBM: every input byte is read once and every output
// byte written once. A row stays in registers between its statistics and its
// output (blocks of 8 columns a thread, consecutive threads holding consecutive
// blocks), so nothing is read twice. (Above 8192 columns the backward's two
// blocks a thread do not fit the 128 registers of a workgroup of 1024: 47 to 259
// of them go through scratch memory, and 4096 x 10240 bf16 takes 76 us, 4.4
// TB/s, where 4096 x 8192 takes 48, 5.6 TB/s.) Squares, products, the statistics
// and dw are summed in fp32; s is normalised before it is rounded to h's type.
//
// Measured: 4096 x 2048 from fp32 with dropout 14.6 us (5.7 TB/s), 16384 x 2560
// from fp32 to e4m3 74 us (5.1 TB/s), the backward of 4096 x 2048 with dropout
// 18.6 us and 3.9 for dw (4.5 TB/s together), dropout of 4096 x 8192 bf16 21.6
// us (6.2 TB/s). A copy of 512 MiB reaches 5.4 TB/s.
#include <algorithm>

#include "row_device.hpp"

namespace twell {
namespace {

template <class TX, class TH, class TO, bool kWaveRow, int kBlocks>
__global__ __launch_bounds__(kWaveRow ? kThreads : kMaxThreads) void add_rmsnorm_kernel(NormArgs a) {
  constexpr int kRows = kWaveRow ? kThreads / 64 : 1;
  __shared__ float red[3][kMaxThreads / 64];
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
  float s[kBlocks][8];
  if (a.residual != nullptr) {
    const TH* r = static_cast<const TH*>(a.residual) + row * d;
    Raw8<TH> rr[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) load_block(r, t + i * kTpr, d, rr[i]);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      unpack8(rx[i], s[i]);
      if (a.drop.threshold != 0) drop8(s[i], t + i * kTpr, static_cast<uint32_t>(row), a.drop);
      float v[8];
      unpack8(rr[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      unpack8(rx[i], s[i]);
      if (a.drop.threshold != 0) drop8(s[i], t + i * kTpr, static_cast<uint32_t>(row), a.drop);
    }
  }
  // A thread's sum of (s k)^2.
  auto squares = [&](float k) {
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(s[i][j] * k, s[i][j] * k, sq);
    return sq;
  };
  const auto plus = [](float p, float q) { return p + q; };
  float sq = squares(1.f);
  if (a.h != nullptr) {
    TH* h = static_cast<TH*>(a.h) + row * d;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) store_block(h, t + i * kTpr, d, s[i], a.stream);
  }
  sq = across_waves<kWaveRow>(wave_sum(sq), red[0], plus);
  const float mean = sq / static_cast<float>(d) + a.eps;
  float rstd = 1.f / sqrtf(mean);
  // Squares leave fp32's range long before s does (|s| of 2^60 gave rstd = 0 and a
  // row of zeros): such a row is summed again, scaled by a power of two.
  if (mean > 0x1p120f || mean < 0x1p-100f) {  // the same for the row's threads
    const float k = mean > 1.f ? 0x1p-100f : 0x1p100f;
    sq = across_waves<kWaveRow>(wave_sum(squares(k)), red[2], plus);
    rstd = k / sqrtf(sq / static_cast<float>(d) + a.eps * k * k);
  }
  if (a.rstd != nullptr && t == 0) a.rstd[row] = rstd;

  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    float w[8];
    if (a.w_f32) {
      Raw8<float> r;
      load_block(static_cast<const float*>(a.weight), t + i * kTpr, d, r);
      unpack8(r, w);
    } else {
      Raw8<uint16_t> r;
      load_block(static_cast<const uint16_t*>(a.weight), t + i * kTpr, d, r);
      unpack8(r, w);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[i][j] = s[i][j] * rstd * w[j];
      if constexpr (sizeof(TO) == 1) amax = max_nan(amax, fabsf(s[i][j]));
    }
  }
  if constexpr (sizeof(TO) == 1) {
    // Columns past d hold zeros (0 * rstd * 0) and cannot raise the maximum;
    // where rstd is not finite they would be NaN, but then the row is too.
    amax = across_waves<kWaveRow>(wave_max(amax), red[1], max_nan);
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

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... (times 4, a wave each, for
// kWaveRow): a thread keeps its columns' sums of dw in registers over all its rows;
// the waves of a workgroup add theirs through LDS in wave order, and each
// workgroup leaves one row of partial sums, which dweight_kernel adds in row
// order: two calls give the same bits.
template <class TG, class TH, class TX, bool kWaveRow, int kBlocks>
__global__ __launch_bounds__(kWaveRow ? kThreads : kMaxThreads) void add_rmsnorm_backward_kernel(
    NormBackwardArgs a) {
  constexpr int kRows = kWaveRow ? kThreads / 64 : 1;
  constexpr int kLdsFloats = kWaveRow ? 64 * 8 * kBlocks : 1;
  __shared__ float red[2][kMaxThreads / 64];
  __shared__ float dws[kLdsFloats];
  const int kTpr = kWaveRow ? 64 : blockDim.x;  // threads of a row
  const int t = kWaveRow ? threadIdx.x & 63 : threadIdx.x;
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  float dw[kBlocks][8];
  Raw8<float> w[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    if (a.w_f32) {
      load_block(static_cast<const float*>(a.weight), t + i * kTpr, d, w[i]);
    } else {
      Raw8<uint16_t> r;
      load_block(static_cast<const uint16_t*>(a.weight), t + i * kTpr, d, r);
      float v[8];
      unpack8(r, v);
      w[i].a = __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]});
      w[i].b = __builtin_bit_cast(u32x4_t, f32x4_t{v[4], v[5], v[6], v[7]});
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  int flip = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  // The next row is requested before this one's sum is waited for.
  Raw8<TG> rg[kBlocks];
  Raw8<TH> rh[kBlocks], rn[kBlocks];
  float next_rstd;
  auto fetch = [&](int64_t row) {
    next_rstd = a.rstd[row];
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
  if (row < a.M) fetch(row);
  for (; row < a.M; row += step) {
    const float rstd = next_rstd;
    float g[kBlocks][8], xh[kBlocks][8], nx[kBlocks][8];
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      float wv[8];
      unpack8(rg[i], g[i]);
      unpack8(rh[i], xh[i]);
      unpack8(rn[i], nx[i]);
      unpack8(w[i], wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rstd;
        dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
        g[i][j] *= wv[j];
        c = fmaf(g[i][j], xh[i][j], c);
      }
    }
    if (row + step < a.M) fetch(row + step);
    // red[flip] alternates, so the next row's writes cannot overtake this
    // row's reads with one barrier a row
    c = across_waves<kWaveRow>(wave_sum(c), red[flip], [](float p, float q) { return p + q; }) * inv_d;
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int b = t + i * kTpr;
      float* v = nx[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(rstd, fmaf(-xh[i][j], c, g[i][j]), v[j]);
      if (a.dres != nullptr) store_block(static_cast<TH*>(a.dres) + row * d, b, d, v, a.stream);
      if (a.dx != nullptr) {
        if (a.drop.threshold != 0) drop8(v, b, static_cast<uint32_t>(row), a.drop);
        store_block(static_cast<TX*>(a.dx) + row * d, b, d, v, a.stream);
      }
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * d;
  if constexpr (kWaveRow) {
    // the four waves add in turn; a block's 8 sums sit at [block][j]
    const int wave = threadIdx.x >> 6;
    for (int k = 0; k < kRows; ++k) {
      if (wave == k) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float* p = &dws[(i * 8 + j) * 64 + t];
            if (k == 0) {
              *p = dw[i][j];
            } else if (k < kRows - 1) {
              *p += dw[i][j];
            } else {
              dw[i][j] += *p;
            }
          }
      }
      __syncthreads();
    }
    if (wave != kRows - 1) return;
  }
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) store_block(part, t + i * kTpr, d, dw[i]);
}

// Flat over the blocks of 8 columns; a workgroup takes kDropBlocks of them.
constexpr int kDropBlocks = 4;

template <class TX, class TY>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropoutArgs a) {
  const uint32_t nb = static_cast<uint32_t>((a.d + 7) / 8);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kDropBlocks);
  const int64_t row0 = first / nb;
  const uint32_t col0 = static_cast<uint32_t>(first - row0 * nb);
  int64_t row[kDropBlocks];
  int b[kDropBlocks];
  Raw8<TX> rx[kDropBlocks];
  Raw8<TY> rr[kDropBlocks];
#pragma unroll
  for (int i = 0; i < kDropBlocks; ++i) {
    const uint32_t at = col0 + i * kThreads + threadIdx.x;  // below nb + 1024
    const uint32_t r = at / nb;
    row[i] = row0 + r;
    b[i] = static_cast<int>(at - r * nb);
    if (row[i] < a.M) {
      load_block(static_cast<const TX*>(a.x) + row[i] * a.d, b[i], a.d, rx[i]);
      if (a.residual != nullptr) load_block(static_cast<const TY*>(a.residual) + row[i] * a.d, b[i], a.d, rr[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kDropBlocks; ++i) {
    if (row[i] >= a.M) continue;
    float v[8];
    unpack8(rx[i], v);
    if (a.drop.threshold != 0) drop8(v, b[i], static_cast<uint32_t>(row[i]), a.drop);
    if (a.residual != nullptr) {
      float r[8];
      unpack8(rr[i], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    store_block(static_cast<TY*>(a.y) + row[i] * a.d, b[i], a.d, v, a.stream);
  }
}

}  // namespace

hipError_t launch_add_rmsnorm(NormArgs a, bool x_f32, bool h_f32, bool out_e4m3, hipStream_t s) {
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
          add_rmsnorm_kernel<TX, TH, uint8_t, kWaveRow, kBlocks><<<grid, threads, 0, s>>>(a);
        } else {
          add_rmsnorm_kernel<TX, TH, uint16_t, kWaveRow, kBlocks><<<grid, threads, 0, s>>>(a);
        }
      });
    });
  });
  return hipGetLastError();
}

// Workgroups of the backward = rows of partial dw sums: 4 rows each (the sums
// are another M / 4 rows to write and read), between one and two workgroups a CU.
int norm_backward_groups(int64_t M, int64_t d) {
  const int64_t rows = d <= 512 ? 4 : 1;
  const int64_t groups = std::min<int64_t>(std::max<int64_t>(M / 4, 256), kBackwardGroups);
  return static_cast<int>(std::min<int64_t>((M + rows - 1) / rows, groups));
}

hipError_t launch_add_rmsnorm_backward(NormBackwardArgs a, bool g_f32, bool h_f32, bool x_f32, float* dweight,
                                       hipStream_t s) {
  a.stream = a.M * a.d * ((a.dres ? (h_f32 ? 4 : 2) : 0) + (a.dx ? (x_f32 ? 4 : 2) : 0)) >= kStreamBytes;
  const int groups = norm_backward_groups(a.M, a.d);
  if (groups > 0) by_shape(a.d, false, [&](auto shape, int threads) {
    constexpr bool kWaveRow = decltype(shape)::wave_row;
    constexpr int kBlocks = decltype(shape)::blocks;
    by_type(g_f32, [&](auto* g) {
      by_type(h_f32, [&](auto* h) {
        by_type(x_f32, [&](auto* x) {
          using TG = std::remove_pointer_t<decltype(g)>;
          using TH = std::remove_pointer_t<decltype(h)>;
          using TX = std::remove_pointer_t<decltype(x)>;
          add_rmsnorm_backward_kernel<TG, TH, TX, kWaveRow, kBlocks><<<groups, threads, 0, s>>>(a);
        });
      });
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  dweight_kernel<<<(a.d + 15) / 16, 1024, 0, s>>>(a.part, groups, a.d, a.d, dweight, nullptr);
  return hipGetLastError();
}

hipError_t launch_dropout(DropoutArgs a, bool x_f32, bool y_f32, hipStream_t s) {
  a.stream = a.M * a.d * (y_f32 ? 4 : 2) >= kStreamBytes;
  const int64_t blocks = a.M * ((a.d + 7) / 8);
  const dim3 grid(static_cast<unsigned>((blocks + kThreads * kDropBlocks - 1) / (kThreads * kDropBlocks)));
  by_type(x_f32, [&](auto* x) {
    by_type(y_f32, [&](auto* y) {
      using TX = std::remove_pointer_t<decltype(x)>;
      using TY = std::remove_pointer_t<decltype(y)>;
      dropout_kernel<TX, TY><<<grid, kThreads, 0, s>>>(a);
    });
  });
  return hipGetLastError();
}

}  // namespace twell
