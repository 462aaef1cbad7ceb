// Products with 4-bit weights and group scales for gfx950:
//
//   y[m, n] = sx[m] sum over k of x[m, k] s[n, k / g] (q[n, k] - z[n, k / g])
//
// and the gated pair h = z > 0 ? z u : 0 of two such products.
//
// A byte s000mmmm read as e4m3 is (-1)^s m 2^-9 exactly for m = 0..15 (m < 8 are
// that format's subnormals, 8..15 its first binade). So the codes of four
// bytes become q - z as sign and magnitude in a few integer operations (see
// Codes), and are then the matrix operand of an e4m3 product as they stand;
// for bf16 one v_cvt_scalef32_pk_bf16_fp8 by 2^9 turns two of them into
// integers. Subtracting z there, not as z sum(x) from the sums, costs 1.25
// operations a weight more and keeps groups exact in which one large weight
// leaves all others at zero: their products are zeros, not large terms that
// cancel (measured on such a gate: error of the layer 2.1e-5 with the sums,
// 3e-6 this way).
// fp32 x is cut into three bf16 parts that add up to it exactly (8 + 8 + 8
// bits). All products are exact in fp32; sums are held in fp32 per group,
// then scaled and added.
//
// v_mfma_f32_16x16x32: 16 rows of x by 16 units, 32 values of K, which lie
// inside one group (groups are 32, 64 or 128). Lane l holds row or unit
// l % 16 and 8 consecutive k at 8 (l / 16); the result has unit l % 16 and
// rows 4 (l / 16) + 0..3. A wave takes K in chunks of 128: lane l loads 16
// consecutive bytes of its unit's row, and a 4 x 4 transposition between the
// four 16-lane quarters (two v_permlane32_swap, two v_permlane16_swap) gives
// register i the codes of K values 32 i + 8 (l / 16) + 0..7. Low nibbles are
// even k, high nibbles odd k, so x operands are put in that order too.
// The waves of a workgroup take the chunks of K in turn and add up through LDS
// in wave order.
#include "block_device.hpp"

namespace twell {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kChunk = 128;

__device__ __forceinline__ f32x4 mfma_bf16(u32x4_t a, u32x4_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_e4m3(u32x2_t a, u32x2_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0, 0,
                                                    0);
}

// Bytes w of 16 lanes' quarters: register i of quarter j becomes register j of
// quarter i.
__device__ __forceinline__ u32x4_t transpose_quarters(u32x4_t w) {
  auto r0 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  auto r1 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  auto s0 = __builtin_amdgcn_permlane16_swap(r0[0], r1[0], false, false);
  auto s1 = __builtin_amdgcn_permlane16_swap(r0[1], r1[1], false, false);
  return u32x4_t{s0[0], s0[1], s1[0], s1[1]};
}

// Two bytes of sign and magnitude (0, 1 or 2, 3 of w) as a pair of bf16 integers.
template <bool kHigh>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.f, kHigh));
}

// The matrix operands of one step of 32 k. Parts of x: bf16 and e4m3 have one.
template <Q4X kX>
struct Step {
  static constexpr int parts = kX == Q4X::f32 ? 3 : 1;
  u32x4_t x[parts];

  // 8 bf16 in memory order, put into the order of the codes.
  __device__ static u32x4_t even_odd(u32x4_t w) {
    return u32x4_t{__builtin_amdgcn_perm(w[1], w[0], 0x05040100u), __builtin_amdgcn_perm(w[3], w[2], 0x05040100u),
                   __builtin_amdgcn_perm(w[1], w[0], 0x07060302u), __builtin_amdgcn_perm(w[3], w[2], 0x07060302u)};
  }

  // Row m of x at k .. k + 7; zeros past M and past K.
  __device__ __forceinline__ void load(const void* base, int m, int M, int64_t K, int64_t k) {
    const int64_t left = K - k;
    const int n = m < M ? (left >= 8 ? 8 : static_cast<int>(left)) : 0;
    if constexpr (kX == Q4X::e4m3) {
      const uint8_t* p = static_cast<const uint8_t*>(base) + m * K + k;
      u32x2_t w = {0u, 0u};
      if (n == 8) {
        __builtin_memcpy(&w, p, 8);
      } else {
        for (int i = 0; i < n; ++i) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
      }
      x[0][0] = __builtin_amdgcn_perm(w[1], w[0], 0x06040200u);
      x[0][1] = __builtin_amdgcn_perm(w[1], w[0], 0x07050301u);
    } else if constexpr (kX == Q4X::bf16) {
      const uint16_t* p = static_cast<const uint16_t*>(base) + m * K + k;
      Raw8<uint16_t> r = {};
      if (n == 8) {
        load8(p, r);
      } else if (n > 0) {
        load8_cut(p, n, r);
      }
      x[0] = even_odd(r.w);
    } else {
      const float* p = static_cast<const float*>(base) + m * K + k;
      Raw8<float> r = {};
      if (n == 8) {
        load8(p, r);
      } else if (n > 0) {
        load8_cut(p, n, r);
      }
      float v[8];
      unpack8(r, v);
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // the top 8 significant bits, and what is left
          h[i] = __float_as_uint(v[i]) & 0xFFFF0000u;
          v[i] -= __uint_as_float(h[i]);
        }
        x[s] = u32x4_t{(h[0] >> 16) | h[2], (h[4] >> 16) | h[6], (h[1] >> 16) | h[3], (h[5] >> 16) | h[7]};
      }
    }
  }
};

// Four codes (bytes 0..15) as q - z in sign and magnitude; zero = 128 - z in
// every byte (z <= 15, so no byte carries into the next).
__device__ __forceinline__ uint32_t sign_magnitude(uint32_t q, uint32_t zero) {
  const uint32_t d = q + zero;                            // 128 + (q - z)
  const uint32_t neg = ~(d >> 7) & 0x01010101u;           // 1 where q < z
  const uint32_t m = (d ^ (0x80808080u - neg)) + neg;     // d ^ 0x80, or (d ^ 0x7F) + 1
  return m | (neg << 7);
}

template <Q4X kX>
struct Codes {
  u32x4_t w;
  __device__ __forceinline__ Codes(uint32_t c, uint32_t zero) {
    const uint32_t lo = sign_magnitude(c & 0x0F0F0F0Fu, zero);
    const uint32_t hi = sign_magnitude((c >> 4) & 0x0F0F0F0Fu, zero);
    if constexpr (kX == Q4X::e4m3) {
      w[0] = lo;
      w[1] = hi;
    } else {
      w = u32x4_t{codes_bf16<false>(lo), codes_bf16<true>(lo), codes_bf16<false>(hi), codes_bf16<true>(hi)};
    }
  }
};

template <Q4X kX>
__device__ __forceinline__ f32x4 product(const Step<kX>& x, u32x4_t w, f32x4 c) {
  if constexpr (kX == Q4X::e4m3) {
    return mfma_e4m3(u32x2_t{x.x[0][0], x.x[0][1]}, u32x2_t{w[0], w[1]}, c);
  } else {
#pragma unroll
    for (int p = 0; p < Step<kX>::parts; ++p) c = mfma_bf16(x.x[p], w, c);
    return c;
  }
}

template <Q4X kX, bool kGated, int kGroup, int kMT, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void q4_kernel(Q4Args a) {
  constexpr int kMats = kGated ? 2 : 1;
  constexpr int kPer = kChunk / kGroup;                   // groups of a chunk
  constexpr float kCode = kX == Q4X::e4m3 ? 512.f : 1.f;  // an e4m3 code stands for (q - z) / 512
  __shared__ float red[kWaves > 1 ? kWaves - 1 : 1][kMats * kMT][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int quarter = lane >> 4, col = lane & 15;
  const int unit = blockIdx.x * 16 + col;
  const int64_t row_of_w = min(unit, a.N - 1);
  const int m0 = blockIdx.y * (16 * kMT);
  const int64_t K = a.K, kb = (K + 1) / 2, G = (K + kGroup - 1) / kGroup;
  const int chunks = static_cast<int>((K + kChunk - 1) / kChunk);

  f32x4 total[kMats][kMT] = {};
  for (int c = wave; c < chunks; c += kWaves) {
    u32x4_t w[kMats];
    float s[kMats][kPer];
    uint32_t z[kMats][kPer];
#pragma unroll
    for (int t = 0; t < kMats; ++t) {
      const Q4Weight& q = t == 0 ? a.w : a.up;
      const uint8_t* p = q.codes + row_of_w * kb;
      const int64_t at = c * 64 + quarter * 16, left = kb - at;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (left >= 16) {
        v = load16_any(p + at);
      } else {
        for (int i = 0; i < left; ++i) v[i >> 2] |= static_cast<uint32_t>(p[at + i]) << (8 * (i & 3));
      }
      w[t] = transpose_quarters(v);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int64_t g = row_of_w * G + min(static_cast<int64_t>(c) * kPer + i, G - 1);  // past K x is zero
        s[t][i] = bf16_lo(q.scales[g]) * kCode;
        z[t][i] = (128u - (q.zeros != nullptr ? q.zeros[g] & 15u : 8u)) * 0x01010101u;
      }
    }
    f32x4 acc[kMats][kMT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      constexpr int kSteps = kGroup / 32;
      const int64_t k = static_cast<int64_t>(c) * kChunk + 32 * i;
      Step<kX> x[kMT];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) x[mt].load(a.x, m0 + 16 * mt + col, a.M, K, k + 8 * quarter);
#pragma unroll
      for (int t = 0; t < kMats; ++t) {
        const Codes<kX> q(w[t][i], z[t][i / kSteps]);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          acc[t][mt] = product<kX>(x[mt], q.w, i % kSteps == 0 ? f32x4{} : acc[t][mt]);
          if (i % kSteps == kSteps - 1) {
#pragma unroll
            for (int r = 0; r < 4; ++r) total[t][mt][r] = fmaf(s[t][i / kSteps], acc[t][mt][r], total[t][mt][r]);
          }
        }
      }
    }
  }

  if constexpr (kWaves > 1) {
    if (wave > 0) {
#pragma unroll
      for (int t = 0; t < kMats; ++t)
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int r = 0; r < 4; ++r) red[wave - 1][t * kMT + mt][r][lane] = total[t][mt][r];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int t = 0; t < kMats; ++t)
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          for (int o = 0; o < kWaves - 1; ++o) total[t][mt][r] += red[o][t * kMT + mt][r][lane];
  }
  if (unit >= a.N) return;
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = m0 + 16 * mt + 4 * quarter + r;
      if (m >= a.M) continue;
      const float sx = kX == Q4X::e4m3 ? a.x_scale[m] : 1.f;
      float v = total[0][mt][r] * sx;
      if constexpr (kGated) v = v > 0.f ? v * (total[kMats - 1][mt][r] * sx) : 0.f;
      const int64_t at = static_cast<int64_t>(m) * a.N + unit;
      if (a.y_f32) {
        static_cast<float*>(a.y)[at] = v;
      } else {
        store1(static_cast<uint16_t*>(a.y) + at, v);
      }
    }
}

// Symmetric round to nearest: s = max|w| / 7 of the group in bf16, code
// round(w / s) + 8. A lane holds 8 consecutive k, a group is 4, 8 or 16 lanes.
__global__ __launch_bounds__(256) void q4_quantize_kernel(const uint16_t* W, int N, int K, int group, uint8_t* codes,
                                                          uint16_t* scales) {
  const int64_t G = (K + group - 1) / group, per_row = G * (group / 8);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t n = id / per_row;
  const int b = static_cast<int>(id - n * per_row);
  float v[8] = {};
  if (n < N) {
    Raw8<uint16_t> r;
    load_block(W + n * K, b, K, r);
    unpack8(r, v);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  for (int o = 1; o < group / 8; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
  if (n >= N) return;
  const uint32_t sb = pack_bf16(amax / 7.f, 0.f);
  const float s = bf16_lo(sb);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = s > 0.f ? fminf(fmaxf(rintf(v[i] / s) + 8.f, 0.f), 15.f) : 8.f;
    w |= static_cast<uint32_t>(q) << (4 * i);
  }
  const int64_t kb = (static_cast<int64_t>(K) + 1) / 2;
  for (int i = 0; i < 4; ++i)
    if (4 * b + i < kb) codes[n * kb + 4 * b + i] = static_cast<uint8_t>(w >> (8 * i));
  if (b % (group / 8) == 0) scales[n * G + b / (group / 8)] = static_cast<uint16_t>(sb);
}

template <Q4X kX, bool kGated, int kGroup>
hipError_t launch_typed(const Q4Args& a, hipStream_t s) {
  const unsigned nx = (a.N + 15) / 16;
  if (a.M <= 16) {
    q4_kernel<kX, kGated, kGroup, 1, 8><<<dim3(nx, 1), 512, 0, s>>>(a);
  } else {
    q4_kernel<kX, kGated, kGroup, 4, 4><<<dim3(nx, (a.M + 63) / 64), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <Q4X kX, bool kGated>
hipError_t launch_group(const Q4Args& a, hipStream_t s) {
  if (a.group == 32) return launch_typed<kX, kGated, 32>(a, s);
  if (a.group == 64) return launch_typed<kX, kGated, 64>(a, s);
  return launch_typed<kX, kGated, 128>(a, s);
}

template <Q4X kX>
hipError_t launch_x(const Q4Args& a, bool gated, hipStream_t s) {
  return gated ? launch_group<kX, true>(a, s) : launch_group<kX, false>(a, s);
}

}  // namespace

hipError_t launch_q4(const Q4Args& a, Q4X x_type, bool gated, hipStream_t s) {
  switch (x_type) {
    case Q4X::bf16:
      return launch_x<Q4X::bf16>(a, gated, s);
    case Q4X::f32:
      return launch_x<Q4X::f32>(a, gated, s);
    default:
      return launch_x<Q4X::e4m3>(a, gated, s);
  }
}

hipError_t launch_q4_quantize(const uint16_t* W, int N, int K, int group, uint8_t* codes, uint16_t* scales,
                              hipStream_t s) {
  const int64_t G = (K + group - 1) / group, lanes = static_cast<int64_t>(N) * G * (group / 8);
  q4_quantize_kernel<<<static_cast<unsigned>((lanes + 255) / 256), 256, 0, s>>>(W, N, K, group, codes, scales);
  return hipGetLastError();
}

}  // namespace twell
