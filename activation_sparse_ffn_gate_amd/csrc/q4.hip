// Products with 4-bit weights and group scales for gfx950:
//
//   y[m, n] = sx[m] sum over k of x[m, k] s[n, k / g] (q[n, k] - z[n, k / g])
//
// and the gated pair h = z > 0 ? z u : 0 of two such products.
//
// A byte s000mmmm read as e4m3 is (-1)^s m 2^-9 exactly for m = 0..15 (m < 8
// are that format's subnormals, 8..15 its first binade), so one
// v_cvt_scalef32_pk_bf16_fp8 by 2^9 turns two codes into bf16 integers. z is
// taken off inside the sums of 32 values of K, not as z sum(x) from a group's:
// that keeps groups exact in which one large weight leaves all others at zero.
// Their products then are zeros or cancel at once, where they would be large
// terms. Where z goes is a choice by which unit has room: as sign and magnitude
// of q - z in the codes (sign_magnitude, 1.25 integer operations a weight) or
// as a second matrix product of the same x by -z (add_step). 16 rows and 32
// rows take the second (24 rows by 8192 units and K 2048: 11.2 us against
// 11.9), 64 and 128 rows, where codes are turned once for 4 or 8 products, the
// first (256 rows by 10240 units and K 2560, with a slower epilogue than now: 39
// us against 42). x in e4m3 is
// turned into bf16 too, exactly: the e4m3 matrix product itself sums with too
// few bits (relative error 1e-5 over 2048 values of K where the bf16 product
// has 6e-8). fp32 x is cut into three bf16 parts that add up to it exactly (8 +
// 8 + 8 bits, down to the 2^-133 that bf16 ends at: all of |x| >= 2^-110). All
// products are exact in fp32; sums are held in fp32 per group, then scaled and
// added.
//
// v_mfma_f32_16x16x32_bf16: 16 rows of x by 16 units, 32 values of K, which
// lie inside one group (groups are 32, 64 or 128). Lane l holds row or unit
// l % 16 and 8 consecutive k at 8 (l / 16); the result has unit l % 16 and
// rows 4 (l / 16) + 0..3. A wave takes K in chunks of 128: lane l loads 16
// consecutive bytes of its unit's row, and a 4 x 4 transposition between the
// four 16-lane quarters (two v_permlane32_swap, two v_permlane16_swap) gives
// register i the codes of K values 32 i + 8 (l / 16) + 0..7. Low nibbles are
// even k, high nibbles odd k, so x operands are put in that order too (0, 2,
// 4, 6, 1, 3, 5, 7 of each 8).
//
// Few rows, or few of both (plan() has the rule): q4_tile_kernel. What bounds it
// is the latency of a few dependent steps (a launch, loads, a barrier, LDS) and
// not the codes' bytes: one row by 8192 units and K 2048 takes 5.1 us a launch in
// a graph, where the 8.7 MB take 1.6 us at the rate of a large copy and an empty
// launch 2.4 us. More: q4_wide_kernel, bound by turning codes into operands and
// the matrix instructions, which share a SIMD's issue (64 vector operations and
// 16 of these matrix instructions take 0.8 of the sum of what they take apart).
#include <algorithm>

#include "block_device.hpp"

namespace twell {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kChunk = 128;

__device__ __forceinline__ f32x4 mfma_bf16(u32x4_t a, u32x4_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
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

// Two e4m3 bytes (0, 1 or 2, 3 of w), times a power of two, as a pair of bf16.
template <bool kHigh>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, kHigh));
}

// 8 bf16 in memory order, put into the order of the codes.
__device__ __forceinline__ u32x4_t even_odd(u32x4_t w) {
  return u32x4_t{__builtin_amdgcn_perm(w[1], w[0], 0x05040100u), __builtin_amdgcn_perm(w[3], w[2], 0x05040100u),
                 __builtin_amdgcn_perm(w[1], w[0], 0x07060302u), __builtin_amdgcn_perm(w[3], w[2], 0x07060302u)};
}

// Three bf16 parts of v that add up to it: the top 8 significant bits, then
// those of what is left.
__device__ __forceinline__ void cut3(float v, uint32_t* part) {
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    part[s] = __float_as_uint(v) & 0xFFFF0000u;
    v -= __uint_as_float(part[s]);
  }
}

// Elements of x of one kind: bytes or words of 8 consecutive k as they lie in
// memory, and the matrix operands (kParts of them) they become. `planes` is
// fp32 that an earlier kernel has cut, here the hidden matrix between the two
// products of the FFN: three planes of parts, each [K / 8][q4_rows(M)] blocks
// of 8 k in the order of the codes (the last block of a cut K ends in zeros),
// so that a wave's operand is contiguous. (Two parts would be a third less to
// move and multiply, but lose up to 2^-18 of a value: relative errors of 1 to 4e-6
// in y, which has under 7e-7 with three.)
template <Q4X kX>
struct XBlock {
  static constexpr int kParts = kX == Q4X::f32 || kX == Q4X::planes ? 3 : 1;
  static constexpr int kWords = kX == Q4X::e4m3 ? 2 : kX == Q4X::bf16 ? 4 : kX == Q4X::f32 ? 8 : 12;
  static constexpr int kBytes = kX == Q4X::e4m3 ? 1 : kX == Q4X::f32 ? 4 : 2;  // of an element
  uint32_t w[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void put(int at, u32x4_t v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[at + i] = v[i];
  }
  __device__ __forceinline__ u32x4_t get(int at) const { return u32x4_t{w[at], w[at + 1], w[at + 2], w[at + 3]}; }

  // The 8 elements at p; planes: the block at p of each plane, `plane` bytes apart.
  __device__ __forceinline__ void load(const uint8_t* p, int64_t plane) {
    if constexpr (kX == Q4X::e4m3) {
      __builtin_memcpy(w, p, 8);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) put(4 * i, load16_any(p + (kX == Q4X::planes ? i * plane : 16 * i)));
    }
  }
  // The first n (0 to 7) elements at p, zeros after them.
  __device__ __forceinline__ void load_cut(const uint8_t* p, int n) {
    clear();
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      if (i >= n) continue;
      if constexpr (kX == Q4X::e4m3) {
        w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
      } else if constexpr (kX == Q4X::f32) {
        w[i] = __float_as_uint(reinterpret_cast<const float*>(p)[i]);
      } else {
        w[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i & 1));
      }
    }
  }
  __device__ __forceinline__ void operands(u32x4_t* x) const {
    if constexpr (kX == Q4X::planes) {
#pragma unroll
      for (int p = 0; p < kParts; ++p) x[p] = get(4 * p);
    } else if constexpr (kX == Q4X::bf16) {
      x[0] = even_odd(get(0));
    } else if constexpr (kX == Q4X::e4m3) {
      const uint32_t e = __builtin_amdgcn_perm(w[1], w[0], 0x06040200u), o = __builtin_amdgcn_perm(w[1], w[0], 0x07050301u);
      x[0] = u32x4_t{pair_bf16<false>(e, 1.f), pair_bf16<true>(e, 1.f), pair_bf16<false>(o, 1.f), pair_bf16<true>(o, 1.f)};
    } else {
      uint32_t h[8][3];
#pragma unroll
      for (int i = 0; i < 8; ++i) cut3(__uint_as_float(w[i]), h[i]);
#pragma unroll
      for (int s = 0; s < 3; ++s)
        x[s] = u32x4_t{(h[0][s] >> 16) | h[2][s], (h[4][s] >> 16) | h[6][s], (h[1][s] >> 16) | h[3][s],
                       (h[5][s] >> 16) | h[7][s]};
    }
  }
};

// Where element (m, k) of x lies, k a multiple of 8, in bytes.
template <Q4X kX>
__device__ __forceinline__ int64_t x_offset(int64_t m, int64_t k, int64_t M, int64_t K) {
  return kX == Q4X::planes ? (k / 8 * q4_rows(M) + m) * 16 : (m * K + k) * XBlock<kX>::kBytes;
}
__host__ __device__ inline int64_t plane_bytes(int64_t M, int64_t K) { return q4_pad(K) * q4_rows(M) * 2; }

// Four codes (bytes 0..15) as q - z in sign and magnitude; zero = 128 - z in
// every byte (z <= 15, so no byte carries into the next).
__device__ __forceinline__ uint32_t sign_magnitude(uint32_t q, uint32_t zero) {
  const uint32_t d = q + zero;                            // 128 + (q - z)
  const uint32_t neg = ~(d >> 7) & 0x01010101u;           // 1 where q < z
  const uint32_t m = (d ^ (0x80808080u - neg)) + neg;     // d ^ 0x80, or (d ^ 0x7F) + 1
  return m | (neg << 7);
}

// The 8 codes of c as the matrix operand q - z.
__device__ __forceinline__ u32x4_t code_operand(uint32_t c, uint32_t zero) {
  const uint32_t lo = sign_magnitude(c & 0x0F0F0F0Fu, zero);
  const uint32_t hi = sign_magnitude((c >> 4) & 0x0F0F0F0Fu, zero);
  return u32x4_t{pair_bf16<false>(lo, 512.f), pair_bf16<true>(lo, 512.f), pair_bf16<false>(hi, 512.f),
                 pair_bf16<true>(hi, 512.f)};
}

// The 8 codes of c as the matrix operand q, beside one that is -z throughout.
__device__ __forceinline__ u32x4_t plain_operand(uint32_t c) {
  const uint32_t lo = c & 0x0F0F0F0Fu, hi = (c >> 4) & 0x0F0F0F0Fu;
  return u32x4_t{pair_bf16<false>(lo, 512.f), pair_bf16<true>(lo, 512.f), pair_bf16<false>(hi, 512.f),
                 pair_bf16<true>(hi, 512.f)};
}

// A code operand with k in memory order.
__device__ __forceinline__ u32x4_t memory_order(u32x4_t q) {
  return u32x4_t{__builtin_amdgcn_perm(q[2], q[0], 0x05040100u), __builtin_amdgcn_perm(q[2], q[0], 0x07060302u),
                 __builtin_amdgcn_perm(q[3], q[1], 0x05040100u), __builtin_amdgcn_perm(q[3], q[1], 0x07060302u)};
}

// A wave's 16 units of a weight: wave-uniform bases and 32-bit offsets of the
// lane's unit (past the matrix: of its last unit, computed and not stored).
struct Units {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;  // nullable
  int64_t kb;            // code bytes of a unit
  int G;                 // groups of a unit
  uint32_t code_off, unit_off;

  __device__ __forceinline__ Units(const Q4Weight& w, int first, int N, int K, int group, int lane) {
    kb = (static_cast<int64_t>(K) + 1) / 2;
    G = static_cast<int>((static_cast<int64_t>(K) + group - 1) / group);
    first = min(first, N - 1);
    codes = w.codes + first * kb;
    scales = w.scales + static_cast<int64_t>(first) * G;
    zeros = w.zeros == nullptr ? nullptr : w.zeros + static_cast<int64_t>(first) * G;
    unit_off = min(lane & 15, N - 1 - first);
    code_off = unit_off * static_cast<uint32_t>(kb) + (lane >> 4) * 16;
  }

  // The lane's 16 code bytes of whole chunk c.
  __device__ __forceinline__ u32x4_t load(int c) const {
    return load16_any(codes + static_cast<int64_t>(c) * 64 + code_off);
  }
  // Of the chunk that K ends in: past it x is zero (or the operand made zero),
  // so any code will do.
  __device__ __forceinline__ u32x4_t load_cut(int c) const {
    const uint32_t row = unit_off * static_cast<uint32_t>(kb), last = row + static_cast<uint32_t>(kb) - 1;
    u32x4_t w = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i >> 2] |= static_cast<uint32_t>(codes[min(code_off + c * 64 + i, last)]) << (8 * (i & 3));
    return w;
  }
  // Scale (high half, bf16) and zero point (low byte) of a unit of the 16 at
  // group g; past K, where x is zero, the last group's.
  __device__ __forceinline__ uint32_t scale(uint32_t u, int g) const {
    const int64_t at = static_cast<int64_t>(u) * G + min(g, G - 1);
    return static_cast<uint32_t>(scales[at]) << 16 | (zeros != nullptr ? zeros[at] & 15u : 8u);
  }
};

// 128 - z of a scale word in every byte, and -z as a pair of bf16 (integers up
// to 15 are exact).
__device__ __forceinline__ uint32_t zero_bytes(uint32_t sz) {
  return __builtin_amdgcn_perm(0u, 128u - (sz & 15u), 0u);
}
__device__ __forceinline__ uint32_t minus_zero(uint32_t sz) {
  const uint32_t f = __float_as_uint(-static_cast<float>(sz & 15u));
  return f >> 16 | f;
}
__device__ __forceinline__ float scale_of(uint32_t sz) { return __uint_as_float(sz & 0xFFFF0000u); }

// One matrix instruction's K of up to 16 rows: acc + x (q - z). With one part
// of x, as q and then -z by the same x: two matrix instructions instead of the
// 12 integer operations of sign_magnitude, as vector operations are what few
// rows have least room for. acc leaves each pair holding the sum over those 32
// values, so what rounding the intermediate sum of x q costs stays that of 32
// terms.
template <int kParts>
__device__ __forceinline__ f32x4 add_step(const u32x4_t* x, uint32_t codes, uint32_t sz, f32x4 acc) {
  if constexpr (kParts == 1) {
    const uint32_t z = minus_zero(sz);
    acc = mfma_bf16(x[0], plain_operand(codes), acc);
    return mfma_bf16(x[0], u32x4_t{z, z, z, z}, acc);
  } else {
    const u32x4_t q = code_operand(codes, zero_bytes(sz));
#pragma unroll
    for (int p = 0; p < kParts; ++p) acc = mfma_bf16(x[p], q, acc);
    return acc;
  }
}

// Scales and zero points of kCols units (16 a wave, waves of the gated pair's
// second weight among them) and kGroups groups from `first_group` on, put into
// LDS as words [group][kCols + 1] by kThreads threads, consecutive ones along
// the groups. Nothing is done with the loaded values before put(), so fetch()
// waits for nothing.
template <int kCols, int kGroups, int kThreads>
struct ScaleStage {
  static constexpr int kEach = (kCols * kGroups + kThreads - 1) / kThreads;
  static constexpr int kStride = kCols + 1;
  static constexpr int kBytes = kGroups * kStride * 4;
  uint16_t s[kEach];
  uint8_t z[kEach];

  // locate(column, group, scale, zero) gives where the two lie.
  template <class Fn>
  __device__ __forceinline__ void fetch(int first_group, Fn&& locate) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int id = min(static_cast<int>(threadIdx.x) + kThreads * i, kCols * kGroups - 1);
      uint64_t scale, zero;  // addresses in global memory
      locate(id / kGroups, first_group + id % kGroups, scale, zero);
      s[i] = *(const __attribute__((address_space(1))) uint16_t*)scale;
      z[i] = *(const __attribute__((address_space(1))) uint8_t*)zero;
    }
  }
  // has(column): whether its weight has zero points.
  template <class Fn>
  __device__ __forceinline__ void put(uint32_t* lds, Fn&& has) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int id = threadIdx.x + kThreads * i;
      if (kCols * kGroups % kThreads == 0 || id < kCols * kGroups)
        lds[id % kGroups * kStride + id / kGroups] =
            static_cast<uint32_t>(s[i]) << 16 | (has(id / kGroups) ? z[i] & 15u : 8u);
    }
  }
};

// Units that are stored: the planes' last block is filled with zeros.
__device__ __forceinline__ int stored_units(const Q4Args& a) {
  return a.y_type == Q4Y::planes ? static_cast<int>(q4_pad(a.N)) : a.N;
}

// One output from its sums z (and u) and its row's scale.
__device__ __forceinline__ float output(const Q4Args& a, float z, float u, float sx) {
  const float v = z * sx;
  return !a.gated ? v : v > 0.f ? v * (u * sx) : 0.f;
}

// Output v of row m, to y as it is or to h's planes.
template <Q4Y kY>
__device__ __forceinline__ void put_y(const Q4Args& a, int64_t m, int unit, float v) {
  if constexpr (kY == Q4Y::f32) {
    static_cast<float*>(a.y)[m * a.N + unit] = v;
  } else if constexpr (kY == Q4Y::bf16) {
    store1(static_cast<uint16_t*>(a.y) + m * a.N + unit, v);
  } else {
    if (unit >= a.N) v = 0.f;
    uint32_t part[3];
    cut3(v, part);
    if (!isfinite(v)) {  // stays what it is
      part[0] = pack_bf16(0.f, v);
      part[1] = part[2] = 0u;
    }
    uint8_t* y = static_cast<uint8_t*>(a.y) + x_offset<Q4X::planes>(m, unit & ~7, a.M, a.N);
    y += (unit & 6) + 8 * (unit & 1);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint16_t*>(y + p * plane_bytes(a.M, a.N)) = static_cast<uint16_t>(part[p] >> 16);
  }
}

// Calls f with the type of y as a constant.
template <class Fn>
__device__ __forceinline__ void by_y(const Q4Args& a, Fn&& f) {
  if (a.y_type == Q4Y::f32) {
    f(std::integral_constant<Q4Y, Q4Y::f32>{});
  } else if (a.y_type == Q4Y::bf16) {
    f(std::integral_constant<Q4Y, Q4Y::bf16>{});
  } else {
    f(std::integral_constant<Q4Y, Q4Y::planes>{});
  }
}

// The end of a wave: unit's sums for rows m + 16 t + 0..3 of each of kTiles
// tiles. With K split over workgroups the sums go to the partials [split][z,
// u][M][N] that q4_join_kernel adds. The rows' scales are loaded before anything
// is stored, since a wait for a load is a wait for the stores before it too.
template <int kTiles>
__device__ __forceinline__ void finish(const Q4Args& a, int unit, int m, const f32x4* z, const f32x4* u) {
  if (a.splits > 1) {
    if (unit >= a.N) return;
    const int64_t size = static_cast<int64_t>(a.M) * a.N;
    float* p = a.part + (blockIdx.z * (a.gated ? 2 : 1)) * size + unit;
#pragma unroll
    for (int i = 0; i < 4 * kTiles; ++i) {
      const int row = m + 16 * (i / 4) + i % 4;
      if (row >= a.M) continue;
      p[static_cast<int64_t>(row) * a.N] = z[i / 4][i % 4];
      if (a.gated) p[size + static_cast<int64_t>(row) * a.N] = u[i / 4][i % 4];
    }
    return;
  }
  if (unit >= stored_units(a)) return;
  float sx[4 * kTiles], v[4 * kTiles];
#pragma unroll
  for (int i = 0; i < 4 * kTiles; ++i) sx[i] = 1.f;
  if (a.x_scale != nullptr) {
#pragma unroll
    for (int i = 0; i < 4 * kTiles; ++i) sx[i] = a.x_scale[min(m + 16 * (i / 4) + i % 4, a.M - 1)];
  }
#pragma unroll
  for (int i = 0; i < 4 * kTiles; ++i) v[i] = output(a, z[i / 4][i % 4], u[i / 4][i % 4], sx[i]);
  by_y(a, [&](auto y) {
#pragma unroll
    for (int i = 0; i < 4 * kTiles; ++i) {
      const int row = m + 16 * (i / 4) + i % 4;
      if (row < a.M) put_y<decltype(y)::value>(a, row, unit, v[i]);
    }
  });
}

__global__ __launch_bounds__(256) void q4_join_kernel(Q4Args a) {
  const int units = stored_units(a);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = id / units;
  const int unit = static_cast<int>(id - m * units);
  if (m >= a.M) return;
  const int64_t size = static_cast<int64_t>(a.M) * a.N;
  const int mats = a.gated ? 2 : 1;
  const float sx = a.x_scale != nullptr ? a.x_scale[m] : 1.f;
  float z = 0.f, u = 0.f;
  if (unit < a.N) {
    const float* p = a.part + m * a.N + unit;
    for (int s = 0; s < a.splits; ++s) {
      z += p[(s * mats) * size];
      if (a.gated) u += p[(s * mats + 1) * size];
    }
  }
  by_y(a, [&](auto y) { put_y<decltype(y)::value>(a, m, unit, output(a, z, u, sx)); });
}

// 16 rows of x a workgroup. It has kWN times 16 units (the gated
// pair: half of them the up weight's) and 8 / kWN waves on each 16, which take
// kDepth chunks of K in a row each. x and the scales go through LDS, kSlice
// values of K at a time, x turned into matrix operands once: blocks of 8 k by
// row, a block's 16 rows followed by 16 bytes so that the writes (16 blocks of
// one row side by side, for whole lines of x) spread over the banks. Each
// request takes a microsecond and a wave computes a chunk in a fraction of one,
// so all of a slice's codes are requested at once, and the next slice's x,
// scales and codes while this one is computed. Loads are unconditional (past K
// of the last whole chunk), so that the compiler can count them. With the codes
// under way while x and the scales are put into LDS the gated pair of 16 rows by
// 8192 units and K 2048 takes 8.8 us, with them waited for first 9.6.
template <Q4X kX, int kWN>
struct TileShape {
  static constexpr int kRows = 16, kWK = 8 / kWN;
  static constexpr int kParts = XBlock<kX>::kParts;
  static constexpr int kSlice = kParts == 1 ? 2048 : 1024;
  static constexpr int kDepth = kSlice / kChunk / kWK;
  static constexpr int kStride = kRows * 16 + 16;  // bytes from a block of 8 k to the next
  static constexpr int kPart = kSlice / 8 * kStride;
  static constexpr int kBlocks = kSlice / 8 * kRows / 512;  // a thread stages
};

template <Q4X kX, int kGroup, int kWN>
__global__ __launch_bounds__(512) void q4_tile_kernel(Q4Args a) {
  using S = TileShape<kX, kWN>;
  using Scales = ScaleStage<16 * kWN, S::kSlice / kGroup, 512>;
  constexpr int kWK = S::kWK, kParts = S::kParts, kDepth = S::kDepth;
  constexpr int kSteps = kGroup / 32;  // matrix instructions of a group
  constexpr int kSliceChunks = S::kSlice / kChunk;
  static_assert(kParts * S::kPart >= 8 * 1024, "the waves' sums fit");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kParts * S::kPart];
  __shared__ uint32_t lds_scale[Scales::kBytes / 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / kWK, wk = wave % kWK;
  const int quarter = lane >> 4, col = lane & 15;
  const int first = (a.gated ? blockIdx.x * (kWN / 2) + wn / 2 : blockIdx.x * kWN + wn) * 16;
  const int full = a.K / kChunk, chunks = (a.K + kChunk - 1) / kChunk;
  const int begin = blockIdx.z * a.split_chunks, end = min(chunks, begin + a.split_chunks);  // begin: whole slices
  const Units units(a.gated && (wn & 1) ? a.up : a.w, first, a.N, a.K, kGroup, lane);

  // A thread stages kBlocks blocks of one row, 256 k apart: 16 threads side by
  // side along K, then the 16 rows; of planes, where rows lie side by side, the
  // other way round.
  constexpr bool kPlanes = kX == Q4X::planes;
  XBlock<kX> raw[S::kBlocks];
  const int m = kPlanes ? threadIdx.x & 15 : threadIdx.x / 16 % S::kRows;  // of the tile
  const int m0 = blockIdx.y * S::kRows, rows = a.M - m0;
  const int k0 = kPlanes ? threadIdx.x / 16 * 8 : 8 * (threadIdx.x & 15) + threadIdx.x / 256 * 128;
  const int64_t k_bytes = kPlanes ? 2 * q4_rows(a.M) : XBlock<kX>::kBytes;  // from k to k + 1, 8 at a time
  const int64_t plane = plane_bytes(a.M, a.K);
  const int k_end = kPlanes ? static_cast<int>(q4_pad(a.K)) : a.K;
  const uint8_t* xp = static_cast<const uint8_t*>(a.x) + k0 * k_bytes;
  xp += x_offset<kX>(m0 + min(m, rows - 1), 0, a.M, a.K);
  auto fetch_x = [&](int slice_k) {
    if (m >= rows) return;  // rows past M are computed from what LDS holds and not stored
#pragma unroll
    for (int i = 0; i < S::kBlocks; ++i) {
      raw[i].clear();
      if (slice_k + k0 + 256 * i + 8 <= k_end) raw[i].load(xp + (slice_k + 256 * i) * k_bytes, plane);
    }
  };
  auto put = [&](const XBlock<kX>& b, int k) {
    u32x4_t x[kParts];
    b.operands(x);
#pragma unroll
    for (int p = 0; p < kParts; ++p) lds_store16(lds, p * S::kPart + k / 8 * S::kStride + m * 16, x[p]);
  };
  auto put_x = [&] {
    if (m >= rows) return;
#pragma unroll
    for (int i = 0; i < S::kBlocks; ++i) put(raw[i], k0 + 256 * i);
  };
  // The block that K ends in, left zero by put_x: by the thread of its row and place.
  auto put_cut = [&](int slice_k) {
    const int cut = (a.K & ~7) - slice_k;
    if (!kPlanes && m < rows && a.K % 8 != 0 && cut >= 0 && cut < S::kSlice && (cut - k0) % 256 == 0) {
      XBlock<kX> b;
      b.load_cut(xp + (slice_k + cut - k0) * k_bytes, a.K & 7);
      put(b, cut);
    }
  };
  // The two weights' bases in scalar registers, so that a lane selects between
  // them and does not load the one it wants. Without zero points the scales'
  // bytes are read in their place and not used.
  const bool w_has = a.w.zeros != nullptr, u_has = a.gated && a.up.zeros != nullptr;
  const uint64_t ws = reinterpret_cast<uint64_t>(a.w.scales), us = reinterpret_cast<uint64_t>(a.up.scales);
  const uint64_t wz = w_has ? reinterpret_cast<uint64_t>(a.w.zeros) : ws;
  const uint64_t uz = u_has ? reinterpret_cast<uint64_t>(a.up.zeros) : us;
  auto is_up = [&](int column) { return a.gated && (column / 16 & 1); };
  Scales scales;
  auto fetch_scales = [&](int slice_k) {
    scales.fetch(slice_k / kGroup, [&](int column, int g, uint64_t& s, uint64_t& z) {
      const int w = column / 16;  // wave of the workgroup's columns
      const int tile = static_cast<int>(blockIdx.x) * (a.gated ? kWN / 2 : kWN) + (a.gated ? w / 2 : w);
      const int64_t at = static_cast<int64_t>(min(tile * 16 + column % 16, a.N - 1)) * units.G + min(g, units.G - 1);
      const uint64_t up = is_up(column) ? ~uint64_t(0) : 0;  // (masks: a choice of addresses becomes a load of one)
      s = (ws ^ ((ws ^ us) & up)) + 2 * at;
      z = (wz ^ ((wz ^ uz) & up)) + at;
    });
  };
  auto stage = [&](int slice_k) {
    put_x();
    scales.put(lds_scale, [&](int column) { return is_up(column) ? u_has : w_has; });
    put_cut(slice_k);
  };

  f32x4 total = {};
  auto add = [&](u32x4_t w, int in_slice) {  // chunk of the slice in LDS
    const u32x4_t v = transpose_quarters(w);
    const uint8_t* xl = lds + (in_slice * 16 + quarter) * S::kStride + col * 16;
    const uint32_t* sl = lds_scale + in_slice * (kChunk / kGroup) * Scales::kStride + wn * 16 + col;
    f32x4 acc;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4_t xs[kParts];
#pragma unroll
      for (int p = 0; p < kParts; ++p) xs[p] = lds_load16(xl, p * S::kPart + 4 * i * S::kStride);
      if (i % kSteps == 0) acc = f32x4{};
      const uint32_t sz = sl[i / kSteps * Scales::kStride];
      acc = add_step<kParts>(xs, v[i], sz, acc);
      if (i % kSteps == kSteps - 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) total[r] = fmaf(scale_of(sz), acc[r], total[r]);
      }
    }
  };

  u32x4_t w[kDepth];
  auto fetch_codes = [&](int i, int s0) { w[i] = units.load(min(s0 + wk * kDepth + i, full - 1)); };
  // x and scales first: loads come back in order, and codes may still be on
  // their way while those are put into LDS
  fetch_x(begin * kChunk);
  fetch_scales(begin * kChunk);
  keep_order();
  if (full > 0) {  // (put in both branches: after them the codes might not have been requested)
#pragma unroll
    for (int i = 0; i < kDepth; ++i) fetch_codes(i, begin);
    stage(begin * kChunk);
  } else {
    stage(begin * kChunk);
  }
  int s0 = begin;
#pragma unroll 1
  for (; s0 + kSliceChunks < end; s0 += kSliceChunks) {  // (so its chunks are whole)
    lds_barrier();
    fetch_x((s0 + kSliceChunks) * kChunk);
    fetch_scales((s0 + kSliceChunks) * kChunk);
    keep_order();
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      add(w[i], wk * kDepth + i);
      fetch_codes(i, s0 + kSliceChunks);
    }
    lds_barrier();  // every wave has read the slice
    stage((s0 + kSliceChunks) * kChunk);
  }
  lds_barrier();
#pragma unroll
  for (int i = 0; i < kDepth; ++i)
    if (s0 + wk * kDepth + i < min(full, end)) add(w[i], wk * kDepth + i);
  if (full < end && wk == (full - s0) / kDepth) add(units.load_cut(full), full - s0);

  __syncthreads();
  float* red = reinterpret_cast<float*>(lds);  // sums of a wave at [wave][r][lane]
  if (wave > 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) red[(wave * 4 + r) * 64 + lane] = total[r];
  }
  __syncthreads();
  if (wk > 0 || (a.gated && (wn & 1))) return;
  f32x4 up = {};
#pragma unroll
  for (int o = 0; o < kWK; ++o)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (o > 0) total[r] += red[((wn * kWK + o) * 4 + r) * 64 + lane];
      if (a.gated) up[r] += red[(((wn + 1) * kWK + o) * 4 + r) * 64 + lane];
    }
  finish<1>(a, first + col, m0 + 4 * quarter, &total, &up);
}

// x [M, K] into planes of matrix operands (1 for e4m3, and bf16 that
// q4_wide_kernel cannot read as it is; 3 for fp32). A wave has 8 blocks of 8 k
// side by side (whole lines of bf16) of 8 rows.
template <Q4X kX>
__global__ __launch_bounds__(256) void q4_planes_kernel(Q4Args a, uint8_t* out) {
  constexpr int kParts = XBlock<kX>::kParts;
  const int lane = threadIdx.x & 63, b = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 8 + (lane & 7);
  const int m = blockIdx.y * 8 + (lane >> 3), k = 8 * b;
  if (k >= a.K || m >= a.M) return;
  const uint8_t* p = static_cast<const uint8_t*>(a.x) + x_offset<kX>(m, k, a.M, a.K);
  XBlock<kX> v;
  if (k + 8 <= a.K) {
    v.load(p, 0);
  } else {
    v.load_cut(p, a.K - k);
  }
  u32x4_t x[kParts];
  v.operands(x);
#pragma unroll
  for (int i = 0; i < kParts; ++i)
    store16_any(out + i * plane_bytes(a.M, a.K) + x_offset<Q4X::planes>(m, k, a.M, a.K), x[i]);
}

// Many rows, from planes of matrix operands (kParts of them), or (kRowMajor)
// bf16 x as it is, where its rows are 16-byte pieces throughout. A workgroup
// has 16 kMT rows and kWN waves of 16 units side by side (for the gated pair
// every other wave has the up weight of its neighbour's units), so that codes
// are turned into operands once for all its rows. x comes through a ring of
// kStages chunks in LDS, written by global_load_lds: before a chunk is computed
// the last of the next kStages - 1 is requested, and its codes with it. One
// barrier a chunk: past it every wave's part of the chunk has landed and every
// wave has read the chunk before, whose place the next request takes. The counted
// wait before it leaves what was requested since under way, but it is not the
// only one: in every pass of the loop over kStages - 1 chunks the compiler waits
// once for all loads, at the loop's head where the codes carried around it are
// copied, and with groups of 32 and 64 again where the words just loaded are cut
// into scales and zero points. So with three stages a request has between one
// and two chunks of time, and not always two. In LDS planes keep
// their order, [block][row], where the 16 rows of an operand lie side by side.
// A row-major chunk is 256 bytes a row, piece p of row r at p ^ (r % 16), so
// that 16 rows' reads of one piece meet different banks; there k comes in
// memory order, and the code operands are put into it. Three chunks in the
// ring, two where a chunk is more than 16 KB, so that two workgroups fit a CU
// (64 rows by 8192 units and K 2048: 14.4 us with three, 15.6 with two). 256
// rows by 10240 units and K 2560 in groups of 32 with zero points take 37 to 39
// us: 13.4 GFLOP at 0.35 PFLOP/s. A chunk costs a wave 214 vector instructions
// beside its 16 matrix ones: 64 to scale the sums of groups of 32 (16 for groups
// of 128, which take 30 us, of 64 33), some 100 to turn its codes; the waits
// above have their part in the difference too.
template <int kParts, bool kRowMajor, int kGroup, int kMT, int kWN>
__global__ __launch_bounds__(64 * kWN, 2) void q4_wide_kernel(Q4Args a) {
  constexpr int kPer = kChunk / kGroup, kSteps = 4 / kPer;
  constexpr int kRows = 16 * kMT, kPart = 256 * kRows;  // bytes of a chunk of one plane
  constexpr int kStages = kParts * kMT <= 4 ? 3 : 2;
  constexpr bool kPair = kParts == 1 && kMT == 2;  // q and then -z by the same x
  constexpr int kDma = 4 * kMT * kParts / kWN;  // a wave's requests of 1 KB a chunk
  constexpr int kRed = kWN / 2 * kMT * 1024;    // up sums of the gated pair
  constexpr int kLds = kStages * kParts * kPart;
  static_assert(kLds >= kRed && kDma * kWN == 4 * kMT * kParts, "LDS and requests");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quarter = lane >> 4, col = lane & 15;
  // Row tiles of the same units are neighbours on one XCD (workgroup b runs on XCD b % 8).
  const int items = gridDim.x, lin = items % 8 == 0 ? blockIdx.x % 8 * (items / 8) + blockIdx.x / 8 : blockIdx.x;
  const int row_tiles = (a.M + kRows - 1) / kRows;
  const int tile = lin / row_tiles, m0 = (lin - tile * row_tiles) * kRows;
  const int first = (a.gated ? tile * (kWN / 2) + wave / 2 : tile * kWN + wave) * 16;
  const int chunks = (a.K + kChunk - 1) / kChunk, full = a.K / kChunk;
  const int begin = blockIdx.z * a.split_chunks, end = min(chunks, begin + a.split_chunks);
  const Units units(a.gated && (wave & 1) ? a.up : a.w, first, a.N, a.K, kGroup, lane);
  const int64_t plane = plane_bytes(a.M, a.K);
  const int ld = static_cast<int>(q4_rows(a.M));
  const int blocks = static_cast<int>(q4_pad(a.K) / 8);

  // Request i of a chunk is KB e of a plane's [block][row] pieces of 16 bytes,
  // or of the rows' pieces.
  const uint8_t* x_rows = static_cast<const uint8_t*>(a.x) + static_cast<int64_t>(m0) * a.K * 2;
  auto request = [&](int c, int slot, int last_block) {
    uint8_t* to = lds + slot * (kParts * kPart);
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int d = wave * kDma + i, p = d / (4 * kMT), e = d % (4 * kMT);
      if constexpr (kRowMajor) {
        const int r = 4 * e + (lane >> 4), piece = (lane ^ r) & 15;
        const uint32_t row = static_cast<uint32_t>(min(r, a.M - 1 - m0)) * (2 * a.K);  // past M: computed, not stored
        const uint8_t* base = x_rows + static_cast<int64_t>(c) * 256;
        const int back = last_block >= 0 ? max(16 * c + piece - last_block, 0) : 0;  // past K: its last piece
        dma16(reinterpret_cast<const uint16_t*>(base + row + (piece - back) * 16), to + e * 1024);
        continue;
      }
      const int b0 = 64 * e / kRows, db = lane / kRows;  // blocks of this KB
      const int b = last_block >= 0 ? min(16 * c + b0 + db, last_block) - db : 16 * c + b0;
      const uint8_t* base = static_cast<const uint8_t*>(a.x) + p * plane + (static_cast<int64_t>(b) * ld + m0) * 16;
      const uint32_t off = (db * ld + (64 * e + lane) % kRows) * 16;
      dma16(reinterpret_cast<const uint16_t*>(base + off), to + p * kPart + e * 1024);
    }
  };

  // A lane's codes, scales and zero points of a chunk; kLoads loads of a whole one.
  struct Codes {
    u32x4_t w;
    uint16_t s[kPer];
    uint8_t z[kPer];
  };
  constexpr int kLoads = 3;
  const uint8_t* zeros = units.zeros != nullptr ? units.zeros : reinterpret_cast<const uint8_t*>(units.scales);
  const uint32_t group_off = units.unit_off * units.G;
  auto load = [&](Codes& s, int c) {
    s.w = units.load(c);
    __builtin_memcpy(s.s, units.scales + c * kPer + group_off, 2 * kPer);
    __builtin_memcpy(s.z, zeros + c * kPer + group_off, kPer);
  };
  auto load_any = [&](Codes& s, int c) {
    if (c < full) {
      load(s, c);
    } else {
      s.w = units.load_cut(c);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t sz = units.scale(units.unit_off, c * kPer + i);
        s.s[i] = static_cast<uint16_t>(sz >> 16);
        s.z[i] = static_cast<uint8_t>(sz);
      }
    }
  };

  f32x4 total[kMT] = {};
  // Chunk c, landed in LDS at `slot`, with its codes. kCut: K may end in it.
  auto compute = [&](int c, int slot, const Codes& w, auto cut) {
    constexpr bool kCut = decltype(cut)::value;
    const u32x4_t v = transpose_quarters(w.w);
    const uint8_t* xl = lds + slot * (kParts * kPart) + (kRowMajor ? col * 256 : quarter * (kRows * 16) + col * 16);
    f32x4 acc[kMT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4_t xs[kMT][kParts];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int p = 0; p < kParts; ++p)
          xs[mt][p] = kRowMajor ? lds_load16(xl, ((4 * i + quarter) ^ col) * 16 + 4096 * mt)
                                : lds_load16(xl, p * kPart + 4 * i * (kRows * 16) + 256 * mt);
      const uint32_t sz = units.zeros != nullptr ? w.z[i / kSteps] : 8u;
      const uint32_t mz = minus_zero(sz);
      u32x4_t q = kPair ? plain_operand(v[i]) : code_operand(v[i], zero_bytes(sz));
      if constexpr (kRowMajor) q = memory_order(q);
      u32x4_t z = {mz, mz, mz, mz};
      if (kCut && c * 16 + 4 * i + quarter >= blocks) q = z = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        if (i % kSteps == 0) acc[mt] = f32x4{};
#pragma unroll
        for (int p = 0; p < kParts; ++p) acc[mt] = mfma_bf16(xs[mt][p], q, acc[mt]);
      }
      if constexpr (kPair) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) acc[mt] = mfma_bf16(xs[mt][0], z, acc[mt]);
      }
      if (i % kSteps == kSteps - 1) {
        const float sc = bf16_lo(w.s[i / kSteps]);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int r = 0; r < 4; ++r) total[mt][r] = fmaf(sc, acc[mt][r], total[mt][r]);
      }
    }
  };

  // Codes of a chunk sit in ahead[(chunk - begin) % kAhead] until it is their
  // turn (the loop is unrolled by kAhead, so those are registers). In the main
  // loop every load is unconditional, so that what is outstanding can be counted:
  // a count too high would read LDS before it is written.
  constexpr int kAhead = kStages - 1;
  Codes ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (begin + i < end) {
      request(begin + i, i, blocks - 1);
      keep_order();
      load_any(ahead[i], begin + i);
      keep_order();
    }
  int c = begin, slot = 0;  // slot of chunk c in the ring
  auto slot_of = [](int s) { return s < kStages ? s : s - kStages; };
#pragma unroll 1
  for (const int last = min(end, full) - 2 * kAhead; c <= last; c += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // behind this chunk's requests are the next kAhead - 1 chunks', each with
      // its codes; 0 also waits for this wave's reads of the chunk before
      keep_order();
      waitcnt<(kAhead - 1) * (kDma + kLoads), 0>();
      raw_barrier();
      const Codes w = ahead[i];
      request(c + i + kAhead, slot_of(slot + kAhead), -1);
      keep_order();
      load(ahead[i], c + i + kAhead);
      keep_order();
      compute(c + i, slot, w, std::false_type{});
      slot = slot_of(slot + 1);
    }
  }
#pragma unroll 1
  for (; c < end; ++c) {
    keep_order();
    waitcnt<0, 0>();
    raw_barrier();
    const Codes w = ahead[0];
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) ahead[i] = ahead[i + 1];
    if (c + kAhead < end) {
      request(c + kAhead, slot_of(slot + kAhead), blocks - 1);
      load_any(ahead[kAhead - 1], c + kAhead);
    }
    compute(c, slot, w, std::true_type{});
    slot = slot_of(slot + 1);
  }

  float* red = reinterpret_cast<float*>(lds);
  if (a.gated) {
    __syncthreads();
    if (wave & 1) {
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[((wave / 2 * kMT + mt) * 4 + r) * 64 + lane] = total[mt][r];
    }
    __syncthreads();
    if (wave & 1) return;
  }
  f32x4 up[kMT] = {};
  if (a.gated) {
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r) up[mt][r] = red[((wave / 2 * kMT + mt) * 4 + r) * 64 + lane];
  }
  finish<kMT>(a, first + col, m0 + 4 * quarter, total, up);
}

// Symmetric round to nearest: s = max|w| / 7 of the group in bf16, code
// round(w / s) + 8. A lane holds 8 consecutive k, a group is 4, 8 or 16 lanes.
// 8192 x 2048 take 18 us, bound by the exact divisions (42 MB would take 8): a
// weight is laid out once.
__global__ __launch_bounds__(256) void q4_quantize_kernel(const uint16_t* W, int N, int K, int group, uint8_t* codes,
                                                          uint16_t* scales) {
  const int64_t G = (K + group - 1) / group;
  const uint32_t per_row = static_cast<uint32_t>(G) * (group / 8);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 256, row0 = first / per_row;
  const uint32_t at = static_cast<uint32_t>(first - row0 * per_row) + threadIdx.x;
  const int64_t n = row0 + at / per_row;
  const int b = static_cast<int>(at % per_row);
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
  uint8_t* c = codes + n * kb + 4 * b;
  if (4 * b + 4 <= kb) {
    __builtin_memcpy(c, &w, 4);
  } else {
    for (int i = 0; i < 4; ++i)
      if (4 * b + i < kb) c[i] = static_cast<uint8_t>(w >> (8 * i));
  }
  if (b % (group / 8) == 0) scales[n * G + b / (group / 8)] = static_cast<uint16_t>(sb);
}

// Parts of x in q4_wide_kernel.
constexpr int wide_parts(Q4X x) { return x == Q4X::f32 || x == Q4X::planes ? 3 : 1; }

// Rows of a workgroup of q4_wide_kernel, and its waves. 128 rows turn codes into
// operands for twice as many as 64 and pay once they give 1.5 workgroups a CU:
// 512 rows by 8192 units and K 2048 (512 workgroups) take 32.5 us against 39.6,
// 384 by 10240 and K 2560 (480) 39 against 53; 256 by 10240 (320) 40.5 against
// 39.2 and 256 by 8192 (256) 27 against 23. Three parts of x have no room for
// 128 in LDS, and for 64 rows only as one workgroup a CU, which therefore has 8
// waves (256 rows by 8192 and K 2048: 41 us, with 4 waves 67); up to 64 rows
// they are taken 32 at a time (40 rows by 1000 and K 500: 11.9 us against 16.9).
int64_t wide_rows(int parts, bool gated, int64_t M, int64_t N) {
  if (M <= 32 || (parts == 3 && M <= 64)) return 32;
  const int64_t units = gated ? 32 : 64;
  return parts == 1 && (N + units - 1) / units * ((M + 127) / 128) >= 384 ? 128 : 64;
}
constexpr int wide_waves(int parts, int64_t rows) { return parts == 3 && rows == 64 ? 8 : 4; }

template <Q4X kX, int kGroup>
void launch_tile(const Q4Args& a, int waves, dim3 grid, hipStream_t s) {
  if (waves == 2) {
    q4_tile_kernel<kX, kGroup, 2><<<grid, 512, 0, s>>>(a);
  } else {
    q4_tile_kernel<kX, kGroup, 1><<<grid, 512, 0, s>>>(a);
  }
}

template <int kParts, bool kRowMajor, int kGroup>
void launch_wide(const Q4Args& a, dim3 grid, hipStream_t s) {
  const int64_t rows = wide_rows(kParts, a.gated, a.M, a.N);
  if (rows == 32) {
    constexpr int kWaves = wide_waves(kParts, 32);
    q4_wide_kernel<kParts, kRowMajor, kGroup, 2, kWaves><<<grid, 64 * kWaves, 0, s>>>(a);
  } else if (rows == 64) {
    constexpr int kWaves = wide_waves(kParts, 64);
    q4_wide_kernel<kParts, kRowMajor, kGroup, 4, kWaves><<<grid, 64 * kWaves, 0, s>>>(a);
  } else if constexpr (kParts == 1) {
    constexpr int kWaves = wide_waves(kParts, 128);
    q4_wide_kernel<1, kRowMajor, kGroup, 8, kWaves><<<grid, 64 * kWaves, 0, s>>>(a);
  }
}

// Calls f with the group as a constant.
template <class Fn>
void by_group(int group, Fn&& f) {
  if (group == 32) {
    f(std::integral_constant<int, 32>{});
  } else if (group == 64) {
    f(std::integral_constant<int, 64>{});
  } else {
    f(std::integral_constant<int, 128>{});
  }
}

// How a product is run: by q4_tile_kernel (`few`) or q4_wide_kernel, with
// `waves` side by side (tile) or in all (wide), `items` workgroups (units times
// rows), and K cut into `splits` parts.
struct Plan {
  bool few;
  int waves, items, splits, split_chunks;
};

// slice: the chunks of K that a workgroup takes at a time.
Plan cut_k(bool few, int waves, int64_t items, int64_t want, int64_t slice, int64_t K) {
  const int64_t chunks = (K + kChunk - 1) / kChunk, slices = (chunks + slice - 1) / slice;
  want = std::max<int64_t>(1, std::min<int64_t>(want, 16));
  Plan p;
  p.few = few;
  p.waves = waves;
  p.items = static_cast<int>(items);
  p.split_chunks = static_cast<int>((slices + want - 1) / want * slice);
  p.splits = static_cast<int>((chunks + p.split_chunks - 1) / p.split_chunks);
  return p;
}

// A split has two slices or more, as the second is requested while the first is
// computed (16 rows by 4096 and K 2560: 6.6 us whole, 8.0 in two splits). Two
// waves side by side where one would give more than a workgroup a CU (16 rows by
// 6144 units and K 2048: 5.8 us against 6.7; by 4096 one is better, 4.6 against
// 5.0), and for the gated pair, which needs two.
Plan plan_tile(Q4X x, bool gated, int64_t M, int64_t N, int64_t K) {
  const int64_t slice = wide_parts(x) > 1 ? 8 : 16, slices = (K + kChunk * slice - 1) / (kChunk * slice);
  for (int waves = gated ? 2 : 1;; ++waves) {
    const int64_t units = 16 * waves / (gated ? 2 : 1);
    const int64_t items = (N + units - 1) / units * ((M + 15) / 16);
    const Plan p = cut_k(true, waves, items, std::min(512 / items, slices / 2), slice, K);
    if (waves == 2 || items * p.splits <= 256) return p;
  }
}

// K is split for a workgroup a CU, or for all that the device holds where each
// still has 1024 values of K: 128 rows by 2048 units and K 8192 take 21.0 us in
// 8 splits and 25.8 in 4, 512 rows 48.6 us in 2 and 74.5 in one. A split of
// less than that costs more in partial sums than it gives (100 rows by 2048 and
// K 2048: 12.7 us in 4 splits, 15.2 in 2, 21.6 in one; so up to a workgroup a
// CU 512 values are enough).
Plan plan_wide(Q4X x, bool gated, int64_t M, int64_t N, int64_t K) {
  const int64_t rows = wide_rows(wide_parts(x), gated, M, N), chunks = (K + kChunk - 1) / kChunk;
  const int waves = wide_waves(wide_parts(x), rows);
  const int64_t units = 16 * waves / (gated ? 2 : 1);
  const int64_t items = (N + units - 1) / units * ((M + rows - 1) / rows);
  const int64_t resident = waves == 8 ? 256 : 512;  // workgroups, at least
  const int64_t want = std::max(std::min(256 / items, chunks / 4), std::min(resident / items, chunks / 8));
  return cut_k(false, waves, items, want, 1, K);
}

// Above 16 rows q4_tile_kernel reads the codes once for every 16 rows, but
// needs no launch before it that turns x into operands, seldom one that joins
// splits, and starts fast: it is taken up to a workgroup a CU (64 rows by 2048 units and K 2048 5.7 us
// against 9.2, 256 by 256 and K 2560 6.4 against 9.5). A CU holds two of those
// with groups of 128 and one part of x (32 rows by 8192 and K 2048: 7.8 us
// against 11.5; 64 by 2048 and K 8192, two slices each, 15.2 against 13.4; with
// groups of 32, of which a CU holds one, 24 by 6000 and K 300 take 11.3 against
// 8.7). Three parts of x make q4_wide_kernel slower still, so there the limit
// is three slices a CU (64 rows by 2048 and K 2048 8.5 us against 12.9, 256 by
// 256 and K 2560 10.8 against 19.5; at five, 160 by 2048 and K 2048 23.2
// against 18.9).
Plan plan(Q4X x, bool gated, int64_t M, int64_t N, int64_t K, int group) {
  const Plan p = plan_tile(x, gated, M, N, K);
  const int64_t groups = static_cast<int64_t>(p.items) * p.splits, work = groups * p.split_chunks;
  if (M <= 16 || groups <= 256) return p;
  if (wide_parts(x) == 1 ? group == 128 && work <= 512 * 16 : work <= 768 * 8) return p;
  return plan_wide(x, gated, M, N, K);
}

// Bytes of x in planes for q4_wide_kernel (0: q4_tile_kernel reads x as it is, or it
// is in planes). Those of bf16 rows that are read as they are stay unused: that
// depends on the address of x.
size_t x_planes_bytes(const Plan& p, Q4X x, int64_t M, int64_t K) {
  return p.few || x == Q4X::planes ? 0 : align256(size_t(wide_parts(x)) * size_t(plane_bytes(M, K)));
}

size_t room(const Plan& p, Q4X x, bool gated, int64_t M, int64_t N, int64_t K) {
  const size_t part = p.splits > 1 ? size_t(p.splits) * (gated ? 2 : 1) * size_t(M) * size_t(N) * 4 : 0;
  return x_planes_bytes(p, x, M, K) + align256(part);
}

}  // namespace

// (which kernel it is depends on the group too: enough for either)
size_t q4_workspace_bytes(Q4X x, bool gated, int64_t M, int64_t N, int64_t K) {
  const size_t tile = room(plan_tile(x, gated, M, N, K), x, gated, M, N, K);
  return M <= 16 ? tile : std::max(tile, room(plan_wide(x, gated, M, N, K), x, gated, M, N, K));
}

hipError_t launch_q4(Q4Args a, Q4X x_type, void* workspace, hipStream_t s) {
  const Plan p = plan(x_type, a.gated, a.M, a.N, a.K, a.group);
  a.splits = p.splits;
  a.split_chunks = p.split_chunks;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t x_bytes = x_planes_bytes(p, x_type, a.M, a.K);
  a.part = reinterpret_cast<float*>(ws + x_bytes);
  dim3 grid(p.items, 1, p.splits);
  if (!p.few) {
    // bf16 rows of whole 16-byte pieces are read as they are
    const bool row_major = x_type == Q4X::bf16 && a.K % 8 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
    if (x_bytes > 0 && !row_major) {
      const dim3 blocks(static_cast<unsigned>((q4_pad(a.K) / 8 + 31) / 32), static_cast<unsigned>((a.M + 7) / 8));
      if (x_type == Q4X::bf16) q4_planes_kernel<Q4X::bf16><<<blocks, 256, 0, s>>>(a, ws);
      if (x_type == Q4X::f32) q4_planes_kernel<Q4X::f32><<<blocks, 256, 0, s>>>(a, ws);
      if (x_type == Q4X::e4m3) q4_planes_kernel<Q4X::e4m3><<<blocks, 256, 0, s>>>(a, ws);
      a.x = ws;
    }
    by_group(a.group, [&](auto g) {
      constexpr int kGroup = decltype(g)::value;
      if (row_major) {
        launch_wide<1, true, kGroup>(a, grid, s);
      } else if (wide_parts(x_type) == 1) {
        launch_wide<1, false, kGroup>(a, grid, s);
      } else {
        launch_wide<3, false, kGroup>(a, grid, s);
      }
    });
  } else {
    grid.y = (a.M + 15) / 16;
    grid.x /= grid.y;
    by_group(a.group, [&](auto g) {
      constexpr int kGroup = decltype(g)::value;
      if (x_type == Q4X::bf16) launch_tile<Q4X::bf16, kGroup>(a, p.waves, grid, s);
      if (x_type == Q4X::f32) launch_tile<Q4X::f32, kGroup>(a, p.waves, grid, s);
      if (x_type == Q4X::e4m3) launch_tile<Q4X::e4m3, kGroup>(a, p.waves, grid, s);
      if (x_type == Q4X::planes) launch_tile<Q4X::planes, kGroup>(a, p.waves, grid, s);
    });
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t outputs = static_cast<int64_t>(a.M) * (a.y_type == Q4Y::planes ? q4_pad(a.N) : a.N);
  q4_join_kernel<<<static_cast<unsigned>((outputs + 255) / 256), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_q4_quantize(const uint16_t* W, int N, int K, int group, uint8_t* codes, uint16_t* scales,
                              hipStream_t s) {
  const int64_t G = (K + group - 1) / group, lanes = static_cast<int64_t>(N) * G * (group / 8);
  q4_quantize_kernel<<<static_cast<unsigned>((lanes + 255) / 256), 256, 0, s>>>(W, N, K, group, codes, scales);
  return hipGetLastError();
}

}  // namespace twell
