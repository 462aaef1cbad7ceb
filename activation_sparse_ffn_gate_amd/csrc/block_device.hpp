// Device helpers of the operators around the FFN (residual norm, dropout,
// 4-bit products): typed loads and stores of 8 elements, and the
// counter-based generator of dropout.
//
// The 8-element accesses are written as memcpy of 16-byte pieces, which the
// compiler turns into dwordx4 loads and stores whatever the address (gfx950
// runs with unaligned access enabled), so rows of odd widths take the same
// path as aligned ones and only a row's last, cut block goes element by
// element.
#pragma once

#include "twell_device.hpp"
#include "twell_internal.hpp"

namespace twell {

__device__ __forceinline__ u32x4_t load16_any(const void* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// kStream: with the non-temporal hint, for outputs that pass the L2 by the time
// they are read.
template <bool kStream = false>
__device__ __forceinline__ void store16_any(void* p, u32x4_t v) {
  typedef u32x4_t any_t __attribute__((aligned(1)));
  if constexpr (kStream) {
    __builtin_nontemporal_store(v, static_cast<any_t*>(p));
  } else {
    *static_cast<any_t*>(p) = v;
  }
}

// Raw 8 elements as they lie in memory: 16 bytes of bf16 or 32 of fp32.
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4_t w;
};
template <>
struct Raw8<float> {
  u32x4_t a, b;
};

__device__ __forceinline__ void load8(const uint16_t* p, Raw8<uint16_t>& r) { r.w = load16_any(p); }
__device__ __forceinline__ void load8(const float* p, Raw8<float>& r) {
  r.a = load16_any(p);
  r.b = load16_any(p + 4);
}

// The first n (1..7) of 8 elements, the others zero.
__device__ __forceinline__ void load8_cut(const uint16_t* p, int n, Raw8<uint16_t>& r) {
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : 0u;
  r.w = u32x4_t{e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16)};
}
__device__ __forceinline__ void load8_cut(const float* p, int n, Raw8<float>& r) {
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < n ? __float_as_uint(p[i]) : 0u;
  r.a = u32x4_t{e[0], e[1], e[2], e[3]};
  r.b = u32x4_t{e[4], e[5], e[6], e[7]};
}

__device__ __forceinline__ void unpack8(const Raw8<uint16_t>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(r.w[i]);
    v[2 * i + 1] = bf16_hi(r.w[i]);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(r.a[i]);
    v[4 + i] = __uint_as_float(r.b[i]);
  }
}

// Memory accesses stay on their side: loads come back in the order of the
// program, and waitcnt<> counts them.
__device__ __forceinline__ void keep_order() { asm volatile("" ::: "memory"); }

// A barrier past which every wave's LDS accesses are done; __syncthreads() would
// also wait for the loads and stores of global memory that are under way.
__device__ __forceinline__ void lds_barrier() {
  keep_order();
  waitcnt<63, 0>();
  raw_barrier();
}

// Two fp32 as a bf16 pair, round to nearest even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2_t v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

template <bool kStream = false>
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  store16_any<kStream>(
      p, u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
}
template <bool kStream = false>
__device__ __forceinline__ void store8(float* p, const float* v) {
  store16_any<kStream>(p, __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]}));
  store16_any<kStream>(p + 4, __builtin_bit_cast(u32x4_t, f32x4_t{v[4], v[5], v[6], v[7]}));
}
// Four fp32 as e4m3 bytes, round to nearest even (values are within +-448).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}
template <bool kStream = false>
__device__ __forceinline__ void store8(uint8_t* p, const float* v) {
  typedef u32x2_t any_t __attribute__((aligned(1)));
  const u32x2_t w = {pack_e4m3(v[0], v[1], v[2], v[3]), pack_e4m3(v[4], v[5], v[6], v[7])};
  if constexpr (kStream) {
    __builtin_nontemporal_store(w, reinterpret_cast<any_t*>(p));
  } else {
    *reinterpret_cast<any_t*>(p) = w;
  }
}

__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, 0.f)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint8_t* p, float v) { *p = static_cast<uint8_t>(pack_e4m3(v, 0.f, 0.f, 0.f)); }

template <class T>
__device__ __forceinline__ void store8_cut(T* p, int n, const float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store1(p + i, v[i]);
}

// Blocks of 8 columns: block b of a row of d columns is whole, cut or absent.
template <class T>
__device__ __forceinline__ void load_block(const T* row, int b, int d, Raw8<T>& r) {
  const int n = d - 8 * b;
  if (n >= 8) {
    load8(row + 8 * b, r);
  } else if (n > 0) {
    load8_cut(row + 8 * b, n, r);
  } else {
    r = Raw8<T>{};
  }
}
template <class T>
__device__ __forceinline__ void store_block(T* row, int b, int d, const float* v, bool stream = false) {
  const int n = d - 8 * b;
  if (n >= 8 && stream) {
    store8<true>(row + 8 * b, v);
  } else if (n >= 8) {
    store8(row + 8 * b, v);
  } else if (n > 0) {
    store8_cut(row + 8 * b, n, v);
  }
}

// ------------------------------------------------------------------ dropout
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): 128 bits from a 128-bit counter and a 64-bit key.
// The counter is (column / 8, row, offset), the key the seed, and the 8
// columns of a block take the 8 16-bit halves of the four words in order, so
// one evaluation serves 8 elements and any kernel that knows an element's row
// and column finds its bits again.
__device__ __forceinline__ u32x4_t philox(uint32_t c0, uint32_t c1, const Dropout& r) {
  uint32_t c2 = r.off_lo, c3 = r.off_hi, k0 = r.seed_lo, k1 = r.seed_hi;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

// v of block b of a row: kept elements scaled, dropped ones an exact zero
// (selected, not multiplied, so a dropped infinity or NaN is gone too).
__device__ __forceinline__ void drop8(float* v, int b, uint32_t row, const Dropout& r) {
  const u32x4_t w = philox(static_cast<uint32_t>(b), row, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] & 0xFFFFu) >= r.threshold ? v[2 * i] * r.scale : 0.f;
    v[2 * i + 1] = (w[i] >> 16) >= r.threshold ? v[2 * i + 1] * r.scale : 0.f;
  }
}

}  // namespace twell
