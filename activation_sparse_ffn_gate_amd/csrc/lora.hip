// Low-rank adapters of many requests beside a shared projection, for gfx950:
//
//   y[m] = base[m] + scaling[a] sx[m] (x[m] A_a^T) B_a^T,   a = index[m]
//
// A_a [R, K] and B_a [N, R] are bf16, a row without an adapter keeps its base. What
// has to be read is each adapter that the batch meets, x, base, and y written: for
// decode batches of many requests the adapters are most of it, for prompts y is.
//
// Two launches: t = x A_a^T in fp32, K split over workgroups and their waves, then y.
// Rows go by tiles of 16, the free dimension of v_mfma_f32_16x16x32_bf16, and within
// a tile each adapter in turn takes the rows that name it (the others' operands are
// zero and their results are not stored), so any order of requests is right and
// neighbours that share an adapter share its loads. Both products have the adapter as the first
// operand and the rows as the second: a lane then holds four consecutive r, or n, of one row.
//   operand lane layout: lane l holds row (l % 16) and the 8 consecutive k values
//   8 (l / 16) .. + 7; accumulator: lane l holds column (l % 16), element v is row 4 (l / 16) + v.
//
// fp32 rows, and t, enter the matrix instructions as three bf16 parts that add up to
// them (exactly down to bf16's 2^-133); e4m3 is exact in bf16. Products are exact and sums are
// fp32 in a fixed order: two calls give the same bits.
#include <algorithm>

#include "block_device.hpp"

namespace twell {
namespace {

constexpr int kTile = 16;          // rows that one matrix instruction takes
constexpr int kShrinkWaves = 4;    // of a workgroup, each with its part of K
constexpr int kExpandWaves = 4;    // of a workgroup, each with its own n
constexpr int kExpandTiles = 4;    // tiles of 16 n that a wave takes

__device__ __forceinline__ f32x4_t mfma_16x16x32(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// 8 fp32 as bf16 parts that add up to them: each part is the rest rounded to nearest.
__device__ __forceinline__ void split8(const float* v, u32x4_t (&part)[3]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = pack_bf16(rest[2 * i], rest[2 * i + 1]);
      part[p][i] = w;
      if (p < 2) {
        rest[2 * i] -= bf16_lo(w);
        rest[2 * i + 1] -= bf16_hi(w);
      }
    }
}

// Operands of 8 consecutive k of a row: how x lies in memory, and as bf16 parts.
template <LoraX kX>
struct Row8;
template <>
struct Row8<LoraX::bf16> {
  static constexpr int kParts = 1;
  using T = uint16_t;
  Raw8<uint16_t> r;
  __device__ __forceinline__ void load(const T* row, int b, int K) { load_block(row, b, K, r); }
  __device__ __forceinline__ void clear() { r = Raw8<uint16_t>{}; }
  __device__ __forceinline__ void parts(u32x4_t (&p)[1]) const { p[0] = r.w; }
};
template <>
struct Row8<LoraX::f32> {
  static constexpr int kParts = 3;
  using T = float;
  Raw8<float> r;
  __device__ __forceinline__ void load(const T* row, int b, int K) { load_block(row, b, K, r); }
  __device__ __forceinline__ void clear() { r = Raw8<float>{}; }
  __device__ __forceinline__ void parts(u32x4_t (&p)[3]) const {
    float v[8];
    unpack8(r, v);
    split8(v, p);
  }
};
template <>
struct Row8<LoraX::e4m3> {
  static constexpr int kParts = 1;
  using T = uint8_t;
  u32x2_t r;
  __device__ __forceinline__ void load(const T* row, int b, int K) {
    const int left = K - 8 * b;
    r = u32x2_t{0u, 0u};
    if (left >= 8) {
      __builtin_memcpy(&r, row + 8 * b, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) r[i / 4] |= static_cast<uint32_t>(row[8 * b + i]) << (8 * (i % 4));
    }
  }
  __device__ __forceinline__ void clear() { r = u32x2_t{0u, 0u}; }
  __device__ __forceinline__ void parts(u32x4_t (&p)[1]) const {
    float v[8];
    unpack_e4m3(r[0], v);
    unpack_e4m3(r[1], v + 4);
    p[0] = u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  }
};

// The adapters of a tile of rows, in the order of the first row that names each.
// f(adapter, rows as bits of the tile's 16) for every `slots`-th of them from `slot` on.
// `mine`: the lane's row's index (lanes 0..15), already -1 where it names no adapter.
template <class Fn>
__device__ __forceinline__ void each_adapter(int mine, int slot, int slots, Fn&& f) {
  uint32_t left = static_cast<uint32_t>(__ballot(mine >= 0)) & 0xFFFFu;
  for (int k = 0; left != 0; ++k) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
    const uint32_t rows = static_cast<uint32_t>(__ballot(mine == a)) & 0xFFFFu;
    left &= ~rows;
    if (k % slots == slot) f(a, rows);
  }
}

__device__ __forceinline__ int row_adapter(const LoraArgs& a, int row) {
  if (row >= a.M) return -1;
  const int i = a.index[row];
  return i >= 0 && i < a.n ? i : -1;
}

__host__ __device__ constexpr int pad16(int r) { return (r + 15) & ~15; }

// grid (tiles, splits, slots): partial sums of t over a split's part of K, the waves' added through LDS in
// wave order. kRanks: tiles of 16 r held at once.
template <LoraX kX, int kRanks>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(LoraArgs a) {
  __shared__ f32x4_t red[kShrinkWaves][kRanks][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = blockIdx.x * kTile + (lane & 15);
  const int k8 = lane >> 4;
  const int mine = row_adapter(a, m);
  const int steps = (a.K + 31) / 32;  // of 32 k, dealt evenly to splits and their waves
  const int parts = a.splits * kShrinkWaves, part = blockIdx.y * kShrinkWaves + wave;
  const int from = static_cast<int>(static_cast<int64_t>(steps) * part / parts);
  const int to = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / parts);
  const int Rp = pad16(a.R);
  using Row = Row8<kX>;
  const typename Row::T* x = static_cast<const typename Row::T*>(a.x) + static_cast<int64_t>(m) * a.K;
  each_adapter(mine, blockIdx.z, a.slots, [&](int adapter, uint32_t rows) {
    const bool in = rows >> (lane & 15) & 1;
    const uint16_t* A = a.A + static_cast<int64_t>(adapter) * a.R * a.K;
    for (int r0 = 0; r0 < Rp; r0 += 16 * kRanks) {
      f32x4_t acc[kRanks];
#pragma unroll
      for (int i = 0; i < kRanks; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int s = from; s < to; ++s) {
        Row xr;
        xr.clear();
        if (in) xr.load(x, 4 * s + k8, a.K);
        Raw8<uint16_t> ar[kRanks];
#pragma unroll
        for (int i = 0; i < kRanks; ++i) {
          const int r = r0 + 16 * i + (lane & 15);
          ar[i] = Raw8<uint16_t>{};
          if (r < a.R) load_block(A + static_cast<int64_t>(r) * a.K, 4 * s + k8, a.K, ar[i]);
        }
        u32x4_t xp[Row::kParts];
        xr.parts(xp);
#pragma unroll
        for (int p = Row::kParts - 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < kRanks; ++i) acc[i] = mfma_16x16x32(ar[i].w, xp[p], acc[i]);
      }
#pragma unroll
      for (int i = 0; i < kRanks; ++i) red[wave][i][lane] = acc[i];
      __syncthreads();
      // wave w joins every kShrinkWaves-th tile of r
#pragma unroll
      for (int i = 0; i < kRanks; ++i) {
        const int r = r0 + 16 * i + 4 * k8;
        if (i % kShrinkWaves != wave || r >= Rp || !in) continue;
        f32x4_t sum = red[0][i][lane];
#pragma unroll
        for (int w = 1; w < kShrinkWaves; ++w) sum += red[w][i][lane];
        float* t = a.t + (static_cast<int64_t>(blockIdx.y) * a.M + m) * Rp + r;
        *reinterpret_cast<f32x4_t*>(t) = sum;
      }
      __syncthreads();
    }
  });
}

// grid (tiles, parts of N, slots): y of the rows of each adapter from t, whose splits are added in order.
template <class TY, int kSteps>
__global__ __launch_bounds__(64 * kExpandWaves) void lora_expand_kernel(LoraArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = blockIdx.x * kTile + (lane & 15);
  const int k8 = lane >> 4;
  const int mine = row_adapter(a, m);
  const int Rp = pad16(a.R);
  const int n0 = (blockIdx.y * kExpandWaves + wave) * 16 * kExpandTiles;
  if (n0 >= a.N) return;  // the whole wave, and no barrier follows
  const TY* base = static_cast<const TY*>(a.base) + static_cast<int64_t>(m) * a.N;
  TY* y = static_cast<TY*>(a.y) + static_cast<int64_t>(m) * a.N;
  // Two tiles of n side by side: row 4 q + v of tile j is n0 + 32 (tile / 2) + 8 q + 4 j + v, so that a
  // lane holds 8 consecutive n of its row in the pair.
  each_adapter(mine, blockIdx.z, a.slots, [&](int adapter, uint32_t rows) {
    const bool in = rows >> (lane & 15) & 1;
    const uint16_t* B = a.B + static_cast<int64_t>(adapter) * a.N * a.R;
    float factor = a.scaling != nullptr ? a.scaling[adapter] : 1.f;
    if (a.x_scale != nullptr && in) factor *= a.x_scale[m];
    u32x4_t tp[kSteps][3];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int r = 32 * s + 8 * k8;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (in && r < Rp) {
        const float* t = a.t + static_cast<int64_t>(m) * Rp + r;
        for (int k = 0; k < a.splits; ++k) {
          const float* from = t + static_cast<int64_t>(k) * a.M * Rp;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += from[i];
        }
      }
      split8(v, tp[s]);
    }
#pragma unroll
    for (int pair = 0; pair < kExpandTiles / 2; ++pair) {
      f32x4_t acc[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        const int row = lane & 15;
        const int n = min(n0 + 32 * pair + 8 * (row >> 2) + 4 * j + (row & 3), a.N - 1);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          Raw8<uint16_t> b;
          load_block(B + static_cast<int64_t>(n) * a.R, 4 * s + k8, a.R, b);
#pragma unroll
          for (int p = 2; p >= 0; --p) acc[j] = mfma_16x16x32(b.w, tp[s][p], acc[j]);
        }
      }
      const int n = n0 + 32 * pair + 8 * k8;
      if (!in || n >= a.N) continue;
      Raw8<TY> raw;
      load_block(base, n / 8, a.N, raw);
      float v[8];
      unpack8(raw, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(factor, acc[j / 4][j % 4], v[j]);
      store_block(y, n / 8, a.N, v);
    }
  });
  // rows without an adapter
  if (blockIdx.z == 0 && a.base != a.y && mine < 0 && m < a.M) {
#pragma unroll
    for (int pair = 0; pair < kExpandTiles / 2; ++pair) {
      const int n = n0 + 32 * pair + 8 * k8;
      if (n >= a.N) continue;
      Raw8<TY> raw;
      load_block(base, n / 8, a.N, raw);
      float v[8];
      unpack8(raw, v);
      store_block(y, n / 8, a.N, v);
    }
  }
}

int lora_splits(int64_t M, int64_t K) {
  const int64_t tiles = (M + kTile - 1) / kTile;
  return static_cast<int>(std::max<int64_t>(std::min<int64_t>(512 / tiles, K / 512), 1));
}

template <LoraX kX>
void shrink(const LoraArgs& a, dim3 grid, hipStream_t s) {
  if (a.R <= 16) {
    lora_shrink_kernel<kX, 1><<<grid, 64 * kShrinkWaves, 0, s>>>(a);
  } else if (a.R <= 32) {
    lora_shrink_kernel<kX, 2><<<grid, 64 * kShrinkWaves, 0, s>>>(a);
  } else {
    lora_shrink_kernel<kX, 4><<<grid, 64 * kShrinkWaves, 0, s>>>(a);
  }
}

template <class TY>
void expand(const LoraArgs& a, dim3 grid, hipStream_t s) {
  if (a.R <= 32) {
    lora_expand_kernel<TY, 1><<<grid, 64 * kExpandWaves, 0, s>>>(a);
  } else if (a.R <= 64) {
    lora_expand_kernel<TY, 2><<<grid, 64 * kExpandWaves, 0, s>>>(a);
  } else if (a.R <= 128) {
    lora_expand_kernel<TY, 4><<<grid, 64 * kExpandWaves, 0, s>>>(a);
  } else {
    lora_expand_kernel<TY, 8><<<grid, 64 * kExpandWaves, 0, s>>>(a);
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R) {
  return align256(static_cast<size_t>(lora_splits(M, K)) * M * pad16(static_cast<int>(R)) * 4);
}

hipError_t launch_lora(LoraArgs a, LoraX x_type, bool y_f32, void* workspace, hipStream_t s) {
  a.t = static_cast<float*>(workspace);
  a.splits = lora_splits(a.M, a.K);
  const int tiles = (a.M + kTile - 1) / kTile;
  a.slots = a.M <= 256 ? std::min(a.M, kTile) : 4;
  const dim3 up(tiles, a.splits, a.slots);
  if (x_type == LoraX::bf16) {
    shrink<LoraX::bf16>(a, up, s);
  } else if (x_type == LoraX::f32) {
    shrink<LoraX::f32>(a, up, s);
  } else {
    shrink<LoraX::e4m3>(a, up, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int per = 16 * kExpandTiles * kExpandWaves;
  const dim3 down(tiles, (a.N + per - 1) / per, a.slots);
  if (y_f32) {
    expand<float>(a, down, s);
  } else {
    expand<uint16_t>(a, down, s);
  }
  return hipGetLastError();
}

}  // namespace twell
