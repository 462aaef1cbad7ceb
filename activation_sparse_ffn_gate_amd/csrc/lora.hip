// Low-rank adapters of many requests beside a shared projection, for gfx950:
//
//   y[m] = base[m] + scaling[a] sx[m] (x[m] A_a^T) B_a^T,   a = index[m]
//
// A_a [R, K] and B_a [N, R] are bf16, a row without an adapter keeps its base. What
// has to be read is each adapter that the batch meets, x, base, and y written: for
// decode batches of many requests the adapters are most of it, for prompts y is.
//
// One launch. A workgroup takes up to 16 rows of one adapter, the free dimension of
// v_mfma_f32_16x16x32_bf16, and a part of N: its waves split K and join t = x A_a^T in fp32
// through LDS, then they split the part's n. Rows of any order are grouped by adapter (below), so
// requests that share one share its loads. Each part of N computes t again, with A out of the L2: as a launch
// of its own that leaves t in memory the same took 9 us for one row (5.3 here), 18 for 64 rows of
// 48 adapters with K 8192 (14.9), 35 for 1100 rows of prompts (20.7). (That was with loads into the operands' layout. Where
// R K is large, t for each part is what these calls wait for: 4 rows with 64 r and K 8192 23 us; a launch for it was
// not measured there.)
//   operand lane layout: lane l holds row (l % 16) and the 8 consecutive k values
//   8 (l / 16) .. + 7; accumulator: lane l holds column (l % 16), element v is row 4 (l / 16) + v.
//
// What bounds it: for a few rows the chain of launch, index and groups (1.8 to 3 us), A and x (1.5), join (0.7),
// y (0.5); for 64 rows of 48 adapters with K 8192 what a CU takes in of A (256 KB in 6.5 us); for 1100 rows
// (N 10240, K 2560, 32 r, 57 MB: 2.8 TB/s) that every 16 rows read B again (12 of 20 us).
//
// fp32 rows, and t, enter the matrix instructions as three bf16 parts that add up to
// them (exactly down to bf16's 2^-133); e4m3 is exact in bf16. Products are exact and sums are
// fp32 in a fixed order: two calls give the same bits.
#include <algorithm>

#include "block_device.hpp"

namespace twell {
namespace {

constexpr int kTile = 16;  // rows that one matrix instruction takes

__device__ __forceinline__ f32x4_t mfma_16x16x32(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// 8 fp32 as bf16 parts that add up to them: 8 bits of each a part, cut off, as to nearest would take values next to the
// largest fp32 to infinity; the last part, 8 bits or fewer, to nearest where it lies under bf16's least step.
__device__ __forceinline__ void split8(const float* v, u32x4_t (&part)[3]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p == 2) {
        part[p][i] = pack_bf16(rest[2 * i], rest[2 * i + 1]);
        continue;
      }
      const uint32_t lo = __float_as_uint(rest[2 * i]), hi = __float_as_uint(rest[2 * i + 1]);
      part[p][i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);  // the upper halves
      rest[2 * i] -= __uint_as_float(lo & 0xFFFF0000u);
      rest[2 * i + 1] -= __uint_as_float(hi & 0xFFFF0000u);
    }
}

// A wave-uniform base and a 32-bit offset of the lane: no 64-bit vector arithmetic.
template <class T>
__device__ __forceinline__ T* at_bytes(T* base, uint32_t off) {
  using Byte = std::conditional_t<std::is_const_v<T>, const char, char>;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(base) + off);
}

// Operands of 8 consecutive k of a row (those past K zero): how x lies in memory, and as bf16 parts.
template <LoraX kX>
struct Row8;
template <>
struct Row8<LoraX::bf16> {
  static constexpr int kParts = 1;
  using T = uint16_t;
  Raw8<uint16_t> r;
  __device__ __forceinline__ void load(const T* row, int b, int K) { load_block(row, b, K, r); }
  __device__ __forceinline__ void parts(u32x4_t (&p)[1]) const { p[0] = r.w; }
};
template <>
struct Row8<LoraX::f32> {
  static constexpr int kParts = 3;
  using T = float;
  Raw8<float> r;
  __device__ __forceinline__ void load(const T* row, int b, int K) { load_block(row, b, K, r); }
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
  __device__ __forceinline__ void load(const T* row, int b, int K) { r = load_bytes(row + 8 * b, K - 8 * b); }
  __device__ __forceinline__ void parts(u32x4_t (&p)[1]) const {
    float v[8];
    unpack_e4m3(r[0], v);
    unpack_e4m3(r[1], v + 4);
    p[0] = u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  }
};

// The work of a launch: rows go in blocks of kBlock, and a block's rows that name one adapter in items of 16, the
// free dimension of the matrix instruction. Every workgroup finds the block's items by itself, and finds what the
// others do: a hash table in LDS holds a mask of the rows of each adapter, a row's rank is how many earlier ones its
// mask has, rows whose rank is a multiple of 16 begin an item, and items are numbered in the order of those rows. (Only
// the places in the table depend on who came first.) Rows without an adapter count as those of one more, its y
// is base.
constexpr int kBlock = 256;
constexpr int kSlots = 2 * kBlock;

struct __attribute__((aligned(16))) Table {  // lies in memory that is used for something else afterwards
  int key[kSlots];  // adapter, -1: free
  uint32_t rows[kSlots][kBlock / 32];
};

struct Items {
  int adapter[kBlock];     // of each item
  int rank[kBlock];        // of its first row among the adapter's
  int begun[kBlock / 64];  // items that begin in each 64 rows
  int rows[kTile];         // of the item in hand, from the block's first
  int taken[kBlock / 64];  // its rows among each 64
};

// A thread's row: its adapter (-1: none, as past the last row and in threads that have no row) and how many
// earlier rows of the block name that.
struct Row {
  int adapter, rank;
};

// Lists the items of the block at row0; returns how many there are.
__device__ __forceinline__ int find_items(const LoraArgs& a, int row0, Table& table, Items& s, Row& row) {
  constexpr int kParts = kBlock / 64;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  row = {-1, 0};
  if (a.M <= kTile) {  // one item an adapter at most: each wave finds them with ballots (one row 6.4 -> 5.8 us)
    int v = -1;
    if (lane < a.M) {
      v = a.index[lane];
      v = v >= 0 && v < a.n ? v : a.n;
    }
    int all = 0;
    for (uint64_t left = __ballot(v >= 0); left != 0; ++all) {
      const int adapter = __builtin_amdgcn_readlane(v, __builtin_ctzll(left));
      const uint64_t same = __ballot(v == adapter);
      left &= ~same;
      if (v == adapter && wave == 0) row = {adapter, static_cast<int>(mask_rank(same))};
      if (t == 0) {
        s.adapter[all] = adapter;
        s.rank[all] = 0;
      }
    }
    lds_barrier();
    return all;
  }
  const bool valid = t < kBlock && row0 + t < a.M;
  const int v = valid ? a.index[row0 + t] : -1;  // under way while the table is cleared
  auto clear = [&](void* p, int bytes, uint32_t w) {
    for (int at = 16 * t; at < bytes; at += 16 * blockDim.x)
      lds_store16(static_cast<uint8_t*>(p), at, u32x4_t{w, w, w, w});
  };
  clear(table.key, sizeof(table.key), ~0u);
  clear(table.rows, sizeof(table.rows), 0u);
  lds_barrier();
  if (valid) row.adapter = v >= 0 && v < a.n ? v : a.n;
  int slot = 0;
  if (row.adapter >= 0) {
    slot = static_cast<int>(static_cast<uint32_t>(row.adapter) * 0x9E3779B1u >> 23);  // Knuth's hash, 9 bits
    static_assert(kSlots == 1 << 9, "bits of the hash");
    for (;;) {  // half of the slots stay free, so this ends
      const int was = atomicCAS(&table.key[slot], -1, row.adapter);
      if (was == -1 || was == row.adapter) break;
      slot = (slot + 1) & (kSlots - 1);
    }
    atomicOr(&table.rows[slot][t >> 5], 1u << (t & 31));
  }
  lds_barrier();
  bool first = false;
  if (row.adapter >= 0) {
#pragma unroll
    for (int w = 0; w < kBlock / 32; ++w) {
      const uint32_t earlier = w < (t >> 5) ? ~0u : w == (t >> 5) ? (1u << (t & 31)) - 1u : 0u;
      row.rank += __popc(table.rows[slot][w] & earlier);
    }
    first = row.rank % kTile == 0;
  }
  const uint64_t begins = __ballot(first);
  if (wave < kParts && lane == 0) s.begun[wave] = __popcll(begins);
  lds_barrier();
  int before = static_cast<int>(mask_rank(begins)), all = 0;
#pragma unroll
  for (int w = 0; w < kParts; ++w) {
    before += w < wave ? s.begun[w] : 0;
    all += s.begun[w];
  }
  if (first) {
    s.adapter[before] = row.adapter;
    s.rank[before] = row.rank;
  }
  lds_barrier();
  return __builtin_amdgcn_readfirstlane(all);
}

// Puts the rows of item k into s.rows; returns how many. Every thread has left what read those of the item before
// (its last barrier).
__device__ __forceinline__ int take_item(Items& s, int k, const Row& row) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int at = row.adapter == s.adapter[k] ? row.rank - s.rank[k] : -1;
  const bool in = at >= 0 && at < kTile;
  if (in) s.rows[at] = threadIdx.x;
  const int taken = __popcll(__ballot(in));
  if (wave < kBlock / 64 && (threadIdx.x & 63) == 0) s.taken[wave] = taken;
  lds_barrier();
  int count = 0;
#pragma unroll
  for (int w = 0; w < kBlock / 64; ++w) count += s.taken[w];
  return __builtin_amdgcn_readfirstlane(count);
}

// What a workgroup does: every at_once-th item of a block of rows, for a part of N. Where there are items for all XCDs the
// parts of one are 8 workgroups apart, which puts them on one XCD, whose L2 then has A and B once (256 rows of 64
// adapters with 64 r 19.4 -> 16 us); a few items' parts go to all XCDs (one row with 64 r 10.5 -> 7.5).
struct Place {
  int block, item, part;
};
__device__ __forceinline__ Place place_of(const LoraArgs& a) {
  const int in = blockIdx.x & ((1 << a.apart) - 1), first = (blockIdx.y << a.apart) + in;
  const int item = a.blocks > 1 ? first / a.blocks : first;
  return {first - item * a.blocks, item, static_cast<int>(blockIdx.x >> a.apart)};
}

// Elements [from, to) of the item's rows from base to y; from is a multiple of 8. A thread's blocks of 8 are requested four
// at a time.
template <class TY>
__device__ __forceinline__ void copy_rows(const LoraArgs& a, const TY* base, TY* y, const Items& s, int count, int from,
                                          int to) {
  const int blocks = (to - from + 7) / 8;
  constexpr int kAtOnce = 4;
  for (int e0 = threadIdx.x; e0 < count * blocks; e0 += kAtOnce * blockDim.x) {
    Raw8<TY> raw[kAtOnce];
    int64_t row[kAtOnce];
    int b[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int e = min(e0 + k * static_cast<int>(blockDim.x), count * blocks - 1);  // past the end: the last one again
      const int r = e / blocks;
      row[k] = static_cast<int64_t>(s.rows[r]) * a.N;
      b[k] = from / 8 + e - r * blocks;
      load_block(base + row[k], b[k], a.N, raw[k]);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      float v[8];
      unpack8(raw[k], v);
      store_block(y + row[k], b[k], a.N, v);
    }
  }
}

// ------------------------------------------------------------------ whole blocks
// What the waves read goes through LDS by DMA, where 4 or 8 lanes take 64 or 128 consecutive bytes: read straight into
// the operands' lane layout, in which consecutive lanes are different rows, a wave's load is 64 lookups in the cache
// instead of 8 or 16, and the calls took 8 us for one row and 28 for 256 rows of 64 adapters (5.4 and 14).
constexpr int kUnit = 64;           // n that a wave takes at a time
constexpr int kWaveLds = 8 * 1024;  // bytes of a wave's buffers up to 32 r; above twice as many

template <LoraX kX, int kTiles>
struct Stage {  // 32 k: kTiles x 16 rows of A, and 16 of x where they enter as they are
  static constexpr bool kPlanes = kX == LoraX::f32;  // x comes by groups of 512 values instead, cut into bf16 parts once
  static constexpr int kXDma = kPlanes ? 0 : 1;
  static constexpr int kBytes = kTiles * 1024 + (kPlanes ? 0 : kX == LoraX::bf16 ? 1024 : 512);
  static constexpr int kGroupBytes = kPlanes ? 5 * 1024 : 0;  // a group as it comes, its three parts
  static constexpr int kLds = kTiles > 2 ? 2 * kWaveLds : kWaveLds + (kPlanes ? 1024 : 0);
  static constexpr int kDepth = (kLds - kGroupBytes) / kBytes > 4 ? 4 : (kLds - kGroupBytes) / kBytes;
  static constexpr int kDma = kTiles + kXDma;
};

// 16-byte pieces of a row that is 64 bytes in LDS (4 pieces), or a line of 128 (8): piece p of row r lies at
// p ^ swizzle(r), so that 16 rows' reads of one piece spread over all banks.
__device__ __forceinline__ constexpr int swizzle4(int r) { return (r >> 2) & 3; }
__device__ __forceinline__ constexpr int swizzle8(int r) { return (r >> 1) & 7; }

// grid: place_of. K and N are multiples of 64, R of 8 and at most 64, K is at most 2^22 (32-bit
// offsets in a block of rows), addresses are multiples of 16.
template <LoraX kX, class TY, int kTiles, int kW>
__global__ __launch_bounds__(64 * kW) void lora_kernel(LoraArgs a) {
  using S = Stage<kX, kTiles>;
  using X = typename Row8<kX>::T;
  constexpr int kSteps = (kTiles + 1) / 2;  // of 32 r
  constexpr int kRow = 32 * kSteps + 4;     // floats of a row of t
  // One LDS object: with more of them the compiler gives each a scope of its own, and then has LDS reads wait for all DMA
  // that is under way, whatever was counted (16 rows with K 4096 10.5 -> 8.2 us, 64 with K 8192 and f32 x 15.4 -> 14.9).
  constexpr int kTsBytes = 4 * kTile * kRow;
  static_assert(kTsBytes % 16 == 0, "items are aligned to 16");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kW * S::kLds + kTsBytes + sizeof(Items)];
  float* ts = reinterpret_cast<float*>(smem + kW * S::kLds);
  Items& items = *reinterpret_cast<Items*>(smem + kW * S::kLds + kTsBytes);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, i = lane & 15;
  uint8_t* mine_lds = smem + wave * S::kLds;
  // The waves' shares of t lie behind their first unit of B, where the second is requested after the join.
  constexpr int kBBytes = 4096 * kSteps;  // of a unit of B: R up to 32 or 64
  static_assert(2 * kBBytes <= S::kLds && kTiles * 1024 <= kBBytes, "two units of B, a share of t");
  auto red = [&](int w, int k) { return reinterpret_cast<float*>(smem + w * S::kLds + kBBytes) + 256 * k; };
  const Place place = place_of(a);
  if (place.item >= a.at_once) return;  // the whole workgroup
  const int row0 = place.block * kBlock;
  const int from = min(a.wave_steps * wave, a.K / 32), to = min(from + a.wave_steps, a.K / 32);
  const int first = a.part_units * place.part, last = min(first + a.part_units, a.N / kUnit);
  const X* x = static_cast<const X*>(a.x) + static_cast<int64_t>(row0) * a.K;
  const TY* base = static_cast<const TY*>(a.base) + static_cast<int64_t>(row0) * a.N;
  TY* y = static_cast<TY*>(a.y) + static_cast<int64_t>(row0) * a.N;
  Row mine;
  const int n_items = find_items(a, row0, *reinterpret_cast<Table*>(smem), items, mine);

  for (int item = place.item; item < n_items; item += a.at_once) {
    const int adapter = __builtin_amdgcn_readfirstlane(items.adapter[item]);
    if (adapter == a.n && a.base == a.y) continue;
    const int count = take_item(items, item, mine);
    if (adapter == a.n) {
      copy_rows(a, base, y, items, count, kUnit * first, kUnit * last);
      lds_barrier();
      continue;
    }
    const uint16_t* A = a.A + static_cast<int64_t>(adapter) * a.R * a.K;
    const uint16_t* B = a.B + static_cast<int64_t>(adapter) * a.N * a.R;
    auto row_of = [&](int r) { return items.rows[r < count ? r : 0]; };  // past the last: read, not stored

    // ---- t: this wave's steps of K
    // fp32 rows: 2^turn of them, at least the item's, by 16 >> turn steps of 32 k make a group of 512 values, 8 a lane. What
    // a row's values cost to cut into parts is then paid once, and not for all 16 columns (four times the vector
    // instructions of everything else there).
    const int turn = count > 1 ? 32 - __builtin_clz(count - 1) : 0;
    const int group_steps = kTile >> turn;
    const int x_row = kX == LoraX::bf16 ? lane >> 2 : kX == LoraX::f32 ? lane >> (6 - turn) : lane >> 1 & 15;
    const int x_k = lane & ((64 >> turn) - 1);  // of a group: 8 k each
    uint32_t a_off[kTiles], x_off;
    {
      const int r = lane >> 2, p = (lane & 3) ^ swizzle4(r);
#pragma unroll
      for (int k = 0; k < kTiles; ++k)  // rows past R: the last one again, and t is cleared there
        a_off[k] = static_cast<uint32_t>(min(16 * k + r, a.R - 1)) * (2u * a.K) + 16u * p;
      const uint32_t from_row = static_cast<uint32_t>(row_of(x_row)) * a.K;
      x_off = kX == LoraX::bf16  ? 2u * from_row + 16u * p
              : kX == LoraX::f32 ? 4u * from_row + 32u * x_k
                                 : from_row + 16u * (lane & 1);
    }
    auto stage = [&](int s, int slot) {
      uint8_t* to_lds = mine_lds + slot * S::kBytes;
#pragma unroll
      for (int k = 0; k < kTiles; ++k) dma16(at_bytes(A + 32 * s, a_off[k]), to_lds + 1024 * k);
      if constexpr (!S::kPlanes) {  // rows past the item's are left out: what their columns hold is not stored
        if ((kX == LoraX::bf16 || lane < 32) && x_row < count)
          dma16(reinterpret_cast<const uint16_t*>(at_bytes(x + 32 * s, x_off)), to_lds + 1024 * kTiles);
      }
    };
    uint8_t* raw = mine_lds + S::kDepth * S::kBytes;  // a group's values, each lane's own 32 bytes in two halves
    uint8_t* planes = raw + 2048;                     // its parts: [part][step][row][4 pieces]
    auto fetch_group = [&](int s) {
      // lanes whose k is past the end read the group's first step again, which nothing takes
      const uint32_t off = s + (x_k >> 2) < a.K / 32 ? x_off : x_off - 32u * (x_k & ~3);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        dma16(reinterpret_cast<const uint16_t*>(at_bytes(x + 32 * s + 4 * k, off)), raw + 1024 * k);
    };
    auto cut_group = [&] {
      const f32x4_t lo = __builtin_bit_cast(f32x4_t, lds_load16(raw, 16 * lane));
      const f32x4_t hi = __builtin_bit_cast(f32x4_t, lds_load16(raw, 1024 + 16 * lane));
      const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      u32x4_t part[3];
      split8(v, part);
      const int at = ((((x_k >> 2) << turn) + x_row) << 2) + ((x_k & 3) ^ swizzle4(x_row));
#pragma unroll
      for (int k = 0; k < 3; ++k) lds_store16(planes, 1024 * k + 16 * at, part[k]);
    };
    f32x4_t acc[kTiles];
#pragma unroll
    for (int k = 0; k < kTiles; ++k) acc[k] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (S::kPlanes && from < to) fetch_group(from);
#pragma unroll
    for (int k = 0; k < S::kDepth; ++k) {
      keep_order();
      if (from + k < to) stage(from + k, k);
    }
    int slot = 0;
    for (int s = from; s < to; ++s) {
      keep_order();  // what was requested so far is what the wait counts
      // Behind this step's stage were requested the next kDepth - 1 (and perhaps a group, which only makes the wait
      // longer); behind this step's group, group_steps stages.
      const int in_group = S::kPlanes ? (s - from) & (group_steps - 1) : 0;
      if (s + S::kDepth > to) {
        waitcnt<0, 15>();
      } else if (S::kPlanes && in_group == 0 && group_steps < S::kDepth) {
        waitcnt<0, 15>();
      } else {
        waitcnt<(S::kDepth - 1) * S::kDma, 15>();
      }
      keep_order();
      if constexpr (S::kPlanes) {
        if (in_group == 0) {
          cut_group();
          keep_order();
          waitcnt<63, 0>();  // the group has been read
          keep_order();
          if (s + group_steps < to) fetch_group(s + group_steps);
        }
      }
      const uint8_t* in = mine_lds + slot * S::kBytes;
      u32x4_t ar[kTiles], xp[Row8<kX>::kParts];
#pragma unroll
      for (int k = 0; k < kTiles; ++k) ar[k] = lds_load16(in + 1024 * k, 64 * i + 16 * (q ^ swizzle4(i)));
      in += 1024 * kTiles;
      if constexpr (kX == LoraX::bf16) {
        xp[0] = lds_load16(in, 64 * i + 16 * (q ^ swizzle4(i)));
      } else if constexpr (kX == LoraX::f32) {
        const int r = min(i, (1 << turn) - 1);
        const int at = (((in_group << turn) + r) << 2) + (q ^ swizzle4(r));
#pragma unroll
        for (int k = 0; k < 3; ++k) xp[k] = lds_load16(planes, 1024 * k + 16 * at);
      } else {
        Row8<kX> r8;
        r8.r = *reinterpret_cast<const u32x2_t*>(in + 32 * i + 8 * q);
        r8.parts(xp);
      }
#pragma unroll
      for (int p = Row8<kX>::kParts - 1; p >= 0; --p)
#pragma unroll
        for (int k = 0; k < kTiles; ++k) acc[k] = mfma_16x16x32(ar[k], xp[p], acc[k]);
      keep_order();
      waitcnt<63, 0>();  // the slot has been read
      keep_order();
      if (s + S::kDepth < to) stage(s + S::kDepth, slot);
      slot = slot + 1 < S::kDepth ? slot + 1 : 0;
    }
    // accumulator: column i is the row of x, element v is r = 16 k + 4 q + v
#pragma unroll
    for (int k = 0; k < kTiles; ++k)
#pragma unroll
      for (int v = 0; v < 4; ++v) red(wave, k)[16 * (4 * q + v) + i] = acc[k][v];

    // ---- y: units of 64 n. Of B, contiguous there, 16-byte piece g = n R / 8 + p lies at
    // piece (g % 8) ^ swizzle8(g / 8) of its 128 bytes.
    auto fetch_b = [&](int unit, uint8_t* to_lds) {
      const uint16_t* from_b = B + static_cast<int64_t>(unit) * kUnit * a.R;
      for (int c = 0; c < a.R / 8; ++c) {
        const int line = 8 * c + (lane >> 3);
        dma16(from_b + 64 * line + 8 * ((lane & 7) ^ swizzle8(line)), to_lds + 1024 * c);
      }
    };
    // Element n0 + 4 i + j of rows 4 q + v.
    struct Base {
      std::conditional_t<sizeof(TY) == 4, u32x4_t, u32x2_t> r[4];
    };
    uint32_t y_off[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
      y_off[v] = (static_cast<uint32_t>(row_of(4 * q + v)) * a.N + 4u * i) * static_cast<uint32_t>(sizeof(TY));
    auto fetch_base = [&](int unit, Base& to_regs) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        __builtin_memcpy(&to_regs.r[v], at_bytes(base + kUnit * unit, y_off[v]), sizeof(to_regs.r[v]));
    };
    constexpr bool kTwo = sizeof(TY) == 2 || kTiles > 2;  // two units' of base fit the registers
    Base held[kTwo ? 2 : 1];
    const int unit0 = first + wave;
    if (unit0 < last) {
      fetch_b(unit0, mine_lds);
      fetch_base(unit0, held[0]);
    }
    float factor[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      factor[v] = a.scaling != nullptr ? a.scaling[adapter] : 1.f;
      if constexpr (kX == LoraX::e4m3) factor[v] *= a.x_scale[row0 + row_of(4 * q + v)];
    }
    lds_barrier();
    for (int e = threadIdx.x; e < kTile * 32 * kSteps; e += 64 * kW) {
      const int r = e >> 4;
      float sum = 0.f;
      if (r < a.R) {
        float part[kW];
#pragma unroll
        for (int w = 0; w < kW; ++w) part[w] = red(w, r >> 4)[16 * (r & 15) + (e & 15)];
#pragma unroll
        for (int w = 0; w < kW; ++w) sum += part[w];
      }
      ts[(e & 15) * kRow + r] = sum;
    }
    lds_barrier();
    u32x4_t tp[kSteps][3];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const uint8_t* from_t = smem + kW * S::kLds;
      const int at = 4 * (i * kRow + 32 * s + 8 * q);
      const f32x4_t lo = __builtin_bit_cast(f32x4_t, lds_load16(from_t, at));
      const f32x4_t hi = __builtin_bit_cast(f32x4_t, lds_load16(from_t, at + 16));
      const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      split8(v, tp[s]);
    }
    const int pieces = a.R / 8;
    auto take = [&](auto in_half, int unit) {
      constexpr int kHalf = decltype(in_half)::value;
      Base& mine_base = held[kTwo ? kHalf : 0];
      const bool more = unit + kW < last;
      if (more) {
        fetch_b(unit + kW, mine_lds + (kHalf ^ 1) * kBBytes);
        if constexpr (kTwo) fetch_base(unit + kW, held[kHalf ^ 1]);
      }
      // For everything, the next unit's too: waiting by count for this unit's alone, 1100 rows with 32 r and bf16 took 24.2
      // us (20.7 so), with f32 36.6 (34.0), 256 rows with 64 r 20.4 (18.5).
      keep_order();
      waitcnt<0, 15>();
      keep_order();
      const uint8_t* in = mine_lds + kHalf * kBBytes;
      f32x4_t out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        out[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int g = (4 * i + j) * pieces + min(4 * s + q, pieces - 1);  // past R: where t is zero
          const u32x4_t b = lds_load16(in, 128 * (g >> 3) + 16 * ((g & 7) ^ swizzle8(g >> 3)));
#pragma unroll
          for (int p = 2; p >= 0; --p) out[j] = mfma_16x16x32(tp[s][p], b, out[j]);
        }
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (4 * q + v >= count) continue;
        TY* p = at_bytes(y + kUnit * unit, y_off[v]);
        if constexpr (sizeof(TY) == 4) {
          f32x4_t b = __builtin_bit_cast(f32x4_t, mine_base.r[v]);
#pragma unroll
          for (int j = 0; j < 4; ++j) b[j] = fmaf(factor[v], out[j][v], b[j]);
          __builtin_memcpy(p, &b, 16);
        } else {
          const u32x2_t b = mine_base.r[v];
          const float f = factor[v];
          const u32x2_t w = {pack_bf16(fmaf(f, out[0][v], bf16_lo(b[0])), fmaf(f, out[1][v], bf16_hi(b[0]))),
                             pack_bf16(fmaf(f, out[2][v], bf16_lo(b[1])), fmaf(f, out[3][v], bf16_hi(b[1])))};
          __builtin_memcpy(p, &w, 8);
        }
      }
      if (!kTwo && more) fetch_base(unit + kW, mine_base);
      keep_order();
      waitcnt<63, 0>();  // this half has been read
      keep_order();
    };
    for (int unit = unit0; unit < last; unit += 2 * kW) {
      take(std::integral_constant<int, 0>{}, unit);
      if (unit + kW < last) take(std::integral_constant<int, 1>{}, unit + kW);
    }
    lds_barrier();  // the next item's rows
  }
}

// ------------------------------------------------------------------ any sizes
// 8 elements from any address: the words that they lie in, each of which holds a byte of them, and the last of these by
// itself. (A load of 16 bytes at an odd element takes as long as several: 1100 rows with 32 r, N 8191 and K 2049 are 61
// us so and 36 here, one row with 16 r 13.6 and 7.7.)
typedef u32x4_t words4_t __attribute__((aligned(4)));
typedef u32x2_t words2_t __attribute__((aligned(4)));

template <class T>
__device__ __forceinline__ const uint8_t* word_of(const T* p) {
  return reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
}
template <class T>
__device__ __forceinline__ uint32_t last_word(const T* p) {
  return *reinterpret_cast<const uint32_t*>(word_of(reinterpret_cast<const uint8_t*>(p + 8) - 1));
}
__device__ __forceinline__ uint32_t shifted(uint32_t hi, uint32_t lo, const void* p) {
  return __builtin_amdgcn_alignbyte(hi, lo, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3));
}

// kAny: at any address; else at multiples of 4.
template <class T, bool kAny>
struct Words8;
template <bool kAny>
struct Words8<uint16_t, kAny> {
  u32x4_t w;
  uint32_t last;
  __device__ __forceinline__ void load(const uint16_t* p) {
    w = *reinterpret_cast<const words4_t*>(word_of(p));
    if constexpr (kAny) last = last_word(p);
  }
  __device__ __forceinline__ void get(const uint16_t* p, Raw8<uint16_t>& r) const {
    r.w = w;
    if constexpr (kAny)
      r.w = u32x4_t{shifted(w[1], w[0], p), shifted(w[2], w[1], p), shifted(w[3], w[2], p), shifted(last, w[3], p)};
  }
};
template <bool kAny>
struct Words8<uint8_t, kAny> {
  u32x2_t w;
  uint32_t last;
  __device__ __forceinline__ void load(const uint8_t* p) {
    w = *reinterpret_cast<const words2_t*>(word_of(p));
    if constexpr (kAny) last = last_word(p);
  }
  __device__ __forceinline__ void get(const uint8_t* p, u32x2_t& r) const {
    r = w;
    if constexpr (kAny) r = u32x2_t{shifted(w[1], w[0], p), shifted(last, w[1], p)};
  }
};
template <bool kAny>
struct Words8<float, kAny> {
  Raw8<float> r;
  __device__ __forceinline__ void load(const float* p) { load8(p, r); }
  __device__ __forceinline__ void get(const float*, Raw8<float>& v) const { v = r; }
};

__device__ __forceinline__ void store_words(float* p, const float* v) { store8(p, v); }
__device__ __forceinline__ void store_words(uint16_t* p, const float* v) {
  if ((reinterpret_cast<uintptr_t>(p) & 3) == 0) {
    store8(p, v);
  } else {
    typedef uint32_t words3_t __attribute__((ext_vector_type(3), aligned(4)));
    store1(p, v[0]);
    *reinterpret_cast<words3_t*>(p + 1) =
        words3_t{pack_bf16(v[1], v[2]), pack_bf16(v[3], v[4]), pack_bf16(v[5], v[6])};
    store1(p + 7, v[7]);
  }
}

// The same with loads into the operands' layout, for widths that are no multiples, more than 64 r and odd addresses.
// Whole steps of K are loaded without conditions, several under way, and what is cut by elements. kAny: some row's
// blocks of 8 are at no multiple of 4 (1100 rows with 32 r are 22 us with N 8200 and K 2056, 36 with 8191 and 2049, 18
// in the kernel above with 8192 and 2048). The next unit's operands under way too need more registers than two
// workgroups a CU have: 64 rows 14.3 -> 17.9 us. grid: place_of.
constexpr int kAnyWaves = 8;

// Steps of 32 k under way in a wave, as many as keep two workgroups a CU up to 32 r.
template <LoraX kX, int kTiles>
constexpr int kAnyAhead = kX == LoraX::f32 ? (kTiles > 1 ? 2 : 3) : (kTiles > 2 ? 2 : kTiles > 1 ? 3 : 5);

template <LoraX kX, class TY, int kTiles, int kSteps, bool kAny>
__global__ __launch_bounds__(64 * kAnyWaves, kSteps == 1 ? 4 : 2) void lora_any_kernel(LoraArgs a) {
  __shared__ f32x4_t red[kAnyWaves][kTiles][64];
  __shared__ u32x4_t parts[kSteps][3][64];
  __shared__ Table table;
  __shared__ __attribute__((aligned(16))) Items items;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k8 = lane >> 4;
  const Place place = place_of(a);
  if (place.item >= a.at_once) return;  // the whole workgroup
  const int row0 = place.block * kBlock;
  const int k_steps = (a.K + 31) / 32;
  const int from = min(a.wave_steps * wave, k_steps), to = min(from + a.wave_steps, k_steps), whole = min(to, a.K / 32);
  // units here are 32 n: two tiles of B side by side, row 4 q + v of tile j being n = 32 unit + 8 q + 4 j + v, so that
  // a lane's accumulators are 8 consecutive n of its row
  const int first = a.part_units * place.part, last = min(first + a.part_units, (a.N + 31) / 32);
  using X = typename Row8<kX>::T;
  const X* x = static_cast<const X*>(a.x) + static_cast<int64_t>(row0) * a.K;
  const TY* base = static_cast<const TY*>(a.base) + static_cast<int64_t>(row0) * a.N;
  TY* y = static_cast<TY*>(a.y) + static_cast<int64_t>(row0) * a.N;
  Row mine;
  const int n_items = find_items(a, row0, table, items, mine);

  for (int item = place.item; item < n_items; item += a.at_once) {
    const int adapter = __builtin_amdgcn_readfirstlane(items.adapter[item]);
    if (adapter == a.n && a.base == a.y) continue;
    const int count = take_item(items, item, mine);
    if (adapter == a.n) {
      copy_rows(a, base, y, items, count, 32 * first, min(32 * last, a.N));
      lds_barrier();
      continue;
    }
    const bool in = (lane & 15) < count;  // other lanes read what the item's first row does, and are not stored
    const int row = items.rows[in ? lane & 15 : 0];
    const X* x_row = x + static_cast<int64_t>(row) * a.K;
    const TY* base_row = base + static_cast<int64_t>(row) * a.N;
    const uint16_t* A = a.A + static_cast<int64_t>(adapter) * a.R * a.K;
    const uint16_t* B = a.B + static_cast<int64_t>(adapter) * a.N * a.R;
    const int64_t B_left = static_cast<int64_t>(a.n - adapter) * a.N * a.R;  // elements, this adapter's and the others'

    // Block b of a row of B as 8 elements from its first r: what is past R belongs to the next row and is cleared after
    // the load, and at the end of the last adapter's words are read one by one, none past the last.
    auto at_b = [&](int unit, int j, int s) {
      const int i = lane & 15, n = min(32 * unit + 8 * (i >> 2) + 4 * j + (i & 3), a.N - 1);  // past N: not stored
      return B + static_cast<int64_t>(n) * a.R + 8 * min(4 * s + k8, (a.R - 1) >> 3);
    };
    constexpr int kAtOnce = kSteps < 4 ? kSteps : 4;
    auto load_b = [&](int unit, int s0, Words8<uint16_t, kAny> (&r)[kAtOnce][2]) {
      if (static_cast<int64_t>(min(32 * unit + 32, a.N)) * a.R + 7 <= B_left) {
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j) r[s][j].load(at_b(unit, j, s0 + s));
      } else {
        const uint8_t* end = word_of(B + B_left - 1);
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint8_t* w = word_of(at_b(unit, j, s0 + s));
            auto word = [&](int i) { return *reinterpret_cast<const uint32_t*>(min(w + 4 * i, end)); };
            r[s][j].w = u32x4_t{word(0), word(1), word(2), word(3)};
            if constexpr (kAny) r[s][j].last = word(4);
          }
      }
    };
    auto get_b = [&](int unit, int j, int s, const Words8<uint16_t, kAny>& words) {
      Raw8<uint16_t> r;
      words.get(at_b(unit, j, s), r);
      const int left = a.R - 8 * (4 * s + k8);
#pragma unroll
      for (int d = 0; d < 4; ++d)
        r.w[d] &= left >= 2 * d + 2 ? 0xffffffffu : left == 2 * d + 1 ? 0x0000ffffu : 0u;
      return r.w;
    };
    auto at_base = [&](int unit) { return base_row + 32 * unit + 8 * k8; };
    auto load_base = [&](int unit, Words8<TY, kAny>& r) {
      if (32 * (unit + 1) <= a.N) {
        r.load(at_base(unit));
      } else if (8 * (4 * unit + k8) + 8 <= a.N) {
        r.load(at_base(unit));
      }
    };

    // t, kTiles tiles of r at a time, each two of which make one step of 32 r
#pragma unroll 1
    for (int r0 = 0; r0 < 32 * kSteps; r0 += 32 * ((kTiles + 1) / 2)) {
      f32x4_t acc[kTiles];
      const uint16_t* a_row[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {  // rows past R: the last one again, and t is cleared there
        a_row[i] = A + static_cast<int64_t>(min(r0 + 16 * i + (lane & 15), a.R - 1)) * a.K;
        acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      auto add = [&](const Row8<kX>& xr, const Raw8<uint16_t> (&ar)[kTiles]) {
        u32x4_t xp[Row8<kX>::kParts];
        xr.parts(xp);
#pragma unroll
        for (int p = Row8<kX>::kParts - 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < kTiles; ++i) acc[i] = mfma_16x16x32(ar[i].w, xp[p], acc[i]);
      };
      Row8<kX> cut_x;
      Raw8<uint16_t> cut_a[kTiles];
      const bool cut = from < to && whole < to;
      if (cut) {
        cut_x.load(x_row, 4 * whole + k8, a.K);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) load_block(a_row[i], 4 * whole + k8, a.K, cut_a[i]);
      }
      constexpr int kAhead = kAnyAhead<kX, kTiles>;
      for (int s0 = from; s0 < whole; s0 += kAhead) {
        Words8<X, kAny> xw[kAhead];
        Words8<uint16_t, kAny> aw[kAhead][kTiles];
        auto at = [&](int s) { return 32 * min(s0 + s, whole - 1) + 8 * k8; };  // past the last: again, not added
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
          xw[s].load(x_row + at(s));
#pragma unroll
          for (int i = 0; i < kTiles; ++i) aw[s][i].load(a_row[i] + at(s));
        }
        keep_order();
#pragma unroll
        for (int s = 0; s < kAhead; ++s)
          if (s0 + s < whole) {
            Row8<kX> xr;
            Raw8<uint16_t> ar[kTiles];
            xw[s].get(x_row, xr.r);
#pragma unroll
            for (int i = 0; i < kTiles; ++i) aw[s][i].get(a_row[i], ar[i]);
            add(xr, ar);
          }
      }
      if (cut) add(cut_x, cut_a);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) red[wave][i][lane] = acc[i];
      lds_barrier();
      if (wave < (kTiles + 1) / 2) {
        // this lane's 8 r of the step: of tile 2 wave + k8 / 2, held by lanes of quarters 2 (k8 % 2) and the next
        const int i = min(2 * wave + (lane >> 5), kTiles - 1), at = (lane & 15) + 32 * (k8 & 1);
        f32x4_t lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll
        for (int w = 0; w < kAnyWaves; ++w) {
          lo += red[w][i][at];
          hi += red[w][i][at + 16];
        }
        const int r = 2 * wave + (lane >> 5) < kTiles ? r0 + 32 * wave + 8 * k8 : a.R;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = r + k < a.R ? (k < 4 ? lo[k % 4] : hi[k % 4]) : 0.f;
        u32x4_t p[3];
        split8(v, p);
#pragma unroll
        for (int k = 0; k < 3; ++k) parts[r0 / 32 + wave][k][lane] = p[k];
      }
      lds_barrier();
    }
    float factor = a.scaling != nullptr ? a.scaling[adapter] : 1.f;
    if (a.x_scale != nullptr) factor *= a.x_scale[row0 + row];
    auto add = [&](int unit, int s0, const Words8<uint16_t, kAny> (&b)[kAtOnce][2], f32x4_t (&acc)[2]) {
#pragma unroll
      for (int s = 0; s < kAtOnce; ++s) {
        u32x4_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) w[j] = get_b(unit, j, s0 + s, b[s][j]);
#pragma unroll
        for (int p = 2; p >= 0; --p) {
          const u32x4_t t = parts[s0 + s][p][lane];
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[j] = mfma_16x16x32(w[j], t, acc[j]);
        }
      }
    };
    auto finish = [&](int unit, const Words8<TY, kAny>& words, const f32x4_t (&acc)[2]) {
      const int n = 8 * (4 * unit + k8);
      if (!in || n >= a.N) return;
      auto result = [&](int j, float v) { return fmaf(factor, acc[j / 4][j % 4], v); };
      TY* y_row = y + static_cast<int64_t>(row) * a.N;
      float v[8];
      Raw8<TY> raw;
      if (n + 8 <= a.N) {
        words.get(at_base(unit), raw);
        unpack8(raw, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = result(j, v[j]);
        if constexpr (kAny) {
          store_words(y_row + n, v);
        } else {
          store8(y_row + n, v);
        }
      } else {
        load8_cut(base_row + n, a.N - n, raw);
        unpack8(raw, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = result(j, v[j]);
        store8_cut(y_row + n, a.N - n, v);
      }
    };
    for (int unit = first + wave; unit < last; unit += kAnyWaves) {
      Words8<TY, kAny> words;
      load_base(unit, words);
      f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int s0 = 0; s0 < kSteps; s0 += kAtOnce) {
        Words8<uint16_t, kAny> b[kAtOnce][2];
        load_b(unit, s0, b);
        keep_order();
        add(unit, s0, b, acc);
      }
      finish(unit, words, acc);
    }
    lds_barrier();  // the next item's rows
  }
}

// Blocks of 8 of every row at multiples of 4.
template <LoraX kX, class TY>
bool at_words(const LoraArgs& a) {
  const uintptr_t addresses = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.A) |
                              reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.base) |
                              reinterpret_cast<uintptr_t>(a.y);
  const int64_t rows = a.K * sizeof(typename Row8<kX>::T) | a.K * 2 | a.R * 2 | a.N * sizeof(TY);
  return ((addresses | rows) & 3) == 0;
}

template <LoraX kX, class TY, bool kAny>
void launch_any(const LoraArgs& a, dim3 grid, hipStream_t s) {
  if (a.R <= 16) {
    lora_any_kernel<kX, TY, 1, 1, kAny><<<grid, 64 * kAnyWaves, 0, s>>>(a);
  } else if (a.R <= 32) {
    lora_any_kernel<kX, TY, 2, 1, kAny><<<grid, 64 * kAnyWaves, 0, s>>>(a);
  } else if (a.R <= 64) {
    lora_any_kernel<kX, TY, 4, 2, kAny><<<grid, 64 * kAnyWaves, 0, s>>>(a);
  } else if (a.R <= 128) {
    lora_any_kernel<kX, TY, 4, 4, kAny><<<grid, 64 * kAnyWaves, 0, s>>>(a);
  } else {
    lora_any_kernel<kX, TY, 4, 8, kAny><<<grid, 64 * kAnyWaves, 0, s>>>(a);
  }
}

template <LoraX kX, class TY>
void launch(const LoraArgs& a, bool even, int waves, dim3 grid, hipStream_t s) {
  if (even) {
    if (waves == 16) {
      if constexpr (kX == LoraX::f32) {
        if (a.R <= 16) {
          lora_kernel<kX, TY, 1, 16><<<grid, 1024, 0, s>>>(a);
        } else {
          lora_kernel<kX, TY, 2, 16><<<grid, 1024, 0, s>>>(a);
        }
      }
    } else if (a.R <= 16) {
      lora_kernel<kX, TY, 1, 8><<<grid, 512, 0, s>>>(a);
    } else if (a.R <= 32) {
      lora_kernel<kX, TY, 2, 8><<<grid, 512, 0, s>>>(a);
    } else {
      lora_kernel<kX, TY, 4, 8><<<grid, 512, 0, s>>>(a);
    }
  } else if (at_words<kX, TY>(a)) {
    launch_any<kX, TY, false>(a, grid, s);
  } else {
    launch_any<kX, TY, true>(a, grid, s);
  }
}

template <class TY>
void launch(const LoraArgs& a, LoraX x_type, bool even, int waves, dim3 grid, hipStream_t s) {
  if (x_type == LoraX::bf16) {
    launch<LoraX::bf16, TY>(a, even, waves, grid, s);
  } else if (x_type == LoraX::f32) {
    launch<LoraX::f32, TY>(a, even, waves, grid, s);
  } else {
    launch<LoraX::e4m3, TY>(a, even, waves, grid, s);
  }
}

}  // namespace

hipError_t launch_lora(LoraArgs a, LoraX x_type, bool y_f32, hipStream_t s) {
  const uintptr_t addresses = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.A) |
                              reinterpret_cast<uintptr_t>(a.B);
  const bool even = a.K % 64 == 0 && a.N % kUnit == 0 && a.R % 8 == 0 && a.R <= 64 && a.K <= (1 << 22) &&
                    addresses % 16 == 0;
  const int units = even ? a.N / kUnit : (a.N + 31) / 32;
  a.blocks = (a.M + kBlock - 1) / kBlock;
  // items of a block at most: whole ones, and a cut one of each adapter (and of none)
  const int rows = std::min(a.M, kBlock);
  const int items = static_cast<int>(std::min<int64_t>(rows, rows / kTile + int64_t(a.n) + 1));
  // Under way at once: 512 workgroups in all, and never fewer than a block of one adapter has. All of them for many
  // adapters, most of which would find nothing, is 1100 rows of 64 adapters 39 us instead of 36.
  a.at_once = std::min(items, std::max(512 / a.blocks, rows / kTile));
  // Parts of N for a workgroup a CU (each computes t, so twice as many is 64 rows of 48 adapters with K 8192 15 -> 20
  // us, half as many is 256 rows of 64 adapters with N 8192 14 -> 25), at least 4 units each.
  const int workgroups = a.blocks * std::min(a.at_once, a.blocks == 1 ? kBlock : rows / kTile + 4);
  const int parts = std::max(std::min(256 / workgroups, (units + 3) / 4), 1);
  // 8 waves, of which two workgroups fit a CU; 16 where few of them have a long K of fp32 rows each, which they cut into
  // parts: 1, 16 and 64 rows with 16 r, N 2048 and K 4096, 5120 and 8192 are 7.4, 10.4, 10.3; 8.5, 11.6, 11.9; 10.9, 15.2, 16.3
  // us with 8 waves and 7.6, 10.5, 10.1; 8.1, 11.7, 11.6; 9.8, 14.2, 14.9 with 16. bf16 rows, with K 8192: 8.3, 11.3, 10.5 and
  // 9.3, 12.6, 11.6; e4m3 9.8, 11.7, 11.7 and 9.6, 13.0, 12.4.
  const int waves =
      even && x_type == LoraX::f32 && a.R <= 32 && workgroups * parts <= 256 && a.K > 4096 ? 16 : 8;
  a.wave_steps = ((a.K + 31) / 32 + waves - 1) / waves;
  a.part_units = (units + parts - 1) / parts;
  a.parts = (units + a.part_units - 1) / a.part_units;
  a.apart = a.blocks * a.at_once >= 32 ? 3 : 0;
  const dim3 grid(a.parts << a.apart, (a.blocks * a.at_once + (1 << a.apart) - 1) >> a.apart);
  if (y_f32) {
    launch<float>(a, x_type, even, waves, grid, s);
  } else {
    launch<uint16_t>(a, x_type, even, waves, grid, s);
  }
  return hipGetLastError();
}

}  // namespace twell
