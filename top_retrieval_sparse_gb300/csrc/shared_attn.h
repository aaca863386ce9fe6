// shared_attn.h -- the step over shared rows: argument block, the list of its work and where
// its partials lie (host <-> device contract inside the library; not part of the C ABI).
#pragma once

#include "cache_ops.h"

namespace tsa {

constexpr int kUnitRows = 256;      // query rows of a unit: two tiles of the tensor core
constexpr int kSharedShares = 152;  // CTAs of the prefix kernel: one an SM
// Cost of a key tile with two query tiles and with one (the products bound the former, the
// rows' bytes the latter).
constexpr int kCostBoth = 4, kCostAlone = 3;

// A group, as the first kernel finds it.
struct SharedGroup {
  int64_t cost0;  // of the groups before it
  int64_t row0;   // first row of its partials
  int32_t b0;     // first sequence
  int32_t rows;   // queries of a KV head: sequences * G
  int32_t P;      // shared rows
  int32_t unit0;  // units of the groups before it
};
struct SharedTotal {
  int64_t cost;
  int32_t shares;  // of the list that take part
  int2 segments[kSharedShares];  // each share's: the number of the first, how many
};
// What a share has of a unit.
struct __align__(16) SharedSegment {
  int32_t b0, P;         // the group's first sequence, its rows
  int32_t seq0, in0;     // sequence and query head of the unit's first query
  int32_t g, rows, rs;   // KV head, queries, rows of a half of the partials
  int32_t both;          // two query tiles
  int32_t copies;        // of the queries in the one tile
  int32_t j0, j1, pad;   // key tiles
  int64_t part;          // its partials: float4's from a.parts
};

struct SharedArgs {
  const uint16_t* q;       // bf16 [B][Hq][128]
  CacheView c;
  const int32_t* lens;
  const int32_t* cu;       // [N + 1] sequences before every group
  const int32_t* shared;   // [N]
  int B, N, Hq, G;
  int inv_g;               // ceil(2^16 / G): r / G = r * inv_g >> 16 for small r
  float scale_log2;
  int box;                 // rows of a copy: 128, or a smaller page
  void* out;               // [B][Hq][128], fp32 or bf16
  int out16;
  float* lse;              // [B][Hq] or nullptr
  int* status;
  // in the workspace
  int32_t* group;          // [B]: a sequence's group, -1: none, kNoGroups: its output is NaN
  int32_t* start;          // [B]: its rows before this one are the group's
  int32_t* leader;         // [B]: the sequence whose cache has them (small caches, else nullptr)
  SharedGroup* groups;     // [N]
  SharedTotal* total;
  SharedSegment* segments; // share after share; number: the share's, plus that of the unit
  int2* spans;             // [units]: a unit's first and last share
  float* own_out;          // [B][Hq][128]: over its own rows
  float* own_lse;          // [B][Hq]
  uint32_t* arrived;       // counters of the decode kernel
  float* parts;            // partials: of each share's first segment, then of the units
};
cudaError_t launch_shared_prep(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_shared_prefix(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const SharedArgs& a, int fmt, cudaStream_t st);
cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t st);

// Rows of partials (of kD + 2 floats) that a share can need, a half of a unit of so many
// queries (while sums are folded the copies in its one tile have theirs), and a group's units.
constexpr int64_t kShareRows = kUnitRows;
// Few queries are laid out 4 or 2 times in their tile of 128 rows, and each copy takes a part
// of the key tile's columns, so that all warps have exponentials to take.
__host__ __device__ inline int tile_copies(int rows) { return rows <= 32 ? 4 : (rows <= 64 ? 2 : 1); }
__host__ __device__ inline int half_rows(int rows) {
  return rows > 128 ? 128 : (rows * tile_copies(rows) + 1) / 2 * 2;
}
__host__ __device__ inline int64_t group_rows(int rows, int Hkv) {
  if (rows == 0) return 0;
  const int full = (rows - 1) / kUnitRows;
  return (int64_t)Hkv * (full * kUnitRows + 2 * half_rows(rows - full * kUnitRows));
}

#ifdef __CUDACC__
// a / b of numbers that are not negative: in 32 bits where they fit (64-bit division takes
// hundreds of cycles).
__device__ __forceinline__ int64_t over(int64_t a, int64_t b) {
  if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
  return (int64_t)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ int64_t share_start(const SharedTotal& t, int share) {
  return over(t.cost * share + t.shares - 1, t.shares);
}

// A unit: queries [256 t, ...) of KV head g of a group.
struct SharedUnit {
  int t, g, rows, tiles, w;  // w: cost of a key tile
  int rs;                    // rows of a half of its partials
  int64_t cost0, row0;
  __device__ bool both() const { return w == kCostBoth; }
};
__device__ __forceinline__ SharedUnit unit_of(const SharedGroup& s, int Hkv, int t, int g) {
  SharedUnit u;
  u.t = t;
  u.g = g;
  u.rows = s.rows - t * kUnitRows < kUnitRows ? s.rows - t * kUnitRows : kUnitRows;
  u.tiles = (s.P + 127) / 128;
  u.w = u.rows > 128 ? kCostBoth : kCostAlone;
  u.rs = half_rows(u.rows);
  u.cost0 = s.cost0 + (int64_t)u.tiles * ((int64_t)t * Hkv * kCostBoth + g * u.w);
  u.row0 = s.row0 + (int64_t)t * Hkv * kUnitRows + (int64_t)g * 2 * u.rs;
  return u;
}
// Floats from a half of a segment's partials to the next: O as [32][rs] pieces of four
// columns, then maxima and sums.
__device__ __forceinline__ int64_t half_floats(int rs) { return (int64_t)rs * (kD + 2); }
// Where a segment's partials begin (a share has at most one that is not its unit's first), in
// pieces of 16 bytes.
__device__ __forceinline__ int64_t segment_part(const SharedUnit& u, int share, bool first) {
  const int64_t row = first ? kSharedShares * kShareRows + u.row0 : share * kShareRows;
  return row * (kD + 2) / 4;
}

#endif

}  // namespace tsa
