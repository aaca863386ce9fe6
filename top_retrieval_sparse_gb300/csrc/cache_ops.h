// cache_ops.h -- argument blocks and launchers of the cache-side kernels:
// rotary positions, the 8-bit cache, window attention (host <-> device
// contract inside the library; not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_internal.cuh"

namespace tsa {

// Rotary table: cos and sin (times the amplitude) of l * w_i for
// l < kRopeLow, then cos and sin of kRopeLow * h * w_i for h < n_hi.
constexpr int kRopeLowBits = 11;
constexpr int kRopeLow = 1 << kRopeLowBits;
struct RopeView {
  const float2* lo;  // [kRopeLow][pairs]; nullptr: no rotation
  const float2* hi;  // [n_hi][pairs]
  int64_t max_pos;
  int pairs;         // rot_dim / 2, a multiple of 8
  int interleaved;
};

struct RopeTableArgs {
  float2* lo;
  float2* hi;
  int n_hi, pairs;
  double amplitude;
  double w[kD / 2];
};
cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t st);

// Rows of [T][H] heads, strides in elements.
struct RowsView {
  uint16_t* p;
  int64_t st, sh;
};

struct RopeArgs {
  RowsView q, qo, k, ko;
  int Hq, Hkv;
  int64_t T;
  const int32_t* positions;
  RopeView rope;
  int inverse;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st);

// A cache that the attention and cache kernels read: byte rows of one KV
// head, contiguous or paged.  Scales (8-bit formats) are indexed by row >>
// block_shift, since a block divides a page and l_cap.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* page_table;
  int64_t l_cap;
  int page_shift, max_pages;
  uint32_t n_pages;
  int Hkv;
  int block_shift;
};
enum CacheFormat : int { kFmtInt8 = 0, kFmtE4m3 = 1, kFmtBf16 = 2 };

// Row index of position i (i < l_cap) of KV head g of sequence b; -1 on a
// page outside the pool.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int b, int g, int64_t i) {
  if (c.page_table) {
    const int32_t page = c.page_table[(int64_t)b * c.max_pages + (i >> c.page_shift)];
    if ((uint32_t)page >= c.n_pages) return -1;
    return (((int64_t)page * c.Hkv + g) << c.page_shift) + (i & ((1 << c.page_shift) - 1));
  }
  return ((int64_t)b * c.Hkv + g) * c.l_cap + i;
}

// Tokens [lo, lo + n) of sequence b in a ragged (cu) or uniform batch;
// false: more than max_n, or not inside [0, T).
__device__ __forceinline__ bool seq_tokens(const int32_t* cu, int max_n, int64_t T, int b,
                                           int64_t& lo, int64_t& n) {
  if (!cu) {
    lo = (int64_t)b * max_n;
    n = max_n;
    return true;
  }
  lo = cu[b];
  n = (int64_t)cu[b + 1] - lo;
  return lo >= 0 && n >= 0 && n <= max_n && lo + n <= T;
}

struct AppendArgs {
  CacheView c;
  int fmt, block;
  RowsView k, v;
  const int32_t* cu;
  int64_t T;
  int max_new;
  const int32_t* lens;
  int B;
  RopeView rope;
  const int32_t* positions;
  int* status;
};
cudaError_t launch_kv8_append(const AppendArgs& a, cudaStream_t st);

struct ReadArgs {
  CacheView c;
  int fmt;
  RowsView k, v;
  const int32_t* cu;
  int64_t T;
  int max_new;
  const int32_t* lens;
  int B;
  int* status;
};
cudaError_t launch_kv8_read(const ReadArgs& a, cudaStream_t st);

// One decode step (attn_decode.cu).
constexpr int kDecodeThreads = 128;
constexpr int kDecodeShares = 4 * 152;                      // most CTAs of a call
constexpr int kDecodeSlot = 2 * kMaxGroup + kMaxGroup * kD; // floats of a partial
struct DecodeArgs {
  const uint16_t* q;       // bf16 [B][Hq][128]
  CacheView c;
  const int32_t* lens;
  int B, Hq;
  int64_t n_init, n_recent;
  float scale_log2;        // scale * log2(e)
  float* out;              // fp32 [B][Hq][128]
  float* lse;              // [B][Hq] or nullptr
  int* status;
  float* partial;          // [2 * kDecodeShares][kDecodeSlot]
  uint32_t* arrived;       // [B * Hkv], zero between calls
};
int attn_decode_ctas(int fmt);  // resident CTAs of an SM
cudaError_t launch_attn_decode(const DecodeArgs& a, int fmt, int grid, cudaStream_t st);

// Many tokens per sequence (window_prefill.cu); the maps are the bf16 pool's
// rows of 128 elements, in boxes of 64 elements by `box` rows.
constexpr int kPreSlot = 2 * 128 + 128 * kD;  // floats of a query tile's partial
// Key tiles between two additions of O to a CTA's sums in the workspace, and how many
// CTAs can have such sums at once (one runs on an SM).
constexpr int kFoldTiles = 128;
constexpr int kFoldPlaces = 152;
struct PrefillArgs {
  RowsView q;
  CacheView c;
  const int32_t* cu;
  int64_t T;
  int max_q;
  const int32_t* lens;
  int Hq, G, inv_g;      // inv_g = ceil(2^16 / G): r / G = r * inv_g >> 16 for r < 128
  int n_init, n_recent;  // clipped to l_cap
  float scale_log2;    // |scale| * log2(e), > 0
  int negate, zero;    // scale < 0: the queries' sign turned; scale = 0: zeros in their place
  int box;
  uint16_t* out;       // bf16 [T][Hq][128]
  float* lse;          // [T][Hq] or nullptr
  int* status;
  int blocks, splits;  // CTAs of a sequence's tokens, and of each one's key tiles
  float* partial;      // [B * Hkv * blocks][splits][2][kPreSlot] (splits > 1)
  float* sums;         // [kFoldPlaces][2][128 * kD], or nullptr: no part has so many tiles
  uint32_t* places;    // [kFoldPlaces], zero between calls
};
cudaError_t launch_window_prefill(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  const PrefillArgs& a, int B, cudaStream_t st);
cudaError_t launch_window_join(const PrefillArgs& a, int B, cudaStream_t st);  // splits > 1

// Launch as a programmatic dependent of the kernel before it on the stream:
// every such kernel calls pdl_wait() before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace tsa
