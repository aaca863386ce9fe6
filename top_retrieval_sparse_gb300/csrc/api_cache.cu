// api_cache.cu -- C ABI of the cache-side operators (declared in
// include/tsa.h): rotary positions, the 8-bit cache, window attention.
//
// Host-side validation, workspace layout and launches.  Nothing here allocates
// device memory, synchronises or prints.
#include <atomic>
#include <cmath>

#include "api_util.h"
#include "cache_ops.h"
#include "shared_attn.h"

using namespace tsa;

namespace {

constexpr double kPi = 3.14159265358979323846;
constexpr double kLog2e = 1.4426950408889634;

// ------------------------------------------------------------- rotation
bool rope_sizes(int rot_dim, int64_t max_pos) {
  return rot_dim >= 16 && rot_dim <= kD && rot_dim % 16 == 0 && max_pos > 0 &&
         max_pos <= (int64_t)1 << 26;
}
int64_t rope_high(int64_t max_pos) { return (max_pos + kRopeLow - 1) / kRopeLow; }

int check_rope(const tsa_rope* r, RopeView& v) {
  v = RopeView{};
  if (!r) return TSA_OK;
  if (!r->table || !aligned(r->table, 16))
    return fail(TSA_ERR_INVALID_ARG, "rope->table NULL or not 16-byte aligned");
  if (!rope_sizes(r->rot_dim, r->max_pos))
    return fail(TSA_ERR_INVALID_ARG, "rope: rot_dim %d or max_pos %lld out of range", r->rot_dim,
                (long long)r->max_pos);
  if (r->layout != TSA_ROPE_HALF && r->layout != TSA_ROPE_INTERLEAVED)
    return fail(TSA_ERR_INVALID_ARG, "rope: unknown layout %d", r->layout);
  v.pairs = r->rot_dim / 2;
  v.lo = static_cast<const float2*>(r->table);
  v.hi = v.lo + (size_t)kRopeLow * v.pairs;
  v.max_pos = r->max_pos;
  v.interleaved = r->layout == TSA_ROPE_INTERLEAVED;
  return TSA_OK;
}

// The axis of every pair of a rotation of rot_dim elements.
int axes_of(const tsa_rope_axes* x, int rot_dim, int (&axis)[kD / 2]) {
  if (!x) return fail(TSA_ERR_INVALID_ARG, "axes is NULL");
  if (x->n < 1 || x->n > 4) return fail(TSA_ERR_INVALID_ARG, "axes: n %d not in [1, 4]", x->n);
  if (x->order != TSA_AXES_BLOCKS && x->order != TSA_AXES_TURNS)
    return fail(TSA_ERR_INVALID_ARG, "axes: unknown order %d", x->order);
  if (x->rates != TSA_RATES_JOINT && x->rates != TSA_RATES_OWN)
    return fail(TSA_ERR_INVALID_ARG, "axes: unknown rates %d", x->rates);
  int left[4] = {}, all = 0;
  for (int a = 0; a < x->n; ++a) {
    if (x->pairs[a] < 1 || x->pairs[a] > kD / 2)
      return fail(TSA_ERR_INVALID_ARG, "axes: pairs[%d] = %d", a, x->pairs[a]);
    all += left[a] = x->pairs[a];
  }
  if (all != rot_dim / 2)
    return fail(TSA_ERR_INVALID_ARG, "axes: %d pairs, the rotation has %d", all, rot_dim / 2);
  for (int i = 0, a = 0; i < all; ++i) {
    while (left[a] == 0) a = (a + 1) % x->n;
    axis[i] = a;
    --left[a];
    if (x->order == TSA_AXES_TURNS) a = (a + 1) % x->n;
  }
  return TSA_OK;
}

int check_axes(const tsa_rope_axes* x, const tsa_rope* rope, int64_t stride, AxesView& v) {
  v = AxesView{};
  int axis[kD / 2] = {};
  const int rc = axes_of(x, rope->rot_dim, axis);
  if (rc) return rc;
  if (stride < 0 || stride >= (int64_t)1 << 40)
    return fail(TSA_ERR_INVALID_ARG, "the positions' stride must be in [0, 2^40)");
  v.n = x->n;
  v.stride = stride;
  for (int i = 0; i < rope->rot_dim / 2; ++i) v.of[i / 8] |= (uint16_t)(axis[i] << (2 * (i % 8)));
  return TSA_OK;
}

// Rows of T tokens and H heads (written rows must not overlap).
int check_rows(const tsa_rows* r, int64_t T, int H, bool written, const char* name, RowsView& v) {
  v = RowsView{};
  if (!r || !r->data) return fail(TSA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(r->data, 16)) return fail(TSA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (r->stride_t < 0 || r->stride_h < 0 || r->stride_t % 8 || r->stride_h % 8)
    return fail(TSA_ERR_INVALID_ARG, "%s: strides must be multiples of 8 and not negative", name);
  if (r->stride_t >= (int64_t)1 << 31 || r->stride_h >= (int64_t)1 << 40)
    return fail(TSA_ERR_INVALID_ARG, "%s: stride out of range", name);
  if (written) {
    const bool by_head = (H <= 1 || r->stride_h >= kD) &&
                         (T <= 1 || r->stride_t >= (H - 1) * r->stride_h + kD);
    const bool by_token = (T <= 1 || r->stride_t >= kD) &&
                          (H <= 1 || r->stride_h >= (T - 1) * r->stride_t + kD);
    if (!by_head && !by_token)
      return fail(TSA_ERR_INVALID_ARG, "%s: the strides make rows overlap", name);
  }
  v.p = static_cast<uint16_t*>(r->data);
  v.st = r->stride_t;
  v.sh = r->stride_h;
  return TSA_OK;
}

int check_tokens(int64_t T, int max_n, const int32_t* cu, int B, const char* what) {
  if (T < 0 || T >= (int64_t)1 << 31) return fail(TSA_ERR_INVALID_ARG, "T out of range");
  if (max_n < 0) return fail(TSA_ERR_INVALID_ARG, "%s < 0", what);
  if (!cu && T != (int64_t)B * max_n)
    return fail(TSA_ERR_INVALID_ARG, "without offsets T must be B * %s (%lld != %d * %d)", what,
                (long long)T, B, max_n);
  return TSA_OK;
}

int check_batch(int B, int Hkv, int d) {
  if (d != kD) return fail(TSA_ERR_INVALID_ARG, "d = %d: only d = 128 is compiled", d);
  if (B < 0 || B > kMostSequences)
    return fail(TSA_ERR_INVALID_ARG, "B = %d: must be in [0, %d]", B, kMostSequences);
  if (Hkv <= 0 || Hkv > 1024)
    return fail(TSA_ERR_INVALID_ARG, "Hkv = %d: must be in [1, 1024]", Hkv);
  return TSA_OK;
}

int check_groups(int B, int Hq, int Hkv) {
  if (Hq <= 0 || Hq % Hkv)
    return fail(TSA_ERR_INVALID_ARG, "Hq %% Hkv != 0 (Hq=%d Hkv=%d)", Hq, Hkv);
  if (Hq / Hkv > kMaxGroup)
    return fail(TSA_ERR_INVALID_ARG, "group size %d > %d", Hq / Hkv, kMaxGroup);
  if ((int64_t)B * Hq > 65535)
    return fail(TSA_ERR_INVALID_ARG, "B*Hq = %lld > 65535", (long long)B * Hq);
  return TSA_OK;
}

// --------------------------------------------------------------- caches
int check_kv8(const tsa_kv8* c, int Hkv, CacheView& v) {
  v = CacheView{};
  if (!c) return fail(TSA_ERR_INVALID_ARG, "cache is NULL");
  if (!c->k || !c->v || !c->k_scale || !c->v_scale)
    return fail(TSA_ERR_INVALID_ARG, "cache codes or scales are NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(TSA_ERR_INVALID_ARG, "cache->k / cache->v must be 16-byte aligned");
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(TSA_ERR_INVALID_ARG, "cache scales must be 4-byte aligned");
  if (c->status && !aligned(c->status, kAlign))
    return fail(TSA_ERR_INVALID_ARG, "cache->status must be 256-byte aligned");
  if (c->format != TSA_KV8_INT8 && c->format != TSA_KV8_E4M3)
    return fail(TSA_ERR_INVALID_ARG, "unknown cache format %d", c->format);
  const int blk = c->block;
  if (blk != 16 && blk != 32 && blk != 64 && blk != 128)
    return fail(TSA_ERR_INVALID_ARG, "block %d: must be 16, 32, 64 or 128", blk);
  if (c->l_cap <= 0 || c->l_cap >= (int64_t)1 << 31)
    return fail(TSA_ERR_INVALID_ARG, "l_cap must be in [1, 2^31)");
  if (c->page_table) {
    const int ps = c->page_size;
    if (ps < 16 || ps > 256 || (ps & (ps - 1)))
      return fail(TSA_ERR_INVALID_ARG, "page_size %d: must be a power of two in [16, 256]", ps);
    if (blk > ps) return fail(TSA_ERR_INVALID_ARG, "block %d > page_size %d", blk, ps);
    if (c->max_pages <= 0 || (int64_t)c->max_pages * ps != c->l_cap)
      return fail(TSA_ERR_INVALID_ARG, "paged cache: l_cap must equal max_pages*page_size");
    if (c->n_pages <= 0) return fail(TSA_ERR_INVALID_ARG, "n_pages must be > 0");
    while ((1 << v.page_shift) < ps) ++v.page_shift;
  } else if (c->l_cap % blk) {
    return fail(TSA_ERR_INVALID_ARG, "block %d does not divide l_cap %lld", blk,
                (long long)c->l_cap);
  }
  while ((1 << v.block_shift) < blk) ++v.block_shift;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.page_table = c->page_table;
  v.l_cap = c->l_cap;
  v.max_pages = c->max_pages;
  v.n_pages = (uint32_t)c->n_pages;
  v.Hkv = Hkv;
  return TSA_OK;
}

int check_cache(const tsa_kv* kv, int Hkv, CacheView& v) {
  v = CacheView{};
  const int rc = validate_kv(kv);
  if (rc) return rc;
  if (kv->l_cap <= 0) return fail(TSA_ERR_INVALID_ARG, "kv->l_cap must be > 0");
  if (kv->page_table)
    while ((1 << v.page_shift) < kv->page_size) ++v.page_shift;
  v.k = static_cast<uint8_t*>(const_cast<void*>(kv->k));
  v.v = static_cast<uint8_t*>(const_cast<void*>(kv->v));
  v.page_table = kv->page_table;
  v.l_cap = kv->l_cap;
  v.max_pages = kv->max_pages;
  v.n_pages = 0x80000000u;  // the pool's size is not known: any page that is not negative
  v.Hkv = Hkv;
  return TSA_OK;
}

int check_window(int64_t n_init, int64_t n_recent, float scale) {
  if (n_init < 0 || n_recent < 0)
    return fail(TSA_ERR_INVALID_ARG, "n_init and n_recent must be >= 0");
  if (!std::isfinite(scale)) return fail(TSA_ERR_INVALID_ARG, "scale must be finite");
  return TSA_OK;
}

// The tensor map of a bf16 pool's rows: boxes of 64 elements by `box` rows with
// the 128-byte swizzle; of a pool of codes: boxes of whole rows as they are (encoded on
// the host; nothing is launched).
int row_map(const void* base, int64_t rows, int box, CUtensorMap* map, bool codes = false) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || !f)
      return fail(TSA_ERR_CUDA, "cuTensorMapEncodeTiled not found: %s", cudaGetErrorString(e));
    fn.store(f, std::memory_order_release);
  }
  const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(codes ? kD : kRowBytes)};
  const cuuint32_t extent[2] = {(cuuint32_t)(codes ? kD : 64), (cuuint32_t)box}, step[2] = {1, 1};
  const CUresult r = reinterpret_cast<Encode>(f)(
      map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
      const_cast<void*>(base), dims, strides, extent, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
      codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(TSA_ERR_CUDA, "tensor map: driver error %d", (int)r);
  return TSA_OK;
}

// Workspace of a decode step: the status word, the shares' partials, then the
// units' arrival counters.  The counters come after a region of fixed size, so
// that whatever sizes share a workspace, they only ever hold counters.
constexpr size_t kDecodePartial = kAlign;
constexpr size_t kDecodeArrived =
    kDecodePartial + (size_t)2 * kDecodeShares * kDecodeSlot * sizeof(float);

// How the prefill kernel cuts a call: CTAs of 2 * floor(128 / G) tokens each, and
// where those are at most half the SMs, each one's key tiles over several.  A
// part saves the tiles that others take (1.3 us each) and costs its partial and a
// share of joining them: at most 8 for full tiles, more for few rows, never below two
// tiles (16 tokens late in a window of 4096, 33 tiles a head: 60 us in one CTA).
struct PrefillCut {
  int64_t blocks, splits, units;
  bool folds;  // a CTA may have more than kFoldTiles key tiles
};
PrefillCut prefill_cut(int B, int Hkv, int G, int64_t max_q, int64_t l_cap, int64_t n_init,
                       int64_t n_recent) {
  PrefillCut c{0, 1, 0, false};
  const int64_t tokens = 2 * (128 / G);
  c.blocks = (max_q + tokens - 1) / tokens;
  c.units = c.blocks * B * Hkv;
  const int64_t sms = 152;  // (not the device's: sizes do not depend on where they are asked)
  const int64_t q = max_q < tokens ? max_q : tokens;
  auto tiles = [&](int64_t rows) { return ((rows < l_cap ? rows : l_cap) + 127) / 128; };
  int64_t n = tiles(n_init < l_cap ? n_init : l_cap) + 1 +
              tiles((n_recent < l_cap ? n_recent : l_cap) + q);
  if (n > tiles(l_cap)) n = tiles(l_cap);
  c.folds = n > kFoldTiles;
  if (c.units < 1 || c.units > sms / 2) return c;
  const int64_t rows = max_q * G < 128 ? max_q * G : 128;
  c.splits = sms / c.units;
  if (c.splits > (n + 1) / 2) c.splits = (n + 1) / 2;
  if (c.splits > 8 * 128 / rows) c.splits = 8 * 128 / rows;
  if (c.splits > 32) c.splits = 32;
  if (c.splits < 1) c.splits = 1;
  c.folds = (n + c.splits - 1) / c.splits > kFoldTiles;
  return c;
}
// Workspace: the status word, which places of the long sums are taken (zero between
// calls of whatever sizes, so at a fixed offset), the partials, the long sums.
constexpr size_t kPrePlaces = kAlign;
constexpr size_t kPrePartial =
    kPrePlaces + (kFoldPlaces * sizeof(uint32_t) + kAlign - 1) / kAlign * kAlign;
size_t prefill_sums(const PrefillCut& c) {
  return kPrePartial + (c.splits > 1 ? (size_t)(c.units * c.splits) * 2 * kPreSlot * sizeof(float)
                                     : 0);
}
size_t prefill_bytes(const PrefillCut& c) {
  return prefill_sums(c) + (c.folds ? (size_t)kFoldPlaces * 2 * 128 * kD * sizeof(float) : 0);
}

// CTAs of a decode step: as many as fit at once, fewer where even the longest sequences
// would not fill the smallest shares (8 slabs of 16 rows).
int decode_grid(int64_t units, int64_t rows, int fmt) {
  const int64_t slabs = units * ((rows + 15) / 16 + 1);
  int64_t grid = num_sms() * attn_decode_ctas(fmt);
  if (grid > kDecodeShares) grid = kDecodeShares;
  if (grid > (slabs + 7) / 8) grid = (slabs + 7) / 8;
  return (int)grid;
}

// Both decode entry points after their cache's checks.
int decode_run(const void* q, const CacheView& c, int fmt, const int32_t* lens, int B, int Hq,
               int Hkv, int64_t n_init, int64_t n_recent, float scale, float* out,
               float* lse_out, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_window(n_init, n_recent, scale);
  if (rc) return rc;
  if (B == 0) return report_ok();
  if (!q || !out || !lens) return fail(TSA_ERR_INVALID_ARG, "q, out and lens must be non-NULL");
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(TSA_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if ((rc = check_workspace(workspace, ws_bytes, tsa_attn_decode_workspace_size(B, Hq, Hkv, kD))))
    return rc;
  // The kernels count rows in 32 bits (more keys than that exceed the memory).
  const int64_t pool = c.page_table ? (fmt == kFmtBf16 ? 0 : (int64_t)c.n_pages << c.page_shift)
                                    : (int64_t)B * c.l_cap;
  if (pool > (int64_t)0xffffffff / Hkv)
    return fail(TSA_ERR_INVALID_ARG, "the cache has 2^32 rows or more");
  DecodeArgs a{};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.q = static_cast<const uint16_t*>(q);
  a.c = c;
  a.lens = lens;
  a.B = B;
  a.Hq = Hq;
  a.n_init = n_init;
  a.n_recent = n_recent;
  a.scale_log2 = (float)((double)scale * kLog2e);
  a.out = out;
  a.lse = lse_out;
  a.status = reinterpret_cast<int*>(ws);
  a.partial = reinterpret_cast<float*>(ws + kDecodePartial);
  a.arrived = reinterpret_cast<uint32_t*>(ws + kDecodeArrived);
  const int64_t cap = c.l_cap;
  const int64_t seen = (n_init < cap ? n_init : cap) + (n_recent < cap ? n_recent : cap) + 32;
  const int grid = decode_grid((int64_t)B * Hkv, seen < cap ? seen : cap, fmt);
  return launched(launch_attn_decode(a, fmt, grid, static_cast<cudaStream_t>(stream)),
                  "attention launch");
}

// Workspace of a step with shared rows.  Nothing but the status word outlasts a call, so
// that calls of whatever sizes may share it.
struct SharedLayout {
  size_t partial, arrived, rows, total_at, groups, segments, spans, own, parts, total;
};
SharedLayout shared_layout(int B, int N, int Hq, int Hkv) {
  SharedLayout l{};
  const size_t row = round_up((size_t)B * Hq * (kD + 1) * sizeof(float));
  // at most: every share's first segment, and the units' (two halves; units of up to 64
  // queries, one of a group and head, have up to four copies of each row)
  const int64_t groups = N < B ? N : B, all = (int64_t)B * Hq, few = groups * Hkv * 64;
  const int64_t units = 2 * all + 6 * (all < few ? all : few) + 2 * groups * Hkv;
  l.partial = kDecodePartial;
  l.arrived = kDecodeArrived;
  l.rows = l.arrived + round_up((size_t)B * Hkv * sizeof(uint32_t));
  l.total_at = l.rows + 3 * round_up((size_t)B * sizeof(int32_t));
  l.groups = l.total_at + round_up(sizeof(SharedTotal));
  l.segments = l.groups + round_up((size_t)N * sizeof(SharedGroup));
  // (a unit has 256 queries, or is its group and head's last)
  const size_t list = kSharedShares + (size_t)B * Hq / kUnitRows + (size_t)Hkv * (N < B ? N : B);
  l.spans = l.segments + round_up(list * sizeof(SharedSegment));
  l.own = l.spans + round_up(list * sizeof(int2));
  l.parts = l.own + row;
  l.total = l.parts +
            round_up((size_t)(kSharedShares * kShareRows + units) * (kD + 2) * sizeof(float));
  return l;
}

// Bytes of keys and values up to which reading the shared rows for every sequence costs less
// than the three kernels that read them once.
constexpr int64_t kSmallCache = (int64_t)64 << 20;

// Both entry points of a step with shared rows after their cache's checks.
int shared_run(const void* q, const CacheView& c, int fmt, const int32_t* lens, int B,
               const int32_t* cu, const int32_t* shared, int N, int Hq, int Hkv, float scale,
               void* out, int out16, float* lse_out, void* workspace, size_t ws_bytes,
               void* stream) {
  int rc = check_window(0, 0, scale);
  if (rc) return rc;
  if (N < 0 || N > 4096) return fail(TSA_ERR_INVALID_ARG, "N = %d: must be in [0, 4096]", N);
  if (B == 0) return report_ok();
  if (!q || !out || !lens) return fail(TSA_ERR_INVALID_ARG, "q, out and lens must be non-NULL");
  if (!cu || (N > 0 && !shared))
    return fail(TSA_ERR_INVALID_ARG, "cu_group and shared must be non-NULL");
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(TSA_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  const SharedLayout l = shared_layout(B, N, Hq, Hkv);
  if ((rc = check_workspace(workspace, ws_bytes, l.total))) return rc;
  const int64_t pool = c.page_table ? (fmt == kFmtBf16 ? 0 : (int64_t)c.n_pages << c.page_shift)
                                    : (int64_t)B * c.l_cap;
  if (pool > (int64_t)0x7fffffff / Hkv)
    return fail(TSA_ERR_INVALID_ARG, "the cache has 2^31 rows or more");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedArgs s{};
  s.q = static_cast<const uint16_t*>(q);
  s.c = c;
  s.lens = lens;
  s.cu = cu;
  s.shared = shared;
  s.B = B;
  s.N = N;
  s.Hq = Hq;
  s.G = Hq / Hkv;
  s.inv_g = (65536 + s.G - 1) / s.G;
  s.scale_log2 = (float)((double)scale * kLog2e);
  s.box = c.page_table && (1 << c.page_shift) < 128 ? 1 << c.page_shift : 128;
  s.out = out;
  s.out16 = out16;
  s.lse = lse_out;
  s.status = reinterpret_cast<int*>(ws);
  const size_t ints = round_up((size_t)B * sizeof(int32_t)), rows = (size_t)B * Hq;
  s.group = reinterpret_cast<int32_t*>(ws + l.rows);
  s.start = reinterpret_cast<int32_t*>(ws + l.rows + ints);
  s.total = reinterpret_cast<SharedTotal*>(ws + l.total_at);
  s.groups = reinterpret_cast<SharedGroup*>(ws + l.groups);
  s.segments = reinterpret_cast<SharedSegment*>(ws + l.segments);
  s.spans = reinterpret_cast<int2*>(ws + l.spans);
  s.own_out = reinterpret_cast<float*>(ws + l.own);
  s.own_lse = s.own_out + rows * kD;
  s.parts = reinterpret_cast<float*>(ws + l.parts);
  s.arrived = reinterpret_cast<uint32_t*>(ws + l.arrived);
  DecodeArgs a{};
  a.q = s.q;
  a.c = c;
  a.B = B;
  a.Hq = Hq;
  a.scale_log2 = s.scale_log2;
  a.status = s.status;
  a.partial = reinterpret_cast<float*>(ws + l.partial);
  a.arrived = s.arrived;
  const int grid = decode_grid((int64_t)B * Hkv, c.l_cap + 16, fmt);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool codes = fmt != kFmtBf16;
  a.lens = lens;
  a.start = s.start;
  // A small cache: every sequence reads the shared rows for itself, mostly from L2.
  if ((int64_t)B * Hkv * c.l_cap * 2 * (codes ? kD : kRowBytes) <= kSmallCache) {
    s.leader = reinterpret_cast<int32_t*>(ws + l.rows + 2 * ints);
    a.leader = s.leader;
    a.group = s.group;
    a.out = static_cast<float*>(out);
    a.out16 = out16;
    a.lse = lse_out;
    if ((rc = launched(launch_shared_prep(s, st), "groups launch"))) return rc;
    return launched(launch_attn_decode(a, fmt, grid, st), "attention launch");
  }
  CUtensorMap kmap, vmap;
  if (N > 0) {
    const int64_t all = c.page_table ? (codes ? pool * Hkv : 0x7fffffff) : (int64_t)B * Hkv * c.l_cap;
    if ((rc = row_map(c.k, all, s.box, &kmap, codes)) ||
        (rc = row_map(c.v, all, s.box, &vmap, codes)))
      return rc;
  }
  if ((rc = launched(launch_shared_prep(s, st), "groups launch"))) return rc;
  if (N > 0 &&
      (rc = launched(launch_shared_prefix(kmap, vmap, s, fmt, st), "attention launch")))
    return rc;
  a.out = s.own_out;
  a.lse = s.own_lse;
  if ((rc = launched(launch_attn_decode(a, fmt, grid, st), "attention launch"))) return rc;
  return launched(launch_shared_join(s, st), "join launch");
}

// The rates w_i of a rotation of `rot` elements.
void rope_rates(const tsa_rope_spec* s, double low, double high, int rot, double* w_out) {
  const bool parts = s->scaling == TSA_ROPE_BY_PARTS, yarn = s->scaling == TSA_ROPE_YARN;
  const int n = rot / 2;
  double theta = s->theta;
  if (s->scaling == TSA_ROPE_NTK) theta *= std::pow(s->factor, rot / (rot - 2.0));
  double lo = 0, hi = 0;
  if (yarn) {
    const double per = rot / (2 * std::log(theta));
    lo = std::floor(per * std::log(s->orig_len / (2 * kPi * high)));
    hi = std::ceil(per * std::log(s->orig_len / (2 * kPi * low)));
    lo = lo < 0 ? 0 : lo;
    hi = hi > rot - 1 ? rot - 1 : hi;
  }
  for (int i = 0; i < n; ++i) {
    double w = std::pow(theta, -2.0 * i / rot);
    if (s->scaling == TSA_ROPE_LINEAR) w /= s->factor;
    if (parts) {
      double t = (s->orig_len * w / (2 * kPi) - low) / (high - low);
      t = t < 0 ? 0 : (t > 1 ? 1 : t);
      w = (1 - t) * w / s->factor + t * w;
    }
    if (yarn) {
      const double span = hi - lo > 0.001 ? hi - lo : 0.001;
      double r = (i - lo) / span;
      r = r < 0 ? 0 : (r > 1 ? 1 : r);
      w = r * w / s->factor + (1 - r) * w;
    }
    w_out[i] = w;
  }
}

// tsa_rope_table and tsa_rope_table_axes (own: the axes' rates, and every pair's axis).
int rope_table(const tsa_rope_spec* s, const tsa_rope_axes* own, const int* axis, void* table,
               size_t bytes, tsa_rope* rope, void* stream) {
  if (!s || !rope) return fail(TSA_ERR_INVALID_ARG, "spec or rope is NULL");
  if (!rope_sizes(s->rot_dim, s->max_pos))
    return fail(TSA_ERR_INVALID_ARG,
                "rot_dim %d must be a multiple of 16 up to 128, max_pos %lld in [1, 2^26]",
                s->rot_dim, (long long)s->max_pos);
  if (s->layout != TSA_ROPE_HALF && s->layout != TSA_ROPE_INTERLEAVED)
    return fail(TSA_ERR_INVALID_ARG, "unknown layout %d", s->layout);
  if (s->scaling < TSA_ROPE_PLAIN || s->scaling > TSA_ROPE_YARN)
    return fail(TSA_ERR_INVALID_ARG, "unknown scaling %d", s->scaling);
  if (!(s->theta > 1.0) || !std::isfinite(s->theta))
    return fail(TSA_ERR_INVALID_ARG, "theta must be finite and > 1");
  if (!std::isfinite(s->amplitude) || s->amplitude < 0)
    return fail(TSA_ERR_INVALID_ARG, "amplitude must be finite and >= 0");
  const bool scaled = s->scaling != TSA_ROPE_PLAIN;
  const bool parts = s->scaling == TSA_ROPE_BY_PARTS, yarn = s->scaling == TSA_ROPE_YARN;
  if (scaled && (!(s->factor >= 1.0) || !std::isfinite(s->factor)))
    return fail(TSA_ERR_INVALID_ARG, "factor must be finite and >= 1");
  double low = s->low, high = s->high;
  if (parts || yarn) {
    if (s->orig_len <= 0) return fail(TSA_ERR_INVALID_ARG, "orig_len must be > 0");
    if (low == 0 && high == 0) {
      low = 1;
      high = parts ? 4 : 32;
    }
    if (!(low > 0) || !(high > low) || !std::isfinite(high))
      return fail(TSA_ERR_INVALID_ARG, "low and high must be finite with 0 < low < high");
  }
  if (!table || !aligned(table, 16))
    return fail(TSA_ERR_INVALID_ARG, "table NULL or not 16-byte aligned");
  if (bytes < tsa_rope_table_size(s->rot_dim, s->max_pos))
    return fail(TSA_ERR_INVALID_ARG, "table too small (%zu < %zu)", bytes,
                tsa_rope_table_size(s->rot_dim, s->max_pos));
  if (own && s->scaling == TSA_ROPE_NTK)
    for (int x = 0; x < own->n; ++x)
      if (own->pairs[x] < 2)
        return fail(TSA_ERR_INVALID_ARG, "axes: this scaling needs 2 pairs of every axis");
  const int rot = s->rot_dim, n = rot / 2;
  RopeTableArgs a{};
  if (own) {
    double w[4][kD / 2];
    int seen[4] = {};
    for (int x = 0; x < own->n; ++x) rope_rates(s, low, high, 2 * own->pairs[x], w[x]);
    for (int i = 0; i < n; ++i) a.w[i] = w[axis[i]][seen[axis[i]]++];
  } else {
    rope_rates(s, low, high, rot, a.w);
  }
  a.amplitude = s->amplitude > 0 ? s->amplitude : (yarn ? 0.1 * std::log(s->factor) + 1.0 : 1.0);
  a.pairs = n;
  a.n_hi = (int)rope_high(s->max_pos);
  a.lo = static_cast<float2*>(table);
  a.hi = a.lo + (size_t)kRopeLow * n;
  rope->table = table;
  rope->max_pos = s->max_pos;
  rope->rot_dim = rot;
  rope->layout = s->layout;
  return launched(launch_rope_table(a, static_cast<cudaStream_t>(stream)), "table launch");
}

// rope_apply, with axes (many) or without.
int rope_run(const tsa_rows* q, const tsa_rows* q_out, int Hq, const tsa_rows* k,
             const tsa_rows* k_out, int Hkv, int64_t T, int d, const int32_t* positions,
             int64_t stride, const tsa_rope* rope, const tsa_rope_axes* axes, bool many,
             int inverse, void* stream) {
  if (d != kD) return fail(TSA_ERR_INVALID_ARG, "d = %d: only d = 128 is compiled", d);
  if (Hq <= 0 || Hq > 8192 || Hkv < 0 || Hkv > 8192)
    return fail(TSA_ERR_INVALID_ARG, "Hq must be in [1, 8192], Hkv in [0, 8192]");
  if (T < 0 || T >= (int64_t)1 << 31) return fail(TSA_ERR_INVALID_ARG, "T out of range");
  RopeArgs a{};
  if (!rope) return fail(TSA_ERR_INVALID_ARG, "rope is NULL");
  int rc = check_rope(rope, a.rope);
  if (rc) return rc;
  if (many && (rc = check_axes(axes, rope, stride, a.axes))) return rc;
  if (T == 0) return report_ok();
  if ((rc = check_rows(q, T, Hq, false, "q", a.q))) return rc;
  if ((rc = check_rows(q_out, T, Hq, true, "q_out", a.qo))) return rc;
  if (a.q.p == a.qo.p && (a.q.st != a.qo.st || a.q.sh != a.qo.sh))
    return fail(TSA_ERR_INVALID_ARG, "q_out over q needs q's strides");
  if (Hkv > 0) {
    if ((rc = check_rows(k, T, Hkv, false, "k", a.k))) return rc;
    if ((rc = check_rows(k_out, T, Hkv, true, "k_out", a.ko))) return rc;
    if (a.k.p == a.ko.p && (a.k.st != a.ko.st || a.k.sh != a.ko.sh))
      return fail(TSA_ERR_INVALID_ARG, "k_out over k needs k's strides");
  }
  if (!positions) return fail(TSA_ERR_INVALID_ARG, "positions is NULL");
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.T = T;
  a.positions = positions;
  a.inverse = inverse != 0;
  return launched(launch_rope(a, static_cast<cudaStream_t>(stream)), "rotation launch");
}

// kv8_append, with axes (many) or without.
int append_run(const tsa_kv8* cache, const tsa_rows* k_new, const tsa_rows* v_new,
               const int32_t* cu_new, int64_t T, int max_new, const int32_t* lens, int B, int Hkv,
               int d, const tsa_rope* rope, const tsa_rope_axes* axes, bool many,
               const int32_t* positions, int64_t stride, void* stream) {
  AppendArgs a{};
  int rc = check_batch(B, Hkv, d);
  if (rc) return rc;
  if ((rc = check_kv8(cache, Hkv, a.c))) return rc;
  if ((rc = check_tokens(T, max_new, cu_new, B, "max_new"))) return rc;
  if ((rc = check_rope(rope, a.rope))) return rc;
  if (many) {
    if (!rope) return fail(TSA_ERR_INVALID_ARG, "axes without rope");
    if ((rc = check_axes(axes, rope, stride, a.axes))) return rc;
  }
  if (B == 0 || T == 0 || max_new == 0) return report_ok();
  if ((rc = check_rows(k_new, T, Hkv, false, "k_new", a.k))) return rc;
  if ((rc = check_rows(v_new, T, Hkv, false, "v_new", a.v))) return rc;
  if (!lens) return fail(TSA_ERR_INVALID_ARG, "lens is NULL");
  if (many && !positions) return fail(TSA_ERR_INVALID_ARG, "axes without positions");
  if ((T / cache->block + 2) * 2 * Hkv >= (int64_t)1 << 31)
    return fail(TSA_ERR_INVALID_ARG, "T * Hkv is too large");
  a.fmt = cache->format == TSA_KV8_INT8 ? kFmtInt8 : kFmtE4m3;
  a.block = cache->block;
  a.cu = cu_new;
  a.T = T;
  a.max_new = max_new;
  a.lens = lens;
  a.B = B;
  a.positions = positions;
  a.status = cache->status;
  return launched(launch_kv8_append(a, static_cast<cudaStream_t>(stream)), "append launch");
}

}  // namespace

extern "C" {

size_t tsa_rope_table_size(int rot_dim, int64_t max_pos) {
  if (!rope_sizes(rot_dim, max_pos)) return 0;
  return (size_t)(kRopeLow + rope_high(max_pos)) * (rot_dim / 2) * sizeof(float2);
}

int tsa_rope_table(const tsa_rope_spec* s, void* table, size_t bytes, tsa_rope* rope,
                   void* stream) {
  return rope_table(s, nullptr, nullptr, table, bytes, rope, stream);
}

int tsa_rope_table_axes(const tsa_rope_spec* s, const tsa_rope_axes* axes, void* table,
                        size_t bytes, tsa_rope* rope, void* stream) {
  if (!s) return fail(TSA_ERR_INVALID_ARG, "spec is NULL");
  int axis[kD / 2] = {};
  if (rope_sizes(s->rot_dim, s->max_pos)) {  // (else refused below)
    const int rc = axes_of(axes, s->rot_dim, axis);
    if (rc) return rc;
  }
  const bool own = axes && axes->rates == TSA_RATES_OWN;
  return rope_table(s, own ? axes : nullptr, axis, table, bytes, rope, stream);
}

int rope_apply(const tsa_rows* q, const tsa_rows* q_out, int Hq, const tsa_rows* k,
               const tsa_rows* k_out, int Hkv, int64_t T, int d, const int32_t* positions,
               const tsa_rope* rope, int inverse, void* stream) {
  return rope_run(q, q_out, Hq, k, k_out, Hkv, T, d, positions, 0, rope, nullptr, false, inverse,
                  stream);
}

int rope_apply_axes(const tsa_rows* q, const tsa_rows* q_out, int Hq, const tsa_rows* k,
                    const tsa_rows* k_out, int Hkv, int64_t T, int d, const int32_t* positions,
                    int64_t stride, const tsa_rope* rope, const tsa_rope_axes* axes, int inverse,
                    void* stream) {
  return rope_run(q, q_out, Hq, k, k_out, Hkv, T, d, positions, stride, rope, axes, true, inverse,
                  stream);
}

int kv8_append(const tsa_kv8* cache, const tsa_rows* k_new, const tsa_rows* v_new,
               const int32_t* cu_new, int64_t T, int max_new, const int32_t* lens, int B, int Hkv,
               int d, const tsa_rope* rope, const int32_t* positions, void* stream) {
  return append_run(cache, k_new, v_new, cu_new, T, max_new, lens, B, Hkv, d, rope, nullptr, false,
                    positions, 0, stream);
}

int kv8_append_axes(const tsa_kv8* cache, const tsa_rows* k_new, const tsa_rows* v_new,
                    const int32_t* cu_new, int64_t T, int max_new, const int32_t* lens, int B,
                    int Hkv, int d, const tsa_rope* rope, const tsa_rope_axes* axes,
                    const int32_t* positions, int64_t stride, void* stream) {
  return append_run(cache, k_new, v_new, cu_new, T, max_new, lens, B, Hkv, d, rope, axes, true,
                    positions, stride, stream);
}

int kv8_read(const tsa_kv8* cache, const tsa_rows* k_out, const tsa_rows* v_out,
             const int32_t* cu, int64_t T, int max_new, const int32_t* lens, int B, int Hkv, int d,
             void* stream) {
  ReadArgs a{};
  int rc = check_batch(B, Hkv, d);
  if (rc) return rc;
  if ((rc = check_kv8(cache, Hkv, a.c))) return rc;
  if ((rc = check_tokens(T, max_new, cu, B, "max_new"))) return rc;
  if (B == 0 || T == 0 || max_new == 0) return report_ok();
  if ((rc = check_rows(k_out, T, Hkv, true, "k_out", a.k))) return rc;
  if ((rc = check_rows(v_out, T, Hkv, true, "v_out", a.v))) return rc;
  if (!lens) return fail(TSA_ERR_INVALID_ARG, "lens is NULL");
  a.fmt = cache->format == TSA_KV8_INT8 ? kFmtInt8 : kFmtE4m3;
  a.cu = cu;
  a.T = T;
  a.max_new = max_new;
  a.lens = lens;
  a.B = B;
  a.status = cache->status;
  return launched(launch_kv8_read(a, static_cast<cudaStream_t>(stream)), "read launch");
}

size_t tsa_attn_decode_workspace_size(int B, int Hq, int Hkv, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || d != kD) return 0;
  return kDecodeArrived + ((size_t)B * Hkv * sizeof(uint32_t) + kAlign - 1) / kAlign * kAlign;
}

int kv8_attn_decode(const void* q, const tsa_kv8* cache, const int32_t* lens, int B, int Hq,
                    int Hkv, int d, int64_t n_init, int64_t n_recent, float scale, float* out,
                    float* lse_out, void* workspace, size_t ws_bytes, void* stream) {
  CacheView c;
  int rc = check_batch(B, Hkv, d);
  if (rc) return rc;
  if ((rc = check_groups(B, Hq, Hkv))) return rc;
  if ((rc = check_kv8(cache, Hkv, c))) return rc;
  return decode_run(q, c, cache->format == TSA_KV8_INT8 ? kFmtInt8 : kFmtE4m3, lens, B, Hq, Hkv,
                    n_init, n_recent, scale, out, lse_out, workspace, ws_bytes, stream);
}

int window_attn_decode(const void* q, const tsa_kv* kv, const int32_t* lens, int B, int Hq,
                       int Hkv, int d, int64_t n_init, int64_t n_recent, float scale, float* out,
                       float* lse_out, void* workspace, size_t ws_bytes, void* stream) {
  CacheView c;
  int rc = check_batch(B, Hkv, d);
  if (rc) return rc;
  if ((rc = check_groups(B, Hq, Hkv))) return rc;
  if ((rc = check_cache(kv, Hkv, c))) return rc;
  return decode_run(q, c, kFmtBf16, lens, B, Hq, Hkv, n_init, n_recent, scale, out, lse_out,
                    workspace, ws_bytes, stream);
}

size_t tsa_shared_attn_workspace_size(int B, int N, int Hq, int Hkv, int d) {
  if (B <= 0 || N < 0 || Hq <= 0 || Hkv <= 0 || d != kD) return 0;
  return shared_layout(B, N, Hq, Hkv).total;
}

int shared_attn_decode(const void* q, const tsa_kv* kv, const int32_t* lens, int B,
                       const int32_t* cu_group, const int32_t* shared, int N, int Hq, int Hkv,
                       int d, float scale, void* out, int out_bf16, float* lse_out,
                       void* workspace, size_t ws_bytes, void* stream) {
  CacheView c;
  int rc = check_batch(B, Hkv, d);
  if (rc) return rc;
  if ((rc = check_groups(B, Hq, Hkv))) return rc;
  if ((rc = check_cache(kv, Hkv, c))) return rc;
  return shared_run(q, c, kFmtBf16, lens, B, cu_group, shared, N, Hq, Hkv, scale, out,
                    out_bf16 != 0, lse_out, workspace, ws_bytes, stream);
}

int kv8_shared_attn_decode(const void* q, const tsa_kv8* cache, const int32_t* lens, int B,
                           const int32_t* cu_group, const int32_t* shared, int N, int Hq,
                           int Hkv, int d, float scale, void* out, int out_bf16, float* lse_out,
                           void* workspace, size_t ws_bytes, void* stream) {
  CacheView c;
  int rc = check_batch(B, Hkv, d);
  if (rc) return rc;
  if ((rc = check_groups(B, Hq, Hkv))) return rc;
  if ((rc = check_kv8(cache, Hkv, c))) return rc;
  return shared_run(q, c, cache->format == TSA_KV8_INT8 ? kFmtInt8 : kFmtE4m3, lens, B, cu_group,
                    shared, N, Hq, Hkv, scale, out, out_bf16 != 0, lse_out, workspace, ws_bytes,
                    stream);
}

size_t window_attn_prefill_workspace_size(int B, int Hq, int Hkv, int d, int max_q, int64_t l_cap,
                                          int64_t n_init, int64_t n_recent) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || d != kD || max_q < 0 || l_cap <= 0 || n_init < 0 ||
      n_recent < 0 || Hq % Hkv || Hq / Hkv > kMaxGroup)
    return 0;
  return prefill_bytes(prefill_cut(B, Hkv, Hq / Hkv, max_q, l_cap, n_init, n_recent));
}

int window_attn_prefill(const tsa_rows* q, const tsa_kv* kv, const int32_t* cu_q, int64_t T,
                        int max_q, const int32_t* lens, int B, int Hq, int Hkv, int d,
                        int64_t n_init, int64_t n_recent, float scale, void* out, float* lse_out,
                        void* workspace, size_t ws_bytes, void* stream) {
  PrefillArgs a{};
  int rc = check_batch(B, Hkv, d);
  if (rc) return rc;
  if ((rc = check_groups(1, Hq, Hkv))) return rc;
  if ((int64_t)B * Hkv > 65535) return fail(TSA_ERR_INVALID_ARG, "B*Hkv > 65535");
  if ((rc = check_cache(kv, Hkv, a.c))) return rc;
  if ((rc = check_tokens(T, max_q, cu_q, B, "max_q"))) return rc;
  if ((rc = check_window(n_init, n_recent, scale))) return rc;
  if (B == 0 || T == 0 || max_q == 0) return report_ok();
  if ((rc = check_rows(q, T, Hq, false, "q", a.q))) return rc;
  if (!out || !lens) return fail(TSA_ERR_INVALID_ARG, "out and lens must be non-NULL");
  if (!aligned(out, 16)) return fail(TSA_ERR_INVALID_ARG, "out must be 16-byte aligned");
  const PrefillCut cut = prefill_cut(B, Hkv, Hq / Hkv, max_q, kv->l_cap, n_init, n_recent);
  if ((rc = check_workspace(workspace, ws_bytes, prefill_bytes(cut)))) return rc;
  CUtensorMap kmap, vmap;
  const int box = kv->page_table && kv->page_size < 128 ? kv->page_size : 128;
  const int64_t rows = kv->page_table ? 0x7fffffff : (int64_t)B * Hkv * kv->l_cap;
  if (rows > 0x7fffffff) return fail(TSA_ERR_INVALID_ARG, "the cache has 2^31 rows or more");
  if ((rc = row_map(kv->k, rows, box, &kmap)) || (rc = row_map(kv->v, rows, box, &vmap))) return rc;
  a.cu = cu_q;
  a.T = T;
  a.max_q = max_q;
  a.lens = lens;
  a.Hq = Hq;
  a.G = Hq / Hkv;
  a.inv_g = (65536 + a.G - 1) / a.G;
  a.n_init = (int)(n_init < kv->l_cap ? n_init : kv->l_cap);
  a.n_recent = (int)(n_recent < kv->l_cap ? n_recent : kv->l_cap);
  a.negate = scale < 0;
  a.zero = scale == 0;
  a.scale_log2 = a.zero ? 1.f : (float)(std::fabs((double)scale) * kLog2e);
  a.box = box;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse_out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<int*>(ws);
  a.partial = reinterpret_cast<float*>(ws + kPrePartial);
  a.sums = cut.folds ? reinterpret_cast<float*>(ws + prefill_sums(cut)) : nullptr;
  a.places = reinterpret_cast<uint32_t*>(ws + kPrePlaces);
  a.splits = (int)cut.splits;
  // no sequence has more than T tokens, whatever max_q says
  const int64_t tokens = 2 * (128 / a.G), most = max_q < T ? max_q : T;
  a.blocks = (int)((most + tokens - 1) / tokens);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = launched(launch_window_prefill(kmap, vmap, a, B, st), "attention launch");
  if (rc || a.splits == 1) return rc;
  return launched(launch_window_join(a, B, st), "join launch");
}

}  // extern "C"
