// shared_prefix.cu -- the shared rows of a decode step's groups: every query of a group over
// the group's rows [0, P), which are read once for up to 256 queries.
//
// Per (group, KV head) the queries are S sequences times G heads, M = S G rows of Q, and
//   S = Q K^T,  W = 2^(S c - m c),  O = W V
// are matrix products of M x 128 by 128 x P and M x P by P x 128, with the running maximum m
// and sum of a softmax.  For M <= 140 or so the rows' bytes bound them, beyond that the
// products do (4 M flop a byte pair of K and V, 280 flop a byte of measured rates).
//
// A unit is 256 queries (two tiles of 128, A and B) of a (group, KV head); its key tiles of
// 128 rows are the work.  All units form one list of costs, which the CTAs, one an SM, take
// in equal contiguous shares, whatever the groups' sizes (they are only known on the
// device).  What a share has of a unit is a segment; each leaves (O, maximum, sum) in the
// workspace, and the joining kernel adds them, and the own rows', in order.
// Where the unit has more than 128 queries, A and B take the same key tiles and one's
// softmax runs under the other's products.  Where it has not, A takes the even and B the
// odd tiles for the same queries, so that a tile's chain of copy, product, softmax, product
// is hidden by the other's all the same.
//
// Up to 64 queries lie two or four times in their tile, and each copy takes a part of every
// tile's columns: the exponentials are then all warps' work, and the copies are joined at
// the segment's end.
//
// Warps.  0 and 3: the matrix instructions of A and of B, 1: the copies, 2: the rows of V
// behind P (zeroed, for whatever they hold 0 * NaN would reach the output), 4-7: softmax of
// A (thread = row = tensor-memory lane), 8-11: of B.  K and V tiles go through a ring of
// five 32 KB slots by TMA (two 64-column boxes with the 128-byte swizzle; a box a page where
// pages are smaller than a tile), which runs on across segments.  A slot is filled again
// when its three readers have given it back: both matrix threads, or one and the zeroing
// warp for the other, and the zeroing warp.  It passes every slot in order and counts the
// tiles; a stream that has passed by tiles of the other waits for that count (kLag).  Weights
// are handed to the second product by quarters of a tile (by halves 22 us more of 409, 256
// queries' worth of samples under 131071 rows).
//
// Registers.  The compiler spills 232 bytes of the form for bf16 caches with fp32 output, 92 of
// that with bf16 output and 76 to 80 of those for 8-bit caches.  Loads and stores of spills are
// 1.8, 0.7 and at most 0.07 % of the instructions that run (counters, the cases below): a
// few a key tile in the first two, a few a segment in the others.
//
// 8-bit caches.  Codes come by TMA into a ring of four 16 KB slots; warps 12-15 widen them to
// fp16 (exact) into three operand slots, zeroing V's rows behind P, and find the blocks'
// scales.  The queries are in fp16 too, each row's exponents shifted.  The keys' scale is a
// factor of the logits, the values' belongs to the weights and is taken out of their sum.
//
// Numbers.  The weights enter the second product in two parts where the output is fp32
// (2^-18 of a weight left out in bf16, 2^-22 in fp16; a third bf16 part has no room in tensor
// memory beside the logits), in one where it is bf16, as in the prompt kernel.  There the
// weights' errors are of the size of the output's own rounding and independent of each
// other: 256 x 7 heads under 131071 rows are 2.4e-3 off 64 bits where rounding alone leaves
// 1.66e-3, and take 396 us; with two parts 1.66e-3 and 558.  e4m3 (one fp16 part has 11 bits): 1.67e-3
// for 1.66e-3, 683 us for 768.
//
// What bounds it (one call, the kernel alone).  64 sequences x 4 heads under 32767 rows of 8
// KV heads, fp32: 46 us for 20 us of bytes and 27 us of matrix instructions (three products
// of a tile); 12 us pass before the first product.  256 x 7 heads under 131071 rows of 4,
// bf16: 306 us, 1570 TFLOP/s; the path from the logits to the first weights is a little
// longer than the other stream's products.  8 groups of 8 x 4 heads under 115K rows of 8, e4m3: 623 us,
// 2.96 TB/s of codes: a tile's chain of barriers, and shared memory (a tile moves 224 KB through
// it: 32 copied in, 32 read and 64 written by the widening warps, 96 read by the products).
// Waits that read the global timer took 17 % more there, loops unrolled past the instruction
// cache 27 %.
#include <cuda_fp16.h>

#include <type_traits>

#include "shared_attn.h"
#include "tcgen.cuh"

namespace tsa {

namespace {

// Slots of the ring of operands, and, for 8-bit caches, of the ring of codes before it.
template <int FMT>
constexpr int kSlots = FMT == kFmtBf16 ? 5 : 3;
constexpr int kRawSlots = 4, kRawBytes = kTile * kD;
template <int FMT>
constexpr int kSharedThreads = FMT == kFmtBf16 ? 384 : 512;
// Registers a scheduler (bf16): 2 * 216 + 72 = 3 * 168.
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
template <int FMT>
constexpr int kSharedSmem = (2 + kSlots<FMT>) * kSlotBytes +
                            (FMT == kFmtBf16 ? 0 : kRawSlots * kRawBytes) + 1024;
constexpr float kLeastScale = 1.f / (1ll << 60);  // the smallest that the cache's writer gives
constexpr float kLeastFactor = 1e-37f;  // of a logit: keys of scale 0 (never written) are masked too
// fp16 weights: 2^7 for the one that raised the maximum, up to 2^15 under it later.
constexpr float kRaised = 7.f, kSlack = 15.f;
// Weights may grow to 2^16 under an old maximum before O is rescaled: bf16 and fp32 keep
// their precision at any size.
constexpr float kRescale = 16.f, kMost = 65536.f;
// Matrix instructions truncate their 32-bit sums, all in one direction (6.3e-9 of a sum of
// one sign for every row and part of a weight): after so many of a stream's tiles O is added,
// with rounding, to the sum in the workspace and begins again.  (fp32, 48 sequences in 6 groups
// of 2K to 131K rows: 16 tiles 246 us and 2.4e-6 off 64 bits, 24 tiles 230 and 2.9e-6, 32 tiles
// 229 and 3.7e-6; 32-bit products and sums are 2.1e-6 off.)
template <int PARTS>
constexpr int kFoldEvery = PARTS == 2 ? 24 : 128;

template <int FMT>
struct SharedBars {
  uint64_t q[2], s[2], p[2][4], o[2], full[kSlots<FMT>], empty[kSlots<FMT>], drain[2], turn[2],
      raw_full[kRawSlots], raw_empty[kRawSlots], scale[kRawSlots];
};

// A barrier tells its last two phases apart and no more, so a wait for a slot is right only once
// the slot's item of the lap before is known to have landed.  A stream that passes by the other's
// tiles (a unit of one key tile is stream A's alone) may be any number of laps ahead of the ring.
// It therefore waits for the slots of a tile only when the zeroing warp, which passes all
// tiles in order, has counted all but kLag of those before it.  With five slots a tile's two
// items lie in those of the two tiles before the last one.  With three its V takes the slot of
// the last tile's K, which has landed when its own K has, since operands of codes land in
// order.
constexpr uint32_t kLag = 1;

// Slot i of the rings' endless rows, and the parity of its barriers there.
template <int FMT>
__device__ __forceinline__ int slot_of(uint32_t i) { return i % kSlots<FMT>; }
template <int FMT>
__device__ __forceinline__ uint32_t lap_of(uint32_t i) { return i / kSlots<FMT> & 1u; }
__device__ __forceinline__ int raw_slot(uint32_t i) { return i % kRawSlots; }
__device__ __forceinline__ uint32_t raw_lap(uint32_t i) { return i / kRawSlots & 1u; }

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two weights in the products' type, and their values.
template <int FMT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return FMT == kFmtBf16 ? bf16x2(lo, hi) : f16x2(lo, hi);
}
template <int FMT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (FMT == kFmtBf16) return make_float2(bf_lo(w), bf_hi(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Four codes as fp16, exactly.
template <int FMT>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == kFmtInt8) {
    lo = codes_lo_f16x2(w);
    hi = codes_hi_f16x2(w);
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
        " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}
// Logarithm of a value scale: exact for powers of two.
__device__ __forceinline__ float lg2_scale(float x) {
  const uint32_t u = __float_as_uint(x);
  return (float)((int)(u >> 23) - 127) + log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
}

template <int FMT, int PARTS>
__global__ void __launch_bounds__(kSharedThreads<FMT>, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, SharedArgs a) {
  constexpr bool Q8 = FMT != kFmtBf16;
  constexpr int SLOTS = kSlots<FMT>;
  constexpr uint32_t kTypes = (1u << 7) | (1u << 10);  // operands in bf16, else fp16
  constexpr uint32_t kQk = Q8 ? kIdesc & ~kTypes : kIdesc, kPv = Q8 ? kIdescV & ~kTypes : kIdescV;
  extern __shared__ uint8_t smem_raw[];
  __shared__ SharedBars<FMT> bar;
  // 8-bit: of a tile's blocks of 16 rows: the keys' scale, the logarithm of the values' scale
  // and its inverse.
  __shared__ float4 scale_s[Q8 ? kRawSlots : 1][8];
  __shared__ float2 run_s[2][64];            // maxima and sums while copies are joined
  __shared__ uint32_t tmem_s;
  __shared__ uint32_t passed_s;              // tiles that the zeroing warp has passed
  __shared__ volatile int abort_s;
  __shared__ volatile int bad_s[8];          // number of a segment that met a bad page
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, ring = base + 2 * kSlotBytes;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q[i], kTile);
      mbar_init(&bar.s[i], 1);
      for (int c = 0; c < 4; ++c) mbar_init(&bar.p[i][c], kTile);
      mbar_init(&bar.o[i], 1);
      mbar_init(&bar.drain[i], 1);
      mbar_init(&bar.turn[i], 1);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&bar.full[i], Q8 ? 4 : 1);
      mbar_init(&bar.empty[i], 3);
    }
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], 4);
      mbar_init(&bar.scale[i], 1);
    }
    fence_mbar_init();
    passed_s = 0u;
    abort_s = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
  }
  if (tid < 8) bad_s[tid] = 0;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&tmem_s))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tmem_s;
  // The whole warp agrees, where what follows is a warp's work.
  auto wait = [&](uint64_t* x, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_long(x, parity, &abort_s)) != 0;
  };
  const int2 list = a.total->segments[blockIdx.x];
  const int n_seg = list.y;
  const SharedSegment* segments = a.segments + list.x;

  if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ softmax
    if (!Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = (warp >> 2) - 1;           // stream A or B
    const int r = tid & 127;                 // row of the stream's tile
    const int r_warp = (warp & 3) * 32, r_half = lane >> 4, piece = lane & 15;
    const uint32_t q_mine = q_at + x * kSlotBytes;
    const uint32_t s_at = tmem + x * kTile + ((uint32_t)(warp & 3) << 21);
    const uint32_t o_at = s_at + 2 * kTile;
    const float sc = a.scale_log2 < 0.f ? -a.scale_log2 : (a.scale_log2 == 0.f ? 1.f : a.scale_log2);
    uint32_t tiles = 0, segs = 0;            // of this stream, so far
    uint32_t seg_tile = 0;                   // tiles of the segments before this one
    bool ok = true;
    for (int number = 0; number < n_seg; ++number) {
      const SharedSegment& u = segments[number];
      const bool both = u.both;
      // The unit's row in this thread's row of the tile.  Few queries are there in copies,
      // each of which takes its part of every tile's columns.
      const int copies = u.copies, lg = copies >> 1, span = kTile >> lg, copy = r >> (7 - lg);
      const int first = both ? x * kTile : 0, unit_rows = u.rows;
      const int row = first + (r & (span - 1));
      const bool live = row < unit_rows;
      const bool warp_live = first + (r_warp & (span - 1)) < unit_rows;
      // bit c: columns 32 c ... are this copy's
      const uint32_t mine_c = copies == 1 ? 15u : (copies == 2 ? 3u << 2 * copy : 1u << copy);
      auto mine_is = [&](int c) { return (mine_c >> c & 1u) != 0u; };
      const int all = u.j1 - u.j0, tile0 = u.j0;
      const int n = both ? all : (all - x + 1) / 2;      // tiles of this stream
      const int P = u.P, rs = u.rs;
      float* mine = a.parts + 4 * u.part + x * half_floats(rs);
      // columns 4 i .. of this thread's sum at sums[i * rs]
      float4* sums = reinterpret_cast<float4*>(mine) + (both ? r : copy * unit_rows + row);
      float m = -INFINITY, l = 0.f;
      float row_sc = sc;                     // 8-bit: with the inverse of the queries' shift
      if (n > 0) {
        // Q, swizzled as the copies would: rows of 128 bytes, piece c at c ^ (row & 7).
        // A half-warp a row, so that a row's 256 bytes are one request.
        {
          const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
          const int seq0 = u.seq0, in0 = u.in0, head0 = u.g * a.G;
          uint4 w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int rr = first + ((r_warp + 2 * i + r_half) & (span - 1));
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (rr < unit_rows && a.scale_log2 != 0.f) {
              const int sq = ((in0 + rr) * a.inv_g) >> 16, h = in0 + rr - sq * a.G;
              w[i] = *reinterpret_cast<const uint4*>(
                  a.q + ((int64_t)(seq0 + sq) * a.Hq + head0 + h) * kD + 8 * piece);
            }
          }
          if constexpr (Q8) {
            // fp16, each row's exponents shifted so that its largest element is in
            // [2^14, 2^15)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              uint32_t* x = &w[i].x;
              float amax = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                amax = fmaxf(amax, fmaxf(fabsf(bf_lo(x[e])), fabsf(bf_hi(x[e]))));
#pragma unroll
              for (int o = 1; o < 16; o <<= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
              int e2 = 141 - (int)(__float_as_uint(amax) >> 23);  // 14 - floor(log2 amax)
              e2 = amax == 0.f ? 0 : (e2 > 126 ? 126 : (e2 < -113 ? -113 : e2));
              const float up = __uint_as_float((uint32_t)(e2 + 127) << 23);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = f16x2(bf_lo(x[e]) * up, bf_hi(x[e]) * up);
              // (this thread's own row is number lane: round lane / 2, half lane % 2)
              const int of = __shfl_sync(0xffffffffu, e2, (lane & 1) * 16);
              if (lane >> 1 == i) row_sc = sc * __uint_as_float((uint32_t)(127 - of) << 23);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int rr = r_warp + 2 * i + r_half;
            const uint32_t at = q_mine + (piece >> 3) * kHalf + rr * 128 +
                                (((piece & 7) ^ (rr & 7)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[i].x ^ flip),
                         "r"(w[i].y ^ flip), "r"(w[i].z ^ flip), "r"(w[i].w ^ flip)
                         : "memory");
          }
        }
        fence_proxy_async();
        mbar_arrive(&bar.q[x]);

        bool more = false;                   // a sum is in the workspace, under `under`
        float under = 0.f;
        // O to the sum in the workspace.  While the maximum is the one that the sum is under,
        // it is added there, without a wait for what is there.
        auto put = [&]() {
          const float f = !more || under == m ? 1.f : ex2(Q8 ? under - m : (under - m) * sc);
          const bool scaled = __any_sync(0xffffffffu, f != 1.f && live);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            __syncwarp();
            load_cols(o_at + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 8 && live; ++i) {
              float4* at = sums + (8 * c + i) * rs;
              float4 y = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              if (more && !scaled) {
                asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(at), "f"(y.x),
                             "f"(y.y), "f"(y.z), "f"(y.w)
                             : "memory");
              } else {
                if (more) {
                  const float4 u = __ldcg(at);
                  y = make_float4(fmaf(u.x, f, y.x), fmaf(u.y, f, y.y), fmaf(u.z, f, y.z),
                                  fmaf(u.w, f, y.w));
                }
                __stcg(at, y);
              }
            }
          }
          more = true;
          under = m;
        };
        // (two forms, so that the usual one's code is in one piece)
        auto tiles_of = [&](auto many) {
        constexpr bool MANY = decltype(many)::value;  // copies > 1
        for (int j0 = 0; j0 < n && ok; j0 += kFoldEvery<PARTS>) {
          const int j1 = j0 + kFoldEvery<PARTS> < n ? j0 + kFoldEvery<PARTS> : n;
          for (int j = j0; j < j1; ++j) {
            const int tile = both ? j : 2 * j + x, k0 = (tile0 + tile) * kTile;
            const uint32_t parity = (tiles + j) & 1;
            ok = wait(&bar.s[x], parity);
            if (__builtin_expect(!ok, 0)) break;
            if (Q8) ok = wait(&bar.scale[raw_slot(seg_tile + tile)], raw_lap(seg_tile + tile));
            if (__builtin_expect(!ok, 0)) break;
            if (!warp_live) {  // nobody reads these rows' weights
#pragma unroll
              for (int c = 0; c < 4; ++c) mbar_arrive(&bar.p[x][c]);
              continue;
            }
            fence_after();
            // (S is there, so O's products before it are done)
            if (__builtin_expect(j == j0 && j > 0, 0)) put();
            // 8-bit: y = log2 of a weight with its row's value scale, block by block of 16; the
            // columns are read twice, 32 at a time, for want of registers.
            [[maybe_unused]] const float4* blocks = scale_s[Q8 ? (seg_tile + tile) % kRawSlots : 0];
            float s[Q8 ? 32 : 128];
            auto columns = [&](int c) {  // 32 c ..., masked
              float(&y)[32] = reinterpret_cast<float(&)[32]>(s[Q8 ? 0 : 32 * c]);
              if (Q8) load_cols(s_at + 32 * c, y);
              if (__builtin_expect(MANY || k0 + kTile > P, 0)) {
                const uint32_t on = !MANY || mine_is(c) ? below(P - k0 - 32 * c) : 0u;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(on & (1u << i))) y[i] = -INFINITY;
              }
            };
            if constexpr (!Q8) {
              load_cols(s_at, s);
#pragma unroll
              for (int c = 0; c < 4; ++c) columns(c);
            }
            // Weights of a quarter of a tile (32 keys) under the maximum `top`; their sum.
            auto weights = [&](int c, float top) {
              const float off = top == -INFINITY ? 0.f : (Q8 ? -top : -top * sc);
              float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              float sum = 0.f;
              if (MANY && !mine_is(c)) {  // another copy's
                const uint32_t none[16] = {};
                store_cols(s_at + (PARTS == 2 ? 32 : 16) * c, none);
                if (PARTS == 2) store_cols(s_at + 32 * c + 16, none);
                return 0.f;
              }
              if (Q8) columns(c);
              const float* y = s + (Q8 ? 0 : 32 * c);
              uint32_t w[16], w2[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float f = sc, o = off;
                if constexpr (Q8) {
                  const float4 k = blocks[2 * c + i / 8];
                  f = fmaxf(row_sc * k.x, kLeastFactor);
                  o = off + k.y;
                  if (i % 8 == 0) add[0] = add[1] = make_float2(0.f, 0.f);
                }
                float2 e = fma2(make_float2(y[2 * i], y[2 * i + 1]), make_float2(f, f),
                                make_float2(o, o));
                e.x = ex2(e.x);
                e.y = ex2(e.y);
                add[i & 1] = add2(add[i & 1], e);
                if constexpr (Q8) {
                  if (i % 8 == 7)
                    sum = fmaf((add[0].x + add[0].y) + (add[1].x + add[1].y),
                               blocks[2 * c + i / 8].z, sum);
                }
                w[i] = pack2<FMT>(e.x, e.y);
                if (PARTS == 2) {
                  const float2 d = fma2(unpack2<FMT>(w[i]), make_float2(-1.f, -1.f), e);
                  w2[i] = pack2<FMT>(d.x, d.y);
                }
              }
              store_cols(s_at + (PARTS == 2 ? 32 : 16) * c, w);
              if (PARTS == 2) store_cols(s_at + 32 * c + 16, w2);
              return Q8 ? sum : (add[0].x + add[0].y) + (add[1].x + add[1].y);
            };
            auto publish = [&](int c) {  // their products may begin
              wait_stores();
              fence_before();
              mbar_arrive(&bar.p[x][c]);
            };
            float l0 = 0.f;
            if constexpr (Q8) {
              // fp16's range is short: every logit is looked at before the weights are taken.
              float top = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                if (MANY && !mine_is(c)) continue;
                columns(c);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float t = s[16 * i];
#pragma unroll
                  for (int e = 1; e < 15; e += 2) t = max3(t, s[16 * i + e], s[16 * i + e + 1]);
                  t = fmaxf(t, s[16 * i + 15]);
                  const float4 k = blocks[2 * c + i];
                  const float f = fmaxf(row_sc * k.x, kLeastFactor);
                  top = fmaxf(top, t == -INFINITY ? t : fmaf(t, f, k.y));
                }
              }
              if (__builtin_expect(__any_sync(0xffffffffu, !(top <= m + kSlack)), 0)) {
                const float to = fmaxf(m, top - kRaised);
                const float f = m == to ? 1.f : ex2(m - to);
                m = to;
                l *= f;
                if (j > j0) {
#pragma unroll 1
                  for (int c = 0; c < 4; ++c) {
                    float o[32];
                    load_cols(o_at + 32 * c, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= f;
                    store_cols(o_at + 32 * c, o);
                  }
                }
              }
            } else {
              // The maximum is off the path from S to the weights.  They are taken under the
              // maximum so far as long as they stay below 2^kRescale: the first quarter's sum
              // tells for itself, the others' logits are looked at.  Where they do not
              // (first tiles, rarely later) the maximum is found, O and the sum are rescaled
              // and the weights taken again.
              bool good = m != -INFINITY || !live;
              if (__builtin_expect(__all_sync(0xffffffffu, good), 1)) {
                float tops[4] = {s[32], s[33], s[34], s[35]};
#pragma unroll
                for (int i = 36; i < 124; i += 8)
#pragma unroll
                  for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], s[i + e], s[i + 4 + e]);
                const float t = max3(fmaxf(tops[0], s[124]), fmaxf(tops[1], s[125]),
                                     max3(tops[2], s[126], fmaxf(tops[3], s[127])));
                l0 = weights(0, m);
                good = (l0 <= kMost && (t - m) * sc <= kRescale) || !live;
              }
              if (__builtin_expect(!__all_sync(0xffffffffu, good), 0)) {
                float tops[4] = {m, m, m, m};
#pragma unroll
                for (int i = 0; i < 128; i += 8)
#pragma unroll
                  for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], s[i + e], s[i + 4 + e]);
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                const float f = m == top ? 1.f : ex2((m - top) * sc);
                m = top;
                l *= f;
                if (j > j0) {
#pragma unroll
                  for (int c = 0; c < 4; ++c) {
                    float o[32];
                    load_cols(o_at + 32 * c, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= f;
                    store_cols(o_at + 32 * c, o);
                  }
                }
                l0 = weights(0, m);
              }
            }
            if (!Q8) publish(0);
            l += l0;
            // (8-bit: one piece of code for all quarters, for the instruction cache's sake)
#pragma unroll (Q8 ? 1 : 3)
            for (int c = Q8 ? 0 : 1; c < 4; ++c) {
              l += weights(c, m);
              publish(c);
            }
          }
        }
        };
        if (copies > 1)
          tiles_of(std::true_type{});
        else
          tiles_of(std::false_type{});
        if (ok) ok = wait(&bar.o[x], segs & 1);
        fence_after();
        if (copies == 1) {
          if (ok && warp_live) put();
        } else {
          // The copies by turns, each adding its rows to the sums so far (in the queries'
          // tile, which the products have read); the last one writes them out.  Every warp
          // of the stream passes all barriers, whatever has gone wrong.
          float4* so_far = reinterpret_cast<float4*>(smem_raw + (q_mine - smem_u32(smem_raw))) + row;
          float4* total = reinterpret_cast<float4*>(mine) + row;
          if (!ok) l = nanf("");
#pragma unroll 1
          for (int k = 0; k < copies; ++k) {
            if (k == copy && warp_live) {
              const float2 was = k > 0 && live ? run_s[x][row] : make_float2(-INFINITY, 0.f);
              const float top = fmaxf(m, was.x);
              auto under_top = [&](float y) { return y == top ? 1.f : ex2(Q8 ? y - top : (y - top) * sc); };
              const float f = under_top(m), f_was = under_top(was.x), f_more = under_top(under);
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float o[32] = {};
                __syncwarp();
                if (ok) load_cols(o_at + 32 * c, o);
                if (live) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    float4 y = make_float4(o[4 * i] * f, o[4 * i + 1] * f, o[4 * i + 2] * f,
                                           o[4 * i + 3] * f);
                    if (more) {
                      const float4 u = __ldcg(sums + (8 * c + i) * rs);
                      y = make_float4(fmaf(u.x, f_more, y.x), fmaf(u.y, f_more, y.y),
                                      fmaf(u.z, f_more, y.z), fmaf(u.w, f_more, y.w));
                    }
                    if (k > 0) {
                      const float4 u = so_far[(8 * c + i) * span];
                      y = make_float4(fmaf(u.x, f_was, y.x), fmaf(u.y, f_was, y.y),
                                      fmaf(u.z, f_was, y.z), fmaf(u.w, f_was, y.w));
                    }
                    if (k < copies - 1)
                      so_far[(8 * c + i) * span] = y;
                    else
                      __stcg(total + (8 * c + i) * rs, y);
                  }
                }
              }
              l = l * f + was.y * f_was;
              m = top;
              if (live) run_s[x][row] = make_float2(m, l);
            }
            asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
          }
        }
        fence_before();
        tiles += n;
        ++segs;
      }
      if (!ok || bad_s[number & 7] == number + 1) {
        l = nanf("");
        m = 0.f;
      }
      if (live && copy == copies - 1) {
        float* stats = mine + (size_t)rs * kD;
        const int at = both ? r : row;
        stats[at] = Q8 ? m : m * sc;
        stats[rs + at] = l;
      }
      seg_tile += all;
    }
  } else {
   if (!Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
   if (warp == 0 || warp == 3) {
    // ------------------------------------------------ matrix instructions
    // One thread for each stream.  With both on the same tiles by turns: O_A(j), S_A(j+1),
    // then O_B(j), S_B(j+1).  One thread's execute in order: S(j+1) may overwrite the
    // weights of j without a wait.
    const int x = warp == 3;
    if (elect_one()) {
      const uint32_t s_at = tmem + x * kTile, o_at = s_at + 2 * kTile;
      const uint64_t qd = operand(q_at + x * kSlotBytes, 16);
      const uint64_t kd = operand(ring, 16), vd = operand(ring, kHalf);
      auto qk = [&](int slot) {
        const uint64_t kx = kd + slot * (kSlotBytes >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          mma_ss(s_at, qd + at, kx + at, kQk, k > 0);
        }
        commit_mma(&bar.s[x]);
        commit_mma(&bar.empty[slot]);
      };
      // so far: tiles and segments of this stream, turns, tiles of the segments
      uint32_t tiles = 0, segs = 0, turns = 0, passed = 0;
      uint32_t seen = 0;                     // of the zeroing warp's count
      bool ok = true;
      for (int seg = 0; ok && seg < n_seg; ++seg) {
        const bool both = segments[seg].both;
        const int j0 = segments[seg].j0, P = segments[seg].P;
        const int all = segments[seg].j1 - j0, n = both ? all : (all - x + 1) / 2;
        auto number = [&](int j) { return passed + (both ? j : 2 * j + x); };
        auto in_reach = [&](uint32_t tile) {  // its slots may be waited for
          return tile <= kLag || wait_count(&passed_s, tile - kLag, seen, &abort_s);
        };
        if (n > 0) {
          const uint32_t i = 2 * number(0);
          ok = wait_long(&bar.q[x], segs & 1, &abort_s) && in_reach(number(0)) &&
               wait_long(&bar.full[slot_of<FMT>(i)], lap_of<FMT>(i), &abort_s);
          if (both && x == 1) ok = ok && wait_long(&bar.turn[1], turns & 1, &abort_s);
          if (ok) {
            fence_after();
            qk(slot_of<FMT>(i));
          }
          if (both) mbar_arrive(&bar.turn[x ^ 1]);
        }
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t tile = number(j), i = 2 * tile + 1;  // V's slot
          ok = wait_long(&bar.full[slot_of<FMT>(i)], lap_of<FMT>(i), &abort_s);
          if (!Q8 && ok && (j0 + (int)(tile - passed) + 1) * kTile > P)
            ok = wait_count(&passed_s, tile + 1, seen, &abort_s);
          const uint64_t vx = vd + slot_of<FMT>(i) * (kSlotBytes >> 4);
          const bool more = j % kFoldEvery<PARTS> > 0;
          const uint32_t parity = (tiles + j) & 1;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ok = ok && wait_long(&bar.p[x][c], parity, &abort_s);
            if (c == 0 && both)
              ok = ok && wait_long(&bar.turn[x], (turns + j + x) & 1, &abort_s);
            if (ok) {
              fence_after();
#pragma unroll
              for (int k = 2 * c; k < 2 * c + 2; ++k) {
                const uint64_t vk = vx + ((k * 16 * 128) >> 4);
                if (PARTS == 2) {
                  const uint32_t w = s_at + 32 * c + 8 * (k & 1);
                  mma_ts(o_at, w, vk, kPv, more || k > 0);
                  mma_ts(o_at, w + 16, vk, kPv, true);
                } else {
                  mma_ts(o_at, s_at + 8 * k, vk, kPv, more || k > 0);
                }
              }
            }
          }
          if (!ok) break;
          commit_mma(&bar.empty[slot_of<FMT>(i)]);
          if (j + 1 < n) {
            const uint32_t k = 2 * number(j + 1);
            ok = in_reach(number(j + 1)) &&
                 wait_long(&bar.full[slot_of<FMT>(k)], lap_of<FMT>(k), &abort_s);
            if (!ok) break;
            qk(slot_of<FMT>(k));
          } else {
            commit_mma(&bar.o[x]);
          }
          if (both) mbar_arrive(&bar.turn[x ^ 1]);
        }
        if (both) {  // (A sees B's last arrival, so that neither's count runs ahead)
          if (x == 0) ok = ok && wait_long(&bar.turn[0], (turns + n) & 1, &abort_s);
          turns += n + 1;
        }
        tiles += n;
        segs += n > 0;
        passed += all;
      }
      if (!ok) {  // nothing may still run on tensor memory when it is given back
        commit_mma(&bar.drain[x]);
        mbar_wait(&bar.drain[x], 0);
        atomicOr(a.status, kStatusTimeout);
      }
    }
    __syncwarp();
   } else if (warp == 1) {
    // -------------------------------------------------------------- copies
    const int box = a.box;                   // rows of a box: 128, or a smaller page
    const int per = kTile / box;             // boxes of a tile
    // (bf16: two halves of 64 columns)
    const int i_box = Q8 ? lane : lane >> 1, half = Q8 ? 0 : lane & 1;
    const uint32_t raw = ring + SLOTS * kSlotBytes;
    uint32_t it = 0;
    bool ok = true;
    for (int number = 0; ok && number < n_seg; ++number) {
      const int b = segments[number].b0, g = segments[number].g, P = segments[number].P;
      const int j0 = segments[number].j0, j1 = segments[number].j1;
      const int32_t* pages =
          a.c.page_table ? a.c.page_table + (int64_t)b * a.c.max_pages : nullptr;
      // Lane's box of key tile j: its first row in the pool, or -1 where nothing of it
      // is seen.
      auto find = [&](int j) -> int64_t {
        if (j >= j1 || i_box >= per) return -1;
        const int r0 = j * kTile + i_box * box;
        if (r0 >= P) return -1;
        if (!pages) return ((int64_t)b * a.c.Hkv + g) * a.c.l_cap + r0;
        const int32_t page = pages[r0 >> a.c.page_shift];
        if ((uint32_t)page >= a.c.n_pages) {
          bad_s[number & 7] = number + 1;
          atomicOr(a.status, kStatusBadLength);
          return -1;
        }
        return (((int64_t)page * a.c.Hkv + g) << a.c.page_shift) +
               (r0 & ((1 << a.c.page_shift) - 1));
      };
      int64_t next = find(j0);
      for (int j = j0; j < j1 && ok; ++j) {
        const int64_t row = next;
        next = find(j + 1);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * box * 128;
        for (int w = 0; w < 2 && ok; ++w) {
          const int sl = Q8 ? raw_slot(it) : slot_of<FMT>(it);
          uint64_t* landed = Q8 ? &bar.raw_full[sl] : &bar.full[sl];
          if (it >= (Q8 ? kRawSlots : SLOTS))
            ok = Q8 ? wait(&bar.raw_empty[sl], raw_lap(it) ^ 1)
                    : wait(&bar.empty[sl], lap_of<FMT>(it) ^ 1);
          if (!ok) break;
          if (Q8) fence_proxy_async();  // (behind the widening warps' reads of the slot)
          if (lane == 0) mbar_expect_tx(landed, bytes);
          __syncwarp();
          if (row >= 0)
            copy_box(Q8 ? raw + sl * kRawBytes + i_box * box * kD
                        : ring + sl * kSlotBytes + half * kHalf + i_box * box * 128,
                     w ? &vmap : &kmap, 64 * half, (int)row, landed);
          ++it;
        }
      }
    }
    if (!ok)  // let the copies in flight land
      for (uint32_t n = Q8 ? kRawSlots : SLOTS, i = it > n ? it - n : 0; i < it; ++i) {
        if (Q8)
          mbar_wait(&bar.raw_full[raw_slot(i)], raw_lap(i));
        else
          mbar_wait(&bar.full[slot_of<FMT>(i)], lap_of<FMT>(i));
      }
   } else if (warp == 2) {
    // ---------------------------------------- rows of V behind the shared ones
    uint32_t tile = 0;
    bool ok = true;
    for (int seg = 0; ok && seg < n_seg; ++seg) {
      const bool both = segments[seg].both;
      const int P = segments[seg].P, j1 = segments[seg].j1;
      for (int j = segments[seg].j0; j < j1 && ok; ++j, ++tile) {
        // every slot is given back for this warp, and for the stream that passes it by
        auto give = [&](uint32_t i) {
          mbar_arrive(&bar.empty[slot_of<FMT>(i)]);
          if (!both) mbar_arrive(&bar.empty[slot_of<FMT>(i)]);
        };
        const uint32_t i = 2 * tile;
        if (lane == 0) {
          ok = wait_long(&bar.full[slot_of<FMT>(i)], lap_of<FMT>(i), &abort_s);
          if (ok) give(i);
          ok = ok && wait_long(&bar.full[slot_of<FMT>(i + 1)], lap_of<FMT>(i + 1), &abort_s);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int left = P - j * kTile;
        if (!Q8 && left < kTile) {
          const uint32_t at = ring + slot_of<FMT>(i + 1) * kSlotBytes + (lane >> 4) * kHalf +
                              (lane & 15) * 8;
          for (int r = left; r < kTile; ++r)
            asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(at + r * 128), "r"(0)
                         : "memory");
          fence_proxy_async();
          __syncwarp();
        }
        if (lane == 0) {
          raise_count(&passed_s, tile + 1);
          give(i + 1);
        }
      }
    }
   } else if (Q8 && warp >= 12) {
    // ------------------------------------------- codes to operands, scales
    // 16 codes a lane and turn: 16 bytes of a row become two pieces of its half of the
    // operand.  Eight lanes take half of a row and the other half of the next one, so that
    // together they touch all banks, in the codes as in the operand.
    const uint32_t raw = ring + SLOTS * kSlotBytes;
    const int mine = tid - 384, row0 = mine >> 2;
    const int ch = (mine & 3) | (row0 & 1) << 2;       // of a row's eight, at even turns
    const uint32_t at0 = ((2 * (mine & 3)) ^ (row0 & 7)) << 4;  // the first piece's place
    uint32_t tile = 0;
    bool ok = true;
    for (int seg = 0; ok && seg < n_seg; ++seg) {
      const int b = segments[seg].b0, g = segments[seg].g, P = segments[seg].P;
      const int j0 = segments[seg].j0, j1 = segments[seg].j1;
      const int32_t* pages =
          a.c.page_table ? a.c.page_table + (int64_t)b * a.c.max_pages : nullptr;
      // Lanes 0-7: the keys' scales of key tile j's eight blocks of 16 rows, 8-15 the values'.
      auto scale_of = [&](int j) {
        const int r0 = j * kTile + 16 * (lane & 7);
        if (warp != 12 || lane >= 16 || j >= j1 || r0 >= P) return 1.f;
        int64_t row = ((int64_t)b * a.c.Hkv + g) * a.c.l_cap + r0;
        if (pages) {
          const int32_t page = pages[r0 >> a.c.page_shift];
          if ((uint32_t)page >= a.c.n_pages) return 1.f;  // (flagged by the copies)
          row = (((int64_t)page * a.c.Hkv + g) << a.c.page_shift) +
                (r0 & ((1 << a.c.page_shift) - 1));
        }
        return (lane < 8 ? a.c.ks : a.c.vs)[row >> a.c.block_shift];
      };
      float next = scale_of(j0);
      for (int j = j0; j < j1 && ok; ++j, ++tile) {
        if (warp == 12) {
          // (a value scale of 0, never written, counts as the least)
          const float vs = fmaxf(__shfl_down_sync(0xffffffffu, next, 8), kLeastScale);
          if (lane < 8)
            scale_s[raw_slot(tile)][lane] = make_float4(next, lg2_scale(vs), 1.f / vs, 0.f);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.scale[raw_slot(tile)]);
          next = scale_of(j + 1);
        }
        const int left = P - j * kTile;
        for (int w = 0; w < 2 && ok; ++w) {
          const uint32_t i = 2 * tile + w;
          ok = wait(&bar.raw_full[raw_slot(i)], raw_lap(i));
          if (!ok) break;
          // The codes wait in registers for the operand's slot.
          const uint32_t from = raw + raw_slot(i) * kRawBytes, to = ring + slot_of<FMT>(i) * kSlotBytes;
          uint4 c[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int piece = ch ^ (n & 1) << 2;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(c[n].x), "=r"(c[n].y), "=r"(c[n].z), "=r"(c[n].w)
                         : "r"(from + (row0 + n / 2 * 32) * kD + piece * 16)
                         : "memory");
          }
          if (i >= SLOTS) ok = wait(&bar.empty[slot_of<FMT>(i)], lap_of<FMT>(i) ^ 1);
          if (!ok) break;
          // (rows 8 apart have the same swizzle)
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            if (n == 2) {
              // The codes' slot is free, but not before all loads have returned: one that is
              // still on its way (the products keep shared memory busy) would find the codes of
              // the next lap, so which lane arrives depends on what they brought.  (The e4m3
              // groups of the header, whole call: arriving right behind the loads took 654 us and
              // tore tiles; here 683, before the first piece 703, before the seventh 693.)
              uint32_t any = 0u;
#pragma unroll
              for (int e = 0; e < 8; ++e) any |= c[e].x | c[e].y | c[e].z | c[e].w;
              const int by = __any_sync(0xffffffffu, any != 0u) ? 0 : 1;
              __syncwarp();
              if (lane == by) mbar_arrive(&bar.raw_empty[raw_slot(i)]);
            }
            const int row = row0 + n / 2 * 32, piece = ch ^ (n & 1) << 2;
            uint4 y, z;
            widen<FMT>(c[n].x, y.x, y.y);
            widen<FMT>(c[n].y, y.z, y.w);
            widen<FMT>(c[n].z, z.x, z.y);
            widen<FMT>(c[n].w, z.z, z.w);
            if (left < kTile && row >= left) y = z = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t half = to + (piece >> 2) * kHalf + row * 128;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(half + at0), "r"(y.x),
                         "r"(y.y), "r"(y.z), "r"(y.w)
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(half + (at0 ^ 16)),
                         "r"(z.x), "r"(z.y), "r"(z.z), "r"(z.w)
                         : "memory");
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.full[slot_of<FMT>(i)]);
        }
      }
    }
   }
  }
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int FMT>
cudaError_t launch_fmt(const CUtensorMap& kmap, const CUtensorMap& vmap, const SharedArgs& a,
                       cudaStream_t st) {
  const auto kernel = a.out16 ? shared_prefix_kernel<FMT, 1> : shared_prefix_kernel<FMT, 2>;
  const cudaError_t e = cudaFuncSetAttribute(
      (const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedSmem<FMT>);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(kSharedShares), dim3(kSharedThreads<FMT>), kSharedSmem<FMT>,
                          st, kmap, vmap, a);
}

}  // namespace

cudaError_t launch_shared_prefix(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const SharedArgs& a, int fmt, cudaStream_t st) {
  if (fmt == kFmtInt8) return launch_fmt<kFmtInt8>(kmap, vmap, a, st);
  if (fmt == kFmtE4m3) return launch_fmt<kFmtE4m3>(kmap, vmap, a, st);
  return launch_fmt<kFmtBf16>(kmap, vmap, a, st);
}

}  // namespace tsa
