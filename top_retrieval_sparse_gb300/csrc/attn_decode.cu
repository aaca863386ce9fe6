// attn_decode.cu -- one decode step of attention over the rows that window
// and sinks leave visible: a bf16 cache, or an 8-bit one with a scale for each
// block of rows and KV head.
//
// Per (sequence, KV head) the G <= 8 query heads share every row that is read:
//   z_i = scale q.k_i,  out = sum_i e^z_i v_i / sum_i e^z_i
// in one pass, with the running maximum and sum of the softmax.  A row is read
// once and used for 4 G flop a byte pair, so bandwidth bounds the kernel as
// long as its instructions keep up.
//
// Split.  The rows are cut into slabs of 16 (aligned, so a slab lies in one page and
// one scale block); the slabs of all sequences and KV heads form one list, which the
// CTAs of a resident grid take in equal contiguous shares, whatever the sequences'
// lengths (they are only known on the device).  A share that holds all of a unit
// (sequence, KV head) writes its output; other shares leave (o, max, sum) in the
// workspace and the last to arrive joins them in share order, so results do not depend
// on the order of arrival.
//
// A warp's slab.  mma.m16n8k16 with the rows as M for the logits (heads are the 8
// columns) and the head dimension as M for the output, so that no column of the
// products is wasted on more than 8 - G heads, and the tensor pipe has time to spare
// (17 % busy).  tcgen05 would want 64 or 128 rows of queries; here there are 8.  Rows
// go from global memory straight into the registers of the fragments: the reduction
// index of a product may be permuted at will as long as both operands agree, so each
// lane takes whole 16-byte pieces.  The next slabs' keys are requested when this slab's
// logits are done, their values when the output products are, which keeps up to 8 KB a
// warp and 12 or 16 warps an SM in flight without shared memory (a ring of asynchronous
// copies in shared memory was slower: a million rows 406 us).
//
// Numbers.  Codes are exact in fp16 (whole numbers to 127, 4-bit significands), and so
// are queries after a shift of their exponents; bf16 rows and queries meet as bf16.
// The softmax weights enter the second product as the sum of two fp16 or three bf16
// parts (2^-22 and 2^-24 of the weight at most), so the result is that of 32-bit
// arithmetic.  Matrix instructions truncate their 32-bit sums, which over the hundreds
// of slabs of a long share would lose 2^-17 (measured at a million rows: 1.0e-5 off 64
// bits, 6e-7 now; four million rows of values of one sign: 1e-4 too small, 9e-6 at most
// now); every 16 slabs they are added to sums in shared memory, with
// rounding.  Value scales differ by block, so the weights carry them: w_i = e^z_i s_i
// relative to the largest such product, while the sum adds w_i / s_i.  (fp16 has steps of
// 2^-24 below 2^-14, so what is under 2^-32 of a warp's largest w is lost from the output
// and not from the sum: at most 2^-32 of that w times the row's code.)  The maximum is
// raised only when a weight would pass 2^15: one vote a slab in place of six shuffles.
//
// What bounds it.  bf16: bandwidth (16 x 65536 rows of 4 KV heads, 308 us, 7.0 TB/s).
// e4m3: a million rows of 8 KV heads 318 us, 6.7 TB/s.  int8: its codes take twice the
// instructions to widen (380 a slab; issue slots 43 % busy), 173 us for the same 16 x
// 65536 rows, 6.2 TB/s; pages of 16 cost 2 % more.
#include <cuda_fp16.h>

#include "cache_ops.h"

namespace tsa {

namespace {

constexpr int kWarps = kDecodeThreads / 32;
// log2 of a weight that raised the maximum, and of the largest one that does
// not: fp16's normal numbers then reach 2^-21 below the first, its smallest
// steps 2^-32.
constexpr float kRaised = 7.f, kSlack = 15.f;
constexpr float kLeastScale = 1.f / (1ll << 60);  // the smallest that the cache's writer gives

__device__ __forceinline__ uint4 ld_row(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ uint4 ld_row_if(const uint8_t* p, bool on) {
  return on ? ld_row(p) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ uint32_t word(const uint4& w, int j) {
  return j == 0 ? w.x : (j == 1 ? w.y : (j == 2 ? w.z : w.w));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Of value scales: the exponent and the logarithm of what is left, so that it is
// exact for powers of two (an error would change a weight, and its share of the sum).
__device__ __forceinline__ float lg2(float x) {
  const uint32_t u = __float_as_uint(x);
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;"
      : "=f"(r)
      : "f"(__uint_as_float((u & 0x7fffffu) | 0x3f800000u)));
  // the exponent's bits under the exponent of 2^23
  return r + (__uint_as_float((u >> 23) | 0x4b000000u) - 8388735.f);
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Codes in bytes 0-1 (lo) or 2-3 (hi) of w as fp16x2, exactly.
template <int FMT>
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  if (FMT == kFmtInt8) return codes_lo_f16x2(w);
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n"
      : "=r"(r) : "r"(w));
  return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  if (FMT == kFmtInt8) return codes_hi_f16x2(w);
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n"
      : "=r"(r) : "r"(w));
  return r;
}

template <int FMT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (FMT == kFmtBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int FMT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (FMT == kFmtBf16) return make_float2(bf_lo(w), bf_hi(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int FMT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (FMT == kFmtBf16)
    mma_bf16(d, a0, a1, a2, a3, b0, b1);
  else
    mma_f16(d, a0, a1, a2, a3, b0, b1);
}

// a / b of numbers that are not negative; 64-bit division takes hundreds of cycles
// and is only needed past 2^32 slabs.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
  return (int64_t)((uint32_t)a / (uint32_t)b);
}

// The visible rows of one sequence as a list of slabs: [0, s0), then from sw.
struct Visible {
  int L, n0, lo, s0, sw, n;
};
__device__ __forceinline__ Visible visible(const DecodeArgs& a, int b) {
  Visible v;
  const int len = a.lens[b], cap = (int)a.c.l_cap;
  v.L = len < 0 ? 0 : (len > cap ? cap : len);
  v.n0 = a.n_init < v.L ? (int)a.n_init : v.L;
  v.lo = a.n_recent < v.L ? v.L - (int)a.n_recent : 0;
  v.s0 = (int)(((uint32_t)v.n0 + 15) >> 4);
  v.sw = v.lo >> 4 > v.s0 ? v.lo >> 4 : v.s0;
  const int se = (int)(((uint32_t)v.L + 15) >> 4);
  v.n = v.s0 + (v.lo < v.L && se > v.sw ? se - v.sw : 0);
  return v;
}

// A partial of one (share, unit): max and sum of every head, then o.
__device__ __forceinline__ float* slot_of(const DecodeArgs& a, int share, int which) {
  return a.partial + (size_t)(2 * share + which) * kDecodeSlot;
}

__device__ __forceinline__ void put_row(const DecodeArgs& a, int b, int head, int lane, float4 o,
                                        float m, float l) {
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
  const int64_t at = (int64_t)b * a.Hq + head;
  *reinterpret_cast<float4*>(a.out + at * kD + 4 * lane) =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (a.lse && lane == 0) {
    // m carries a value scale and l its inverse (2^60 at most), so the exponents are
    // added first: log2(l) as one number would be off by up to 2^-18.
    const uint32_t u = __float_as_uint(l);
    const float e = (float)((int)(u >> 23) - 127);
    const float f = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
    a.lse[at] = l == 0.f ? -INFINITY
                         : (l < INFINITY ? ((m + e) + log2f(f)) * 0.6931471805599453f : l);
  }
}

// Slabs that a warp works on at once, and CTAs of 4 warps an SM: rows of 8 KB
// a turn for bf16 and e4m3 (their rows wait in 64 registers a lane, 12 warps an SM);
// int8 codes take twice e4m3's instructions to widen, and 16 warps of one slab
// each hide those better (16 x 65536 rows, both before slabs' usual case was put first:
// int8 183 us against 187 with two slabs; e4m3 177 against 173).
__host__ __device__ constexpr int slabs_of(int fmt) { return fmt == kFmtE4m3 ? 2 : 1; }
__host__ __device__ constexpr int ctas_of(int fmt) { return fmt == kFmtInt8 ? 4 : 3; }

template <int FMT>
__global__ void __launch_bounds__(kDecodeThreads, ctas_of(FMT)) attn_decode_kernel(DecodeArgs a) {
  constexpr bool B16 = FMT == kFmtBf16;
  constexpr int NS = slabs_of(FMT);      // slabs a warp works on at once
  constexpr int KW = B16 ? 4 : 2;        // 16-byte pieces of a key row a lane takes
  constexpr int VW = B16 ? 2 : 1;        // and of a value row
  constexpr int ROW = B16 ? 2 * kD : kD; // bytes of a row
  constexpr int PARTS = B16 ? 3 : 2;     // 16-bit parts of a softmax weight
  constexpr int kFold = 8 / NS * 2;      // turns between folds: 16 slabs or 8 pairs
  extern __shared__ int64_t prefix[];    // [B + 1] slabs before each sequence
  __shared__ __align__(16) float acc_s[kWarps][kMaxGroup][kD];
  __shared__ float stat_s[kWarps][2][kMaxGroup];
  __shared__ int64_t scan_s[kWarps];
  __shared__ int last_s;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gr = lane >> 2, tq = lane & 3;
  const int Hkv = a.c.Hkv, G = a.Hq / Hkv;

  // The list of all slabs, sequence by sequence.  Up to 32 sequences every warp
  // makes it for itself (all write the same values), else the warps share it.
  if (tid == 0) prefix[0] = 0;
  const int step = a.B <= 32 ? 32 : kDecodeThreads, me = a.B <= 32 ? lane : tid;
  int64_t carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += step) {
    const int b = b0 + me;
    int64_t n = 0;
    if (b < a.B) {
      const Visible v = visible(a, b);
      n = (int64_t)v.n * Hkv;
      if (blockIdx.x == 0 && v.L != a.lens[b]) atomicOr(a.status, kStatusBadLength);
      if (n == 0 && b % gridDim.x == blockIdx.x)  // nothing visible
        for (int h = 0; h < a.Hq; ++h) {
          float* o = a.out + ((int64_t)b * a.Hq + h) * kD;
          for (int j = 0; j < kD; ++j) o[j] = 0.f;
          if (a.lse) a.lse[(int64_t)b * a.Hq + h] = -INFINITY;
        }
    }
    int64_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (a.B <= 32) {
      if (b < a.B) prefix[b + 1] = x;
      if (lane == 0) prefix[0] = 0;
      carry = __shfl_sync(0xffffffffu, x, 31);
      __syncwarp();
      break;
    }
    if (lane == 31) scan_s[warp] = x;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) x += scan_s[w];
    }
    if (b < a.B) prefix[b + 1] = carry + x;
    for (int w = 0; w < kWarps; ++w) carry += scan_s[w];
    __syncthreads();
  }
  const int64_t total = carry;
  constexpr int kLeast = kWarps * 2;  // slabs of the smallest share (a power of two)
  int64_t share = quotient(total + gridDim.x - 1, gridDim.x);
  share = (share + kLeast - 1) & ~(int64_t)(kLeast - 1);
  if (share < kLeast) share = kLeast;
  int64_t at = (int64_t)blockIdx.x * share;
  const int64_t end = at + share < total ? at + share : total;
  if (at >= end) return;
  int b = 0;
  for (int hi = a.B; hi - b > 1;) {  // the last sequence that starts at or before `at`
    const int mid = (b + hi) >> 1;
    if (prefix[mid] <= at) b = mid; else hi = mid;
  }

  bool first = true;
  while (at < end) {
    while (prefix[b + 1] <= at) ++b;
    const Visible vis = visible(a, b);
    const int g = (int)quotient(at - prefix[b], vis.n);
    // the unit in the list, and the slabs of it that are this share's
    const int64_t u0 = prefix[b] + (int64_t)g * vis.n, u1 = u0 + vis.n;
    const int k0 = (int)(at - u0), k1 = (int)((u1 < end ? u1 : end) - u0);

    // Query fragments (columns: heads), exact in the product's type.
    uint32_t qf[8][2];
    float qs0 = a.scale_log2, qs1 = a.scale_log2;
    {
      const uint16_t* qp = a.q + ((int64_t)b * a.Hq + g * G + (gr < G ? gr : 0)) * kD;
      float amax = 0.f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int d = B16 ? 8 * (tq + 4 * (s >> 1)) + 4 * (s & 1)
                          : 16 * (tq + 4 * (s >> 2)) + 4 * (s & 3);
        uint2 w = *reinterpret_cast<const uint2*>(qp + d);
        if (gr >= G) w = make_uint2(0u, 0u);
        qf[s][0] = w.x;
        qf[s][1] = w.y;
        if (!B16)
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf_lo(w.x)), fabsf(bf_hi(w.x))),
                                   fmaxf(fabsf(bf_lo(w.y)), fabsf(bf_hi(w.y)))));
      }
      if (!B16) {
        // exponents shifted so that the head's largest element is in [2^14, 2^15)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int e = 141 - (int)(__float_as_uint(amax) >> 23);  // 14 - floor(log2 amax)
        e = amax == 0.f ? 0 : (e > 126 ? 126 : (e < -113 ? -113 : e));
        const float up = __uint_as_float((uint32_t)(e + 127) << 23);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[s][i] = pack2<FMT>(bf_lo(qf[s][i]) * up, bf_hi(qf[s][i]) * up);
        qs0 *= __shfl_sync(0xffffffffu, down, 8 * tq);
        qs1 *= __shfl_sync(0xffffffffu, down, 8 * tq + 4);
      }
    }

    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    bool bad = false;
    // kFold turns' sums, a lane's own 16 bytes for each of acc's rows
    float4* fold = reinterpret_cast<float4*>(&acc_s[warp][0][0]) + lane;
    bool folded = false;
    int turns = 0;

    uint4 kr[NS][2][KW], vr[NS][4][VW];
    // Rows fit 32 bits: 2^32 rows of keys alone are more than the memory.
    uint32_t row[NS], seen[NS], seen_now[NS];
    float ks[NS], vs[NS], ks_now[NS], vs_now[NS];
    int32_t page[NS] = {};
    const int32_t* pages = a.c.page_table ? a.c.page_table + (int64_t)b * a.c.max_pages : nullptr;
    const uint32_t unit_row = (uint32_t)(((int64_t)b * Hkv + g) * a.c.l_cap);
    const uint8_t* k_lane = a.c.k + gr * ROW + 16 * tq;
    const uint8_t* v_lane = a.c.v + 2 * tq * ROW + 16 * VW * gr;

    // All rows are seen of the sinks' slabs but the last, and of the window's but
    // the first and the last: those three take the long way.
    const int inside = vis.s0 + 1, shift = vis.sw - vis.s0;
    const uint32_t insides = vis.n - 1 > inside ? vis.n - 1 - inside : 0;
    auto first_row = [&](int k) {
      return (int)((uint32_t)(k < vis.s0 ? k : k + shift) << 4);
    };
    auto want_pages = [&](int k) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
        if (pages && k + s < k1) page[s] = pages[first_row(k + s) >> a.c.page_shift];
    };
    auto find_rows = [&](int k) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int i = first_row(k + s);
        seen[s] = 0xffffu;
        if (__builtin_expect(((uint32_t)(k + s - inside) >= insides && k + s >= vis.s0 - 1) ||
                                 k + s >= k1, 0)) {
          seen[s] = 0u;
          if (k + s < k1)
            for (int j = 0; j < 16; ++j)
              if ((j < vis.n0 - i || j >= vis.lo - i) && j < vis.L - i) seen[s] |= 1u << j;
        }
        row[s] = unit_row + (uint32_t)i;
        if (pages) {
          row[s] = (((uint32_t)page[s] * (uint32_t)Hkv + (uint32_t)g) << a.c.page_shift) +
                   ((uint32_t)i & ((1u << a.c.page_shift) - 1u));
          if (__builtin_expect((uint32_t)page[s] >= a.c.n_pages, 0)) {
            bad |= seen[s] != 0u;
            seen[s] = 0u;
          }
        }
        if (__builtin_expect(seen[s] == 0u, 0)) row[s] = 0u;  // (nothing is read)
      }
    };
    auto want_keys = [&]() {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint8_t* p = k_lane + (uint64_t)row[s] * ROW;
        if (__builtin_expect(seen[s] == 0xffffu, 1)) {
#pragma unroll
          for (int c = 0; c < KW; ++c) {
            kr[s][0][c] = ld_row(p + 64 * c);
            kr[s][1][c] = ld_row(p + 8 * ROW + 64 * c);
          }
        } else {
#pragma unroll
          for (int c = 0; c < KW; ++c) {
            kr[s][0][c] = ld_row_if(p + 64 * c, (seen[s] >> gr) & 1u);
            kr[s][1][c] = ld_row_if(p + 8 * ROW + 64 * c, (seen[s] >> (gr + 8)) & 1u);
          }
        }
        if (!B16) {
          ks[s] = vs[s] = 1.f;
          if (__builtin_expect(seen[s] != 0u, 1)) {
            ks[s] = a.c.ks[row[s] >> a.c.block_shift];
            vs[s] = a.c.vs[row[s] >> a.c.block_shift];
          }
        }
      }
    };
    auto want_values = [&]() {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint8_t* p = v_lane + (uint64_t)row[s] * ROW;
        // rows 2tq, 2tq + 1, 2tq + 8, 2tq + 9
        if (__builtin_expect(seen[s] == 0xffffu, 1)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < VW; ++c)
              vr[s][i][c] = ld_row(p + ((i & 1) + 8 * (i >> 1)) * ROW + 16 * c);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < VW; ++c) {
              const int r = (i & 1) + 8 * (i >> 1);
              vr[s][i][c] = ld_row_if(p + r * ROW + 16 * c, (seen[s] >> (2 * tq + r)) & 1u);
            }
        }
      }
    };

    constexpr int stride = kWarps * NS;
    int k = k0 + warp * NS;
    want_pages(k);
    find_rows(k);
    want_pages(k + stride);
    want_keys();
    want_values();
    for (; k < k1; k += stride) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        seen_now[s] = seen[s];
        ks_now[s] = ks[s];
        // (a cache that was zeroed and not written here has scales of 0, which have no
        // logarithm: its values count as codes of the least scale, 4e-16 at most)
        vs_now[s] = fmaxf(vs[s], kLeastScale);
      }
      find_rows(k + stride);
      want_pages(k + 2 * stride);

      // Logits: lane holds rows gr and gr + 8 of heads 2tq and 2tq + 1.
      float z[NS][4];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        float ze[4] = {0.f, 0.f, 0.f, 0.f}, zo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          float(&d)[4] = t & 1 ? zo : ze;
          if (B16) {
            const int c = t >> 1, j = 2 * (t & 1);
            mma<FMT>(d, word(kr[s][0][c], j), word(kr[s][1][c], j), word(kr[s][0][c], j + 1),
                     word(kr[s][1][c], j + 1), qf[t][0], qf[t][1]);
          } else {
            const uint32_t w0 = word(kr[s][0][t >> 2], t & 3);
            const uint32_t w1 = word(kr[s][1][t >> 2], t & 3);
            mma<FMT>(d, codes_lo<FMT>(w0), codes_lo<FMT>(w1), codes_hi<FMT>(w0),
                     codes_hi<FMT>(w1), qf[t][0], qf[t][1]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) z[s][j] = ze[j] + zo[j];
      }
      want_keys();

      // y = log2 of the weights' products with their value scale
      float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const float f0 = B16 ? qs0 : qs0 * ks_now[s], f1 = B16 ? qs1 : qs1 * ks_now[s];
        const float add = B16 ? 0.f : lg2(vs_now[s]);
        z[s][0] = fmaf(z[s][0], f0, add);
        z[s][1] = fmaf(z[s][1], f1, add);
        z[s][2] = fmaf(z[s][2], f0, add);
        z[s][3] = fmaf(z[s][3], f1, add);
        if (__builtin_expect(seen_now[s] != 0xffffu, 0)) {
          if (!((seen_now[s] >> gr) & 1u)) z[s][0] = z[s][1] = -INFINITY;
          if (!((seen_now[s] >> (gr + 8)) & 1u)) z[s][2] = z[s][3] = -INFINITY;
        }
        top0 = fmaxf(top0, fmaxf(z[s][0], z[s][2]));
        top1 = fmaxf(top1, fmaxf(z[s][1], z[s][3]));
      }
      if (__builtin_expect(
              __any_sync(0xffffffffu, top0 > m0 + kSlack || top1 > m1 + kSlack), 0)) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
        }
        const float n0 = fmaxf(m0, top0 - kRaised), n1 = fmaxf(m1, top1 - kRaised);
        const float f0 = m0 == n0 ? 1.f : ex2(m0 - n0), f1 = m1 == n1 ? 1.f : ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i][0] *= f0;
          acc[i][1] *= f1;
          acc[i][2] *= f0;
          acc[i][3] *= f1;
          if (folded) {
            float4 f = fold[32 * i];
            f.x *= f0; f.y *= f1; f.z *= f0; f.w *= f1;
            fold[32 * i] = f;
          }
        }
      }
      const float c0 = m0 == -INFINITY ? 0.f : m0, c1 = m1 == -INFINITY ? 0.f : m1;
      // Weights in parts, transposed to the product's B layout (rows 2tq,
      // 2tq + 1 and 2tq + 8, 2tq + 9 of head gr).
      uint32_t wt[NS][PARTS][2];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        float p[4] = {ex2(z[s][0] - c0), ex2(z[s][1] - c1), ex2(z[s][2] - c0),
                      ex2(z[s][3] - c1)};
        const float un = B16 ? 1.f : rcp(vs_now[s]);
        l0 = fmaf(p[0] + p[2], un, l0);
        l1 = fmaf(p[1] + p[3], un, l1);
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
          const uint32_t x = pack2<FMT>(p[0], p[1]), y = pack2<FMT>(p[2], p[3]);
          wt[s][i][0] = transpose8(x);
          wt[s][i][1] = transpose8(y);
          const float2 fx = unpack2<FMT>(x), fy = unpack2<FMT>(y);
          p[0] -= fx.x; p[1] -= fx.y; p[2] -= fy.x; p[3] -= fy.y;
        }
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {  // dimensions 16 gr + 2i .. + 3
          uint32_t x[2][4];
          if (B16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = (i + h) >> 2, j = (i + h) & 3;
              const uint32_t a0 = word(vr[s][0][c], j), a1 = word(vr[s][1][c], j);
              const uint32_t a2 = word(vr[s][2][c], j), a3 = word(vr[s][3][c], j);
              x[h][0] = prmt(a0, a1, 0x5410);
              x[h][1] = prmt(a0, a1, 0x7632);
              x[h][2] = prmt(a2, a3, 0x5410);
              x[h][3] = prmt(a2, a3, 0x7632);
            }
          } else {
            const int j = i >> 1;
            const uint32_t a0 = word(vr[s][0][0], j), a1 = word(vr[s][1][0], j);
            const uint32_t a2 = word(vr[s][2][0], j), a3 = word(vr[s][3][0], j);
            const uint32_t t0 = prmt(a0, a1, 0x5140), t1 = prmt(a0, a1, 0x7362);
            const uint32_t t2 = prmt(a2, a3, 0x5140), t3 = prmt(a2, a3, 0x7362);
            x[0][0] = codes_lo<FMT>(t0); x[0][1] = codes_hi<FMT>(t0);
            x[0][2] = codes_lo<FMT>(t2); x[0][3] = codes_hi<FMT>(t2);
            x[1][0] = codes_lo<FMT>(t1); x[1][1] = codes_hi<FMT>(t1);
            x[1][2] = codes_lo<FMT>(t3); x[1][3] = codes_hi<FMT>(t3);
          }
#pragma unroll
          for (int j = 0; j < PARTS; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma<FMT>(acc[i + h], x[h][0], x[h][1], x[h][2], x[h][3], wt[s][j][0], wt[s][j][1]);
        }
      }
      want_values();
      if (++turns == kFold) {  // the sums so far go to shared memory, with rounding
        turns = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float4 f = folded ? fold[32 * i] : make_float4(0.f, 0.f, 0.f, 0.f);
          f.x += acc[i][0]; f.y += acc[i][1]; f.z += acc[i][2]; f.w += acc[i][3];
          fold[32 * i] = f;
          acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        }
        folded = true;
      }
    }
    if (folded) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = fold[32 * i];
        acc[i][0] += f.x; acc[i][1] += f.y; acc[i][2] += f.z; acc[i][3] += f.w;
      }
      __syncwarp();
    }

    // Join the warps.
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if (bad) {
      if (lane == 0) atomicOr(a.status, kStatusBadLength);
      l0 = l1 = nanf("");
    }
    if (gr == 0) {
      stat_s[warp][0][2 * tq] = m0;
      stat_s[warp][0][2 * tq + 1] = m1;
      stat_s[warp][1][2 * tq] = l0;
      stat_s[warp][1][2 * tq + 1] = l1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc_s[warp][2 * tq][16 * gr + 2 * i] = acc[i][0];
      acc_s[warp][2 * tq + 1][16 * gr + 2 * i] = acc[i][1];
      acc_s[warp][2 * tq][16 * gr + 2 * i + 1] = acc[i][2];
      acc_s[warp][2 * tq + 1][16 * gr + 2 * i + 1] = acc[i][3];
    }
    __syncthreads();
    const bool all = k0 == 0 && k1 == vis.n;  // the whole unit
    float* slot = slot_of(a, blockIdx.x, first ? 0 : 1);
    for (int h = warp; h < G; h += kWarps) {
      float m = -INFINITY, l = 0.f;
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stat_s[w][0][h]);
      const float c = m == -INFINITY ? 0.f : m;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(stat_s[w][0][h] - c);
        l = fmaf(stat_s[w][1][h], f, l);
        const float4 x = *reinterpret_cast<const float4*>(&acc_s[w][h][4 * lane]);
        o.x = fmaf(x.x, f, o.x); o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z); o.w = fmaf(x.w, f, o.w);
      }
      if (all) {
        put_row(a, b, g * G + h, lane, o, m, l);
      } else {
        if (lane == 0) {
          slot[h] = m;
          slot[kMaxGroup + h] = l;
        }
        *reinterpret_cast<float4*>(slot + 2 * kMaxGroup + h * kD + 4 * lane) = o;
      }
    }
    if (!all) {
      // The shares of the unit are s0 .. s1; the last to get here joins them.
      const int s0 = (int)quotient(u0, share), s1 = (int)quotient(u1 - 1, share);
      const int which0 = u0 == s0 * share ? 0 : 1;  // the unit's slot of share s0; 0 of the others
      uint32_t* ctr = a.arrived + (int64_t)b * Hkv + g;
      __threadfence();
      __syncthreads();
      if (tid == 0) last_s = atomicAdd(ctr, 1u) == (uint32_t)(s1 - s0);
      __syncthreads();
      if (last_s) {
        __threadfence();
        for (int h = warp; h < G; h += kWarps) {
          // lanes look at the shares' maxima and sums, then at the outputs'
          // dimensions; every load of a pass is independent of the others
          auto part = [&](int s) { return slot_of(a, s, s > s0 ? 0 : which0); };
          float m = -INFINITY, l = 0.f;
          for (int s = s0 + lane; s <= s1; s += 32) m = fmaxf(m, __ldcg(part(s) + h));
          m = warp_max(m);
          const float c = m == -INFINITY ? 0.f : m;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int t = s0; t <= s1; t += 32) {
            const int n = s1 - t + 1 < 32 ? s1 - t + 1 : 32;
            float f = 0.f;
            if (lane < n) {
              f = ex2(__ldcg(part(t + lane) + h) - c);
              l = fmaf(__ldcg(part(t + lane) + kMaxGroup + h), f, l);
            }
#pragma unroll 16
            for (int s = 0; s < n; ++s) {
              const float w = __shfl_sync(0xffffffffu, f, s);
              const float4 x = __ldcg(reinterpret_cast<const float4*>(
                  part(t + s) + 2 * kMaxGroup + h * kD + 4 * lane));
              o.x = fmaf(x.x, w, o.x); o.y = fmaf(x.y, w, o.y);
              o.z = fmaf(x.z, w, o.z); o.w = fmaf(x.w, w, o.w);
            }
          }
          l = warp_sum(l);
          put_row(a, b, g * G + h, lane, o, m, l);
        }
        if (tid == 0) *ctr = 0u;  // ready for the next call
      }
    }
    __syncthreads();  // the shared arrays are free again
    first = false;
    at = u0 + k1;
  }
}

}  // namespace

int attn_decode_ctas(int fmt) { return ctas_of(fmt); }

cudaError_t launch_attn_decode(const DecodeArgs& a, int fmt, int grid, cudaStream_t st) {
  const size_t smem = (size_t)(a.B + 1) * sizeof(int64_t);
  const dim3 g(grid), th(kDecodeThreads);
  const auto kernel = fmt == kFmtInt8   ? attn_decode_kernel<kFmtInt8>
                      : fmt == kFmtE4m3 ? attn_decode_kernel<kFmtE4m3>
                                        : attn_decode_kernel<kFmtBf16>;
  if (smem > 24 * 1024) {  // with the static arrays: past the default limit
    const cudaError_t e = cudaFuncSetAttribute(
        (const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kernel, g, th, smem, st, a);
}

}  // namespace tsa
