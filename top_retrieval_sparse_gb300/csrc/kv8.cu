// kv8.cu -- the 8-bit KV cache: written (with the keys' rotation) and read.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "rope.cuh"

namespace tsa {

namespace {

enum { kStraight = 0, kTurnHalf = 1, kTurnInterleaved = 2 };

// Threads of an append CTA: one team of warps, so that none waits at another's
// barriers (128K tokens of 8 heads, blocks of 64: 157 us with two teams a CTA, 117 us with
// one); teams of one warp have no barriers, and there are eight.
__host__ __device__ constexpr int append_threads(int blk) { return blk == 16 ? 256 : 2 * blk; }

// 2^e for the smallest e >= -60 with top * 2^e >= amax (finite, >= 0), top = 127
// or 448 = 1.984375 * 2^6 or 1.75 * 2^8: from amax's exponent and mantissa.
__device__ __forceinline__ float scale_for(float amax, int fmt) {
  const uint32_t u = __float_as_uint(amax), m = u & 0x7fffffu;
  int e = (int)(u >> 23) - 127 - (fmt == kFmtInt8 ? 6 : 8) +
          (m > (fmt == kFmtInt8 ? 0x7e0000u : 0x600000u));
  e = e < -60 ? -60 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The larger magnitude, NaN if either is.
__device__ __forceinline__ float max_abs(float m, float x) {
  float r;
  asm("{\n .reg .f32 t;\n abs.f32 t, %2;\n max.NaN.f32 %0, %1, t;\n}\n"
      : "=f"(r) : "f"(m), "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {  // of bf16 pairs
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
  return r;
}

// Codes of eight values.  int8: 1.5 * 2^23 + 128 is added, which rounds to whole
// numbers (ties to even) and leaves code + 128 in the low byte: one fused operation
// where every value is finite (CLEAN: the scale then holds them); else infinities
// saturate and NaN becomes 0.
template <int FMT, bool CLEAN>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  if constexpr (FMT == kFmtInt8) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (CLEAN) {
        b[e] = __float_as_uint(fmaf(x[e], inv, 12583040.f));
      } else {
        float y = x[e] * inv;
        y = y == y ? fminf(fmaxf(y, -127.f), 127.f) : 0.f;
        b[e] = __float_as_uint(y + 12583040.f);
      }
    }
    const uint32_t lo0 = __byte_perm(b[0], b[1], 0x0040), hi0 = __byte_perm(b[2], b[3], 0x0040);
    const uint32_t lo1 = __byte_perm(b[4], b[5], 0x0040), hi1 = __byte_perm(b[6], b[7], 0x0040);
    return make_uint2(__byte_perm(lo0, hi0, 0x5410), __byte_perm(lo1, hi1, 0x5410));
  } else {
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      h[e] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e] * inv, x[2 * e + 1] * inv),
                                      __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  }
}

// Values of eight codes (exact).  int8: a byte under the exponent of 2^23 is the
// number 2^23 + code + 128.
template <int FMT>
__device__ __forceinline__ void decode8(uint2 w, float scale, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = h ? w.y : w.x;
    if constexpr (FMT == kFmtInt8) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[4 * h + e] =
            (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + e)) - 8388736.f) * scale;
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const __half2_raw r =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * e)), __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        x[4 * h + 2 * e] = f.x * scale;
        x[4 * h + 2 * e + 1] = f.y * scale;
      }
    }
  }
}

// Bandwidth-bound: a row's 256 bytes are read once and written as 128.  The new
// rows of one (block, KV head, K or V) stay in the registers of BLK / 16 warps (a team; 16
// rows a warp, eight lanes a row, 128 bytes a lane in flight) between the search for
// their largest magnitude and their coding.  Neighbouring teams take the heads of one
// block, whose rows are neighbours in memory.  Keys are rotated (KIND) by angles from the
// table in L2, 512 bytes a row, which each head's team reads for itself: sharing them
// between the heads in shared memory made a CTA go through the heads one after another
// over strided reads (227 us for 128K tokens of 8 heads, 194 us so).  128K tokens without a
// rotation: 117 us, 6.9 TB/s; with it the rotated rows in 32 bits beside the rows as read
// and the angles reach the limit of 128 registers (16 warps an SM; 80 to 112 bytes a
// thread spill, 204 at blocks of 16), and what those warps wait for bounds it.
template <int FMT, int BLK, int KIND>
__global__ void __launch_bounds__(append_threads(BLK), (KIND ? 512 : 768) / append_threads(BLK))
    kv8_append_kernel(AppendArgs a, int nb) {
  constexpr int TW = BLK / 16, TEAMS = append_threads(BLK) / 32 / TW;
  __shared__ float red[append_threads(BLK) / 32];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y;
  int64_t tok, n;
  const int64_t L = a.lens[b];
  const bool good = seq_tokens(a.cu, a.max_new, a.T, b, tok, n);
  if (!good || L < n || L > a.c.l_cap) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
    return;
  }
  if (n == 0) return;
  const int64_t start = L - n;
  const int warp = threadIdx.x >> 5, team = warp / TW, lane = threadIdx.x & 31, l = lane & 7;
  const int row_in = (warp % TW) * 16 + (lane >> 3);  // rows row_in + 4 i of the block
  // Team's item: head g of K, then of V, of block j (counted from start's).
  const uint32_t item = blockIdx.x * TEAMS + team, half = item / a.c.Hkv;
  const int g = (int)(item - half * a.c.Hkv);
  const bool values = half & 1;
  const int64_t j = half >> 1, p0 = (start / BLK + j) * BLK;  // the block's first position
  const int64_t tok0 = tok + p0 - start;                      // token of its row 0
  // rows [r0, r1) are new
  const int r0 = start > p0 ? (int)(start - p0) : 0;
  const int r1 = j >= nb || p0 >= L ? 0 : (L - p0 < BLK ? (int)(L - p0) : BLK);
  const bool turn = KIND && !values;
  RopeLane ln = {2 * l, 2 * l + 1, -1};
  if (turn) ln = rope_lane(a.rope, l);
  const RowsView& in = values ? a.v : a.k;
  uint8_t* codes = values ? a.c.v : a.c.k;
  float* scales = values ? a.c.vs : a.c.ks;
  int64_t row0 = -1;                                  // of the block in the pool
  float old = 0.f;
  if (r1 > 0) {
    row0 = cache_row(a.c, b, g, p0);
    if (row0 < 0 && lane == 0 && a.status) atomicOr(a.status, kStatusBadLength);
  }
  const bool live = row0 >= 0;
  if (live) old = scales[row0 / BLK];
  uint4 w[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row_in + 4 * i;
    w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (live && r >= r0 && r < r1) {
      const uint16_t* p = in.p + (tok0 + r) * in.st + g * in.sh;
      w[i][0] = *reinterpret_cast<const uint4*>(p + 8 * ln.a);
      w[i][1] = *reinterpret_cast<const uint4*>(p + 8 * ln.b);
    }
  }
  // Rotated rows in 32 bits (KIND); otherwise they are widened where they are used.
  // A block's own positions share the table's high angle (128 divides kRopeLow), and
  // the low ones are asked for with the rows, not after them.
  float x[KIND ? 4 : 1][16];
  if constexpr (KIND != kStraight) {
    const bool own = turn && live && !a.positions && p0 + r1 <= a.rope.max_pos;
    float4 lo[4][4], hi[4];
    if (own && ln.pair >= 0) {
      const int n8 = a.rope.pairs >> 3;
      const float4* h = reinterpret_cast<const float4*>(
                            a.rope.hi + (p0 >> kRopeLowBits) * a.rope.pairs) + l;
      const float4* q = reinterpret_cast<const float4*>(
                            a.rope.lo + ((p0 & (kRopeLow - 1)) + row_in) * a.rope.pairs) + l;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = h[n8 * e];
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i][e] = q[2 * a.rope.pairs * i + n8 * e];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row_in + 4 * i;
      float u[8], v[8];
      unpack8(w[i][0], u);
      unpack8(w[i][1], v);
      if (ln.pair >= 0 && live && r >= r0 && r < r1) {
        float2 cs[8];
        if (own) {
#pragma unroll
          for (int e = 0; e < 4; ++e) rope_sum(lo[i][e], hi[e], cs[2 * e], cs[2 * e + 1]);
        } else {
          const int64_t at = a.positions ? (int64_t)a.positions[tok0 + r] : p0 + r;
          rope_angles(a.rope, at, l, cs);
          if (l == 0 && (at < 0 || at >= a.rope.max_pos) && a.status)
            atomicOr(a.status, kStatusBadLength);
        }
        rope_turn(KIND == kTurnInterleaved, cs, u, v);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] = u[e];
        x[i][8 + e] = v[e];
      }
    }
  }
  auto row_values = [&](int i, float (&u)[8], float (&v)[8]) {
    if constexpr (KIND != kStraight) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[e] = x[i][e];
        v[e] = x[i][8 + e];
      }
    } else {
      unpack8(w[i][0], u);
      unpack8(w[i][1], v);
    }
  };
  // Largest magnitude, NaN or infinite where a value is (rows that are not new are
  // zeros here).
  float amax = 0.f;
  if constexpr (KIND != kStraight) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = max_abs(amax, x[i][e]);
  } else {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        m = max_abs2(max_abs2(max_abs2(max_abs2(m, w[i][h].x), w[i][h].y), w[i][h].z), w[i][h].w);
    amax = max_abs(bf_lo(m), bf_hi(m));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_abs(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const bool clean = amax <= 3.402823466e38f;  // of this warp
  if (!clean) {                                // once more, of what is finite
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u[8], v[8];
      row_values(i, u, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float mu = fabsf(u[e]), mv = fabsf(v[e]);
        if (mu <= 3.402823466e38f) amax = fmaxf(amax, mu);
        if (mv <= 3.402823466e38f) amax = fmaxf(amax, mv);
      }
    }
    amax = warp_max(amax);
  }
  if (TW > 1) {
    if (lane == 0) red[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TW; ++i) amax = fmaxf(amax, red[team * TW + i]);
  }
  if (!live) return;
  const float need = scale_for(amax, FMT);
  const bool older = r0 > 0;                   // older rows live in the block
  const float s = older ? fmaxf(old, need) : need;
  const float inv = 1.f / s;                   // exact: a power of two
  uint8_t* out = codes + row0 * kD;
  if (older && s != old) {                     // grown: the older rows once more
    for (int r = row_in; r < r0 && r < (warp % TW + 1) * 16; r += 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2* at = reinterpret_cast<uint2*>(out + r * kD + 8 * (h ? ln.b : ln.a));
        float y[8];
        decode8<FMT>(*at, old, y);
        *at = encode8<FMT, true>(y, inv);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row_in + 4 * i;
    if (r >= r0 && r < r1) {
      float u[8], v[8];
      row_values(i, u, v);
      const uint2 cu = clean ? encode8<FMT, true>(u, inv) : encode8<FMT, false>(u, inv);
      const uint2 cv = clean ? encode8<FMT, true>(v, inv) : encode8<FMT, false>(v, inv);
      if (KIND == kTurnHalf && ln.b != ln.a + 1) {
        *reinterpret_cast<uint2*>(out + r * kD + 8 * ln.a) = cu;
        *reinterpret_cast<uint2*>(out + r * kD + 8 * ln.b) = cv;
      } else {
        *reinterpret_cast<uint4*>(out + r * kD + 8 * ln.a) = make_uint4(cu.x, cu.y, cv.x, cv.y);
      }
    }
  }
  // (every lane of the team has read the old scale before the barrier above; a
  // team of one warp is in step)
  __syncwarp();
  if (warp % TW == 0 && lane == 0) scales[row0 / BLK] = s;
}

constexpr int kReadRows = 64;  // rows of a CTA of kv8_read_kernel

// Bandwidth-bound: eight lanes a row, 16 codes a lane, keys and values of two
// rows in flight a lane.  No early start for the next kernel: what is read
// back may be a cache that the key scan streams before its wait.
template <int FMT>
__global__ void __launch_bounds__(256) kv8_read_kernel(ReadArgs a) {
  pdl_wait();
  const int b = blockIdx.z, g = blockIdx.y, l = threadIdx.x & 7;
  int64_t tok, n;
  const bool good = seq_tokens(a.cu, a.max_new, a.T, b, tok, n);
  if (!good) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
    if (tok < 0 || tok + n > a.T) return;
    n = n < 0 ? 0 : (n > a.max_new ? a.max_new : n);
  }
  const int64_t j0 = (int64_t)blockIdx.x * kReadRows + (threadIdx.x >> 3);
  if (j0 >= n) return;
  const int64_t L = a.lens[b];
  const bool bad_len = !good || L < 0 || L > a.c.l_cap;
  int64_t row[2];
  uint4 code[2][2];
  float scale[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t j = j0 + 32 * i, pos = L - n + j;
    row[i] = bad_len || pos < 0 || j >= n ? -1 : cache_row(a.c, b, g, pos);
    if (row[i] >= 0) {
      code[i][0] = *reinterpret_cast<const uint4*>(a.c.k + row[i] * kD + 16 * l);
      code[i][1] = *reinterpret_cast<const uint4*>(a.c.v + row[i] * kD + 16 * l);
      scale[i][0] = a.c.ks[row[i] >> a.c.block_shift];
      scale[i][1] = a.c.vs[row[i] >> a.c.block_shift];
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t j = j0 + 32 * i, pos = L - n + j, t = tok + j;
    if (j >= n) break;
    const bool nan = row[i] < 0 && (bad_len || pos >= 0);
    if (nan && l == 0 && a.status) atomicOr(a.status, kStatusBadLength);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const RowsView& out = w ? a.v : a.k;
      const uint32_t blank = nan ? 0x7fff7fffu : 0u;
      uint4 lo = make_uint4(blank, blank, blank, blank), hi = lo;
      if (row[i] >= 0) {
        float x[8];
        decode8<FMT>(make_uint2(code[i][w].x, code[i][w].y), scale[i][w], x);
        lo = pack8(x);
        decode8<FMT>(make_uint2(code[i][w].z, code[i][w].w), scale[i][w], x);
        hi = pack8(x);
      }
      uint4* to = reinterpret_cast<uint4*>(out.p + t * out.st + g * out.sh + 16 * l);
      to[0] = lo;
      to[1] = hi;
    }
  }
}

template <int FMT, int BLK, int KIND>
cudaError_t append_kind(const AppendArgs& a, cudaStream_t st) {
  constexpr int THREADS = append_threads(BLK), TEAMS = THREADS / 32 / (BLK / 16);
  // blocks that a sequence can touch
  const int nb = (int)(((a.max_new < a.T ? a.max_new : a.T) + BLK - 2) / BLK + 1);
  const dim3 grid((unsigned)(((int64_t)nb * 2 * a.c.Hkv + TEAMS - 1) / TEAMS), a.B);
  return launch_dependent(kv8_append_kernel<FMT, BLK, KIND>, grid, dim3(THREADS), 0, st, a, nb);
}

template <int FMT, int BLK>
cudaError_t append_block(const AppendArgs& a, cudaStream_t st) {
  if (!a.rope.lo) return append_kind<FMT, BLK, kStraight>(a, st);
  return a.rope.interleaved ? append_kind<FMT, BLK, kTurnInterleaved>(a, st)
                            : append_kind<FMT, BLK, kTurnHalf>(a, st);
}

template <int FMT>
cudaError_t append_fmt(const AppendArgs& a, cudaStream_t st) {
  switch (a.block) {
    case 16: return append_block<FMT, 16>(a, st);
    case 32: return append_block<FMT, 32>(a, st);
    case 64: return append_block<FMT, 64>(a, st);
    default: return append_block<FMT, 128>(a, st);
  }
}

}  // namespace

cudaError_t launch_kv8_append(const AppendArgs& a, cudaStream_t st) {
  return a.fmt == kFmtInt8 ? append_fmt<kFmtInt8>(a, st) : append_fmt<kFmtE4m3>(a, st);
}

cudaError_t launch_kv8_read(const ReadArgs& a, cudaStream_t st) {
  const int64_t most = a.max_new < a.T ? a.max_new : a.T;
  const dim3 grid((unsigned)((most + kReadRows - 1) / kReadRows), a.c.Hkv, a.B), th(256);
  return a.fmt == kFmtInt8 ? launch_dependent(kv8_read_kernel<kFmtInt8>, grid, th, 0, st, a)
                           : launch_dependent(kv8_read_kernel<kFmtE4m3>, grid, th, 0, st, a);
}

}  // namespace tsa
