// kv8.cu -- the 8-bit KV cache: written (with the keys' rotation) and read.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "rope.cuh"

namespace tsa {

namespace {

constexpr int kAppendThreads = 256;

// Smallest e >= -60 with top * 2^e >= amax (finite), top = 127 or 448:
// amax = m * 2^x with m in [1, 2) and top = 1.984375 * 2^6 or 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float amax, int fmt) {
  if (!(amax > 0.f)) return ldexpf(1.f, -60);
  int x;
  const float m = 2.f * frexpf(amax, &x);  // in [1, 2), amax = m * 2^(x - 1)
  --x;
  int e = fmt == kFmtInt8 ? (m <= 1.984375f ? x - 6 : x - 5) : (m <= 1.75f ? x - 8 : x - 7);
  if (e < -60) e = -60;
  return ldexpf(1.f, e);
}

// Codes of eight values.  int8: 1.5 * 2^23 + 128 is added, which rounds to whole
// numbers (ties to even) and leaves code + 128 in the low byte; infinities
// saturate and NaN becomes 0.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  if constexpr (FMT == kFmtInt8) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y = x[e] * inv;
      y = y == y ? fminf(fmaxf(y, -127.f), 127.f) : 0.f;
      b[e] = __float_as_uint(y + 12583040.f);
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

template <int FMT>
__device__ __forceinline__ void decode8(uint2 w, float scale, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = ((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 0xffu;
    if (FMT == kFmtInt8) {
      x[e] = (float)((int)b - 128) * scale;
    } else {
      const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
      x[e] = __half2float(__half(h)) * scale;
    }
  }
}

// Bandwidth-bound: a row's 256 bytes are read once and written as 128.  The new
// rows of one (block, KV head, K or V) stay in the registers of BLK / 16 warps (a team;
// 16 rows a warp, eight lanes a row, 128 bytes a lane in flight) between the search
// for their largest magnitude and their coding.  With ROT the keys' angles are the same for
// every KV head, so a CTA puts those of the block's rows into shared memory once
// and its teams go through `heads` heads; blockIdx.x < nb is then the keys of block
// blockIdx.x, and the rest are the values, a team each, as without a rotation.
template <int FMT, int BLK, bool ROT>
__global__ void __launch_bounds__(kAppendThreads, ROT ? 2 : 3)
    kv8_append_kernel(AppendArgs a, int nb, int heads) {
  constexpr int TW = BLK / 16, TEAMS = kAppendThreads / 32 / TW;
  extern __shared__ float2 angle_s[];       // [BLK][pairs] (ROT)
  __shared__ float red[kAppendThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, Hkv = a.c.Hkv;
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

  // This CTA's items: (block, head, K or V) of its teams.
  const int parts = (Hkv + heads - 1) / heads;        // CTAs of a block's keys
  const bool turn = ROT && (int)blockIdx.x < nb * parts;
  int64_t j = 0;                                      // block, counted from start's
  int g0 = 0, g1 = 0, which = 0;                      // team's heads: g0, g0 + TEAMS, ... < g1
  if (turn) {
    j = blockIdx.x / parts;
    g0 = (blockIdx.x % parts) * heads;
    g1 = g0 + heads < Hkv ? g0 + heads : Hkv;
    g0 += team;
  } else {
    // item i: head i % Hkv of block i / Hkv; K then V within a block without ROT
    const int64_t i = (int64_t)(blockIdx.x - (ROT ? nb * parts : 0)) * TEAMS + team;
    which = ROT ? 1 : (int)((i / Hkv) & 1);
    j = ROT ? i / Hkv : i / (2 * Hkv);
    g0 = (int)(i % Hkv);
    g1 = g0 + 1;
  }
  const int64_t p0 = (start / BLK + j) * BLK;         // the block's first position
  const bool any = j < nb && p0 < L;
  RopeLane ln = {2 * l, 2 * l + 1, -1};
  if (ROT && turn) {
    if (!any) return;                                 // the whole CTA: one block
    ln = rope_lane(a.rope, l);
    for (int e = threadIdx.x; e < BLK * a.rope.pairs; e += kAppendThreads) {
      const int64_t pos = p0 + e / a.rope.pairs;
      if (pos < start || pos >= L) continue;
      const int64_t at = a.positions ? (int64_t)a.positions[tok + pos - start] : pos;
      angle_s[e] = rope_angle(a.rope, at, e % a.rope.pairs);
      if ((at < 0 || at >= a.rope.max_pos) && a.status) atomicOr(a.status, kStatusBadLength);
    }
    __syncthreads();
  }
  const RowsView& in = which ? a.v : a.k;
  uint8_t* codes = which ? a.c.v : a.c.k;
  float* scales = which ? a.c.vs : a.c.ks;
  const int turns = ROT && turn ? (heads + TEAMS - 1) / TEAMS : 1;
  for (int it = 0; it < turns; ++it) {
    const int g = g0 + it * TEAMS;
    int64_t row0 = -1;
    if (any && g < g1) {
      row0 = cache_row(a.c, b, g, p0);
      if (row0 < 0 && lane == 0 && a.status) atomicOr(a.status, kStatusBadLength);
    }
    const bool live = row0 >= 0;
    float x[ROT ? 4 : 1][16];  // rotated rows; without ROT they are widened again below
    float amax = 0.f, had = 0.f;
    uint4 w[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t pos = p0 + row_in + 4 * i;
      w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (live && pos >= start && pos < L) {
        const uint16_t* p = in.p + (tok + pos - start) * in.st + g * in.sh;
        w[i][0] = *reinterpret_cast<const uint4*>(p + 8 * ln.a);
        w[i][1] = *reinterpret_cast<const uint4*>(p + 8 * ln.b);
      }
    }
    if (live) had = scales[row0 / BLK];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u[8], v[8];
      unpack8(w[i][0], u);
      unpack8(w[i][1], v);
      if (ROT && turn) {
        const int64_t pos = p0 + row_in + 4 * i;
        if (live && ln.pair >= 0 && pos >= start && pos < L) {
          float2 cs[8];
          const float4* at =
              reinterpret_cast<const float4*>(angle_s + (row_in + 4 * i) * a.rope.pairs + ln.pair);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 q = at[e];
            cs[2 * e] = make_float2(q.x, q.y);
            cs[2 * e + 1] = make_float2(q.z, q.w);
          }
          if (a.rope.interleaved)
            rope_turn(true, cs, u, v);
          else
            rope_turn(false, cs, u, v);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (ROT) {
          x[i][e] = u[e];
          x[i][8 + e] = v[e];
        }
        const float mu = fabsf(u[e]), mv = fabsf(v[e]);
        if (mu <= 3.402823466e38f) amax = fmaxf(amax, mu);
        if (mv <= 3.402823466e38f) amax = fmaxf(amax, mv);
      }
    }
    amax = warp_max(amax);
    if (TW > 1) {
      __syncthreads();  // the turn before has read red
      if (lane == 0) red[warp] = amax;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TW; ++i) amax = fmaxf(amax, red[team * TW + i]);
    }
    if (!live) continue;
    const float need = scale_for(amax, FMT);
    const bool older = p0 < start;         // older rows live in the block
    const float s = older ? fmaxf(had, need) : need;
    const float inv = 1.f / s;             // exact: a power of two
    if (older && s != had) {               // grown: the older rows once more
      for (int64_t r = row_in; r < start - p0 && r < (warp % TW) * 16 + 16; r += 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint2* at = reinterpret_cast<uint2*>(codes + (row0 + r) * kD + 8 * (h ? ln.b : ln.a));
          float y[8];
          decode8<FMT>(*at, had, y);
          *at = encode8<FMT>(y, inv);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = row_in + 4 * i, pos = p0 + r;
      if (pos >= start && pos < L) {
        float u[8], v[8];
        if constexpr (ROT) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            u[e] = x[i][e];
            v[e] = x[i][8 + e];
          }
        } else {
          unpack8(w[i][0], u);
          unpack8(w[i][1], v);
        }
        const uint2 cu = encode8<FMT>(u, inv), cv = encode8<FMT>(v, inv);
        uint8_t* at = codes + (row0 + r) * kD;
        if (ln.b == ln.a + 1) {
          *reinterpret_cast<uint4*>(at + 8 * ln.a) = make_uint4(cu.x, cu.y, cv.x, cv.y);
        } else {
          *reinterpret_cast<uint2*>(at + 8 * ln.a) = cu;
          *reinterpret_cast<uint2*>(at + 8 * ln.b) = cv;
        }
      }
    }
    // (every lane of the team has read `had` before the barriers above; a team of
    // one warp is in step)
    __syncwarp();
    if (warp % TW == 0 && lane == 0) scales[row0 / BLK] = s;
  }
}

// A half-warp per (token, KV head).  No early start for the next kernel: what
// is read back may be a cache that the key scan streams before its wait.
template <int FMT>
__global__ void __launch_bounds__(256) kv8_read_kernel(ReadArgs a) {
  pdl_wait();
  const int b = blockIdx.z, g = blockIdx.y;
  const int c = threadIdx.x & 15;
  int64_t tok, n;
  const bool good = seq_tokens(a.cu, a.max_new, a.T, b, tok, n);
  const int64_t j = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (!good) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
    if (tok < 0 || tok + n > a.T) return;
    n = n < 0 ? 0 : (n > a.max_new ? a.max_new : n);
  }
  if (j >= n) return;
  const int64_t L = a.lens[b];
  const int64_t pos = L - n + j;
  const bool bad_len = !good || L < 0 || L > a.c.l_cap;
  const int64_t row = bad_len || pos < 0 ? -1 : cache_row(a.c, b, g, pos);
  uint4 wk = make_uint4(0u, 0u, 0u, 0u), wv = wk;
  if (row >= 0) {
    float x[8];
    decode8<FMT>(*reinterpret_cast<const uint2*>(a.c.k + row * kD + 8 * c),
                 a.c.ks[row >> a.c.block_shift], x);
    wk = pack8(x);
    decode8<FMT>(*reinterpret_cast<const uint2*>(a.c.v + row * kD + 8 * c),
                 a.c.vs[row >> a.c.block_shift], x);
    wv = pack8(x);
  } else if (bad_len || pos >= 0) {
    wk = wv = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
    if (c == 0 && a.status) atomicOr(a.status, kStatusBadLength);
  }
  const int64_t t = tok + j;
  *reinterpret_cast<uint4*>(a.k.p + t * a.k.st + g * a.k.sh + 8 * c) = wk;
  *reinterpret_cast<uint4*>(a.v.p + t * a.v.st + g * a.v.sh + 8 * c) = wv;
}

template <int FMT, int BLK>
cudaError_t append_block(const AppendArgs& a, cudaStream_t st) {
  constexpr int TEAMS = kAppendThreads / 32 / (BLK / 16);
  const int Hkv = a.c.Hkv;
  // blocks that a sequence can touch
  const int nb = (int)(((a.max_new < a.T ? a.max_new : a.T) + BLK - 2) / BLK + 1);
  const dim3 th(kAppendThreads);
  if (!a.rope.lo) {
    const dim3 grid((unsigned)(((int64_t)nb * 2 * Hkv + TEAMS - 1) / TEAMS), a.B);
    return launch_dependent(kv8_append_kernel<FMT, BLK, false>, grid, th, 0, st, a, nb, 1);
  }
  // All heads of a block's keys in one CTA where the blocks fill the machine,
  // else a turn of the teams a CTA (single tokens: latency counts).
  const int heads = (int64_t)nb * a.B >= 4 * 152 || Hkv < TEAMS ? Hkv : TEAMS;
  const int parts = (Hkv + heads - 1) / heads;
  const dim3 grid((unsigned)(nb * parts + ((int64_t)nb * Hkv + TEAMS - 1) / TEAMS), a.B);
  const size_t smem = (size_t)BLK * a.rope.pairs * sizeof(float2);
  const cudaError_t e =
      cudaFuncSetAttribute((const void*)kv8_append_kernel<FMT, BLK, true>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(BLK * kD * 4));
  if (e != cudaSuccess) return e;
  return launch_dependent(kv8_append_kernel<FMT, BLK, true>, grid, th, smem, st, a, nb, heads);
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
  const dim3 grid((unsigned)((most + 15) / 16), a.c.Hkv, a.B), th(256);
  return a.fmt == kFmtInt8 ? launch_dependent(kv8_read_kernel<kFmtInt8>, grid, th, 0, st, a)
                           : launch_dependent(kv8_read_kernel<kFmtE4m3>, grid, th, 0, st, a);
}

}  // namespace tsa
