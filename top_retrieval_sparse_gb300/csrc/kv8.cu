// kv8.cu -- the 8-bit KV cache: written (with the keys' rotation) and read.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "rope.cuh"

namespace tsa {

namespace {

constexpr int kAppendThreads = 256;                // 16 half-warps, a row each
constexpr int kAppendRows = kAppendThreads / 16;

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

template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = x[e] * inv;
    if (FMT == kFmtInt8) {
      int c = __float2int_rn(y);  // infinities saturate, NaN gives 0
      c = c < -127 ? -127 : (c > 127 ? 127 : c);
      b[e] = (uint32_t)(c + 128);
    } else {
      b[e] = __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
    }
  }
  return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24,
                    b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
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

// One CTA per (touched block, KV head and K or V, sequence): the new rows of
// the block stay in registers between the search for their largest magnitude
// and their coding.
template <int FMT, int BLK>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(AppendArgs a) {
  constexpr int NR = (BLK + kAppendRows - 1) / kAppendRows;
  __shared__ float red[kAppendThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, g = blockIdx.y >> 1, which = blockIdx.y & 1;
  int64_t tok, n;
  const int64_t L = a.lens[b];
  const bool good = seq_tokens(a.cu, a.max_new, a.T, b, tok, n);
  if (!good || L < n || L > a.c.l_cap) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
    return;
  }
  if (n == 0) return;
  const int64_t start = L - n;
  const int64_t p0 = (start / BLK + blockIdx.x) * BLK;  // the block's first position
  if (p0 >= L) return;
  const int64_t row0 = cache_row(a.c, b, g, p0);
  if (row0 < 0) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
    return;
  }
  const int hw = threadIdx.x >> 4, c = threadIdx.x & 15;
  const uint32_t mask = 0xffffu << (threadIdx.x & 16);
  const RowsView& in = which ? a.v : a.k;
  uint8_t* codes = which ? a.c.v : a.c.k;
  float* scales = which ? a.c.vs : a.c.ks;
  const bool turn = !which && a.rope.lo != nullptr;
  const int pair = turn ? rope_pair(a.rope, c) : -1;
  float x[NR][8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int64_t pos = p0 + hw + i * kAppendRows;
    const bool mine = pos >= start && pos < L && (BLK >= kAppendRows || hw < BLK);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    const int64_t t = tok + pos - start;
    if (mine) w = *reinterpret_cast<const uint4*>(in.p + t * in.st + g * in.sh + 8 * c);
    unpack8(w, x[i]);
    if (turn) {
      float2 cs[8];
      const int64_t at = !mine ? 0 : (a.positions ? (int64_t)a.positions[t] : pos);
      if (mine && c == 0 && a.status && (at < 0 || at >= a.rope.max_pos))
        atomicOr(a.status, kStatusBadLength);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        cs[e] = mine && pair >= 0 && pair + e < a.rope.pairs ? rope_angle(a.rope, at, pair + e)
                                                             : make_float2(1.f, 0.f);
      rope_turn(a.rope, c, mask, cs, x[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = fabsf(x[i][e]);
      if (mine && m <= 3.402823466e38f) amax = fmaxf(amax, m);
    }
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  const float had = scales[row0 / BLK];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, red[i]);
  const float need = scale_for(amax, FMT);
  const bool shared_block = p0 < start;  // older rows live in it
  const float s = shared_block ? fmaxf(had, need) : need;
  const float inv = 1.f / s;             // exact: a power of two
  if (shared_block && s != had) {        // grown: the older rows once more
    for (int64_t r = hw; r < start - p0; r += kAppendRows) {
      uint2* at = reinterpret_cast<uint2*>(codes + (row0 + r) * kD + 8 * c);
      float y[8];
      decode8<FMT>(*at, had, y);
      *at = encode8<FMT>(y, inv);
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int64_t r = hw + i * kAppendRows, pos = p0 + r;
    if (pos >= start && pos < L && (BLK >= kAppendRows || hw < BLK))
      *reinterpret_cast<uint2*>(codes + (row0 + r) * kD + 8 * c) = encode8<FMT>(x[i], inv);
  }
  if (threadIdx.x == 0) scales[row0 / BLK] = s;
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

template <int FMT>
cudaError_t append_fmt(const AppendArgs& a, cudaStream_t st) {
  const int nb = (int)(((int64_t)a.max_new + a.block - 2) / a.block + 1);
  const dim3 grid(nb, 2 * a.c.Hkv, a.B), th(kAppendThreads);
  switch (a.block) {
    case 16: return launch_dependent(kv8_append_kernel<FMT, 16>, grid, th, 0, st, a);
    case 32: return launch_dependent(kv8_append_kernel<FMT, 32>, grid, th, 0, st, a);
    case 64: return launch_dependent(kv8_append_kernel<FMT, 64>, grid, th, 0, st, a);
    default: return launch_dependent(kv8_append_kernel<FMT, 128>, grid, th, 0, st, a);
  }
}

}  // namespace

cudaError_t launch_kv8_append(const AppendArgs& a, cudaStream_t st) {
  return a.fmt == kFmtInt8 ? append_fmt<kFmtInt8>(a, st) : append_fmt<kFmtE4m3>(a, st);
}

cudaError_t launch_kv8_read(const ReadArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)a.max_new + 15) / 16), a.c.Hkv, a.B), th(256);
  return a.fmt == kFmtInt8 ? launch_dependent(kv8_read_kernel<kFmtInt8>, grid, th, 0, st, a)
                           : launch_dependent(kv8_read_kernel<kFmtE4m3>, grid, th, 0, st, a);
}

}  // namespace tsa
