// attn_plain.cu -- attention over the rows that window and sinks leave
// visible, one warp per (token, query head), 32-bit throughout.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cache_ops.h"

namespace tsa {

namespace {

template <int FMT>
__device__ __forceinline__ void load4(const uint8_t* base, int64_t row, int lane, float (&x)[4]) {
  if (FMT == kFmtBf16) {
    const uint2 w = *reinterpret_cast<const uint2*>(base + row * (2 * kD) + 8 * lane);
    x[0] = bf_lo(w.x); x[1] = bf_hi(w.x); x[2] = bf_lo(w.y); x[3] = bf_hi(w.y);
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(base + row * kD + 4 * lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t u = (w >> (8 * e)) & 0xffu;
      x[e] = FMT == kFmtInt8
                 ? (float)((int)u - 128)
                 : __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)u, __NV_E4M3)));
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) attn_plain_kernel(AttnArgs a) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t j = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int h = blockIdx.y, b = blockIdx.z;
  int64_t tok = b, n = 1;
  bool bad = false;
  if (a.max_q > 0 && !seq_tokens(a.cu, a.max_q, a.T, b, tok, n)) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadLength);
    if (tok < 0 || n < 0 || tok + n > a.T) return;
    if (n > a.max_q) n = a.max_q;
    bad = true;
  }
  if (j >= n) return;
  int64_t L = a.lens[b];
  if (L < 0 || L > a.c.l_cap) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadLength);
    L = L < 0 ? 0 : a.c.l_cap;
  }
  const int64_t end = L - n + j + 1;  // rows [0, end) are at or before the query
  const int g = h / (a.Hq / a.c.Hkv);
  const int64_t t = tok + j;
  float q[4];
  {
    const uint2 w =
        *reinterpret_cast<const uint2*>(a.q.p + t * a.q.st + h * a.q.sh + 4 * lane);
    q[0] = bf_lo(w.x); q[1] = bf_hi(w.x); q[2] = bf_lo(w.y); q[3] = bf_hi(w.y);
  }
  // Sums of 256 rows first, then of those: one running sum over a long cache
  // would lose what a row adds to it.
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  float l1 = 0.f, o1[4] = {0.f, 0.f, 0.f, 0.f};
  int rows = 0;
  if (end > 0) {
    const int64_t n0 = a.n_init < end ? a.n_init : end;
    int64_t lo = end - a.n_recent;
    if (lo < n0) lo = n0;
    for (int64_t i = 0; i < end; ++i) {
      if (i == n0) i = lo;
      if (i >= end) break;
      const int64_t row = cache_row(a.c, b, g, i);
      if (row < 0) {
        bad = true;
        break;
      }
      float k[4], v[4];
      load4<FMT>(a.c.k, row, lane, k);
      load4<FMT>(a.c.v, row, lane, v);
      float z = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * a.scale_log2;
      float sv = 1.f;
      if (FMT != kFmtBf16) {
        z *= a.c.ks[row >> a.c.block_shift];
        sv = a.c.vs[row >> a.c.block_shift];
      }
      const float mn = fmaxf(m, z);
      const float f = exp2f(m - mn), p = exp2f(z - mn);
      const bool fold = (++rows & 255) == 0;
      m = mn;
      l1 = l1 * f + p;
      l *= f;
      if (fold) l += l1, l1 = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o1[e] = o1[e] * f + p * sv * v[e];
        o[e] *= f;
        if (fold) o[e] += o1[e], o1[e] = 0.f;
      }
    }
  }
  l += l1;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] += o1[e];
  const float inv = bad ? nanf("") : (l > 0.f ? 1.f / l : 0.f);
  if (bad && lane == 0) atomicOr(a.status, kStatusBadLength);
  const int64_t at = (t * a.Hq + h) * kD + 4 * lane;
  if (a.out32) {
    *reinterpret_cast<float4*>(a.out32 + at) =
        make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  } else {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(a.out16 + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (a.lse && lane == 0)
    a.lse[t * a.Hq + h] = bad ? nanf("") : (l > 0.f ? (m + log2f(l)) * 0.6931471805599453f
                                                    : -INFINITY);
}

}  // namespace

cudaError_t launch_attn_plain(const AttnArgs& a, cudaStream_t st) {
  const dim3 grid(a.max_q > 0 ? (a.max_q + 7) / 8 : 1, a.Hq, a.B), th(256);
  if (a.fmt == kFmtInt8) return launch_dependent(attn_plain_kernel<kFmtInt8>, grid, th, 0, st, a);
  if (a.fmt == kFmtE4m3) return launch_dependent(attn_plain_kernel<kFmtE4m3>, grid, th, 0, st, a);
  return launch_dependent(attn_plain_kernel<kFmtBf16>, grid, th, 0, st, a);
}

}  // namespace tsa
