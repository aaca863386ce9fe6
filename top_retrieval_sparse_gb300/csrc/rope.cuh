// rope.cuh -- the rotation of one head row by a half-warp: lane c of 16 holds
// elements [8c, 8c + 8).
#pragma once

#include "cache_ops.h"

namespace tsa {

// cos and sin of position t, pair i: the sum of the two table angles,
// (cos(x + y), sin(x + y)) from (cos x, sin x) and (cos y, sin y).  Each factor
// is within half a step of 32 bits, so each result is within about 2^-23.
__device__ __forceinline__ float2 rope_angle(const RopeView& r, int64_t t, int i) {
  if (t < 0 || t >= r.max_pos) return make_float2(nanf(""), nanf(""));
  const float2 a = r.lo[(t & (kRopeLow - 1)) * r.pairs + i];
  const float2 b = r.hi[(t >> kRopeLowBits) * r.pairs + i];
  return make_float2(a.x * b.x - a.y * b.y, a.y * b.x + a.x * b.y);
}

// First pair of lane c's chunk; -1: the chunk is past rot_dim.
__device__ __forceinline__ int rope_pair(const RopeView& r, int c) {
  const int n8 = r.pairs >> 3;
  if (c >= 2 * n8) return -1;
  return r.interleaved ? 4 * c : 8 * (c < n8 ? c : c - n8);
}

// Rotates the row: x is lane c's chunk; cs[e] the (cos, sin) of pair
// rope_pair(c) + e (8 of them in the half layout, 4 in the interleaved one).
// All 16 lanes of the half-warp call it (mask: theirs).
__device__ __forceinline__ void rope_turn(const RopeView& r, int c, uint32_t mask,
                                          const float2 (&cs)[8], float (&x)[8]) {
  const int n8 = r.pairs >> 3;
  if (r.interleaved) {
    if (c < 2 * n8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = x[2 * e], b = x[2 * e + 1];
        x[2 * e] = a * cs[e].x - b * cs[e].y;
        x[2 * e + 1] = b * cs[e].x + a * cs[e].y;
      }
    }
    return;
  }
  const int src = c < n8 ? c + n8 : (c < 2 * n8 ? c - n8 : c);
  const float sgn = c < n8 ? -1.f : 1.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float o = __shfl_sync(mask, x[e], src, 16);
    if (c < 2 * n8) x[e] = x[e] * cs[e].x + sgn * (o * cs[e].y);
  }
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf_lo(u[e]);
    x[2 * e + 1] = bf_hi(u[e]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    u[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

}  // namespace tsa
