// rope.cuh -- the rotation of one head row by eight lanes.
#pragma once

#include "cache_ops.h"

namespace tsa {

// Place of pair i in a table row of n pairs: lane i / 8 of a row's lanes (below)
// takes its eight pairs as four pieces of 16 bytes, and the lanes' pieces of one load
// lie side by side.
__host__ __device__ __forceinline__ int rope_place(int i, int n) {
  return 2 * ((n >> 3) * ((i & 7) >> 1) + (i >> 3)) + (i & 1);
}

// The angles of two pairs from a piece of the low row and of the high row.
__device__ __forceinline__ void rope_sum(const float4& a, const float4& b, float2& c0,
                                         float2& c1) {
  c0 = make_float2(a.x * b.x - a.y * b.y, a.y * b.x + a.x * b.y);
  c1 = make_float2(a.z * b.z - a.w * b.w, a.w * b.z + a.z * b.w);
}

// cos and sin of position t for the eight pairs of lane l (l < pairs / 8): the sum
// of the two table angles, (cos(x + y), sin(x + y)) from (cos x, sin x) and (cos y,
// sin y).  Each factor is within half a step of 32 bits, so each result is within
// about 2^-23.
__device__ __forceinline__ void rope_angles(const RopeView& r, int64_t t, int l,
                                            float2 (&cs)[8]) {
  if (t < 0 || t >= r.max_pos) {
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = make_float2(nanf(""), nanf(""));
    return;
  }
  const int n8 = r.pairs >> 3;
  const float4* lo = reinterpret_cast<const float4*>(r.lo + (t & (kRopeLow - 1)) * r.pairs) + l;
  const float4* hi = reinterpret_cast<const float4*>(r.hi + (t >> kRopeLowBits) * r.pairs) + l;
#pragma unroll
  for (int e = 0; e < 4; ++e) rope_sum(lo[n8 * e], hi[n8 * e], cs[2 * e], cs[2 * e + 1]);
}

// A row is turned by eight lanes, 16 elements each as two pieces of 8 (lane l's
// pieces `a` and `b`, numbered in the row), such that a lane holds both elements of its
// eight pairs: the pieces of both halves in the half layout, neighbours in the
// interleaved one.  Lanes past rot_dim hold two pieces that are only copied
// (their pairs: -1).
struct RopeLane {
  int a, b, pair;
};
__device__ __forceinline__ RopeLane rope_lane(const RopeView& r, int l) {
  const int n8 = r.pairs >> 3;  // lanes that turn
  RopeLane x;
  x.pair = l < n8 ? 8 * l : -1;
  x.a = r.interleaved || l >= n8 ? 2 * l : l;
  x.b = r.interleaved || l >= n8 ? 2 * l + 1 : l + n8;
  return x;
}
__device__ __forceinline__ void rope_turn(bool interleaved, const float2 (&cs)[8], float (&x)[8],
                                          float (&y)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // pair e: (x_e, y_e), or elements 2e and 2e + 1 of x then y
    float& p = interleaved ? (e < 4 ? x[2 * (e & 3)] : y[2 * (e & 3)]) : x[e];
    float& q = interleaved ? (e < 4 ? x[2 * (e & 3) + 1] : y[2 * (e & 3) + 1]) : y[e];
    const float u = p, v = q;
    p = u * cs[e].x - v * cs[e].y;
    q = v * cs[e].x + u * cs[e].y;
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
