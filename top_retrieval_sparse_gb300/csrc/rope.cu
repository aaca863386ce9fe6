// rope.cu -- rotary positions: the angle table and the rotation of q and k.
#include "rope.cuh"

namespace tsa {

namespace {

__global__ void rope_table_kernel(RopeTableArgs a) {
  const int64_t n = (int64_t)(kRopeLow + a.n_hi) * a.pairs;
  for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n;
       e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = e / a.pairs;
    const int i = (int)(e % a.pairs);
    const bool low = row < kRopeLow;
    const double t = low ? (double)row : (double)(row - kRopeLow) * kRopeLow;
    double s, c;
    sincos(t * a.w[i], &s, &c);
    const double m = low ? a.amplitude : 1.0;
    const float2 v = make_float2((float)(c * m), (float)(s * m));
    if (low)
      a.lo[e] = v;
    else
      a.hi[e - (int64_t)kRopeLow * a.pairs] = v;
  }
}

constexpr int kRopeThreads = 256;

// One CTA per token: 64 threads combine the token's angles once, then every
// half-warp turns rows.  It does not let the next kernel start early: the
// key scan reads q and the keys before its dependency wait.
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  __shared__ float2 cs_s[kD / 2];
  pdl_wait();
  const int64_t t = blockIdx.x;
  if (threadIdx.x < a.rope.pairs) {
    float2 v = rope_angle(a.rope, a.positions[t], threadIdx.x);
    if (a.inverse) v.y = -v.y;
    cs_s[threadIdx.x] = v;
  }
  __syncthreads();
  const int c = threadIdx.x & 15;
  const uint32_t mask = 0xffffu << (threadIdx.x & 16);
  const int p0 = rope_pair(a.rope, c);
  float2 cs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    cs[e] = p0 >= 0 && p0 + e < a.rope.pairs ? cs_s[p0 + e] : make_float2(1.f, 0.f);
  for (int h = threadIdx.x >> 4; h < a.Hq + a.Hkv; h += kRopeThreads / 16) {
    const bool isq = h < a.Hq;
    const RowsView& in = isq ? a.q : a.k;
    const RowsView& out = isq ? a.qo : a.ko;
    const int hh = isq ? h : h - a.Hq;
    float x[8];
    unpack8(*reinterpret_cast<const uint4*>(in.p + t * in.st + hh * in.sh + 8 * c), x);
    rope_turn(a.rope, c, mask, cs, x);
    *reinterpret_cast<uint4*>(out.p + t * out.st + hh * out.sh + 8 * c) = pack8(x);
  }
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t st) {
  const int64_t n = (int64_t)(kRopeLow + a.n_hi) * a.pairs;
  int64_t grid = (n + 255) / 256;
  if (grid > 2048) grid = 2048;
  rope_table_kernel<<<(unsigned)grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  return launch_dependent(rope_kernel, dim3((unsigned)a.T), dim3(kRopeThreads), 0, st, a);
}

}  // namespace tsa
