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
    const int64_t at = row * a.pairs + rope_place(i, a.pairs);
    const bool low = row < kRopeLow;
    const double t = low ? (double)row : (double)(row - kRopeLow) * kRopeLow;
    double s, c;
    sincos(t * a.w[i], &s, &c);
    const double m = low ? a.amplitude : 1.0;
    const float2 v = make_float2((float)(c * m), (float)(s * m));
    if (low)
      a.lo[at] = v;
    else
      a.hi[at - (int64_t)kRopeLow * a.pairs] = v;
  }
}

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 5;   // rows of eight lanes in flight

// Bandwidth-bound: 2 bytes read and written an element for 3 flop.  Eight lanes
// keep their token's angles in registers (8 pairs a lane) and turn every WAYS-th
// head of it, kRopeBatch rows in flight at a time: with four tokens a CTA the angles, 1
// KB of table from L2, serve 40 rows of 512 bytes moved; with one (few tokens) a
// token's heads are spread over the whole CTA.  A lane holds both elements of its
// pairs, so no values change lanes.  A prompt of 32768 tokens, 32 + 8 heads: 113 us,
// 5.9 TB/s (144 us with 16 lanes a row and shuffles).  It does not let the next kernel start
// early: the key scan reads q and the keys before its dependency wait.  Three axes, 32767
// tokens: 121 us (155 us where every lane loaded its own eight pairs' angles).
template <int TOKENS, bool INTER, bool AXES>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  constexpr int WAYS = kRopeThreads / 8 / TOKENS;
  // Several axes: neighbouring pairs may turn by different positions, so a thread finds one
  // pair's angle of the CTA's tokens, and the lanes take theirs from here, in the order of
  // the table's rows.
  __shared__ float4 angle_s[AXES ? TOKENS : 1][kD / 4];
  pdl_wait();
  const int slot = threadIdx.x >> 3;
  const int64_t t = (int64_t)blockIdx.x * TOKENS + slot / WAYS;
  if (AXES) {
    for (int i = threadIdx.x; i < TOKENS * a.rope.pairs; i += kRopeThreads) {
      const int token = i / a.rope.pairs, pair = i - token * a.rope.pairs;
      const int64_t at = (int64_t)blockIdx.x * TOKENS + token;
      if (at < a.T) {
        const uint32_t axis = a.axes.of[pair >> 3] >> (2 * (pair & 7)) & 3u;
        reinterpret_cast<float2*>(angle_s[token])[rope_place(pair, kD / 2)] =
            rope_angle(a.rope, a.positions[at + axis * a.axes.stride], pair);
      }
    }
    __syncthreads();
  }
  if (t >= a.T) return;
  const int H = a.Hq + a.Hkv;
  const RopeLane ln = rope_lane(a.rope, threadIdx.x & 7);
  const uint16_t* qi = a.q.p + t * a.q.st + 8 * ln.a;
  const uint16_t* ki = a.k.p + t * a.k.st + 8 * ln.a;
  uint16_t* qo = a.qo.p + t * a.qo.st + 8 * ln.a;
  uint16_t* ko = a.ko.p + t * a.ko.st + 8 * ln.a;
  const int second = 8 * (ln.b - ln.a);
  float2 cs[8];
  if (ln.pair >= 0) {
    if (AXES) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 x = angle_s[slot / WAYS][8 * e + (threadIdx.x & 7)];
        cs[2 * e] = make_float2(x.x, x.y);
        cs[2 * e + 1] = make_float2(x.z, x.w);
      }
    } else {
      rope_angles(a.rope, a.positions[t], threadIdx.x & 7, cs);
    }
    if (a.inverse)
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e].y = -cs[e].y;
  }
  for (int h0 = slot % WAYS; h0 < H; h0 += WAYS * kRopeBatch) {
    uint4 w[kRopeBatch][2];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int h = h0 + i * WAYS;
      if (h < H) {
        const uint16_t* p = h < a.Hq ? qi + h * a.q.sh : ki + (h - a.Hq) * a.k.sh;
        w[i][0] = *reinterpret_cast<const uint4*>(p);
        w[i][1] = *reinterpret_cast<const uint4*>(p + second);
      }
    }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int h = h0 + i * WAYS;
      if (h < H) {
        if (ln.pair >= 0) {
          float x[8], y[8];
          unpack8(w[i][0], x);
          unpack8(w[i][1], y);
          rope_turn(INTER, cs, x, y);
          w[i][0] = pack8(x);
          w[i][1] = pack8(y);
        }
        uint16_t* p = h < a.Hq ? qo + h * a.qo.sh : ko + (h - a.Hq) * a.ko.sh;
        *reinterpret_cast<uint4*>(p) = w[i][0];
        *reinterpret_cast<uint4*>(p + second) = w[i][1];
      }
    }
  }
}

template <bool INTER, bool AXES>
cudaError_t launch_layout(const RopeArgs& a, cudaStream_t st) {
  // Four tokens a CTA from two CTAs an SM on; below that latency counts.
  const dim3 th(kRopeThreads);
  if (a.T < 4 * 2 * 152)
    return launch_dependent(rope_kernel<1, INTER, AXES>, dim3((unsigned)a.T), th, 0, st, a);
  return launch_dependent(rope_kernel<4, INTER, AXES>, dim3((unsigned)((a.T + 3) / 4)), th, 0, st,
                          a);
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
  if (a.axes.n > 0)
    return a.rope.interleaved ? launch_layout<true, true>(a, st) : launch_layout<false, true>(a, st);
  return a.rope.interleaved ? launch_layout<true, false>(a, st)
                            : launch_layout<false, false>(a, st);
}

}  // namespace tsa
