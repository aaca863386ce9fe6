// shared_attn.cu -- one decode step of a batch whose sequences share their first rows.
//
// Sequence b of group n attends over the group's rows [0, P_n), which lie in the cache of
// its first sequence, and over its own rows [P_n, L_b):
//   z_i = scale q_b.k_i,  out_b = sum_i e^z_i v_i / sum_i e^z_i
// The two parts are computed apart, each with its maximum and sum, and joined.
#include "cache_ops.h"

namespace tsa {

namespace {

// Who shares what with whom, and the decode kernel's counters cleared.
__global__ void __launch_bounds__(256) shared_prep_kernel(SharedArgs a) {
  pdl_wait();
  pdl_trigger();
  const int tid = blockIdx.x * 256 + threadIdx.x;
  const int B = a.B, N = a.N;
  // The offsets must rise within [0, B].
  int bad = 0;
  for (int n = threadIdx.x; n < N; n += 256)
    bad |= a.cu[n] < 0 || a.cu[n] > a.cu[n + 1] || a.cu[n + 1] > B;
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(a.status, kStatusBadLength);
  for (int64_t i = tid; i < (int64_t)B * a.c.Hkv; i += (int64_t)gridDim.x * 256) a.arrived[i] = 0u;
  const int b = tid;
  if (b >= B) return;
  int n = -1, start = 0, leader = b;
  if (bad) {
    n = kNoGroups;
  } else if (N > 0 && b >= a.cu[0] && b < a.cu[N]) {
    int lo = 0, hi = N;  // the last group that starts at or before b
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= b) lo = mid; else hi = mid;
    }
    n = lo;
    leader = a.cu[n];
    const int P = a.shared[n];
    start = P < 0 ? 0 : (P > a.c.l_cap ? (int)a.c.l_cap : P);
    const int L = a.lens[b];
    if (start != P || (L > 0 && L < start)) atomicOr(a.status, kStatusBadLength);
    if (L < start) start = 0;  // nothing of the group's (the join knows)
  }
  a.group[b] = n;
  a.start[b] = start;
  a.leader[b] = leader;
  a.zero[b] = 0;
  a.self[b] = b;
}

// A row (sequence, query head) a warp.
__global__ void __launch_bounds__(256) shared_join_kernel(SharedArgs a) {
  pdl_wait();
  if (!a.out16) pdl_trigger();  // (bf16 outputs may be queries of a key scan)
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)a.B * a.Hq) return;
  const int b = (int)(row / a.Hq), n = a.group[b];
  const float l0 = a.sh_lse[row], l1 = a.own_lse[row];
  const float m = fmaxf(l0, l1);
  float w0 = 0.f, w1 = 0.f, lse = -INFINITY;
  if (m != -INFINITY) {
    const float e0 = expf(l0 - m), e1 = expf(l1 - m);
    const float inv = 1.f / (e0 + e1);
    w0 = e0 * inv;
    w1 = e1 * inv;
    lse = m + logf(e0 + e1);
  }
  const float4 x = reinterpret_cast<const float4*>(a.sh_out + row * kD)[lane];
  const float4 y = reinterpret_cast<const float4*>(a.own_out + row * kD)[lane];
  float4 o = make_float4(x.x * w0 + y.x * w1, x.y * w0 + y.y * w1, x.z * w0 + y.z * w1,
                         x.w * w0 + y.w * w1);
  const int L = a.lens[b];
  bool nan = n == kNoGroups || l0 != l0 || l1 != l1;
  if (n >= 0 && L > 0) nan |= L < a.shared[n];
  if (nan) {
    lse = nanf("");
    o = make_float4(lse, lse, lse, lse);
  }
  if (a.out16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kD)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kD)[lane] = o;
  }
  if (a.lse && lane == 0) a.lse[row] = lse;
}

}  // namespace

cudaError_t launch_shared_prep(const SharedArgs& a, cudaStream_t st) {
  return launch_dependent(shared_prep_kernel, dim3((a.B + 255) / 256), dim3(256), 0, st, a);
}
cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.B * a.Hq;
  return launch_dependent(shared_join_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, a);
}

}  // namespace tsa
