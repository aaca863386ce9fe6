// shared_attn.cu -- one decode step of a batch whose sequences share their first rows: what
// stands before and behind the attention kernels.
//
// Sequence b of group n attends over the group's rows [0, P_n), which lie in the cache of
// its first sequence, and over its own rows [P_n, L_b):
//   z_i = scale q_b.k_i,  out_b = sum_i e^z_i v_i / sum_i e^z_i
// The shared rows' part comes from shared_prefix.cu in partials, the own rows' from the
// decode kernel of attn_decode.cu; each carries its maximum and sum, and they are joined.
#include "shared_attn.h"

namespace tsa {

namespace {

constexpr int kPrepThreads = 1024;
constexpr int kMostGroups = 4096;

// Exclusive prefix over the block's threads, and the whole sum.
__device__ int64_t block_prefix(int64_t x, int64_t* scratch, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = y;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < kPrepThreads / 32; ++w) {
    if (w == warp) before = total;
    total += scratch[w];
  }
  return before + y - x;
}

// The groups' work in a list, and who shares what with whom (the first CTA); the decode
// kernel's counters cleared (the others).
__global__ void __launch_bounds__(kPrepThreads) shared_prep_kernel(SharedArgs a) {
  __shared__ int32_t cu_s[kMostGroups + 1];
  __shared__ int64_t scan_s[kPrepThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int B = a.B, N = a.N, Hkv = a.c.Hkv;
  if (blockIdx.x > 0) {
    const int64_t i = (int64_t)(blockIdx.x - 1) * kPrepThreads + tid;
    if (i < (int64_t)B * Hkv) a.arrived[i] = 0u;
    return;
  }
  for (int n = tid; n <= N; n += kPrepThreads) cu_s[n] = a.cu[n];
  __syncthreads();
  // The offsets must rise within [0, B].
  int bad = 0;
  for (int n = tid; n < N; n += kPrepThreads)
    bad |= cu_s[n] < 0 || cu_s[n] > cu_s[n + 1] || cu_s[n + 1] > B;
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(a.status, kStatusBadLength);
  int64_t cost = 0, rows = 0;
  int columns = 0, groups = 0;  // of groups with work
  for (int n0 = 0; n0 < N; n0 += kPrepThreads) {
    const int n = n0 + tid;
    SharedGroup s{};
    int64_t c = 0, r = 0, total;
    bool some = false;
    if (n < N && !bad) {
      const int P = a.shared[n];
      s.b0 = cu_s[n];
      s.P = P < 0 ? 0 : (P > a.c.l_cap ? (int)a.c.l_cap : P);
      s.rows = s.P > 0 ? (cu_s[n + 1] - cu_s[n]) * a.G : 0;
      if (P != s.P) atomicOr(a.status, kStatusBadLength);
      if (s.rows > 0) {
        const int last = (s.rows - 1) / kUnitRows;
        const int w = s.rows - last * kUnitRows > 128 ? kCostBoth : kCostAlone;
        c = (int64_t)((s.P + 127) / 128) * Hkv * ((int64_t)last * kCostBoth + w);
        r = group_rows(s.rows, Hkv);
        columns += last + 1;
        some = true;
      }
    }
    s.cost0 = cost + block_prefix(c, scan_s, total);
    cost += total;
    s.row0 = rows + block_prefix(r, scan_s, total);
    rows += total;
    if (n < N) a.groups[n] = s;
    groups += __syncthreads_count(some);
  }
  if (groups == 1 && columns > 0) {  // (the one thread that met it)
    // CTAs in step: a whole number of them for every column of queries, so that columns
    // read the same rows at the same time.  Kept where at most a tenth of the CTAs is idle.
    const int even = columns <= kSharedShares ? kSharedShares / columns * columns : 0;
    scan_s[0] = even * 10 >= kSharedShares * 9 ? even : kSharedShares;
  }
  if (groups != 1 && tid == 0) scan_s[0] = kSharedShares;
  __syncthreads();
  if (tid == 0) {
    int64_t shares = scan_s[0];
    if (shares > cost / kCostBoth) shares = cost / kCostBoth;
    a.total->cost = cost;
    a.total->shares = shares < 1 ? 1 : (int)shares;
  }
  for (int b = tid; b < B; b += kPrepThreads) {
    int n = -1, start = 0;
    if (bad) {
      n = kNoGroups;
    } else if (N > 0 && b >= cu_s[0] && b < cu_s[N]) {
      int lo = 0, hi = N;  // the last group that starts at or before b
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_s[mid] <= b) lo = mid; else hi = mid;
      }
      n = lo;
      const int P = a.shared[n], L = a.lens[b];
      start = P < 0 ? 0 : (P > a.c.l_cap ? (int)a.c.l_cap : P);
      if (L > 0 && L < start) atomicOr(a.status, kStatusBadLength);
      if (L < start) start = 0;  // nothing of the group's (the join knows)
    }
    a.group[b] = n;
    a.start[b] = start;
    if (a.leader) {
      a.leader[b] = n >= 0 ? cu_s[n] : b;
      a.zero[b] = 0;
    }
  }
}

// Four columns of a row (sequence, query head) a thread: the partials of the segments of its
// unit in the order of the list, then the own rows'.
__global__ void __launch_bounds__(256) shared_join_kernel(SharedArgs a) {
  pdl_wait();
  if (!a.out16) pdl_trigger();  // (bf16 outputs may be queries of a key scan)
  const int b = blockIdx.x, Hkv = a.c.Hkv, G = a.G;
  const int item = blockIdx.y * 256 + threadIdx.x;
  if (item >= a.Hq * 32) return;
  // neighbouring threads: a KV head's query heads, whose partials are neighbours
  const int h = item % G, c = item / G % 32, g = item / (32 * G);
  const int64_t row = (int64_t)b * a.Hq + g * G + h;
  const int n = a.group[b], L = a.lens[b];
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  bool nan = n == kNoGroups;
  auto add = [&](float pm, float pl, const float4* from) {
    if (pl == 0.f) return;  // (has seen nothing and left no sums)
    const float top = fmaxf(m, pm), f = m == -INFINITY ? 0.f : exp2f(m - top), e = exp2f(pm - top);
    const float4 x = *from;
    o = make_float4(fmaf(o.x, f, x.x * e), fmaf(o.y, f, x.y * e), fmaf(o.z, f, x.z * e),
                    fmaf(o.w, f, x.w * e));
    l = fmaf(l, f, pl * e);
    m = top;
  };
  if (n >= 0 && L > 0) {
    const int P = a.shared[n];
    nan |= L < P;
    if (L >= P && P > 0 && a.leader) {
      const float lse = a.sh_lse[row];
      add(lse * 1.4426950408889634f, lse == -INFINITY ? 0.f : (lse != lse ? lse : 1.f),
          reinterpret_cast<const float4*>(a.sh_out + row * kD) + c);
    } else if (L >= P && P > 0) {
      const SharedGroup s = a.groups[n];
      const SharedTotal t = *a.total;
      const int r0 = (b - s.b0) * G + h, column = r0 / kUnitRows, r = r0 - column * kUnitRows;
      const SharedUnit u = unit_of(s, Hkv, column, g);
      const bool both = u.both();
      const int64_t half = half_floats(u.rs);
      const int s0 = (int)(u.cost0 * t.shares / t.cost);
      for (int share = s0, j0 = 0; j0 < u.tiles; ++share) {
        const float* p = segment_parts(a, u, share, j0);
        if (both) {
          p += (r >> 7) * half;
          const float* stats = p + (int64_t)u.rs * kD + (r & 127);
          add(stats[0], stats[u.rs],
              reinterpret_cast<const float4*>(p) + (int64_t)c * u.rs + (r & 127));
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x, p += half) {
            const float* stats = p + (int64_t)u.rs * kD + r;
            add(stats[0], stats[u.rs], reinterpret_cast<const float4*>(p) + (int64_t)c * u.rs + r);
          }
        }
        const int64_t next = share_start(t, share + 1) - u.cost0;
        j0 = (int)((next + u.w - 1) / u.w);
      }
    }
  }
  {
    const float lse = a.own_lse[row];
    add(lse * 1.4426950408889634f, lse == -INFINITY ? 0.f : (lse != lse ? lse : 1.f),
        reinterpret_cast<const float4*>(a.own_out + row * kD) + c);
  }
  nan |= l != l;
  const float inv = nan ? nanf("") : (l > 0.f ? 1.f / l : 0.f);
  if (nan) o = make_float4(1.f, 1.f, 1.f, 1.f);
  o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
  if (a.out16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kD)[c] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kD)[c] = o;
  }
  if (a.lse && c == 0)
    a.lse[row] = nan ? inv : (l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY);
}

}  // namespace

cudaError_t launch_shared_prep(const SharedArgs& a, cudaStream_t st) {
  const int64_t counters = (int64_t)a.B * a.c.Hkv;
  const dim3 grid((unsigned)(1 + (counters + kPrepThreads - 1) / kPrepThreads));
  return launch_dependent(shared_prep_kernel, grid, dim3(kPrepThreads), 0, st, a);
}
cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t st) {
  const dim3 grid(a.B, (a.Hq * 32 + 255) / 256);
  return launch_dependent(shared_join_kernel, grid, dim3(256), 0, st, a);
}

}  // namespace tsa
