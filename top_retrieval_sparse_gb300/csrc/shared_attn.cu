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

constexpr int kPrepThreads = 256;
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

// The segments of a share, in order: costs [at, end) of the list.
__device__ void list_share(const SharedArgs& a, const SharedTotal& t, int share) {
  const int Hkv = a.c.Hkv;
  int count = 0, first = 0;
  if (share < t.shares && t.cost > 0) {
    int64_t at = share_start(t, share);
    const int64_t end = share_start(t, share + 1);
    int n = 0;
    for (int hi = a.N; hi - n > 1;) {  // the last group that starts at or before `at`
      const int mid = (n + hi) >> 1;
      if (a.groups[mid].cost0 <= at) n = mid; else hi = mid;
    }
    SharedGroup s = a.groups[n];
    while (at < end) {
      const int64_t tiles = (s.P + 127) / 128, column = tiles * Hkv * kCostBoth;
      int64_t g = Hkv;
      SharedUnit u;
      if (s.rows > 0) {
        const int last = (s.rows - 1) / kUnitRows;  // all columns but this one are full
        int64_t k = over(at - s.cost0, column);
        if (k > last) k = last;
        const int w = s.rows - (int)k * kUnitRows > 128 ? kCostBoth : kCostAlone;
        g = over(at - s.cost0 - k * column, tiles * w);
        if (g < Hkv) u = unit_of(s, Hkv, (int)k, (int)g);
      }
      if (g >= Hkv) {
        if (++n >= a.N) break;
        s = a.groups[n];
        continue;
      }
      SharedSegment x;
      x.j0 = (int)over(at - u.cost0 + u.w - 1, u.w);
      const int64_t j1 = over(end - u.cost0 + u.w - 1, u.w);
      x.j1 = j1 < u.tiles ? (int)j1 : u.tiles;
      at = u.cost0 + (int64_t)u.tiles * u.w;
      if (x.j0 >= x.j1) continue;  // (begins behind the last tile's start)
      const int row = u.t * kUnitRows;
      x.b0 = s.b0;
      x.P = s.P;
      x.seq0 = s.b0 + row / a.G;
      x.in0 = row % a.G;
      x.g = u.g;
      x.rows = u.rows;
      x.rs = u.rs;
      x.both = u.both();
      x.copies = u.both() ? 1 : tile_copies(u.rows);
      x.part = segment_part(u, share, x.j0 == 0);
      const int number = share + s.unit0 + u.t * Hkv + u.g;
      if (count == 0) first = number;
      if (x.j0 == 0) a.spans[number - share].x = share;
      if (x.j1 == u.tiles) a.spans[number - share].y = share;
      a.segments[number] = x;
      ++count;
    }
  }
  a.total->segments[share] = make_int2(first, count);
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
    for (int64_t i = (int64_t)(blockIdx.x - 1) * kPrepThreads + tid; i < (int64_t)B * Hkv;
         i += (int64_t)(gridDim.x - 1) * kPrepThreads)
      a.arrived[i] = 0u;
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
  int64_t cost = 0, rows = 0, units = 0;
  int columns = 0, groups = 0;  // of groups with work
  for (int n0 = 0; n0 < N; n0 += kPrepThreads) {
    const int n = n0 + tid;
    SharedGroup s{};
    int64_t c = 0, r = 0, k = 0, total;
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
        k = (int64_t)(last + 1) * Hkv;
        some = true;
      }
    }
    s.cost0 = cost + block_prefix(c, scan_s, total);
    cost += total;
    s.row0 = rows + block_prefix(r, scan_s, total);
    rows += total;
    s.unit0 = (int)(units + block_prefix(k, scan_s, total));
    units += total;
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
  SharedTotal total;
  total.cost = cost;
  {
    int64_t shares = scan_s[0];
    if (shares > cost / kCostBoth) shares = cost / kCostBoth;
    total.shares = shares < 1 ? 1 : (int)shares;
  }
  if (tid == 0) {
    a.total->cost = total.cost;
    a.total->shares = total.shares;
  }
  if (!a.leader)
    for (int share = tid; share < kSharedShares; share += kPrepThreads) list_share(a, total, share);
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
      if (a.leader) a.leader[b] = cu_s[n];
      if (L > 0 && L < start) {
        atomicOr(a.status, kStatusBadLength);
        n = kNoGroups;
      }
      if (L < start) start = 0;
    }
    a.group[b] = n;
    a.start[b] = start;
    if (a.leader && n < 0) a.leader[b] = b;
  }
}

constexpr int kJoinThreads = 512;
constexpr int kMostParts = 2 * kSharedShares;

// A (sequence, KV head) a CTA.  First a warp a query head: the maxima and sums of the row's
// partials, lanes over them, and each one's weight.  Then four columns of a row a thread
// (neighbouring threads the query heads of one KV head, whose partials are neighbours), the
// loads of eight partials in flight; with few query heads several threads share the partials.
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(SharedArgs a) {
  __shared__ float weight_s[kMaxGroup][kMostParts];
  __shared__ int place_s[kMaxGroup][kMostParts];   // of the partial's columns, in pieces of 16 bytes
  __shared__ int count_s[kMaxGroup], rs_s[kMaxGroup];
  __shared__ float own_s[kMaxGroup], inv_s[kMaxGroup];
  __shared__ float4 sum_s[kJoinThreads];
  pdl_wait();
  if (!a.out16) pdl_trigger();  // (bf16 outputs may be queries of a key scan)
  const int b = blockIdx.x, g = blockIdx.y, Hkv = a.c.Hkv, G = a.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = a.group[b], L = a.lens[b];
  const int64_t row0 = (int64_t)b * a.Hq + g * G;
  if (warp < G) {
    const int h = warp;
    const float own_lse = a.own_lse[row0 + h];
    float m = -INFINITY, l = 0.f;
    int parts = 0, rs = 0;
    bool nan = n == kNoGroups;
    if (n >= 0 && L > 0) {
      const SharedGroup s = a.groups[n];
      if (s.rows > 0) {
        const int r0 = (b - s.b0) * G + h, column = r0 / kUnitRows, r = r0 - column * kUnitRows;
        const int2 shares = a.spans[s.unit0 + column * Hkv + g];
        const SharedUnit u = unit_of(s, Hkv, column, g);
        const bool both = u.both();
        const int half = (int)(half_floats(u.rs) / 4), s0 = shares.x;
        parts = (shares.y - s0 + 1) * (both ? 1 : 2);
        rs = u.rs;
        float l_all = 0.f;
        for (int e = lane; e < parts; e += 32) {
          const int share = s0 + (both ? e : e >> 1), at = both ? r & 127 : r;
          const int place = (int)segment_part(u, share, share == s0) + (both ? r >> 7 : e & 1) * half;
          const float* stats = a.parts + (int64_t)place * 4 + u.rs * kD + at;
          const float pm = stats[0], pl = stats[u.rs];
          place_s[h][e] = place + at;
          // (one that has seen nothing has left no sums)
          weight_s[h][e] = pl == 0.f ? -INFINITY : pm;
          const float top = fmaxf(m, pl == 0.f ? -INFINITY : pm);
          if (pl != 0.f) {
            l_all = (m == -INFINITY ? 0.f : l_all * exp2f(m - top)) + pl * exp2f(pm - top);
            m = top;
          }
        }
        l = l_all;
      }
    }
    // of all lanes, and of the own rows
    float top = warp_max(m);
    const float own_m = own_lse == -INFINITY ? -INFINITY : own_lse * 1.4426950408889634f;
    if (own_lse == own_lse) top = fmaxf(top, own_m);
    float all = warp_sum(m == -INFINITY ? 0.f : l * exp2f(m - top));
    const float own = own_lse == -INFINITY ? 0.f : exp2f(own_m - top);  // (NaN stays)
    all += own;
    nan |= all != all;
    __syncwarp();
    for (int e = lane; e < parts; e += 32)
      weight_s[h][e] = weight_s[h][e] == -INFINITY ? 0.f : exp2f(weight_s[h][e] - top);
    if (lane == 0) {
      count_s[h] = nan ? 0 : parts;
      rs_s[h] = rs;
      own_s[h] = own;
      inv_s[h] = nan ? nanf("") : (all > 0.f ? 1.f / all : 0.f);
      if (a.lse) {
        // (8-bit: the sum may carry an inverse scale of up to 2^60, so the exponents are
        // added first)
        const uint32_t u = __float_as_uint(all);
        const float e = (float)((int)(u >> 23) - 127);
        const float f = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
        a.lse[row0 + h] = nan ? nanf("")
                              : (all > 0.f ? ((top + e) + log2f(f)) * 0.6931471805599453f
                                           : -INFINITY);
      }
    }
  }
  __syncthreads();
  const int per = 32 * G, ways = kJoinThreads / per;  // threads of all columns, and of each
  const int h = threadIdx.x % G, c = threadIdx.x / G & 31, way = threadIdx.x / per;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (way < ways) {
    const float4* parts = reinterpret_cast<const float4*>(a.parts);
    const int count = count_s[h], rs = rs_s[h];
#pragma unroll 8
    for (int e = way; e < count; e += ways) {
      const float w = weight_s[h][e];
      float4 x = __ldcg(parts + place_s[h][e] + (int64_t)c * rs);
      if (!(w > 0.f)) x = make_float4(0.f, 0.f, 0.f, 0.f);  // (whatever lies there)
      o.x = fmaf(x.x, w, o.x); o.y = fmaf(x.y, w, o.y);
      o.z = fmaf(x.z, w, o.z); o.w = fmaf(x.w, w, o.w);
    }
    if (way == 0 && own_s[h] > 0.f) {
      const float w = own_s[h];
      const float4 x = reinterpret_cast<const float4*>(a.own_out + (row0 + h) * kD)[c];
      o.x = fmaf(x.x, w, o.x); o.y = fmaf(x.y, w, o.y);
      o.z = fmaf(x.z, w, o.z); o.w = fmaf(x.w, w, o.w);
    }
  }
  if (ways > 1) {
    sum_s[threadIdx.x] = o;
    __syncthreads();
    for (int i = 1; i < ways && way == 0; ++i) {
      const float4 x = sum_s[threadIdx.x + i * per];
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
    }
  }
  if (way > 0) return;
  const float inv = inv_s[h];
  if (inv != inv) o = make_float4(1.f, 1.f, 1.f, 1.f);
  o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
  if (a.out16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (row0 + h) * kD)[c] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    reinterpret_cast<float4*>(static_cast<float*>(a.out) + (row0 + h) * kD)[c] = o;
  }
}

}  // namespace

cudaError_t launch_shared_prep(const SharedArgs& a, cudaStream_t st) {
  const int64_t counters = ((int64_t)a.B * a.c.Hkv + kPrepThreads - 1) / kPrepThreads;
  const dim3 grid((unsigned)(1 + (counters < 64 ? counters : 64)));
  return launch_dependent(shared_prep_kernel, grid, dim3(kPrepThreads), 0, st, a);
}
cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t st) {
  return launch_dependent(shared_join_kernel, dim3(a.B, a.c.Hkv), dim3(kJoinThreads), 0, st, a);
}

}  // namespace tsa
