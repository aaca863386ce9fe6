// pages.cu -- the pages of a paged cache: taken, given back, shared between sequences,
// moved to the front of the pool, copied.
//
// The state is a count of table entries for every page (0: free) and the sequences'
// tables (-1: no page).  A call takes the lowest free pages, sequence by sequence, so
// that its result does not depend on the order in which its threads run: one kernel
// takes a snapshot (a bit for every free page, how many of every 256, what every sequence
// needs), the next one finds every entry's page by its rank in it.  Nothing is read back
// by the host, and a call whose needs exceed the free pages changes nothing.
//
// The last kernel of a call does not let its successor start early: the key scan looks
// pages up and streams keys before its dependency wait.
//
// What bounds them: latency (two or three launches over a few KB to a few MB: 3 to 8 us each,
// 12 us for a decode step's pages taken and given back), but for the copy.
#include "pages.h"

namespace tsa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Pages of a snapshot CTA: 8 counts of 256 pages, 8 words each.
constexpr int kSnap = 8 * kPagesChunk;

// Sum over the block, the same in every thread.
__device__ int block_sum(int x, int* scratch) {
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += scratch[w];
  return s;
}
// Exclusive prefix of x over the block's threads, and the whole sum.
__device__ int block_prefix(int x, int* scratch, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = y;
  __syncthreads();
  total = 0;
  int before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = total;
    total += scratch[w];
  }
  return before + y - x;
}
// The n-th set bit of w (n < popc(w)).
__device__ __forceinline__ int nth_bit(uint32_t w, int n) {
  int at = 0;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const int c = __popc(w & ((1u << s) - 1u));
    if (n >= c) {
      n -= c;
      at += s;
      w >>= s;
    }
  }
  return at;
}

// Entries of a row whose pages hold a position of [lo, hi).
struct Range {
  int j0, j1;
};
__device__ __forceinline__ Range entries_of(const PagesArgs& a, int b) {
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  int64_t lo = a.lo[b], hi = a.hi[b];
  lo = lo < 0 ? 0 : lo;
  hi = hi > cap ? cap : hi;
  if (lo >= hi) return {0, 0};
  return {(int)(lo >> a.page_shift), (int)((hi + (1 << a.page_shift) - 1) >> a.page_shift)};
}

// A pair of a fork, checked: shared entries [0, full) and whether a page is copied.
struct Fork {
  int parent, child, full;
  bool good, part;
};
__device__ __forceinline__ Fork fork_of(const PagesArgs& a, int i) {
  Fork f;
  f.parent = a.parents[i];
  f.child = a.children[i];
  const int n = a.lens[i];
  f.good = (uint32_t)f.parent < (uint32_t)a.B && (uint32_t)f.child < (uint32_t)a.B && n >= 0 &&
           (int64_t)n <= (int64_t)a.max_pages << a.page_shift;
  f.full = n >> a.page_shift;
  f.part = (n & ((1 << a.page_shift) - 1)) != 0;
  return f;
}

// The snapshot: the first CTAs a bit for every free page and the count of every chunk,
// the others what a sequence (take) or a pair (fork) needs; -1: a pair that is wrong.
template <int KIND>
__global__ void __launch_bounds__(kThreads) pages_snapshot_kernel(PagesArgs a) {
  __shared__ int scratch[kWarps];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pool = (a.n_pages + kSnap - 1) / kSnap;
  if ((int)blockIdx.x < pool) {
    const int first = blockIdx.x * kSnap + warp * kPagesChunk;
    int r[8], n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = first + 32 * i + lane;
      r[i] = p < a.n_pages ? a.refs[p] : 1;
    }
    uint32_t mine = 0u;  // lane i keeps word i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = __ballot_sync(0xffffffffu, r[i] == 0);
      n += __popc(w);
      if (lane == i) mine = w;
    }
    if (first < a.n_pages) {
      if (lane < 8) a.free_bits[first / 32 + lane] = mine;
      if (lane == 0) a.free_n[first / kPagesChunk] = n;
    }
    return;
  }
  const int i = blockIdx.x - pool;
  if constexpr (KIND == kPagesTake) {
    const Range r = entries_of(a, i);
    const int32_t* row = a.table + (int64_t)i * a.max_pages;
    int n = 0;
#pragma unroll 4
    for (int j = r.j0 + threadIdx.x; j < r.j1; j += kThreads) n += row[j] < 0;
    n = block_sum(n, scratch);
    if (threadIdx.x == 0) {
      a.need[i] = n;
      const int64_t cap = (int64_t)a.max_pages << a.page_shift;
      if (a.lo[i] < 0 || a.hi[i] > cap) atomicOr(a.status, kStatusBadLength);
    }
  } else if constexpr (KIND == kPagesFork) {
    const Fork f = fork_of(a, i);
    int bad = !f.good;
    if (f.good) {
      // a child once, and no parent of the same call
      for (int k = threadIdx.x; k < a.n; k += kThreads)
        bad |= a.parents[k] == f.child || (k != i && a.children[k] == f.child);
      const int32_t* row = a.table + (int64_t)f.parent * a.max_pages;
#pragma unroll 4
      for (int j = threadIdx.x; j < f.full + f.part; j += kThreads) {
        const int page = row[j];
        bad |= page >= a.n_pages || (page >= 0 && a.refs[page] == 0);
      }
      bad = block_sum(bad, scratch);
    }
    if (threadIdx.x == 0) {
      int n = -1;
      if (!bad) n = f.part && a.table[(int64_t)f.parent * a.max_pages + f.full] >= 0;
      a.need[i] = n;
    }
  }
}

// Whether a page of the pool was free in the snapshot.
__device__ __forceinline__ bool is_free(const PagesArgs& a, int page) {
  return (a.free_bits[page / 32] >> (page % 32)) & 1u;
}
// Counts before every chunk into shared memory; returns how many pages are free.
__device__ int chunk_prefix(const PagesArgs& a, int* before, int* scratch) {
  const int chunks = (a.n_pages + kPagesChunk - 1) / kPagesChunk;
  int all = 0;
  for (int c0 = 0; c0 < chunks; c0 += kThreads) {
    const int c = c0 + threadIdx.x;
    int total;
    const int x = block_prefix(c < chunks ? a.free_n[c] : 0, scratch, total);
    if (c < chunks) before[c] = all + x;
    all += total;
  }
  if (threadIdx.x == 0) before[chunks] = all;
  __syncthreads();
  return all;
}
// The free page of rank r (r < how many there are).
__device__ int free_page(const PagesArgs& a, const int* before, int r) {
  int lo = 0, hi = (a.n_pages + kPagesChunk - 1) / kPagesChunk;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= r) lo = mid; else hi = mid;
  }
  r -= before[lo];
  const uint4* p = reinterpret_cast<const uint4*>(a.free_bits + lo * (kPagesChunk / 32));
  const uint4 x = p[0], y = p[1];
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  int at = 0;
  uint32_t word = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = __popc(w[i]);
    if (!found) {
      if (r < c) {
        found = true;
        word = w[i];
        at = i;
      } else {
        r -= c;
      }
    }
  }
  return lo * kPagesChunk + 32 * at + nth_bit(word, r);
}

// What the sequences or pairs before number i need, and what all do; bad: one is wrong.
__device__ int need_before(const PagesArgs& a, int n, int i, int* scratch, int& total, int& bad) {
  int before = 0, all = 0, wrong = 0;
  for (int k = threadIdx.x; k < n; k += kThreads) {
    const int x = a.need[k];
    wrong |= x < 0;
    all += x < 0 ? 0 : x;
    if (k < i) before += x < 0 ? 0 : x;
  }
  total = block_sum(all, scratch);
  bad = block_sum(wrong, scratch);
  return block_sum(before, scratch);
}

// A sequence a CTA: its entries without a page take theirs, in order.
__global__ void __launch_bounds__(kThreads) pages_take_kernel(PagesArgs a) {
  extern __shared__ int before[];
  __shared__ int scratch[kWarps];
  pdl_wait();
  const int b = blockIdx.x;
  int total, bad;
  int rank = need_before(a, a.B, b, scratch, total, bad);
  const int free = chunk_prefix(a, before, scratch);
  if (total > free) {
    if (b == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadLength);
    return;
  }
  if (a.need[b] == 0) return;
  const Range r = entries_of(a, b);
  int32_t* row = a.table + (int64_t)b * a.max_pages;
  for (int j0 = r.j0; j0 < r.j1; j0 += kThreads) {
    const int j = j0 + threadIdx.x;
    const bool want = j < r.j1 && row[j] < 0;
    int n;
    const int at = rank + block_prefix(want, scratch, n);
    if (want) {
      const int p = free_page(a, before, at);
      row[j] = p;
      a.refs[p] = 1;
    }
    rank += n;
  }
}

// One entry's page less counted; false: it was not.
__device__ __forceinline__ bool let_go(const PagesArgs& a, int page) {
  if (page >= a.n_pages) return false;
  if (atomicSub(a.refs + page, 1) > 0) return true;
  atomicAdd(a.refs + page, 1);
  return false;
}

// Entries whose pages lie in [lo, hi) altogether.
__global__ void __launch_bounds__(kThreads) pages_free_kernel(PagesArgs a) {
  pdl_wait();
  const int b = blockIdx.y;
  const int ps = 1 << a.page_shift;
  const int64_t lo = a.lo[b] < 0 ? 0 : a.lo[b], hi = a.hi[b];
  const int64_t j0 = (lo + ps - 1) >> a.page_shift;
  int64_t j1 = hi < 0 ? 0 : hi >> a.page_shift;
  if (j1 > a.max_pages) j1 = a.max_pages;
  int32_t* row = a.table + (int64_t)b * a.max_pages;
  bool bad = false;
#pragma unroll 4
  for (int64_t j = j0 + blockIdx.x * kThreads + threadIdx.x; j < j1;
       j += (int64_t)gridDim.x * kThreads) {
    const int page = row[j];
    if (page < 0) continue;
    bad |= !let_go(a, page);
    row[j] = -1;
  }
  if (bad) atomicOr(a.status, kStatusBadLength);
}

// A pair, kThreads columns of the child's row.
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(PagesArgs a) {
  extern __shared__ int before[];
  __shared__ int scratch[kWarps];
  __shared__ int fresh_s;
  pdl_wait();
  const int i = blockIdx.y;
  int total, bad;
  const int rank = need_before(a, a.n, i, scratch, total, bad);
  const int free = chunk_prefix(a, before, scratch);
  if (bad || total > free) {
    if (threadIdx.x == 0 && blockIdx.x == 0) {
      if (i == 0) atomicOr(a.status, kStatusBadLength);
      a.src[i] = a.dst[i] = -1;
    }
    return;
  }
  const Fork f = fork_of(a, i);
  const bool copies = a.need[i] > 0;
  if (threadIdx.x == 0) fresh_s = copies ? free_page(a, before, rank) : -1;
  __syncthreads();
  const int fresh = fresh_s;
  const int32_t* from = a.table + (int64_t)f.parent * a.max_pages;
  int32_t* to = a.table + (int64_t)f.child * a.max_pages;
  if (threadIdx.x == 0 && blockIdx.x == 0) {
    a.src[i] = copies ? from[f.full] : -1;
    a.dst[i] = fresh;
  }
  bool wrong = false;
#pragma unroll 4
  for (int j = blockIdx.x * kThreads + threadIdx.x; j < a.max_pages; j += gridDim.x * kThreads) {
    const int was = to[j];
    const int now = j < f.full ? from[j] : (j == f.full ? fresh : -1);
    // (an entry of a page that counted as free: it may be the one given out here)
    const bool stale = was >= 0 && was < a.n_pages && is_free(a, was);
    if (was == now && !stale) continue;
    if (now >= 0) atomicAdd(a.refs + now, 1);
    if (was >= 0) wrong |= stale || !let_go(a, was);
    to[j] = now < 0 ? -1 : now;
  }
  if (wrong) atomicOr(a.status, kStatusBadLength);
}

// Free pages below page p, from the chunks' prefix.
__device__ int free_below(const PagesArgs& a, const int* before, int p) {
  const int c = p / kPagesChunk;
  int n = before[c];
  if (p % kPagesChunk == 0) return n;
  for (int w = c * (kPagesChunk / 32); w < p / 32; ++w) n += __popc(a.free_bits[w]);
  if (p % 32) n += __popc(a.free_bits[p / 32] & ((1u << (p % 32)) - 1u));
  return n;
}

// With n_live pages in use: the k-th hole below n_live takes the k-th page above.
__global__ void __launch_bounds__(kThreads) pages_moves_kernel(PagesArgs a) {
  extern __shared__ int before[];
  __shared__ int scratch[kWarps];
  pdl_wait();
  pdl_trigger();
  const int live = a.n_pages - chunk_prefix(a, before, scratch);
  const int holes = free_below(a, before, live);  // (every thread: the same words)
  const int pairs = a.n_pages / 2;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.count[0] = holes;
    a.live[0] = live;
  }
  for (int k = holes + blockIdx.x * kThreads + threadIdx.x; k < pairs;
       k += gridDim.x * kThreads)
    a.src[k] = a.dst[k] = -1;
  for (int p = blockIdx.x * kThreads + threadIdx.x; p < a.n_pages; p += gridDim.x * kThreads) {
    const bool free = is_free(a, p);
    if (p < live) {
      if (free) a.dst[free_below(a, before, p)] = p;
    } else if (!free) {
      const int k = (p - live) - (free_below(a, before, p) - holes);
      a.src[k] = p;
      a.rank[p] = k;
    }
  }
}
// The tables' entries and the counts follow the pages.
__global__ void __launch_bounds__(kThreads) pages_follow_kernel(PagesArgs a) {
  pdl_wait();
  const int live = a.live[0], holes = a.count[0];
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t k = at; k < holes; k += step) {
    const int s = a.src[k];
    a.refs[a.dst[k]] = a.refs[s];
    a.refs[s] = 0;
  }
  bool bad = false;
#pragma unroll 4
  for (int64_t e = at; e < (int64_t)a.B * a.max_pages; e += step) {
    const int page = a.table[e];
    if (page < 0) continue;
    // (a page outside the pool, or one that counts as free: below `live` a hole that another
    // page moves into)
    if (page >= a.n_pages || is_free(a, page))
      bad = true;
    else if (page >= live)
      a.table[e] = a.dst[a.rank[page]];
  }
  if (bad) atomicOr(a.status, kStatusBadLength);
}

constexpr int kTileBytes = kThreads * 64;  // of a page that a CTA copies at a time

// Bandwidth-bound: a tile of 16 KB a CTA and turn, four pieces of 16 bytes a thread in
// flight, 2048 threads an SM: 0.4 GB of pages of 64 KB moved in 125 us, 6.3 TB/s.
__global__ void __launch_bounds__(kThreads) pages_copy_kernel(const __grid_constant__ CopyArgs a) {
  pdl_wait();
  const int n = a.count ? min(max(*a.count, 0), a.n) : a.n;
  const int tiles = a.tile0[a.bufs];
  const int64_t all = (int64_t)n * tiles;
  bool bad = false;
  for (int64_t it = blockIdx.x; it < all; it += gridDim.x) {
    const int pair = (int)(it / tiles), t = (int)(it - (int64_t)pair * tiles);
    const int src = a.src[pair], dst = a.dst[pair];
    if (src < 0) continue;
    if (src >= a.n_pages || (uint32_t)dst >= (uint32_t)a.n_pages) {
      bad = true;
      continue;
    }
    int lo = 0, hi = a.bufs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.tile0[mid] <= t) lo = mid; else hi = mid;
    }
    const int64_t bytes = a.bytes[lo], at = (int64_t)(t - a.tile0[lo]) * kTileBytes;
    const uint8_t* from = a.data[lo] + src * bytes + at;
    uint8_t* to = a.data[lo] + dst * bytes + at;
    const int left = (int)(bytes - at < kTileBytes ? bytes - at : kTileBytes);
    if (((bytes | reinterpret_cast<uintptr_t>(a.data[lo])) & 15) == 0) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = (i * kThreads + threadIdx.x) * 16;
        if (o < left) w[i] = __ldcs(reinterpret_cast<const uint4*>(from + o));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = (i * kThreads + threadIdx.x) * 16;
        if (o < left) *reinterpret_cast<uint4*>(to + o) = w[i];
      }
    } else {
      for (int o = threadIdx.x * 4; o < left; o += kThreads * 4)
        *reinterpret_cast<uint32_t*>(to + o) = *reinterpret_cast<const uint32_t*>(from + o);
    }
  }
  if (bad && threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadLength);
}

size_t prefix_bytes(int n_pages) {
  return ((size_t)(n_pages + kPagesChunk - 1) / kPagesChunk + 1) * sizeof(int);
}
template <typename K>
cudaError_t with_prefix(K kernel, dim3 grid, const PagesArgs& a, cudaStream_t st) {
  const size_t smem = prefix_bytes(a.n_pages);
  if (smem > 47 * 1024) {
    // (the most that any call asks for: the limit belongs to the kernel, and another host
    // thread's smaller one would refuse this launch)
    const cudaError_t e =
        cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)prefix_bytes(kMostPages));
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kernel, grid, dim3(kThreads), smem, st, a);
}

}  // namespace

cudaError_t launch_pages_snapshot(const PagesArgs& a, int kind, cudaStream_t st) {
  const int pool = (a.n_pages + kSnap - 1) / kSnap;
  const dim3 th(kThreads);
  if (kind == kPagesTake)
    return launch_dependent(pages_snapshot_kernel<kPagesTake>, dim3(pool + a.B), th, 0, st, a);
  if (kind == kPagesFork)
    return launch_dependent(pages_snapshot_kernel<kPagesFork>, dim3(pool + a.n), th, 0, st, a);
  return launch_dependent(pages_snapshot_kernel<kPagesCompact>, dim3(pool), th, 0, st, a);
}
cudaError_t launch_pages_take(const PagesArgs& a, cudaStream_t st) {
  return with_prefix(pages_take_kernel, dim3(a.B), a, st);
}
cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t st) {
  // four entries a thread, or more in very long rows
  const int cols = (a.max_pages + 4 * kThreads - 1) / (4 * kThreads);
  return launch_dependent(pages_free_kernel, dim3(cols < 64 ? cols : 64, a.B), dim3(kThreads), 0,
                          st, a);
}
cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t st) {
  const int cols = (a.max_pages + 4 * kThreads - 1) / (4 * kThreads);
  return with_prefix(pages_fork_kernel, dim3(cols < 64 ? cols : 64, a.n), a, st);
}
cudaError_t launch_pages_moves(const PagesArgs& a, cudaStream_t st) {
  const int grid = (a.n_pages + kThreads - 1) / kThreads;
  return with_prefix(pages_moves_kernel, dim3(grid < 304 ? grid : 304), a, st);
}
cudaError_t launch_pages_follow(const PagesArgs& a, cudaStream_t st) {
  const int64_t all = (int64_t)a.B * a.max_pages;
  int64_t grid = ((all > a.n_pages ? all : a.n_pages) + 4 * kThreads - 1) / (4 * kThreads);
  if (grid > 1216) grid = 1216;
  return launch_dependent(pages_follow_kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, a);
}

int pages_copy_tiles(int64_t bytes) { return (int)((bytes + kTileBytes - 1) / kTileBytes); }

cudaError_t launch_pages_copy(const CopyArgs& a, int sms, cudaStream_t st) {
  int64_t grid = (int64_t)a.n * a.tile0[a.bufs];
  if (grid > 8 * sms) grid = 8 * sms;
  return launch_dependent(pages_copy_kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, a);
}

}  // namespace tsa
