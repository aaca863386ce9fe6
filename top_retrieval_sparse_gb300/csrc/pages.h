// pages.h -- argument blocks and launchers of the page kernels (host <-> device
// contract inside the library; not part of the C ABI).
#pragma once

#include "cache_ops.h"

namespace tsa {

constexpr int kPagesChunk = 256;  // pages of a count in the snapshot
// More pages than this (134 million positions in pages of 16) would not fit the
// snapshot's prefix in shared memory.
constexpr int kMostPages = 1 << 23;
enum PagesKind : int { kPagesTake = 0, kPagesFork = 1, kPagesCompact = 2 };

struct PagesArgs {
  int32_t* table;            // [B][max_pages]
  int32_t* refs;             // [n_pages]
  int B, max_pages, n_pages, page_shift;
  const int32_t* lo;         // take, free: positions [B]
  const int32_t* hi;
  const int32_t* parents;    // fork: [n]
  const int32_t* children;
  const int32_t* lens;
  int n;
  int32_t* src;              // fork: [n], compact: [n_pages / 2]
  int32_t* dst;
  int32_t* count;            // compact: [1]
  int* status;
  // the snapshot, in the workspace
  uint32_t* free_bits;       // [chunks][8]
  int32_t* free_n;           // [chunks]
  int32_t* need;             // [B] or [n]
  int32_t* rank;             // [n_pages]: number of a page's move
  int32_t* live;             // [1]
};
cudaError_t launch_pages_snapshot(const PagesArgs& a, int kind, cudaStream_t st);
cudaError_t launch_pages_take(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_moves(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_follow(const PagesArgs& a, cudaStream_t st);

constexpr int kCopyBufs = 128;   // buffers of a launch
struct CopyArgs {
  uint8_t* data[kCopyBufs];      // [n_pages][bytes]
  int64_t bytes[kCopyBufs];
  int32_t tile0[kCopyBufs + 1];  // tiles of a page before every buffer's
  int bufs, n, n_pages;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;          // nullptr: n
  int* status;                   // or nullptr
};
int pages_copy_tiles(int64_t bytes);
cudaError_t launch_pages_copy(const CopyArgs& a, int sms, cudaStream_t st);

}  // namespace tsa
