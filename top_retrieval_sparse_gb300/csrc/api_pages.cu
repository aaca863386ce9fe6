// api_pages.cu -- C ABI of the page operators (declared in include/tsa.h): host-side
// validation, workspace layout and launches.  Nothing here allocates device memory,
// synchronises or prints.
#include "api_util.h"
#include "pages.h"

using namespace tsa;

namespace {

bool pages_sizes(int B, int max_pages, int n_pages) {
  return B >= 0 && B <= 4096 && max_pages > 0 && n_pages > 0 && n_pages <= kMostPages &&
         (int64_t)B * max_pages < (int64_t)1 << 31;
}

// Workspace: the status word, then what a call keeps between its kernels.
struct Layout {
  size_t live, need, free_n, free_bits, rank, total;
};
Layout layout_of(int B, int n_pages) {
  const size_t chunks = ((size_t)n_pages + kPagesChunk - 1) / kPagesChunk;
  Layout l{};
  l.live = kAlign;
  l.need = l.live + kAlign;
  l.free_n = l.need + round_up((size_t)(B > 0 ? B : 1) * 4);
  l.free_bits = l.free_n + round_up(chunks * 4);
  l.rank = l.free_bits + round_up(chunks * (kPagesChunk / 8));
  l.total = l.rank + round_up((size_t)n_pages * 4);
  return l;
}

int check_pages(const tsa_pages* p, void* ws, size_t bytes, PagesArgs& a) {
  a = PagesArgs{};
  if (!p) return fail(TSA_ERR_INVALID_ARG, "pages is NULL");
  const int ps = p->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)))
    return fail(TSA_ERR_INVALID_ARG, "page_size %d: must be a power of two in [16, 256]", ps);
  if (!pages_sizes(p->B, p->max_pages, p->n_pages))
    return fail(TSA_ERR_INVALID_ARG,
                "B %d must be in [0, 4096], n_pages %d in [1, 2^23], max_pages %d > 0, B * "
                "max_pages < 2^31", p->B, p->n_pages, p->max_pages);
  if ((int64_t)p->max_pages * ps >= (int64_t)1 << 31)
    return fail(TSA_ERR_INVALID_ARG, "max_pages * page_size must be < 2^31");
  if ((!p->table && p->B > 0) || !p->refs)
    return fail(TSA_ERR_INVALID_ARG, "table and refs must be non-NULL");
  if (!aligned(p->table, 4) || !aligned(p->refs, 4))
    return fail(TSA_ERR_INVALID_ARG, "table and refs must be 4-byte aligned");
  const Layout l = layout_of(p->B, p->n_pages);
  const int rc = check_workspace(ws, bytes, l.total);
  if (rc) return rc;
  a.table = p->table;
  a.refs = p->refs;
  a.B = p->B;
  a.max_pages = p->max_pages;
  a.n_pages = p->n_pages;
  while ((1 << a.page_shift) < ps) ++a.page_shift;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.status = reinterpret_cast<int*>(w);
  a.live = reinterpret_cast<int32_t*>(w + l.live);
  a.need = reinterpret_cast<int32_t*>(w + l.need);
  a.free_n = reinterpret_cast<int32_t*>(w + l.free_n);
  a.free_bits = reinterpret_cast<uint32_t*>(w + l.free_bits);
  a.rank = reinterpret_cast<int32_t*>(w + l.rank);
  return TSA_OK;
}

}  // namespace

extern "C" {

size_t tsa_pages_workspace_size(int B, int max_pages, int n_pages) {
  return pages_sizes(B, max_pages, n_pages) ? layout_of(B, n_pages).total : 0;
}

int pages_alloc(const tsa_pages* pages, const int32_t* lo, const int32_t* hi, void* workspace,
                size_t ws_bytes, void* stream) {
  PagesArgs a;
  int rc = check_pages(pages, workspace, ws_bytes, a);
  if (rc) return rc;
  if (a.B == 0) return report_ok();
  if (!lo || !hi) return fail(TSA_ERR_INVALID_ARG, "lo and hi must be non-NULL");
  a.lo = lo;
  a.hi = hi;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((rc = launched(launch_pages_snapshot(a, kPagesTake, st), "snapshot launch"))) return rc;
  return launched(launch_pages_take(a, st), "alloc launch");
}

int pages_free(const tsa_pages* pages, const int32_t* lo, const int32_t* hi, void* workspace,
               size_t ws_bytes, void* stream) {
  PagesArgs a;
  const int rc = check_pages(pages, workspace, ws_bytes, a);
  if (rc) return rc;
  if (a.B == 0) return report_ok();
  if (!lo || !hi) return fail(TSA_ERR_INVALID_ARG, "lo and hi must be non-NULL");
  a.lo = lo;
  a.hi = hi;
  return launched(launch_pages_free(a, static_cast<cudaStream_t>(stream)), "free launch");
}

int pages_fork(const tsa_pages* pages, const int32_t* parents, const int32_t* children,
               const int32_t* lens, int n, int32_t* src, int32_t* dst, void* workspace,
               size_t ws_bytes, void* stream) {
  PagesArgs a;
  int rc = check_pages(pages, workspace, ws_bytes, a);
  if (rc) return rc;
  if (n < 0 || n > a.B)
    return fail(TSA_ERR_INVALID_ARG, "n = %d: must be in [0, B = %d]", n, a.B);
  if (n == 0) return report_ok();
  if (!parents || !children || !lens || !src || !dst)
    return fail(TSA_ERR_INVALID_ARG, "parents, children, lens, src and dst must be non-NULL");
  a.parents = parents;
  a.children = children;
  a.lens = lens;
  a.n = n;
  a.src = src;
  a.dst = dst;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((rc = launched(launch_pages_snapshot(a, kPagesFork, st), "snapshot launch"))) return rc;
  return launched(launch_pages_fork(a, st), "fork launch");
}

int pages_compact(const tsa_pages* pages, int32_t* src, int32_t* dst, int32_t* count,
                  void* workspace, size_t ws_bytes, void* stream) {
  PagesArgs a;
  int rc = check_pages(pages, workspace, ws_bytes, a);
  if (rc) return rc;
  if (!count || (a.n_pages > 1 && (!src || !dst)))
    return fail(TSA_ERR_INVALID_ARG, "src, dst and count must be non-NULL");
  a.src = src;
  a.dst = dst;
  a.count = count;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((rc = launched(launch_pages_snapshot(a, kPagesCompact, st), "snapshot launch"))) return rc;
  if ((rc = launched(launch_pages_moves(a, st), "compact launch"))) return rc;
  return launched(launch_pages_follow(a, st), "compact launch");
}

int pages_copy(const tsa_page_buf* bufs, int n_bufs, int n_pages, const int32_t* src,
               const int32_t* dst, const int32_t* count, int n, int32_t* status, void* stream) {
  if (n_bufs < 0 || (n_bufs > 0 && !bufs))
    return fail(TSA_ERR_INVALID_ARG, "bufs NULL or n_bufs < 0");
  if (n_pages <= 0) return fail(TSA_ERR_INVALID_ARG, "n_pages must be > 0");
  if (n < 0) return fail(TSA_ERR_INVALID_ARG, "n < 0");
  if (status && !aligned(status, kAlign))
    return fail(TSA_ERR_INVALID_ARG, "status must be 256-byte aligned");
  for (int i = 0; i < n_bufs; ++i)
    if (!bufs[i].data || !aligned(bufs[i].data, 4) || bufs[i].bytes <= 0 || bufs[i].bytes % 4 ||
        bufs[i].bytes > (int64_t)1 << 32)
      return fail(TSA_ERR_INVALID_ARG,
                  "bufs[%d]: data NULL or not 4-byte aligned, or bytes not a multiple of 4 in [4, "
                  "2^32]", i);
  if (n == 0 || n_bufs == 0) return report_ok();
  if (!src || !dst) return fail(TSA_ERR_INVALID_ARG, "src and dst must be non-NULL");
  for (int i0 = 0; i0 < n_bufs; i0 += kCopyBufs) {
    CopyArgs a{};
    a.bufs = n_bufs - i0 < kCopyBufs ? n_bufs - i0 : kCopyBufs;
    a.n = n;
    a.n_pages = n_pages;
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.status = status;
    for (int i = 0; i < a.bufs; ++i) {
      a.data[i] = static_cast<uint8_t*>(bufs[i0 + i].data);
      a.bytes[i] = bufs[i0 + i].bytes;
      a.tile0[i + 1] = a.tile0[i] + pages_copy_tiles(a.bytes[i]);
    }
    const int rc = launched(launch_pages_copy(a, num_sms(), static_cast<cudaStream_t>(stream)),
                            "copy launch");
    if (rc) return rc;
  }
  return report_ok();
}

}  // extern "C"
