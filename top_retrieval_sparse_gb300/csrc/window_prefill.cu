// window_prefill.cu -- attention of many new tokens per sequence over a bf16
// cache: a query at position p sees the rows j <= p with j < n_init or
// j > p - n_recent.
//
// Per KV head the G query heads of a token share its rows, so a 128-row tile of the
// tensor core holds the heads of 128 / G tokens.  A CTA takes two such tiles (A and
// B) over the key tiles of 128 rows that any of their queries sees:
//   S = Q K^T (tcgen05, fp32 in tensor memory), P = 2^(S c - m c) (bf16, over
//   S's columns), O += P V (tcgen05, fp32 in tensor memory)
// with the running maximum m and sum of the softmax in registers, a row a thread.
// Both products of a key tile are 2 x 128^3: the tensor core bounds the kernel, as long
// as the exponentials of one tile run under the other tile's products; hence two.
//
// Warps.  0 and 3: the matrix instructions of A and of B, 1: the copies, 2: zeroing
// of V (first, so that the scheduler prefers them), 4-7: softmax of tile A (thread =
// row = tensor-memory lane), 8-11: of B.  K and V tiles go through a ring of five 32 KB
// slots by TMA (two 64-column boxes with the 128-byte swizzle; a box a page where pages
// are smaller than a tile).  A tile's matrix instructions come in the order O(j),
// S(j+1), O(j+1) ..., from one thread, so that they execute in that order: S(j+1) may
// overwrite P(j) without a wait.  A commit covers all of a thread's, so a softmax that
// sees S(j) also knows O(j-1) done, and may rescale O; it does so only where the
// weights have grown by more than 2^16.
// A slot is filled again when all its readers have given it back: the matrix threads
// (for the last of their instructions) and the zeroing warp, which passes every slot
// in order, K's too.  A wait tells a barrier's last two phases apart and no more, so
// nobody may fall behind by two laps of the ring; this count is what excludes it.
//
// Weights are rounded to bf16 for the second product, as its operands are of one type and
// V is bf16: half a step of 2^-8 each, both ways.  Against 64 bits the output is off by 2.0e-3
// to 2.4e-3 where 32-bit weights rounded once are off by 1.5e-3 to 1.7e-3; a second part
// would take half as many matrix instructions again.
//
// What bounds it: 32K tokens, 32/8 heads, window 4096 + 128 sinks take 1.27 ms in single
// calls (1660 TFLOP/s of visible pairs, 0.86 of the measured burst of a library matrix
// product) and 1.37 ms under a sustained load (1550, 0.89 of its sustained rate); a full
// causal 32K prompt 4.9 ms, 1800 TFLOP/s.  A step of two tiles takes 2400 to 2500 cycles for
// 2048 of matrix instructions; what is left is the path from S to P where it is longer
// than the other tile's products, 12K cycles of a CTA's 95K for its queries and its
// output, and key tiles that the window's edges only partly need.
//
// Few queries (fewer CTAs than half the SMs) share the key tiles of a CTA's queries out
// over several; each leaves (O, maximum, sum) in the workspace, and a second kernel
// joins them, a warp a row (the last CTA to arrive doing it took 10 us).
//
// Long sums.  Matrix instructions truncate their 32-bit sums, all in one direction: values
// of one sign came out 6.3e-9 of themselves too small for every row (6.6e-3 for a million,
// more than bf16's rounding).  So every kFoldTiles tiles a row's O is added, with rounding,
// to a sum in the workspace that carries its own maximum, and begins again from nothing:
// 128 tiles lose 1e-4 at most and cost a full causal 32K prompt 5.14 -> 5.18 ms under a
// sustained load (64 tiles 5.26), 704 tokens after a million rows 10.7 -> 10.9 ms.  The sums are of the CTAs
// that run, not of the call: 20 MB that stay in L2.
//
// Masks cost nothing but at the edges of what is seen: there the rows' columns are
// masked one by one, and rows of V that no query of the CTA sees are zeroed in
// shared memory (whatever they hold, 0 * NaN would reach the output).
#include <cuda.h>

#include "cache_ops.h"

namespace tsa {

namespace {

constexpr int kTile = 128;                       // rows of a key tile and of a query tile
constexpr int kHalf = kTile * 128;               // bytes of 64 columns of a tile
constexpr int kSlotBytes = 2 * kHalf;
constexpr int kSlots = 5;
constexpr int kPreThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // 2 * 216 + 72 = 3 * 168 a scheduler
constexpr int kPreSmem = (2 + kSlots) * kSlotBytes + 1024;
// Weights may grow to 2^16 under an old maximum before O is rescaled: bf16 and
// fp32 keep their precision at any size, and 2^16 is far from overflow.
constexpr float kRescale = 16.f, kMost = 65536.f;

// Instruction descriptors: fp32 accumulator, bf16 operands, 128 x 128; B of the
// second product (V) with its rows (keys) as the reduction index.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((128u / 8) << 17) |
                            ((128u / 16) << 24);
constexpr uint32_t kIdescV = kIdesc | (1u << 16);

// Shared-memory operand, 128-byte swizzle: eight rows of 128 bytes are 1024
// apart (stride offset); `lead` separates the two halves of 64 columns where they are
// the outer index (V).
// An operand further on is the same descriptor with its address field (16 bytes a
// count) advanced.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(on));
  return on != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// Arrives on the barrier when every matrix instruction so far is complete.
__device__ __forceinline__ void commit_mma(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_stores() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// 128 columns of this thread's row; the wait is part of it, so that nothing uses
// the registers before they hold the values.
__device__ __forceinline__ void load_cols(uint32_t addr, float (&x)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, "
      "%47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
      "%62, %63, %64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, "
      "%77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, "
      "%92, %93, %94, %95, %96, %97, %98, %99, %100, %101, %102, %103, %104, %105, "
      "%106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, "
      "%118, %119, %120, %121, %122, %123, %124, %125, %126, %127"
      "}, [%128];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), 
        "=f"(x[7]), "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), 
        "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]), "=f"(x[19]), 
        "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), 
        "=f"(x[26]), "=f"(x[27]), "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31]), 
        "=f"(x[32]), "=f"(x[33]), "=f"(x[34]), "=f"(x[35]), "=f"(x[36]), "=f"(x[37]), 
        "=f"(x[38]), "=f"(x[39]), "=f"(x[40]), "=f"(x[41]), "=f"(x[42]), "=f"(x[43]), 
        "=f"(x[44]), "=f"(x[45]), "=f"(x[46]), "=f"(x[47]), "=f"(x[48]), "=f"(x[49]), 
        "=f"(x[50]), "=f"(x[51]), "=f"(x[52]), "=f"(x[53]), "=f"(x[54]), "=f"(x[55]), 
        "=f"(x[56]), "=f"(x[57]), "=f"(x[58]), "=f"(x[59]), "=f"(x[60]), "=f"(x[61]), 
        "=f"(x[62]), "=f"(x[63]), "=f"(x[64]), "=f"(x[65]), "=f"(x[66]), "=f"(x[67]), 
        "=f"(x[68]), "=f"(x[69]), "=f"(x[70]), "=f"(x[71]), "=f"(x[72]), "=f"(x[73]), 
        "=f"(x[74]), "=f"(x[75]), "=f"(x[76]), "=f"(x[77]), "=f"(x[78]), "=f"(x[79]), 
        "=f"(x[80]), "=f"(x[81]), "=f"(x[82]), "=f"(x[83]), "=f"(x[84]), "=f"(x[85]), 
        "=f"(x[86]), "=f"(x[87]), "=f"(x[88]), "=f"(x[89]), "=f"(x[90]), "=f"(x[91]), 
        "=f"(x[92]), "=f"(x[93]), "=f"(x[94]), "=f"(x[95]), "=f"(x[96]), "=f"(x[97]), 
        "=f"(x[98]), "=f"(x[99]), "=f"(x[100]), "=f"(x[101]), "=f"(x[102]), "=f"(x[103]), 
        "=f"(x[104]), "=f"(x[105]), "=f"(x[106]), "=f"(x[107]), "=f"(x[108]), "=f"(x[109]), 
        "=f"(x[110]), "=f"(x[111]), "=f"(x[112]), "=f"(x[113]), "=f"(x[114]), "=f"(x[115]), 
        "=f"(x[116]), "=f"(x[117]), "=f"(x[118]), "=f"(x[119]), "=f"(x[120]), "=f"(x[121]), 
        "=f"(x[122]), "=f"(x[123]), "=f"(x[124]), "=f"(x[125]), "=f"(x[126]), "=f"(x[127])
      : "r"(addr)
      : "memory");
}
// 32 columns of this thread's row; the wait is part of it, so that nothing uses
// the registers before they hold the values.
__device__ __forceinline__ void load_cols(uint32_t addr, float (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), 
        "=f"(x[7]), "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), 
        "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]), "=f"(x[19]), 
        "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), 
        "=f"(x[26]), "=f"(x[27]), "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void store_cols(uint32_t addr, const float (&x)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32"
      "};" ::"r"(addr),
        "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), 
        "f"(x[8]), "f"(x[9]), "f"(x[10]), "f"(x[11]), "f"(x[12]), "f"(x[13]), "f"(x[14]), 
        "f"(x[15]), "f"(x[16]), "f"(x[17]), "f"(x[18]), "f"(x[19]), "f"(x[20]), "f"(x[21]), 
        "f"(x[22]), "f"(x[23]), "f"(x[24]), "f"(x[25]), "f"(x[26]), "f"(x[27]), "f"(x[28]), 
        "f"(x[29]), "f"(x[30]), "f"(x[31])
      : "memory");
}
__device__ __forceinline__ void store_cols(uint32_t addr, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
      "};" ::"r"(addr),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), 
        "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), 
        "r"(x[15])
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (a.x * b + c, a.y * b + c) and the sum of pairs, two lanes an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Bits [0, n) of a word, any n.
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a CTA's queries see: rows [0, n0) and [lo, end), as a list of `all` key tiles:
// [0, s0) and from sw; the CTA takes n of them from number `from` on.
struct Span {
  int n0, lo, end, s0, sw, all, from, n;
  __device__ int tile(int j) const {
    j += from;
    return j < s0 ? j : sw + (j - s0);
  }
  // Tile j may hold rows that nothing sees.
  __device__ bool edge(int j) const {
    j += from;
    return j == s0 - 1 || j == s0 || j == all - 1;
  }
  __device__ bool sees(int r) const { return r < end && (r < n0 || r >= lo); }
};

// A place for a CTA's sums that no other CTA uses: its SM's, as a rule (a CTA fills an
// SM, so there are as many places as CTAs).  -1: none came free (bounded).
__device__ int take_place(uint32_t* used) {
  uint32_t sm;
  asm volatile("mov.u32 %0, %%smid;" : "=r"(sm));
  for (uint32_t i = 0; i < 1u << 20; ++i) {
    const int at = (int)((sm + i) % kFoldPlaces);
    if (atomicExch(used + at, 1u) == 0u) {
      __threadfence();
      return at;
    }
  }
  return -1;
}

// A bounded wait.  One try in line; the loop with the clock and the abort flag
// is kept out of the way of the usual path.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  if (mbar_wait_or_abort(bar, parity, abort)) return true;
  *abort = 1;
  return false;
}

struct Barriers {
  uint64_t q[2], s[2], p[2][2], o[2], full[kSlots], empty[kSlots], clean[kSlots], drain[2],
      turn[2];
};

// LONG: some CTA may have more than kFoldTiles key tiles (a.sums is there).  The other form
// is 1.7 % faster without the test for it (32K tokens in a window of 4096: 1.43 -> 1.41 ms).
template <bool LONG>
__global__ void __launch_bounds__(kPreThreads, 1)
    window_prefill_kernel(const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, PrefillArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bar;
  __shared__ uint32_t tmem_s;
  __shared__ volatile int abort_s;
  __shared__ volatile int bad_s;
  __shared__ volatile int place_s;           // of the long sums; set before the first copies
  __shared__ float under_s[2][kTile];        // the maximum a row's sum outside is under
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.z, g = blockIdx.y;
  const int G = a.G, TQ = kTile / G;
  pdl_wait();
  // Only the joining kernel may start early: the output is bf16, and the key scan
  // reads its queries before its dependency wait.
  if (a.splits > 1) pdl_trigger();

  // This CTA's tokens [t0, t1) of sequence b, the last blocks first.
  int64_t tok, n64;
  bool bad_count = !seq_tokens(a.cu, a.max_q, a.T, b, tok, n64);
  if (bad_count) {
    if (tid == 0) atomicOr(a.status, kStatusBadLength);
    if (tok < 0 || n64 < 0 || tok + n64 > a.T) return;
    if (n64 > a.max_q) n64 = a.max_q;
  }
  const int n = (int)n64;
  const int block = a.blocks - 1 - (int)blockIdx.x / a.splits;
  const int t0 = block * 2 * TQ;
  if (t0 >= n) return;
  const int t1 = t0 + 2 * TQ < n ? t0 + 2 * TQ : n;
  int L = a.lens[b];
  if (L < 0 || L > a.c.l_cap) {
    if (tid == 0) atomicOr(a.status, kStatusBadLength);
    L = L < 0 ? 0 : (int)a.c.l_cap;
  }
  const int p0 = L - n + t0;                 // position of the first token
  const int ni = a.n_init, nr = a.n_recent;  // both at most l_cap
  Span v;
  v.end = L - n + t1;                        // rows at or before the last token
  if (v.end < 0) v.end = 0;
  v.n0 = ni < v.end ? ni : v.end;
  v.lo = nr == 0 ? v.end : (p0 < nr ? 0 : p0 + 1 - nr);  // of the first token (p0 < v.end)
  if (v.lo > v.end) v.lo = v.end;
  v.s0 = (v.n0 + kTile - 1) / kTile;
  v.sw = v.lo / kTile > v.s0 ? v.lo / kTile : v.s0;
  const int se = (v.end + kTile - 1) / kTile;
  v.all = v.s0 + (v.lo < v.end && se > v.sw ? se - v.sw : 0);
  const int part = blockIdx.x % a.splits;    // of the key tiles
  v.from = (int)((int64_t)v.all * part / a.splits);
  v.n = (int)((int64_t)v.all * (part + 1) / a.splits) - v.from;
  const bool two = t1 - t0 > TQ;             // tile B has tokens

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, ring = base + 2 * kSlotBytes;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q[i], kTile);
      mbar_init(&bar.s[i], 1);
      mbar_init(&bar.p[i][0], kTile);
      mbar_init(&bar.p[i][1], kTile);
      mbar_init(&bar.o[i], 1);
      mbar_init(&bar.drain[i], 1);
      mbar_init(&bar.turn[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], two ? 3 : 2);  // matrix threads, zeroing warp
      mbar_init(&bar.clean[i], 1);
    }
    fence_mbar_init();
    abort_s = 0;
    bad_s = bad_count;
    if (LONG) place_s = -1;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&tmem_s))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_s;
  // The whole warp agrees, where what follows is a warp's work.
  auto wait = [&](uint64_t* x, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_for(x, parity, &abort_s)) != 0;
  };

  if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = (warp >> 2) - 1;           // tile A or B
    const int r = tid & 127;
    const int my_t = t0 + x * TQ + r / G, h = g * G + r % G;
    const bool live = r < TQ * G && my_t < t1;
    // position (rows past the tokens: unused; below 0 nothing is seen)
    const int p = L - n + my_t < 0 ? -1 : L - n + my_t;
    if (x == 0 || two) {
      // Q, swizzled as the copies would: rows of 128 bytes, piece c at c ^ (row & 7).
      // A half-warp a row, so that a row's 256 bytes are one request; all of them in
      // flight before the first is stored.
      const int r_warp = (warp & 3) * 32, r_half = lane >> 4, piece = lane & 15;
      const uint32_t q_mine = q_at + x * kSlotBytes;
      {
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
        uint4 w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int rr = r_warp + 2 * i + r_half, tt = (rr * a.inv_g) >> 16;
          w[i] = make_uint4(0u, 0u, 0u, 0u);
          if (tt < TQ && t0 + x * TQ + tt < t1 && !a.zero)
            w[i] = *reinterpret_cast<const uint4*>(
                a.q.p + (tok + t0 + x * TQ + tt) * a.q.st + (g * G + rr - tt * G) * a.q.sh +
                8 * piece);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int rr = r_warp + 2 * i + r_half;
          const uint32_t at = q_mine + (piece >> 3) * kHalf + rr * 128 +
                              (((piece & 7) ^ (rr & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[i].x ^ flip),
                       "r"(w[i].y ^ flip), "r"(w[i].z ^ flip), "r"(w[i].w ^ flip)
                       : "memory");
        }
      }
      fence_proxy_async();
      mbar_arrive(&bar.q[x]);

      const uint32_t s_at = tmem + x * kTile + ((uint32_t)(warp & 3) << 21);
      const uint32_t o_at = s_at + 2 * kTile;
      const float sc = a.scale_log2;
      float m = -INFINITY, l = 0.f;
      // Columns 32 c + 4 i of that sum (neighbouring rows side by side).
      auto outside = [&](int c, int i) {
        return reinterpret_cast<float4*>(a.sums) +
               (((size_t)place_s * 2 + x) * (kD / 4) + 8 * c + i) * kTile + r;
      };
      // 32 columns of O, the sum outside (if any of it is there yet) added.
      auto whole_sums = [&](int c, bool more, float f, float (&o)[32]) {
        load_cols(o_at + 32 * c, o);
        if (more) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 u = __ldcg(outside(c, i));
            o[4 * i] = fmaf(u.x, f, o[4 * i]);
            o[4 * i + 1] = fmaf(u.y, f, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(u.z, f, o[4 * i + 2]);
            o[4 * i + 3] = fmaf(u.w, f, o[4 * i + 3]);
          }
        }
      };
      // The tile's queries see all of a key tile k0 iff every one of them does.
      const int first = L - n + t0 + x * TQ;
      const int last = L - n + (t0 + (x + 1) * TQ < t1 ? t0 + (x + 1) * TQ : t1) - 1;
      bool ok = true;
      for (int j = 0; j < v.n; ++j) {
        const int k0 = v.tile(j) * kTile;
        const bool whole = k0 + kTile - 1 <= first && (ni - k0 >= kTile || k0 > last - nr);
        ok = wait(&bar.s[x], j & 1);
        if (__builtin_expect(!ok, 0)) break;
        fence_after();
        if (LONG && __builtin_expect(j % kFoldTiles == 0 && j > 0 && place_s >= 0, 0)) {
          const bool more = j > kFoldTiles;
          const float was = more ? under_s[x][r] : m, f = was == m ? 1.f : ex2((was - m) * sc);
          under_s[x][r] = m;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            whole_sums(c, more, f, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              __stcg(outside(c, i),
                     make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
          }
        }
        float s[128];
        load_cols(s_at, s);
        // (the unlikely blocks out of the usual path's instruction stream: 1.29 -> 1.27 ms)
        if (__builtin_expect(!whole, 0)) {
          // columns [0, hi) but [lo, mid): behind the query, between sinks and window
          const int hi = p - k0 + 1, lo = ni - k0, mid = p - nr + 1 - k0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t on = below(hi - 32 * c) & ~(below(mid - 32 * c) & ~below(lo - 32 * c));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(on & (1u << i))) s[32 * c + i] = -INFINITY;
          }
        }
        // Weights of half a tile (64 keys) under the maximum `top`; their sum.
        auto weights = [&](int half, float top) {
          const float off = top == -INFINITY ? 0.f : -top * sc;
          float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 2 * half; c < 2 * half + 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 e = fma2(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]),
                              make_float2(sc, sc), make_float2(off, off));
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              add[i & 1] = add2(add[i & 1], e);
              w[i] = bf16x2(e.x, e.y);
            }
            store_cols(s_at + 16 * c, w);
          }
          return (add[0].x + add[0].y) + (add[1].x + add[1].y);
        };
        auto publish = [&](int half) {  // their products may begin
          wait_stores();
          fence_before();
          mbar_arrive(&bar.p[x][half]);
        };
        // The maximum is off the path from S to P.  Weights are taken under the
        // maximum so far as long as they stay below 2^kRescale: the first half's sum
        // tells for itself, the second half's logits are looked at.  Where they do not
        // (first tiles, rarely later) the maximum is found, O and the sum are rescaled and
        // the weights taken again.
        float l0 = 0.f;
        bool good = m != -INFINITY || !live;  // rows without a query have no say
        if (__builtin_expect(__all_sync(0xffffffffu, good), 1)) {
          float tops[4] = {s[64], s[65], s[66], s[67]};
#pragma unroll
          for (int i = 68; i < 124; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], s[i + e], s[i + 4 + e]);
          const float t = max3(fmaxf(tops[0], s[124]), fmaxf(tops[1], s[125]),
                               max3(tops[2], s[126], fmaxf(tops[3], s[127])));
          l0 = weights(0, m);
          good = (l0 <= kMost && (t - m) * sc <= kRescale) || !live;
        }
        if (__builtin_expect(!__all_sync(0xffffffffu, good), 0)) {
          float tops[4] = {m, m, m, m};
#pragma unroll
          for (int i = 0; i < 128; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], s[i + e], s[i + 4 + e]);
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
          const float f = m == top ? 1.f : ex2((m - top) * sc);
          m = top;
          l *= f;
          if (j > 0) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float o[32];
              load_cols(o_at + 32 * c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f;
              store_cols(o_at + 32 * c, o);
            }
          }
          l0 = weights(0, m);
        }
        publish(0);
        l += l0 + weights(1, m);
        publish(1);
      }
      // O / l; rows without a visible key: 0 and -inf
      if (ok && v.n > 0) {
        ok = wait(&bar.o[x], 0);
        fence_after();
      }
      const bool folds = LONG && place_s >= 0;
      const float was = folds ? under_s[x][r] : m, fs = was == m ? 1.f : ex2((was - m) * sc);
      if (!ok || bad_s) {
        l = nanf("");
        if (m == -INFINITY) m = 0.f;
      }
      if (a.splits > 1) {  // a partial for the kernel that joins them
        const size_t unit = ((size_t)b * a.c.Hkv + g) * a.blocks + block;
        float* mine = a.partial + ((unit * a.splits + part) * 2 + x) * kPreSlot;
        if (live) {
          mine[r] = m * sc;
          mine[kTile + r] = l;
        }
        if (v.n > 0 && ok) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float o[32];
            whole_sums(c, folds, fs, o);
            if (live)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(mine + 2 * kTile + r * kD + 32 * c + 4 * i) =
                    make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
      const bool sums = v.n > 0 && ok, write = a.splits == 1;
      const bool nan = l != l;
      const float inv = nan ? l : (l > 0.f ? 1.f / l : 0.f);
      // A row's 256 bytes go through the warp's own rows of Q's tile, which the
      // products have read, so that a half-warp stores them in one request.
      if (write && sums) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float o[32];
          whole_sums(c, folds, fs, o);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             q_mine + r * 256 + (((4 * c + i) ^ (r & 7)) << 4)),
                         "r"(bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv)),
                         "r"(bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv)),
                         "r"(bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv)),
                         "r"(bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv))
                         : "memory");
        }
        __syncwarp();
      }
      // without sums every row of the CTA is blank: 0, or NaN after a failure
      const uint32_t blank = nan ? 0x7fff7fffu : 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int rr = r_warp + 2 * i + r_half, tt = (rr * a.inv_g) >> 16;
        uint4 w = make_uint4(blank, blank, blank, blank);
        if (sums)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                       : "r"(q_mine + rr * 256 + ((piece ^ (rr & 7)) << 4))
                       : "memory");
        if (write && tt < TQ && t0 + x * TQ + tt < t1)
          *reinterpret_cast<uint4*>(a.out +
                                    ((tok + t0 + x * TQ + tt) * a.Hq + g * G + rr - tt * G) * kD +
                                    8 * piece) = w;
      }
      if (write && live && a.lse)
        a.lse[(tok + my_t) * a.Hq + h] =
            nan ? l : (l > 0.f ? (m * sc + log2f(l)) * 0.6931471805599453f : -INFINITY);
    }
  } else {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
   if (warp == 0 || warp == 3) {
    // ------------------------------------------------ matrix instructions
    // One thread for each query tile (issuing all of them is more than one
    // thread can do in time), by turns: O_A(j), S_A(j+1), then O_B(j), S_B(j+1),
    // so that one tile's softmax runs under the other's products.  K tile j is in
    // the ring's slot of 2j, V tile j in that of 2j + 1.
    const int x = warp == 3;
    if ((x == 0 || two) && elect_one()) {
      const uint32_t s_at = tmem + x * kTile, o_at = s_at + 2 * kTile;
      const uint64_t qd = operand(q_at + x * kSlotBytes, 16);
      const uint64_t kd = operand(ring, 16), vd = operand(ring, kHalf);
      auto qk = [&](int slot) {
        const uint64_t kx = kd + slot * (kSlotBytes >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          mma_ss(s_at, qd + at, kx + at, kIdesc, k > 0);
        }
        commit_mma(&bar.s[x]);
        commit_mma(&bar.empty[slot]);
      };
      bool ok = true;
      if (v.n > 0) {
        ok = wait_for(&bar.q[x], 0, &abort_s) && wait_for(&bar.full[0], 0, &abort_s);
        if (ok && x == 1) ok = wait_for(&bar.turn[1], 0, &abort_s);
        if (ok) qk(0);
        mbar_arrive(&bar.turn[x ^ 1]);
      }
      int slot = 1, lap = 0;                 // of V tile j
      for (int j = 0; j < v.n && ok; ++j) {
        ok = wait_for(&bar.full[slot], lap, &abort_s);
        if (ok && v.edge(j))
          ok = wait_for(&bar.clean[j % kSlots], (j / kSlots) & 1, &abort_s);
        const uint64_t vx = vd + slot * (kSlotBytes >> 4);
        // O begins again every kFoldTiles tiles
        const bool more = LONG ? j % kFoldTiles > 0 || (j > 0 && place_s < 0) : j > 0;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          ok = ok && wait_for(&bar.p[x][part], j & 1, &abort_s);
          if (part == 0 && two) ok = ok && wait_for(&bar.turn[x], (j + x) & 1, &abort_s);
          if (ok) {
            fence_after();
#pragma unroll
            for (int k = 4 * part; k < 4 * part + 4; ++k)
              mma_ts(o_at, s_at + 8 * k, vx + ((k * 16 * 128) >> 4), kIdescV, more || k > 0);
          }
        }
        if (!ok) break;
        commit_mma(&bar.empty[slot]);
        if (++slot == kSlots) slot = 0, lap ^= 1;
        if (j + 1 < v.n) {
          ok = wait_for(&bar.full[slot], lap, &abort_s);
          if (!ok) break;
          qk(slot);
          mbar_arrive(&bar.turn[x ^ 1]);
          if (++slot == kSlots) slot = 0, lap ^= 1;
        } else {
          commit_mma(&bar.o[x]);
          mbar_arrive(&bar.turn[x ^ 1]);
        }
      }
      if (!ok) {  // nothing may still run on tensor memory when it is given back
        commit_mma(&bar.drain[x]);
        mbar_wait(&bar.drain[x], 0);
        atomicOr(a.status, kStatusTimeout);
      }
    }
    __syncwarp();
   } else if (warp == 1) {
    // -------------------------------------------------------------- copies
    const int box = a.box;                   // rows of a box: 128, or a smaller page
    const int per = kTile / box;             // boxes of a tile
    const int i_box = lane >> 1, half = lane & 1;
    const int32_t* pages = a.c.page_table ? a.c.page_table + (int64_t)b * a.c.max_pages : nullptr;
    // Lane's box of tile j: its first row in the pool, or -1 where nothing of it
    // is seen.
    auto find = [&](int j) -> int64_t {
      if (j >= v.n || i_box >= per) return -1;
      const int r0 = v.tile(j) * kTile + i_box * box;
      const bool any = r0 < v.end && (r0 < v.n0 || r0 + box > v.lo);
      if (!any) return -1;
      if (!pages) return ((int64_t)b * a.c.Hkv + g) * a.c.l_cap + r0;
      const int32_t page = pages[r0 >> a.c.page_shift];
      if ((uint32_t)page >= a.c.n_pages) {
        bad_s = 1;
        atomicOr(a.status, kStatusBadLength);
        return -1;
      }
      return (((int64_t)page * a.c.Hkv + g) << a.c.page_shift) + (r0 & ((1 << a.c.page_shift) - 1));
    };
    if (LONG && v.n > kFoldTiles && lane == 0) {
      const int at = take_place(a.places);
      place_s = at;
      if (at < 0) {
        bad_s = 1;
        atomicOr(a.status, kStatusTimeout);
      }
    }
    if (LONG) __syncwarp();
    int64_t next = find(0);
    int issued = 0;
    bool ok = true;
    for (int j = 0; j < v.n && ok; ++j) {
      const int64_t row = next;
      next = find(j + 1);
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * box * 128;
      for (int w = 0; w < 2 && ok; ++w) {
        const int it = 2 * j + w, sl = it % kSlots;
        if (it >= kSlots) ok = wait(&bar.empty[sl], (it / kSlots - 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&bar.full[sl], bytes);
        __syncwarp();
        if (row >= 0)
          copy_box(ring + sl * kSlotBytes + half * kHalf + i_box * box * 128, w ? &vmap : &kmap,
                   64 * half, (int)row, &bar.full[sl]);
        issued = it + 1;
      }
    }
    if (!ok)  // let the copies in flight land
      for (int it = issued > kSlots ? issued - kSlots : 0; it < issued; ++it)
        mbar_wait(&bar.full[it % kSlots], (it / kSlots) & 1);
   } else if (warp == 2) {
    // ---------------------------------------- rows of V that nothing sees
    bool ok = true;
    for (int j = 0; j < v.n && ok; ++j) {
      const int it = 2 * j + 1, k0 = v.tile(j) * kTile;
      if (lane == 0) {
        ok = wait_for(&bar.full[(it - 1) % kSlots], ((it - 1) / kSlots) & 1, &abort_s);
        if (ok) mbar_arrive(&bar.empty[(it - 1) % kSlots]);
        ok = ok && wait_for(&bar.full[it % kSlots], (it / kSlots) & 1, &abort_s);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (k0 + kTile > v.end || (k0 + kTile > v.n0 && k0 < v.lo)) {
        __syncwarp();
        const uint32_t at =
            ring + (it % kSlots) * kSlotBytes + (lane >> 4) * kHalf + (lane & 15) * 8;
        for (int r = 0; r < kTile; ++r)
          if (!v.sees(k0 + r))
            asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(at + r * 128), "r"(0)
                         : "memory");
        fence_proxy_async();
        __syncwarp();
      }
      if (lane == 0) {
        mbar_arrive(&bar.clean[j % kSlots]);
        mbar_arrive(&bar.empty[it % kSlots]);
      }
    }
   }
  }
  fence_before();
  __syncthreads();
  if (LONG && tid == 0 && place_s >= 0) {  // the place is free again
    __threadfence();
    atomicExch(a.places + place_s, 0u);
  }
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Joins the partials of a row (token, query head): a warp a row, lanes over the
// partials' maxima and sums, then over the columns.
__global__ void __launch_bounds__(256) window_join_kernel(PrefillArgs a) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  int64_t tok, n;
  if (!seq_tokens(a.cu, a.max_q, a.T, b, tok, n)) {
    if (tok < 0 || n < 0 || tok + n > a.T) return;
    if (n > a.max_q) n = a.max_q;
  }
  const int64_t j = item / a.Hq;
  const int h = (int)(item % a.Hq), g = h / a.G, TQ = kTile / a.G;
  if (j >= n) return;
  const int block = (int)(j / (2 * TQ)), in = (int)(j % (2 * TQ)), x = in / TQ;
  const int r = (in % TQ) * a.G + h % a.G;
  const size_t unit = ((size_t)b * a.c.Hkv + g) * a.blocks + block;
  const float* p = a.partial + (unit * a.splits * 2 + x) * kPreSlot;
  const size_t step = 2 * (size_t)kPreSlot;  // to the next part; there are at most 32
  const float m = lane < a.splits ? p[lane * step + r] : -INFINITY;
  const float top = warp_max(m);
  const float f = m == -INFINITY ? 0.f : ex2(m - top);
  const float l = warp_sum(lane < a.splits ? p[lane * step + kTile + r] * f : 0.f);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < a.splits; ++k) {
    const float w = __shfl_sync(0xffffffffu, f, k);
    if (w > 0.f) {  // (a part that has seen nothing has left no sums)
      const float4 u =
          *reinterpret_cast<const float4*>(p + k * step + 2 * kTile + r * kD + 4 * lane);
      o.x = fmaf(u.x, w, o.x); o.y = fmaf(u.y, w, o.y);
      o.z = fmaf(u.z, w, o.z); o.w = fmaf(u.w, w, o.w);
    }
  }
  const bool nan = l != l;
  const float inv = nan ? l : (l > 0.f ? 1.f / l : 0.f);
  const int64_t at = (tok + j) * a.Hq + h;
  *reinterpret_cast<uint2*>(a.out + at * kD + 4 * lane) =
      make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
  if (a.lse && lane == 0)
    a.lse[at] = nan ? l : (l > 0.f ? (top + log2f(l)) * 0.6931471805599453f : -INFINITY);
}

}  // namespace

cudaError_t launch_window_prefill(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                  const PrefillArgs& a, int B, cudaStream_t st) {
  const auto kernel = a.sums ? window_prefill_kernel<true> : window_prefill_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute((const void*)kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kPreSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.blocks * a.splits), a.c.Hkv, B);
  return launch_dependent(kernel, grid, dim3(kPreThreads), kPreSmem, st, kmap, vmap, a);
}

cudaError_t launch_window_join(const PrefillArgs& a, int B, cudaStream_t st) {
  const int64_t rows = (a.max_q < a.T ? a.max_q : a.T) * a.Hq;  // of a sequence
  return launch_dependent(window_join_kernel, dim3((unsigned)((rows + 7) / 8), 1, B), dim3(256), 0,
                          st, a);
}

}  // namespace tsa
