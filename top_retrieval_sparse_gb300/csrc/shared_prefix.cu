// shared_prefix.cu -- the shared rows of a decode step's groups: every query of a group over
// the group's rows [0, P), which are read once for up to 256 queries.
//
// Per (group, KV head) the queries are S sequences times G heads, M = S G rows of Q, and
//   S = Q K^T,  W = 2^(S c - m c),  O = W V
// are matrix products of M x 128 by 128 x P and M x P by P x 128, with the running maximum m
// and sum of a softmax.  For M <= 140 or so the rows' bytes bound them, beyond that the
// products do (4 M flop a byte pair of K and V, 280 flop a byte of measured rates).
//
// A unit is 256 queries (two tiles of 128, A and B) of a (group, KV head); its key tiles of
// 128 rows are the work.  All units form one list of costs, which the CTAs, one an SM, take
// in equal contiguous shares, whatever the groups' sizes (they are only known on the
// device).  What a share has of a unit is a segment; each leaves (O, maximum, sum) in the
// workspace, and the joining kernel adds them, and the own rows', in order.
// Where the unit has more than 128 queries, A and B take the same key tiles and one's
// softmax runs under the other's products.  Where it has not, A takes the even and B the
// odd tiles for the same queries, so that a tile's chain of copy, product, softmax, product
// is hidden by the other's all the same.
//
// Warps.  0 and 3: the matrix instructions of A and of B, 1: the copies, 2: the rows of V
// behind P (zeroed, for whatever they hold 0 * NaN would reach the output), 4-7: softmax of
// A (thread = row = tensor-memory lane), 8-11: of B.  K and V tiles go through a ring of
// five 32 KB slots by TMA (two 64-column boxes with the 128-byte swizzle; a box a page where
// pages are smaller than a tile), which runs on across segments.  A slot is filled again
// when its three readers have given it back: both matrix threads, or one and the zeroing
// warp for the other, and the zeroing warp.  It passes every slot in order, so nobody falls
// behind by two laps and a barrier's parity is never taken for another lap's.
#include "shared_attn.h"
#include "tcgen.cuh"

namespace tsa {

namespace {

constexpr int kSlots = 5;
constexpr int kSharedThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // 2 * 216 + 72 = 3 * 168 a scheduler
constexpr int kSharedSmem = (2 + kSlots) * kSlotBytes + 1024;
// Weights may grow to 2^16 under an old maximum before O is rescaled: bf16 and fp32 keep
// their precision at any size.
constexpr float kRescale = 16.f, kMost = 65536.f;
// Matrix instructions truncate their 32-bit sums, all in one direction (6.3e-9 of a sum of
// one sign for every row and part of a weight): after so many of a stream's tiles O is added,
// with rounding, to the sum in the workspace and begins again.
template <int PARTS>
constexpr int kFoldEvery = PARTS == 2 ? 32 : 128;

struct SharedBars {
  uint64_t q[2], s[2], p[2][2], o[2], full[kSlots], empty[kSlots], clean[kSlots], drain[2],
      turn[2];
};

// Slot i of the ring's endless row, and the parity of its barriers there.
__device__ __forceinline__ int slot_of(uint32_t i) { return i % kSlots; }
__device__ __forceinline__ uint32_t lap_of(uint32_t i) { return i / kSlots & 1u; }

template <int PARTS>
__global__ void __launch_bounds__(kSharedThreads, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, SharedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ SharedBars bar;
  __shared__ uint32_t tmem_s;
  __shared__ volatile int abort_s;
  __shared__ volatile int bad_s[8];          // number of a segment that met a bad page
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
      mbar_init(&bar.empty[i], 3);
      mbar_init(&bar.clean[i], 1);
    }
    fence_mbar_init();
    abort_s = 0;
  }
  if (tid < 8) bad_s[tid] = 0;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&tmem_s))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tmem_s;
  // The whole warp agrees, where what follows is a warp's work.
  auto wait = [&](uint64_t* x, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_for(x, parity, &abort_s)) != 0;
  };
  SharedWalk walk(a, blockIdx.x);

  if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = (warp >> 2) - 1;           // stream A or B
    const int r = tid & 127;                 // row of the stream's tile
    const int r_warp = (warp & 3) * 32, r_half = lane >> 4, piece = lane & 15;
    const uint32_t q_mine = q_at + x * kSlotBytes;
    const uint32_t s_at = tmem + x * kTile + ((uint32_t)(warp & 3) << 21);
    const uint32_t o_at = s_at + 2 * kTile;
    const float sc = a.scale_log2 < 0.f ? -a.scale_log2 : (a.scale_log2 == 0.f ? 1.f : a.scale_log2);
    uint32_t tiles = 0, segs = 0;            // of this stream, so far
    bool ok = true;
    for (int number = 1; walk.next(); ++number) {
      const SharedUnit& u = walk.u;
      const bool both = u.both();
      const int first = both ? x * kTile : 0;            // the stream's first row of the unit
      const bool live = first + r < u.rows;
      const bool warp_live = first + r_warp < u.rows;
      const int all = walk.j1 - walk.j0;
      const int n = both ? all : (all - x + 1) / 2;      // tiles of this stream
      const int P = walk.s.P, rs = u.rs;
      float* mine = segment_parts(a, u, blockIdx.x, walk.j0) + x * half_floats(rs);
      float4* sums = reinterpret_cast<float4*>(mine) + r;  // columns 4 i .. at sums[i * rs]
      float m = -INFINITY, l = 0.f;
      if (n > 0 && ok) {
        // Q, swizzled as the copies would: rows of 128 bytes, piece c at c ^ (row & 7).
        // A half-warp a row, so that a row's 256 bytes are one request.
        {
          const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
          const int seq0 = u.t * kUnitRows / a.G, in0 = u.t * kUnitRows - seq0 * a.G;
          uint4 w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int rr = first + r_warp + 2 * i + r_half;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (rr < u.rows && a.scale_log2 != 0.f) {
              const int sq = ((in0 + rr) * a.inv_g) >> 16, h = in0 + rr - sq * a.G;
              w[i] = *reinterpret_cast<const uint4*>(
                  a.q + ((int64_t)(walk.s.b0 + seq0 + sq) * a.Hq + u.g * a.G + h) * kD + 8 * piece);
            }
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

        bool more = false;                   // a sum is in the workspace, under `under`
        float under = 0.f;
        // 32 columns of O, and the sum in the workspace.
        auto whole = [&](int c, float f, float (&o)[32]) {
          load_cols(o_at + 32 * c, o);
          if (more && live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 u = __ldcg(sums + (8 * c + i) * rs);
              o[4 * i] = fmaf(u.x, f, o[4 * i]);
              o[4 * i + 1] = fmaf(u.y, f, o[4 * i + 1]);
              o[4 * i + 2] = fmaf(u.z, f, o[4 * i + 2]);
              o[4 * i + 3] = fmaf(u.w, f, o[4 * i + 3]);
            }
          }
        };
        auto put = [&]() {
          const float f = !more || under == m ? 1.f : ex2((under - m) * sc);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            whole(c, f, o);
            if (live)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                __stcg(sums + (8 * c + i) * rs,
                       make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
          }
          more = true;
          under = m;
        };
        for (int j0 = 0; j0 < n && ok; j0 += kFoldEvery<PARTS>) {
          const int j1 = j0 + kFoldEvery<PARTS> < n ? j0 + kFoldEvery<PARTS> : n;
          for (int j = j0; j < j1; ++j) {
            const int k0 = (walk.j0 + (both ? j : 2 * j + x)) * kTile;
            const uint32_t parity = (tiles + j) & 1;
            ok = wait(&bar.s[x], parity);
            if (__builtin_expect(!ok, 0)) break;
            if (!warp_live) {  // nobody reads these rows' weights
              mbar_arrive(&bar.p[x][0]);
              mbar_arrive(&bar.p[x][1]);
              continue;
            }
            fence_after();
            // (S is there, so O's products before it are done)
            if (__builtin_expect(j == j0 && j > 0, 0)) put();
            float s[128];
            load_cols(s_at, s);
            if (__builtin_expect(k0 + kTile > P, 0)) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t on = below(P - k0 - 32 * c);
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
                uint32_t w[16], w2[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float2 e = fma2(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]),
                                  make_float2(sc, sc), make_float2(off, off));
                  e.x = ex2(e.x);
                  e.y = ex2(e.y);
                  add[i & 1] = add2(add[i & 1], e);
                  w[i] = bf16x2(e.x, e.y);
                  if (PARTS == 2) {
                    const float2 h = make_float2(bf_lo(w[i]), bf_hi(w[i]));
                    const float2 d = fma2(h, make_float2(-1.f, -1.f), e);
                    w2[i] = bf16x2(d.x, d.y);
                  }
                }
                store_cols(s_at + (PARTS == 2 ? 32 : 16) * c, w);
                if (PARTS == 2) store_cols(s_at + 32 * c + 16, w2);
              }
              return (add[0].x + add[0].y) + (add[1].x + add[1].y);
            };
            auto publish = [&](int half) {  // their products may begin
              wait_stores();
              fence_before();
              mbar_arrive(&bar.p[x][half]);
            };
            // The maximum is off the path from S to the weights.  They are taken under the
            // maximum so far as long as they stay below 2^kRescale: the first half's sum
            // tells for itself, the second half's logits are looked at.  Where they do not
            // (first tiles, rarely later) the maximum is found, O and the sum are rescaled
            // and the weights taken again.
            float l0 = 0.f;
            bool good = m != -INFINITY || !live;
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
              if (j > j0) {
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
        }
        if (ok) ok = wait(&bar.o[x], segs & 1);
        if (ok && warp_live) {
          fence_after();
          put();
          fence_before();
        }
        tiles += n;
        ++segs;
      }
      if (!ok || bad_s[number & 7] == number) {
        l = nanf("");
        m = 0.f;
      }
      if (live) {
        float* stats = mine + (size_t)rs * kD;
        stats[r] = m * sc;
        stats[rs + r] = l;
      }
    }
  } else {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
   if (warp == 0 || warp == 3) {
    // ------------------------------------------------ matrix instructions
    // One thread for each stream.  With both on the same tiles by turns: O_A(j), S_A(j+1),
    // then O_B(j), S_B(j+1).  One thread's execute in order: S(j+1) may overwrite the
    // weights of j without a wait.
    const int x = warp == 3;
    if (elect_one()) {
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
      // so far: tiles and segments of this stream, turns, tiles of the segments
      uint32_t tiles = 0, segs = 0, turns = 0, passed = 0;
      bool ok = true;
      while (ok && walk.next()) {
        const bool both = walk.u.both();
        const int all = walk.j1 - walk.j0, n = both ? all : (all - x + 1) / 2;
        auto number = [&](int j) { return passed + (both ? j : 2 * j + x); };
        if (n > 0) {
          const uint32_t i = 2 * number(0);
          ok = wait_for(&bar.q[x], segs & 1, &abort_s) &&
               wait_for(&bar.full[slot_of(i)], lap_of(i), &abort_s);
          if (both && x == 1) ok = ok && wait_for(&bar.turn[1], turns & 1, &abort_s);
          if (ok) {
            fence_after();
            qk(slot_of(i));
          }
          if (both) mbar_arrive(&bar.turn[x ^ 1]);
        }
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t tile = number(j), i = 2 * tile + 1;  // V's slot
          ok = wait_for(&bar.full[slot_of(i)], lap_of(i), &abort_s);
          if (ok && (walk.j0 + (int)(tile - passed) + 1) * kTile > walk.s.P)
            ok = wait_for(&bar.clean[slot_of(tile)], lap_of(tile), &abort_s);
          const uint64_t vx = vd + slot_of(i) * (kSlotBytes >> 4);
          const bool more = j % kFoldEvery<PARTS> > 0;
          const uint32_t parity = (tiles + j) & 1;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && wait_for(&bar.p[x][half], parity, &abort_s);
            if (half == 0 && both)
              ok = ok && wait_for(&bar.turn[x], (turns + j + x) & 1, &abort_s);
            if (ok) {
              fence_after();
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k) {
                const uint64_t vk = vx + ((k * 16 * 128) >> 4);
                if (PARTS == 2) {
                  const uint32_t w = s_at + 32 * (k >> 1) + 8 * (k & 1);
                  mma_ts(o_at, w, vk, kIdescV, more || k > 0);
                  mma_ts(o_at, w + 16, vk, kIdescV, true);
                } else {
                  mma_ts(o_at, s_at + 8 * k, vk, kIdescV, more || k > 0);
                }
              }
            }
          }
          if (!ok) break;
          commit_mma(&bar.empty[slot_of(i)]);
          if (j + 1 < n) {
            const uint32_t k = 2 * number(j + 1);
            ok = wait_for(&bar.full[slot_of(k)], lap_of(k), &abort_s);
            if (!ok) break;
            qk(slot_of(k));
          } else {
            commit_mma(&bar.o[x]);
          }
          if (both) mbar_arrive(&bar.turn[x ^ 1]);
        }
        if (both) {  // (A sees B's last arrival, so that neither's count runs ahead)
          if (x == 0) ok = ok && wait_for(&bar.turn[0], (turns + n) & 1, &abort_s);
          turns += n + 1;
        }
        tiles += n;
        segs += n > 0;
        passed += all;
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
    uint32_t it = 0;
    bool ok = true;
    for (int number = 1; ok && walk.next(); ++number) {
      const int b = walk.s.b0, g = walk.u.g, P = walk.s.P;
      const int32_t* pages =
          a.c.page_table ? a.c.page_table + (int64_t)b * a.c.max_pages : nullptr;
      // Lane's box of key tile j: its first row in the pool, or -1 where nothing of it
      // is seen.
      auto find = [&](int j) -> int64_t {
        if (j >= walk.j1 || i_box >= per) return -1;
        const int r0 = j * kTile + i_box * box;
        if (r0 >= P) return -1;
        if (!pages) return ((int64_t)b * a.c.Hkv + g) * a.c.l_cap + r0;
        const int32_t page = pages[r0 >> a.c.page_shift];
        if ((uint32_t)page >= a.c.n_pages) {
          bad_s[number & 7] = number;
          atomicOr(a.status, kStatusBadLength);
          return -1;
        }
        return (((int64_t)page * a.c.Hkv + g) << a.c.page_shift) +
               (r0 & ((1 << a.c.page_shift) - 1));
      };
      int64_t next = find(walk.j0);
      for (int j = walk.j0; j < walk.j1 && ok; ++j) {
        const int64_t row = next;
        next = find(j + 1);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * box * 128;
        for (int w = 0; w < 2 && ok; ++w) {
          const int sl = slot_of(it);
          if (it >= kSlots) ok = wait(&bar.empty[sl], lap_of(it) ^ 1);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&bar.full[sl], bytes);
          __syncwarp();
          if (row >= 0)
            copy_box(ring + sl * kSlotBytes + half * kHalf + i_box * box * 128, w ? &vmap : &kmap,
                     64 * half, (int)row, &bar.full[sl]);
          ++it;
        }
      }
    }
    if (!ok)  // let the copies in flight land
      for (uint32_t i = it > kSlots ? it - kSlots : 0; i < it; ++i)
        mbar_wait(&bar.full[slot_of(i)], lap_of(i));
   } else if (warp == 2) {
    // ---------------------------------------- rows of V behind the shared ones
    uint32_t tile = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const bool both = walk.u.both();
      for (int j = walk.j0; j < walk.j1 && ok; ++j, ++tile) {
        // every slot is given back for this warp, and for the stream that passes it by
        auto give = [&](uint32_t i) {
          mbar_arrive(&bar.empty[slot_of(i)]);
          if (!both) mbar_arrive(&bar.empty[slot_of(i)]);
        };
        const uint32_t i = 2 * tile;
        if (lane == 0) {
          ok = wait_for(&bar.full[slot_of(i)], lap_of(i), &abort_s);
          if (ok) give(i);
          ok = ok && wait_for(&bar.full[slot_of(i + 1)], lap_of(i + 1), &abort_s);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int left = walk.s.P - j * kTile;
        if (left < kTile) {
          const uint32_t at = ring + slot_of(i + 1) * kSlotBytes + (lane >> 4) * kHalf +
                              (lane & 15) * 8;
          for (int r = left; r < kTile; ++r)
            asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(at + r * 128), "r"(0)
                         : "memory");
          fence_proxy_async();
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive(&bar.clean[slot_of(tile)]);
          give(i + 1);
        }
      }
    }
   }
  }
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

}  // namespace

cudaError_t launch_shared_prefix(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const SharedArgs& a, cudaStream_t st) {
  const auto kernel = a.out16 ? shared_prefix_kernel<1> : shared_prefix_kernel<2>;
  const cudaError_t e = cudaFuncSetAttribute(
      (const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(kSharedShares), dim3(kSharedThreads), kSharedSmem, st, kmap,
                          vmap, a);
}

}  // namespace tsa
