/*
 * tsa.h -- C ABI of libtsa: decode-step top-K sparse attention on one GB300.
 *
 * One decode step of one attention layer: for every query head, score the
 * query against every key of the cache, keep the exact top-K keys outside a
 * static window of initial + recent tokens, attend over those K rows and over
 * the window separately, and merge the two partial results with the
 * log-sum-exp rescale.  A second entry point runs ReTopK's reuse path, which
 * recalls candidate keys from a per-head cache of past queries instead of
 * scanning every key on most steps.  Beside them stand the operators that a
 * program needs around the cache: rotary positions, an 8-bit cache (written with
 * rotated keys, read back, attended), and attention with a sliding window and
 * sinks for one token or many.
 *
 * Sources (page title, section / equation):
 *   [RA]  "RetrievalAttention: Accelerating Long-Context LLM Inference via
 *         Vector Retrieval": Eq. 1, Eq. 2, Eq. 3, Eq. 4-5, the "Flat"
 *         exact-KNN baseline, "CPU-GPU Co-Execution" (static pattern W),
 *         Appendix B.2 Algorithm 1 (per-step window update).
 *   [RTK] "Recall Before You Rank: Similarity-Guided Top-K Reuse for
 *         Efficient Long-Context Attention" (ReTopK): sections 1-5 of the
 *         method (query-support cache, similar-query recall, candidate set,
 *         exact re-ranking, fallback and refresh) and "GPU Kernel".
 *   [RA-review] the English review of RetrievalAttention: Appendix C "CPU
 *         memory minimization" and the future-work item "Scalar
 *         quantization of KV vectors with accuracy-preservation
 *         guarantees" (8-bit scalar quantisation of the keys).
 *
 * Conventions shared by every entry point
 *   - Element types: q, K, V are bf16 (IEEE binary16-brain, 2 bytes);
 *     outputs are fp32; indices are int32 token positions (0-based).
 *   - Head dimension d must be 128 (the only compiled size).
 *   - GQA: query head h reads KV head h / (Hq / Hkv); Hq % Hkv == 0,
 *     Hq / Hkv <= 8, B * Hkv <= 512 and B * Hq <= 65535.
 *   - Ownership: the caller allocates every buffer (device memory unless
 *     stated) and the workspace, and owns the stream.  No entry point
 *     allocates, frees or prints, and none but tsa_workspace_status
 *     synchronises; launches are asynchronous on `stream` (a cudaStream_t;
 *     NULL = legacy default stream).
 *   - Errors: every call returns a tsa_status.  Arguments are validated on
 *     the host before any launch; on an error nothing is launched and
 *     tsa_last_error() describes the problem (thread-local).  Launch
 *     failures are reported as TSA_ERR_CUDA.  Faults inside a kernel surface
 *     through the stream as usual CUDA errors.  What the kernels detect
 *     themselves (a bounded wait that expired, a length outside the cache)
 *     goes into a sticky status word in the workspace, which
 *     tsa_workspace_status() reads after the calls have run.
 *   - Concurrency: calls that share a workspace or a ReTopK state must be
 *     ordered on one stream.
 */
#ifndef TSA_H
#define TSA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define TSA_API __attribute__((visibility("default")))
#else
#define TSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tsa_status {
  TSA_OK = 0,
  TSA_ERR_INVALID_ARG = -1, /* a size, pointer or layout argument is invalid */
  TSA_ERR_WORKSPACE = -2,   /* workspace pointer NULL/misaligned or too small */
  TSA_ERR_CUDA = -3,        /* a CUDA runtime call or launch failed           */
  TSA_ERR_STATE = -4,       /* ReTopK state handle invalid or not initialised */
  TSA_ERR_DEVICE_CHECK = -5,/* a device-side check flagged bad input          */
  TSA_ERR_TIMEOUT = -6      /* a bounded device wait expired (status word)    */
} tsa_status;

/* KV cache of one layer.
 *
 * Contiguous layout (page_table == NULL):
 *   k, v: bf16 [B][Hkv][l_cap][128]; sequence b, KV head g, position i at
 *   element ((b*Hkv + g)*l_cap + i)*128.
 * Paged layout (page_table != NULL):
 *   k, v: bf16 [num_pages][Hkv][page_size][128]; page_table: int32
 *   [B][max_pages] (device); position i of sequence b lives in page
 *   page_table[b*max_pages + i/page_size] at row i % page_size.
 *   page_size is a power of two in [16, 256]; l_cap = max_pages*page_size.
 * Base pointers must be 16-byte aligned.  Positions >= the sequence length
 * are never read. */
typedef struct tsa_kv {
  const void* k;
  const void* v;
  const int32_t* page_table;
  int32_t page_size;
  int32_t max_pages;
  int64_t l_cap;
} tsa_kv;

/* Human-readable description of the last error on this thread ("" if none). */
TSA_API const char* tsa_last_error(void);

/* Version string of the library build. */
TSA_API const char* tsa_version(void);

/* Number of kernels this library has launched in this process so far (all
 * threads, all entry points; a memset of workspace counters is not a
 * kernel and is not counted). */
TSA_API unsigned long long tsa_kernel_launches(void);

/* Per-stage timing (optional, thread-local).  With n >= 4 cudaEvent_t
 * handles (cast to void*), every later sparse_attn_decode / retopk_step call
 * on this thread records, on the call's stream, events[0] before its first
 * kernel, events[1] after the key scan, events[2] at once after events[1]
 * (the selection is the finish kernel's) and events[3] after the finish
 * kernel (selection, attention and merge; on ReTopK steps also the reuse
 * heads' rescoring and the FIFO push).  Events between kernels cost the overlap of their
 * launches.  events == NULL (or n == 0) turns it off.  The events stay owned
 * by the caller. */
TSA_API int tsa_set_stage_events(void* const* events, int n);

/* Per-CTA kernel timeline (optional, thread-local).  `buf` is device memory
 * (64-byte aligned) holding a uint32 record count at offset 0, which the
 * caller zeroes, followed from offset 64 by records of 48 bytes:
 *   uint32 kernel (1 key scan, 4 ReTopK selector, 7 finish (selection +
 *   attention), 8 finish phases; 2, 3, 5 and 6 are unused), uint32 CTA
 *   (linear block index), uint32 SM id, uint32 info (kernel 7: pairs the
 *   scan emitted for the head; kernel 8: bit 31 re-emission, bits 16-30
 *   the threshold bin, bits 0-15 the emission bin used; else 0),
 *   uint64 t[4] (%globaltimer ns: start, two kernel-specific phase marks
 *   or 0, exit; kernel 4: start, dependency wait over, candidate bitmap
 *   built, exit; kernel 8: start, threshold bin found, list read, rows
 *   gathered).
 * Later calls on this thread append one record per CTA while it fits.
 * buf == NULL (or too small) turns tracing off. */
TSA_API int tsa_set_trace(void* buf, size_t bytes);

/* ------------------------------------------------------------------ */
/* sparse_attn_decode -- [RA] Eq. 1-5 with an exact ("Flat") top-K Omega.
 *
 * For each sequence b (length L_b = lens[b], the newest token included)
 * and query head h:
 *   z_i   = scale * q_h . k_i                       for i < L_b   (Eq. 1)
 *   W     = [0, n_init) u [L_b - n_recent, L_b), clipped        (static W)
 *   Omega = the K positions of [0, L_b) \ W with the largest z,
 *           ties to the smaller position; all of it if smaller than K
 *   o_W, o_Omega: softmax-weighted V over W and Omega (Eq. 3)
 *   out   = g1 o_W + g2 o_Omega, lse = log sum_{W u Omega} e^z  (Eq. 4-5)
 *
 * q:          bf16 [B][Hq][128] (device)
 * kv:         the cache (see tsa_kv); read only
 * lens:       int32 [B] (device), 0 <= lens[b] <= kv->l_cap
 * K:          top-K budget (>= 0); n_init, n_recent >= 0
 * scale:      logit scale (1/sqrt(128) for standard attention)
 * out:        fp32 [B][Hq][128] (device)
 * lse_out:    fp32 [B][Hq] or NULL; -inf when W u Omega is empty
 * topk_idx:   int32 [B][Hq][K] or NULL: Omega in unspecified order, padded
 *             with -1 when fewer than K positions exist
 * topk_score: fp32 [B][Hq][K] or NULL: z of topk_idx (padding: -inf)
 * workspace:  device scratch of at least tsa_decode_workspace_size() bytes,
 *             256-byte aligned, zero-filled (e.g. cudaMemsetAsync 0) before
 *             its first use.  Every call leaves it ready for the next call
 *             with the same B, Hq, Hkv, l_cap, K, n_init and n_recent, so
 *             it is reused as is; zero it again before other sizes and after
 *             a call that failed.  It also keeps per-head state
 *             that speeds up the next call (never its result): use one
 *             workspace per layer.
 * Device-detected errors (read them with tsa_workspace_status):
 *   - every wait inside the kernels is bounded (1 s); if one expires the
 *     kernel gives up, the call's out / lse / topk_score are NaN and
 *     topk_idx is -1, the workspace stays consistent, and the status word
 *     keeps TSA_ERR_TIMEOUT: every later call on the workspace also outputs
 *     NaN until tsa_workspace_status(..., clear = 1) has cleared it;
 *   - a lens[b] outside [0, l_cap] is clamped to that range and reported as
 *     TSA_ERR_DEVICE_CHECK (the outputs are those of the clamped length).
 * Returns TSA_OK or an error; see the conventions above. */
TSA_API size_t tsa_decode_workspace_size(int B, int Hq, int Hkv, int d, int64_t l_cap,
                                 int K, int n_init, int n_recent);

TSA_API int sparse_attn_decode(const void* q, const tsa_kv* kv, const int32_t* lens,
                       int B, int Hq, int Hkv, int d, int K, int n_init,
                       int n_recent, float scale, float* out, float* lse_out,
                       int32_t* topk_idx, float* topk_score, void* workspace,
                       size_t ws_bytes, void* stream);

/* sparse_attn_decode_noalloc -- sparse_attn_decode without a caller
 * workspace.  The pages have no counterpart: this is a library service.
 *
 * For callers that cannot allocate device memory when they decode: a serving
 * engine that gives nearly all device memory to its KV-cache pool at start-up
 * and allows no later allocation, or a host for which cudaMalloc (it may
 * synchronise the device) is off limits inside the decode loop.  The scratch
 * lives in one array of tsa_noalloc_scratch_bytes() (32 MiB) of device
 * memory per device, which the library's module holds from the time it is
 * loaded on that device until the process exits.
 *
 * Same arguments and results as sparse_attn_decode, minus the workspace.
 *   - Problems whose tsa_decode_workspace_size() exceeds the array are
 *     rejected with TSA_ERR_WORKSPACE (nothing launched).  The size grows as
 *     B*Hq*16*(l_cap + 65536) bytes plus 12 KiB per head: B*Hq = 4 fits
 *     caches up to about 458 K positions, B*Hq = 16 about 65 K, and
 *     B*Hq >= 32 fits none.
 *   - The arguments are checked as in sparse_attn_decode before the array
 *     or the stream is touched.
 *   - Each call clears the array's status word with its counters, so a
 *     timeout shows as NaN outputs of that call only.
 *   - The first call on a device looks the array's device address up
 *     (cudaGetSymbolAddress, with that device current), which may load the
 *     library's module; make that first call before any stream capture.
 *   - Every call on a device, from any thread or stream, uses the same
 *     array, which keeps the previous call's contents; each call clears the
 *     counters that must start at zero on its stream.  Calls that overlap on
 *     the GPU race: order them on one stream.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library call. */
TSA_API size_t tsa_noalloc_scratch_bytes(void);

TSA_API int sparse_attn_decode_noalloc(const void* q, const tsa_kv* kv,
                       const int32_t* lens, int B, int Hq, int Hkv, int d, int K,
                       int n_init, int n_recent, float scale, float* out,
                       float* lse_out, int32_t* topk_idx, float* topk_score,
                       void* stream);

/* ------------------------------------------------------------------ */
/* int8 key codes and the quantised decode -- [RA-review] Appendix C "CPU
 * memory minimization" (8-bit scalar quantisation of the key vectors,
 * scheme left open) and the future-work item "Scalar quantization of KV
 * vectors with accuracy-preservation guarantees" (per-channel symmetric is
 * the scheme used here; the worry there -- quantised keys shift the top-K --
 * is removed by rescoring: the result is that of the bf16 keys).
 *
 * tsa_kq8: a quantised copy of a cache's keys, caller memory.
 *   codes: uint8, the row geometry of kv->k with one byte per element
 *          (contiguous [B][Hkv][l_cap][128], or paged [pages][Hkv]
 *          [page_size][128] through kv->page_table); the code c in
 *          [-127, 127] of k_ij is stored as the byte c + 128.  16-byte
 *          aligned.
 *   scale: fp32 [B][Hkv][128], the step s_j of each channel.
 *   err:   fp32 [B][Hkv][128], an upper bound of |k_ij - s_j c_ij| over
 *          every coded row of the channel.
 *   Per channel: s_j = maxabs_j / 127 (binary32 division, maxabs over the
 *   fitted rows), c_ij = clamp(rint(k_ij / s_j), -127, 127) (binary32
 *   quotient, ties to even; c = 0 where s_j = 0). */
typedef struct tsa_kq8 {
  void* codes;
  float* scale;
  float* err;
} tsa_kq8;

/* tsa_quantize_keys -- codes of a cache's keys.
 *   fit = 1: for each (sequence b, KV head, channel) s_j from the rows
 *            [0, lens[b]), then codes and err of those rows (n_tail unused);
 *   fit = 0: codes of the last n_tail rows [lens[b] - n_tail, lens[b])
 *            (clipped at 0) with the stored scales; err is raised to cover
 *            them (a value past 127 s_j saturates; its error counts).
 * lens: int32 [B] (device), 0 <= lens[b] <= kv->l_cap.  Launches up to three
 * kernels (and two memsets with fit) on `stream`; reads kv->k only.
 * Returns TSA_OK or an error (nothing launched on an argument error). */
TSA_API int tsa_quantize_keys(const tsa_kv* kv, const tsa_kq8* kq, const int32_t* lens,
                              int B, int Hkv, int d, int64_t n_tail, int fit,
                              void* stream);

/* sparse_attn_decode_q8 -- sparse_attn_decode with the pool scanned through
 * the key codes (128 bytes a key row instead of 256).
 *
 * Same arguments, contract and results as sparse_attn_decode: the selected
 * set Omega, topk_idx / topk_score (the logits of the bf16 keys, bit for bit
 * those sparse_attn_decode reports) and, up to the order of fp32 sums, out and
 * lse.  The codes must cover rows [0, lens[b] - n_new) of every sequence
 * when the call starts; the call first codes the last n_new rows (as
 * tsa_quantize_keys with fit = 0), so a decode loop that appends one key a
 * step passes n_new = 1.
 * How: per query head a bound eps on |z_i - z^_i| (z^ the logit of the codes)
 * is computed from err, the scales and the query; the scan emits the pool
 * positions with z^ >= k^ (the head's emission key); the finish kernel
 * rescores every emitted position on the bf16 keys and keeps those with
 * z >= k^ + eps, which are all the pool positions with such a logit; when
 * they are fewer than K it rescans the head's bf16 keys (slow, exact).
 * workspace: tsa_decode_q8_workspace_size() bytes, same rules as
 * sparse_attn_decode's (a q8 workspace is not interchangeable with a plain
 * one). */
TSA_API size_t tsa_decode_q8_workspace_size(int B, int Hq, int Hkv, int d, int64_t l_cap,
                                            int K, int n_init, int n_recent);

TSA_API int sparse_attn_decode_q8(const void* q, const tsa_kv* kv, const tsa_kq8* kq,
                                  int n_new, const int32_t* lens, int B, int Hq, int Hkv,
                                  int d, int K, int n_init, int n_recent, float scale,
                                  float* out, float* lse_out, int32_t* topk_idx,
                                  float* topk_score, void* workspace, size_t ws_bytes,
                                  void* stream);

/* tsa_workspace_status -- the device-side status of a decode or ReTopK
 * workspace.  The pages have no counterpart: this is error reporting.
 *
 * Synchronises `stream` (the only entry point that does), then reads the
 * workspace's status word (written by the kernels of earlier calls on it):
 *   TSA_OK               nothing was flagged;
 *   TSA_ERR_TIMEOUT      a bounded wait expired in some call (its outputs,
 *                        and those of every later call, are NaN);
 *   TSA_ERR_DEVICE_CHECK a device-side check flagged bad input (a sequence
 *                        length outside [0, l_cap], clamped).
 * With clear != 0 the word is reset to zero, so the next call runs normally
 * (the rest of the workspace needs no reset).  workspace: the pointer given
 * to sparse_attn_decode or retopk_step (256-byte aligned). */
TSA_API int tsa_workspace_status(void* workspace, int clear, void* stream);

/* tsa_inject_scan_stall -- fault injection for tests of the error path.
 *
 * Makes the next sparse_attn_decode or retopk_step call on this thread
 * wait at most wait_limit_ns (1 .. 1e9) in its key scan, and makes the
 * scan's first CTA withhold the copy of its first key tile, so that the
 * bounded waits of that CTA expire: the call then reports TSA_ERR_TIMEOUT
 * through tsa_workspace_status, with NaN outputs, and the device stays
 * usable.  One call only; 0 cancels a pending injection.  Nothing is
 * launched by this function. */
TSA_API int tsa_inject_scan_stall(long long wait_limit_ns);

/* sparse_attn_decode_shard -- one shard of a sequence split over devices
 * ([RA] Eq. 4-5: partial attentions over disjoint sets merge exactly).
 *
 * The cache `kv` (B = 1) holds positions [pos_offset, pos_offset +
 * shard_len) of a sequence of global_len positions, local row i being global
 * position pos_offset + i.  For each query head this computes, over the
 * shard's rows, what sparse_attn_decode computes over a whole cache, with the
 * static window taken in global positions ([0, n_init) u [global_len -
 * n_recent, global_len), met by the shard in a prefix and a suffix of it):
 *   topk_idx / topk_score: the shard's local top-K outside the window, as
 *     LOCAL row indices (add pos_offset for global positions) and logits;
 *   out / lse_out: attention over the shard's window rows and that local
 *     top-K (Eq. 4-5).
 * A split decode step: every shard runs this, the shards exchange their K
 * (logit, global position) pairs per head, every shard keeps the pairs of the
 * global top-K that it holds and runs attend_set over them plus its window
 * rows, and lse_merge folds the shards' (out, lse).
 * q: bf16 [Hq][128]; out fp32 [Hq][128]; lse_out fp32 [Hq] or NULL;
 * topk_idx int32 [Hq][K] or NULL; topk_score fp32 [Hq][K] or NULL.
 * 0 <= shard_len <= kv->l_cap, pos_offset >= 0, pos_offset + shard_len <=
 * global_len.  workspace: tsa_decode_workspace_size(1, Hq, Hkv, d, l_cap, K,
 * n_init, n_recent) bytes, as for sparse_attn_decode. */
TSA_API int sparse_attn_decode_shard(const void* q, const tsa_kv* kv, int64_t shard_len,
                                     int64_t pos_offset, int64_t global_len, int Hq, int Hkv,
                                     int d, int K, int n_init, int n_recent, float scale,
                                     float* out, float* lse_out, int32_t* topk_idx,
                                     float* topk_score, void* workspace, size_t ws_bytes,
                                     void* stream);

/* attend_set -- attention over a given set of rows ([RA] Eq. 3: the partial
 * o_Omega over a set Omega chosen elsewhere).
 *
 * For each sequence b and query head h: z_i = scale * q_h . k_i for the
 * counts[b][h] positions positions[b][h][0 .. counts-1] (rows of this
 * cache), out = softmax(z) . V over them, lse = log sum e^z (an empty set:
 * out 0, lse -inf).  No window is added; each listed row counts once per
 * listing.  q: bf16 [B][Hq][128]; positions: int32 [B][Hq][M] (device),
 * entries past counts ignored; counts: int32 [B][Hq] (device), 0..M;
 * out fp32 [B][Hq][128]; lse_out fp32 [B][Hq] or NULL.  A position outside
 * [0, kv->l_cap) is never read: it is left out and reported as
 * TSA_ERR_DEVICE_CHECK by tsa_workspace_status.  1 <= M <= 2^24.
 * workspace: tsa_attend_set_workspace_size(B, Hq, M) bytes, 256-byte
 * aligned, zero-filled before its first use (calls leave it ready). */
TSA_API size_t tsa_attend_set_workspace_size(int B, int Hq, int M);
TSA_API int attend_set(const void* q, const tsa_kv* kv, int B, int Hq, int Hkv, int d,
                       const int32_t* positions, const int32_t* counts, int M, float scale,
                       float* out, float* lse_out, void* workspace, size_t ws_bytes,
                       void* stream);

/* ------------------------------------------------------------------ */
/* Rotary positions.
 *
 * For a head row x and a position t, every pair i < rot_dim/2 of elements is
 * turned by the angle t * w_i and multiplied by the amplitude:
 *   (a, b) -> amplitude * (a cos - b sin, b cos + a sin),
 * (a, b) = (x_i, x_{i + rot_dim/2}) in the half layout and (x_2i, x_{2i+1}) in
 * the interleaved one; elements from rot_dim on are copied.  The rates are
 * w_i = theta^(-2i/rot_dim), changed for contexts longer than those a model
 * was trained on (factor >= 1, orig_len the original context):
 *   TSA_ROPE_PLAIN     as they are
 *   TSA_ROPE_LINEAR    w_i / factor
 *   TSA_ROPE_NTK       theta * factor^(rot_dim / (rot_dim - 2)) for theta
 *   TSA_ROPE_BY_PARTS  by the turns n_i = orig_len w_i / 2pi over the original
 *                      context: t = clamp((n_i - low) / (high - low), 0, 1),
 *                      w_i -> (1 - t) w_i / factor + t w_i (default low 1, high 4)
 *   TSA_ROPE_YARN      by the pair: lo, hi = floor, ceil of
 *                      rot_dim ln(orig_len / (2pi beta)) / (2 ln theta) at
 *                      beta = high and low (default low 1, high 32), clipped to
 *                      [0, rot_dim - 1]; r = clamp((i - lo) / (hi - lo), 0, 1)
 *                      (0.001 for hi - lo where they meet),
 *                      w_i -> r w_i / factor + (1 - r) w_i;
 *                      amplitude 0.1 ln(factor) + 1 unless given
 * Angles are taken in 64 bits, so far positions lose nothing. */
enum { TSA_ROPE_HALF = 0, TSA_ROPE_INTERLEAVED = 1 };
enum {
  TSA_ROPE_PLAIN = 0, TSA_ROPE_LINEAR = 1, TSA_ROPE_NTK = 2, TSA_ROPE_BY_PARTS = 3,
  TSA_ROPE_YARN = 4
};
typedef struct tsa_rope_spec {
  double theta;      /* base, > 1 */
  double factor;     /* >= 1; only read by the scaled kinds */
  double low, high;  /* both 0: the kind's defaults */
  double amplitude;  /* 0: the kind's default (1 but for yarn) */
  int64_t orig_len;  /* > 0 for TSA_ROPE_BY_PARTS and TSA_ROPE_YARN */
  int64_t max_pos;   /* positions [0, max_pos) are covered; <= 2^26 */
  int32_t rot_dim;   /* a multiple of 16, at most 128 */
  int32_t layout;    /* TSA_ROPE_HALF or TSA_ROPE_INTERLEAVED */
  int32_t scaling;   /* TSA_ROPE_PLAIN .. TSA_ROPE_YARN */
} tsa_rope_spec;

/* A table of the spec's angles, caller device memory (16-byte aligned) of
 * tsa_rope_table_size() bytes.  It holds cos and sin of l w_i for l < 2048 and
 * of 2048 h w_i, and the kernels add the two angles: 1 MiB for rot_dim 128 and a
 * million positions, which stays in L2, where a row per position would be
 * 512 MiB. */
typedef struct tsa_rope {
  const void* table;
  int64_t max_pos;
  int32_t rot_dim;
  int32_t layout;
} tsa_rope;

/* Bytes of the table (0 for sizes that tsa_rope_table refuses). */
TSA_API size_t tsa_rope_table_size(int rot_dim, int64_t max_pos);
/* Fills `table` (one kernel on `stream`) and *rope, which names it. */
TSA_API int tsa_rope_table(const tsa_rope_spec* spec, void* table, size_t bytes,
                           tsa_rope* rope, void* stream);

/* Rows of T tokens and H heads: element (t, h, j) at data + t*stride_t +
 * h*stride_h + j (bf16; strides in elements, multiples of 8; data 16-byte
 * aligned), so that a slice of a fused projection is taken as it is.  Rows that
 * are written must not overlap one another. */
typedef struct tsa_rows {
  void* data;
  int64_t stride_t;
  int64_t stride_h;
} tsa_rows;

/* rope_apply -- rotates the q rows [T][Hq] and the k rows [T][Hkv] of T tokens.
 *
 * positions: int32 [T] (device).  inverse != 0 turns by the opposite angle (the
 * amplitude stays), which is the gradient of the forward rotation and, with
 * amplitude 1, its inverse.  k and k_out may be NULL with Hkv = 0.  An output may
 * be its input (same data and strides); other overlaps are not allowed.  A
 * position outside [0, max_pos) gives NaN in the row's first rot_dim elements.
 * Each output is rounded once, from 32 bits. */
TSA_API int rope_apply(const tsa_rows* q, const tsa_rows* q_out, int Hq, const tsa_rows* k,
                       const tsa_rows* k_out, int Hkv, int64_t T, int d,
                       const int32_t* positions, const tsa_rope* rope, int inverse,
                       void* stream);

/* ------------------------------------------------------------------ */
/* 8-bit KV cache: keys and values in one byte an element, with one scale for
 * each block of `block` consecutive positions and KV head (K and V apart).
 *
 * Geometry as tsa_kv, one byte an element:
 *   contiguous  k, v: [B][Hkv][l_cap][128]; scales fp32 [B][Hkv][l_cap/block]
 *   paged       k, v: [n_pages][Hkv][page_size][128] through page_table int32
 *               [B][max_pages]; scales fp32 [n_pages][Hkv][page_size/block]
 * block: 16, 32, 64 or 128, dividing l_cap (contiguous) or page_size (paged).
 * A value is scale * code:
 *   TSA_KV8_INT8  whole numbers in [-127, 127], stored as the byte code + 128
 *   TSA_KV8_E4M3  8-bit floats (4 exponent and 3 mantissa bits, no infinities)
 * A scale is a power of two, the smallest 2^e with 127 * 2^e (int8) or 448 *
 * 2^e (e4m3) at or above the block's largest finite magnitude, e >= -60.  Powers
 * of two make every division here exact: a code is the value rounded once (to
 * nearest, ties to even), and every stored value is exact in bf16.
 * Codes are 16-byte aligned.  status: NULL, or one 256-byte aligned device int
 * that kernels flag bad lengths, pages and positions in (sticky; read and clear
 * it with tsa_workspace_status). */
enum { TSA_KV8_INT8 = 0, TSA_KV8_E4M3 = 1 };
typedef struct tsa_kv8 {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  int32_t* status;
  int64_t l_cap;
  int32_t page_size;
  int32_t max_pages;
  int32_t n_pages;   /* pages of the pool (paged only) */
  int32_t block;
  int32_t format;
} tsa_kv8;

/* kv8_append -- writes new tokens' K and V into the cache.
 *
 * k_new, v_new: bf16 rows [T][Hkv]; sequence b's are tokens [cu_new[b],
 * cu_new[b+1]) (int32 [B+1], device), or, with cu_new NULL, [b*max_new,
 * (b+1)*max_new).  max_new: the most new tokens of a sequence (a sequence with
 * more is flagged and nothing of it is written).  lens: int32 [B] (device), the
 * lengths after the call: the n_b tokens go to positions [lens[b] - n_b, lens[b]).
 * rope: NULL, or the rotation of the keys, applied in 32 bits on the way (one
 * rounding in all); positions: int32 [T] (device) or NULL for the cache's own.
 * Blocks that begin with a new token take their scale from the new rows.  The
 * block that older rows share takes the larger of its scale and the new rows',
 * and where it grows the older rows' codes are rounded again to it.  Rows from
 * lens[b] on are left as they were.  Infinities are stored as the largest code,
 * NaN as 0 (int8) or NaN (e4m3).  A sequence with lens[b] outside [n_b, l_cap], or rows
 * on a page outside [0, n_pages), are not written, and flagged.  Sequences of one
 * call must not share the pages that they write. */
TSA_API int kv8_append(const tsa_kv8* cache, const tsa_rows* k_new, const tsa_rows* v_new,
                       const int32_t* cu_new, int64_t T, int max_new, const int32_t* lens, int B,
                       int Hkv, int d, const tsa_rope* rope, const int32_t* positions,
                       void* stream);

/* kv8_read -- the last n_b positions of every sequence, back in bf16 (exact).
 *
 * Row counts and places as in kv8_append: token cu[b] + j of k_out and v_out
 * (bf16 rows [T][Hkv]) is position lens[b] - n_b + j.  Positions below 0 give
 * rows of zeros; lens[b] outside [0, l_cap] or a page outside [0, n_pages) gives
 * NaN, and is flagged.  Rows of a sequence past max_new are left as they were. */
TSA_API int kv8_read(const tsa_kv8* cache, const tsa_rows* k_out, const tsa_rows* v_out,
                     const int32_t* cu, int64_t T, int max_new, const int32_t* lens, int B,
                     int Hkv, int d, void* stream);

/* ------------------------------------------------------------------ */
/* Attention with a sliding window and sinks, and attention over the 8-bit
 * cache.  A query at position p sees the positions j <= p with j < n_init (the
 * sinks) or j > p - n_recent (the window): the static W of sparse_attn_decode.
 * n_recent >= p + 1 sees everything before it.  Rows that no query of the call
 * sees are not used, whatever they hold, and pages that hold no visible row are
 * not looked up.  Rows that some query of a sequence sees must be finite.
 *
 * kv8_attn_decode / window_attn_decode: one step, the query of sequence b at
 * position lens[b] - 1.
 *   q: bf16 [B][Hq][128]; lens: int32 [B] (device);
 *   out: fp32 [B][Hq][128] = softmax(scale q.k) . v over the visible rows;
 *   lse_out: fp32 [B][Hq] or NULL (log sum e^z): (out, lse) is a partial that
 *     lse_merge takes.  No visible row: out 0, lse -inf.
 *   A value scale below 2^-60 (0: a cache that was zeroed and not written there)
 *     counts as 2^-60.
 *   Products and sums are as those of 32-bit arithmetic: codes, keys and
 *   queries enter the tensor cores exactly, the softmax weights in parts that
 *   add up to 22 bits (kv8) or 24.  kv8: out takes a row's weight times value scale in
 *   steps of 2^-31 of the largest such product that the same warp has met (lse does
 *   not), and logits are rounded together with log2 of their block's value scale.
 *   Limits: Hq / Hkv <= 8, B <= 4096, Hkv <= 1024, B * Hq <= 65535.
 *   workspace: tsa_attn_decode_workspace_size() bytes, 256-byte aligned,
 *   zero-filled before its first use; calls leave it ready for any call that it
 *   is large enough for (of either entry point).
 * Device-detected errors (tsa_workspace_status on the workspace): a lens[b]
 * outside [0, l_cap] is clamped and flagged; a visible row on a page outside
 * [0, n_pages) (kv8), or on a negative page (tsa_kv), makes the sequence's out and
 * lse NaN and is flagged. */
TSA_API size_t tsa_attn_decode_workspace_size(int B, int Hq, int Hkv, int d);
TSA_API int kv8_attn_decode(const void* q, const tsa_kv8* cache, const int32_t* lens, int B,
                            int Hq, int Hkv, int d, int64_t n_init, int64_t n_recent,
                            float scale, float* out, float* lse_out, void* workspace,
                            size_t ws_bytes, void* stream);
TSA_API int window_attn_decode(const void* q, const tsa_kv* kv, const int32_t* lens, int B,
                               int Hq, int Hkv, int d, int64_t n_init, int64_t n_recent,
                               float scale, float* out, float* lse_out, void* workspace,
                               size_t ws_bytes, void* stream);

/* window_attn_prefill -- the same for many new tokens per sequence, over a
 * bf16 cache that holds them already (prompts, chunks of prompts).
 *
 * q: bf16 rows [T][Hq]; sequence b's are tokens [cu_q[b], cu_q[b+1]) (int32
 * [B+1], device), or [b*max_q, (b+1)*max_q) with cu_q NULL; token j of n_b has
 * position lens[b] - n_b + j (below 0: it sees nothing).  max_q: the most tokens
 * of a sequence (a sequence with more is flagged, its outputs NaN up to max_q).
 * out: bf16 [T][Hq][128], rounded once from 32-bit sums (the softmax weights
 * enter the products in bf16; the sums of at most 16384 rows are truncated, by 1e-4
 * of them at most, and added with rounding); lse_out: fp32 [T][Hq] or NULL.  Rows from cu_q[B]
 * on are left as they were.
 * workspace: window_attn_prefill_workspace_size() bytes (from the same max_q,
 * l_cap and window), 256-byte aligned, zero-filled before its first use; calls
 * leave it ready for any call of this entry point that it is large enough for.
 * Device-detected errors (on the workspace): a lens[b] outside [0, l_cap] is
 * clamped and flagged; a visible row on a negative page is flagged and gives NaN to
 * every query computed with it (a block of tokens of that KV head's query heads);
 * offsets outside [0, T] are flagged and nothing of their sequence is written.
 * Limits: Hq / Hkv <= 8, B <= 4096, B * Hkv <= 65535. */
TSA_API size_t window_attn_prefill_workspace_size(int B, int Hq, int Hkv, int d, int max_q,
                                                  int64_t l_cap, int64_t n_init,
                                                  int64_t n_recent);
TSA_API int window_attn_prefill(const tsa_rows* q, const tsa_kv* kv, const int32_t* cu_q,
                                int64_t T, int max_q, const int32_t* lens, int B, int Hq,
                                int Hkv, int d, int64_t n_init, int64_t n_recent, float scale,
                                void* out, float* lse_out, void* workspace, size_t ws_bytes,
                                void* stream);

/* ------------------------------------------------------------------ */
/* lse_merge -- [RA] Eq. 4-5 on precomputed partials.
 *
 * For each row r < rows, merges two attention partials over disjoint key
 * sets, each given as (o, lse) with lse = log sum e^z over its set:
 *   lse = log(e^lse_a + e^lse_b)
 *   o   = e^(lse_a - lse) o_a + e^(lse_b - lse) o_b
 * A partial with lse = -inf is empty and gets weight 0; if both are empty
 * the row's o is 0 and lse is -inf.
 * o_a, o_b, o_out: fp32 [rows][d]; lse_a, lse_b, lse_out: fp32 [rows]
 * (device).  o_out may alias o_a or o_b; lse_out may alias lse_a or lse_b.
 * d: 1 .. 1024. */
TSA_API int lse_merge(const float* o_a, const float* lse_a, const float* o_b,
              const float* lse_b, float* o_out, float* lse_out, int rows,
              int d, void* stream);

/* ------------------------------------------------------------------ */
/* ReTopK -- [RTK] per-head query-support reuse for one sequence.
 *
 * State (per layer): for every query head a FIFO of C entries (qbar, S):
 * qbar a normalised past query (fp32 [128]), S its final top-K positions.
 * Step t (counted from 0 by the state) with query q and cache length L_t:
 *   qbar_t = q / |q|;  rho_c = qbar_t . qbar_c  for the C entries
 *   exact path if max rho < tau  or  t % T_r == 0:
 *       S_t = exact top-K of all L_t keys (no window)
 *   reuse path otherwise:
 *       R_t = the R entries of largest rho (ties: older entry first)
 *       A_t = Unique(U_{c in R_t} S_c  u  [L_t - W, L_t))      (ascending)
 *       S_t = top-K of A_t by e_i = scale * q . k_i (ties: smaller
 *             position); all of A_t when |A_t| <= K
 *   out = softmax(e_{S_t}) . V_{S_t}   (no window merge)
 *   push (qbar_t, S_t) into the FIFO, evicting the oldest entry.
 *
 * The state lives in caller-owned device memory of retopk_state_size()
 * bytes (256-byte aligned); the opaque host handle holds sizes, pointers,
 * the step counter and the FIFO head. */
typedef struct tsa_retopk tsa_retopk;

TSA_API size_t retopk_state_size(int Hq, int d, int K, int C);

/* Create a handle over `state_mem`.  Hyper-parameters: 1 <= R <= C <= 64,
 * K >= 1, W >= 0, T_r >= 1, R*K + W <= 8192, tau any float (tau > 1: always
 * exact; tau <= -1 with a large T_r: reuse after step 0).  max_len bounds
 * every later L_t and sizes the workspace: the candidate union is a bitmap
 * over the positions with a second level of one bit per 32-bit word; one CTA
 * keeps both in shared memory up to 1.5 M positions (192 KiB), and for
 * longer caches the bitmap lives in the workspace (max_len / 8 bytes per
 * query head) with only the second level in shared memory: max_len <=
 * 50331648.  Nothing is launched. */
TSA_API int retopk_create(tsa_retopk** st, int Hq, int Hkv, int d, int K, int C,
                  int R, int W, float tau, int T_r, int64_t max_len,
                  void* state_mem, size_t state_bytes);

/* Fill the FIFO from the last C prefill queries: prefill_q bf16 [C][Hq][128]
 * (row c is the query of prefill position L0-C+c; c = 0 is the oldest
 * entry) and their supports prefill_supports int32 [C][Hq][K] with sizes
 * prefill_counts int32 [C][Hq] (entries past a count are ignored).  All
 * device pointers.  Resets the step counter to 0. */
TSA_API int retopk_init(tsa_retopk* st, const void* prefill_q,
                const int32_t* prefill_supports, const int32_t* prefill_counts,
                void* stream);

/* Workspace needed by retopk_step for caches up to max_len keys: device
 * scratch, 256-byte aligned, zero-filled before the handle's first step.
 * Like the decode workspace it keeps per-head state that speeds up the next
 * step (never its result), so one workspace serves one handle. */
TSA_API size_t retopk_workspace_size(const tsa_retopk* st);

/* One decode step (see above).  q: bf16 [Hq][128]; kv: this layer's cache
 * with B = 1 (lens are the host value `len`, 1 <= len <= min(kv->l_cap,
 * max_len)); out: fp32 [Hq][128].  Optional outputs (NULL to skip):
 *   support_out int32 [Hq][K] (S_t, unspecified order, -1 padded; a copy
 *     of the FIFO entry this step pushed),
 *   path_out int32 [Hq] (1 exact, 0 reuse),
 *   mcand_out int32 [Hq] (|A_t| on the reuse path, len on the exact path),
 *   cand_out int32 [Hq][R*K+W] (A_t ascending, -1 padded; reuse heads only),
 *   lse_out fp32 [Hq].
 * Advances the step counter and the FIFO head.  (The same as
 * retopk_step_batched with one handle.)  If a bounded wait of the
 * step's key scan expires (see tsa_workspace_status), out and lse are NaN
 * and the FIFO entry is not rewritten (it keeps an older entry): restore
 * the state memory and counters from a copy taken before the step to redo
 * it. */
TSA_API int retopk_step(tsa_retopk* st, const void* q, const tsa_kv* kv, int64_t len,
                float scale, float* out, int32_t* support_out,
                int32_t* path_out, int32_t* mcand_out, int32_t* cand_out,
                float* lse_out, void* workspace, size_t ws_bytes,
                void* stream);

/* retopk_prefill_supports -- the FIFO's initial supports ([RTK] method
 * section 1: the cache starts from the last C prefill queries; the same exact
 * prefill-query top-K is [RA]'s attention-aware index, phase 1).
 *
 * For the last C prefill queries of one sequence -- query c (0 = oldest) at
 * position p_c = L0 - C + c -- and every query head h: the exact top-K of
 * z_i = scale * q_{c,h} . k_i over the causal prefix i in [0, p_c] (no
 * window), ties to the smaller position.  One call runs one key scan and one
 * selection for all C * Hq (query, head) pairs: the queries are a batch of C
 * sequences that all read this sequence's cache (each still reads its own
 * prefix of keys).
 * q_prefill:  bf16 [C][Hq][128] (device), the layout retopk_init takes
 * kv:         the sequence's cache (B = 1), L0 <= kv->l_cap, C <= L0
 * supports:   int32 [C][Hq][K] (device): the positions, unspecified order,
 *             padded with -1 past min(K, p_c + 1)
 * counts:     int32 [C][Hq] (device) or NULL: min(K, p_c + 1)
 * workspace:  retopk_prefill_workspace_size() bytes, 256-byte aligned,
 *             zero-filled before its first use; like the decode workspace
 *             it keeps per-head emission state between calls (a first call
 *             emits every key and costs more).
 * Limits as sparse_attn_decode with B = C (C * Hkv <= 512, C * Hq <= 65535).
 * Device-detected errors: tsa_workspace_status. */
TSA_API size_t retopk_prefill_workspace_size(int C, int Hq, int Hkv, int d, int64_t l_cap,
                                             int K);
TSA_API int retopk_prefill_supports(const void* q_prefill, const tsa_kv* kv, int64_t L0, int C,
                                    int Hq, int Hkv, int d, int K, float scale,
                                    int32_t* supports, int32_t* counts, void* workspace,
                                    size_t ws_bytes, void* stream);

/* retopk_step_batched -- one decode step of n sequences at once, each with
 * its own ReTopK state (continuous batching: any set of initialised handles,
 * in any order, may form a call; a sequence joins after retopk_init on its
 * handle and retires by no longer being passed).
 *
 * handles: n distinct handles (1 <= n <= 64) with equal Hq, Hkv, K, C, R, W,
 *   tau, T_r and max_len; each keeps its own step counter and FIFO head
 *   (both advance by one).
 * q: bf16 [n][Hq][128]; kv: the n sequences' caches in call order (B = n:
 *   contiguous [n][Hkv][l_cap][128], or paged with page-table rows in call
 *   order); lens: host int64 [n], 1 <= lens[b] <= min(l_cap, max_len).
 * Per sequence b everything is as for retopk_step (its path decisions, A_t,
 * S_t, output and FIFO push use only its own state and cache).  Outputs are
 * retopk_step's with a leading [n] (out fp32 [n][Hq][128]; support_out int32
 * [n][Hq][K]; path_out, mcand_out int32 [n][Hq]; cand_out int32
 * [n][Hq][R*K+W]; lse_out fp32 [n][Hq]; optional ones NULL to skip).
 * workspace: retopk_batched_workspace_size(handles[0], n_max) bytes for any
 *   n <= n_max, 256-byte aligned, zero-filled before its first use; it keeps
 *   per-row emission state (only the cost depends on it).  Its layout follows
 *   from ws_bytes (the most sequences it holds), so pass the same ws_bytes
 *   with a workspace on every call. */
TSA_API size_t retopk_batched_workspace_size(const tsa_retopk* proto, int n_max);
TSA_API int retopk_step_batched(tsa_retopk* const* handles, int n, const void* q,
                                const tsa_kv* kv, const int64_t* lens, float scale, float* out,
                                int32_t* support_out, int32_t* path_out, int32_t* mcand_out,
                                int32_t* cand_out, float* lse_out, void* workspace,
                                size_t ws_bytes, void* stream);

/* Host-side counters of the handle (for checkpointing). */
TSA_API int retopk_get_counters(const tsa_retopk* st, int64_t* t, int32_t* fifo_head);
TSA_API int retopk_set_counters(tsa_retopk* st, int64_t t, int32_t fifo_head);

/* Free the host handle only; the state memory belongs to the caller. */
TSA_API int retopk_destroy(tsa_retopk* st);

#ifdef __cplusplus
}
#endif
#endif
