/*
 * dosa_indexer.h -- exact Top-K selection for the DSA sparse-attention indexer
 * on AMD Instinct MI355X (gfx950).
 *
 * The operation (DoSA pages: podcast transcript of "DOSA: Dots Sparse
 * Attention", Method section, problem formulation; the DSA indexer score):
 * every query t carries H indexer heads with query vectors q[t,h,:] and
 * signed weights w[t,h]; all heads share one key k[s,:] per token.  The score
 * of key s for query t is
 *
 *     S(t,s) = sum_h w[t,h] * max(0, q[t,h,:] . k[s,:])
 *
 * and each query keeps the K visible keys of highest score.  Causality: query
 * i of sequence b sits at position kv_lens[b] - q_lens[b] + i and sees the
 * keys at positions 0..position.  Ties are broken towards the lower position.
 * When fewer than K keys are visible, all of them are returned followed by -1.
 *
 * Two entry points compute the same set:
 *   dsa_indexer_topk   scores every visible key (dense scoring with a
 *                      streaming Top-K; the plain method).
 *   dosa_indexer_topk  the DoSA way (same pages, Method section: seed subset
 *                      threshold, certificate built from nonnegative head
 *                      projections, a joint residual bound and an
 *                      activation-informed negative-head aggregate; zicq.com
 *                      summary, items 1-3; picx.dev item, sections 02-03):
 *                      a seed pass scores a seed subset exactly and takes its
 *                      K-th score as a threshold tau; a bound pass computes a
 *                      conservative upper bound per key; keys whose bound is
 *                      below tau are dropped; survivors are compacted and
 *                      scored with all heads; then the exact Top-K.  The
 *                      selected set is identical to dsa_indexer_topk's, bit
 *                      for bit, for every configuration.
 *
 * Layouts (all row-major, all pointers below are DEVICE pointers unless said):
 *   q        [total_q, H, d] of q_dtype; queries of the batch back to back
 *            (total_q = sum q_lens).
 *   q_scale  [total_q] fp32, required iff q_dtype == DOSA_FP8_E4M3FN (one
 *            scale per query token across all heads); ignored otherwise.
 *   w        [total_q, H] fp32 (any sign).
 *   k        contiguous (page_table == NULL): [total_k, d] of k_dtype,
 *            sequence b's keys at rows sum(kv_lens[0..b-1]) + position;
 *            paged: [num_pages, page_size, d], logical key j of sequence b in
 *            pool page page_table[b*max_pages + j/page_size], slot j%page_size.
 *   k_scale  per key token fp32 ([total_k] or [num_pages, page_size]),
 *            required iff k_dtype == DOSA_FP8_E4M3FN.
 *   fp8 values are OCP E4M3FN; the value of a code is scale * decode(code).
 *   q_lens, kv_lens  HOST int32 [batch], 0 <= q_lens[b] <= kv_lens[b].
 *   out_idx  [total_q, topk] int32: logical key positions, -1 padding.
 *   out_score [total_q, topk] fp32 or NULL: the fp32 score of each returned
 *            key (-inf padding).
 *   Row order inside out_idx is unspecified unless DOSA_SORTED is set (then
 *   score descending, position ascending); it is deterministic run to run.
 *
 * Supported: d in {64, 128}; H a multiple of 8 in [8, 64]; 1 <= topk <= 4096;
 * (q_dtype, k_dtype) in {(F32,F32), (BF16,BF16), (FP8,FP8), (BF16,FP8)};
 * contiguous keys: sum(kv_lens) < 2^31 and kv_lens[b] * d * sizeof(k) < 2^32;
 * sum(q_lens) < 2^31.  Other shapes return DOSA_ERR_UNSUPPORTED.
 * Inputs must be finite.
 *
 * Ownership and synchronisation: the caller owns every buffer, including the
 * workspace (size from dosa_workspace_size).  The library allocates no device
 * memory and keeps no data between calls; everything is ordered on `stream`
 * (a hipStream_t, NULL = default stream) and no call waits for the device.
 * A pruned call with query tiles that runs the probe (see DOSA_NO_PROBE),
 * has at least 2^26 causal pairs and whose dense alternative fits in two
 * workgroups per CU forks the certificate stages onto
 * a side stream the library creates once per device (default priority, kept
 * until the process ends) and joins it back into `stream` before its final
 * selection, so `stream` order covers the whole call (graph capture too).
 * Outputs, workspace contents and stats are valid once the stream has
 * completed.  Calls on distinct workspaces/streams may run concurrently;
 * their certificate stages then share the device's side stream.
 *
 * Errors: 0 on success or a negative dosa_status.  On error nothing has been
 * enqueued.  No C++ exception crosses this interface.
 */
#ifndef DOSA_INDEXER_H_
#define DOSA_INDEXER_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DOSA_F32 = 0,
  DOSA_BF16 = 1,
  DOSA_FP8_E4M3FN = 2
} dosa_dtype;

typedef enum {
  DOSA_OK = 0,
  DOSA_ERR_INVALID_ARG = -1,     /* null pointer, bad length, q_lens > kv_lens, ... */
  DOSA_ERR_UNSUPPORTED = -2,     /* dtype combination, d, H or topk outside the supported set */
  DOSA_ERR_WORKSPACE = -3,       /* workspace NULL or smaller than dosa_workspace_size */
  DOSA_ERR_HIP = -4              /* a HIP runtime call or kernel launch failed */
} dosa_status;

/* flags */
#define DOSA_NO_PRUNE 0x1u        /* dosa_indexer_topk: skip the bound pass (every key survives) */
#define DOSA_SORTED 0x2u          /* rows of out_idx in (score desc, position asc) order */
#define DOSA_SEPARABLE_RHO 0x4u   /* residual bound sum_h w_h ||r_h|| instead of the joint bound */
#define DOSA_NO_NEGATIVE 0x8u     /* drop the negative-head aggregate from the bound */
#define DOSA_KEY_BLOCKS 0x20u     /* dosa_indexer_topk: key-block test in the bound pass (calls with query
                                     tiles): per 64-key block a centre, radius and largest norm give one
                                     bound for all its keys (certificates over key blocks, the DoSA
                                     transcript's Conclusion); a block below tau for every query of a
                                     32-query bound tile is never loaded.  Off by default: on the
                                     correlated 128K recipe it skips 5.6% of the tiles and the test
                                     costs more than that saves */
#define DOSA_NO_PROBE 0x10u       /* dosa_indexer_topk: no probe, always the certificate pipeline
                                     (by default a call with >= 8 query tiles first plans its last
                                     tile -- a decode-like call with >= 8 sequences its groups, up
                                     to 256 of them --
                                     with the threshold estimated from the plan's sampled seed-window
                                     keys and, if the certificate prunes no query there, scores every
                                     key densely; the result is the same either way) */
#define DOSA_TWO_ROUNDS 0x40u     /* dosa_indexer_topk, calls with query tiles: the threshold is
                                     refined once within the call (the DoSA transcript, Method: the
                                     stages repeat over tiles of keys as the standings refine).
                                     Round 1 bounds and scores the newer half of each tile's bounded
                                     keys against the seed threshold; the K-th largest exact score
                                     of the seed and round-1 candidates (a valid lower bound of the
                                     K-th score: K distinct keys reach it) becomes the threshold of
                                     round 2 over the older half.  debug_tau keeps round 1's
                                     threshold; debug_mask bits of round-2 keys are against the
                                     raised one */
#define DOSA_GROUP_LISTS 0x80u    /* dosa_indexer_topk, calls with query tiles: every tile's survivors
                                     go to the per-group streams (each query group's own compacted
                                     list, scored one wavefront per group; a group holds the queries
                                     one wavefront scores together: 4 for fp8, 2 for bf16, 1 for
                                     fp32 at H = 64, d = 128) instead of the shared stream (the
                                     tile's union list, whose keys serve all its queries), the two
                                     kinds of survivor stream of the DoSA transcript (Method: GPU
                                     kernel design).  By default compaction picks the union unless
                                     it is 8x the groups' lists together.  The result is the same
                                     either way; the workspace reserves one list of every bounded
                                     key per group */

/* Knobs of dosa_indexer_topk.  None of them changes the selected set; they
 * only change how much work the certificate saves. */
typedef struct {
  int32_t num_proxies;      /* positive heads evaluated exactly in the bound: 0..3 (default 3;
                               the bound kernels give each query 4 MFMA rows: p proxy rows and
                               4 - p rows for the negative-head aggregate) */
  int32_t seed_window;      /* seed = the last seed_window visible keys ... (default 4*topk, >= 64) */
  int32_t seed_prefix;      /* ... plus the first seed_prefix keys (default 64) */
  int32_t buffer_cap;       /* entries per candidate region (each query has one region per key
                               range scored in parallel); 0 = automatic (default): about
                               1.3*topk*(1 + ln(range/topk)) + 256 for the longest range, so
                               that regions rarely overflow; else >= topk + 64 */
  int32_t key_splits;       /* key ranges scored in parallel per query group; 0 = automatic */
  float neg_support_frac;   /* negative head joins the aggregate if positive on >= this
                               fraction of the sampled seed keys (default 0.5) */
  uint32_t flags;           /* DOSA_* flags */
  float* debug_ub;          /* optional DEVICE [total_q, max_kv] fp32: certificate value per
                               bounded key (untouched elsewhere); for testing only */
  float* debug_tau;         /* optional DEVICE [total_q] fp32: each query's seed threshold tau
                               (the K-th largest exactly scored seed score, -inf with fewer than
                               K seeds); written only when the call runs the certificate
                               pipeline (always with DOSA_NO_PROBE); for testing only */
  uint64_t* debug_mask;     /* optional DEVICE [total_q, ceil(max_kv/64)] u64, zeroed by the
                               caller: bit s%64 of word s/64 is OR-ed in for every bounded key s
                               whose certificate reached tau for that query (every bounded key
                               of a query whose plan found nothing to prune); seed keys are not
                               marked; for testing only */
  const int32_t* seed_idx;  /* optional DEVICE [total_q, seed_count] int32: extra seed keys per query,
                               scored exactly and used for tau only -- e.g. the previous decode
                               step's Top-K (the DoSA transcript, Experiments: decode reuses the
                               scores of recently selected keys) or a candidate set shared by a
                               group of nearby queries (the PIVOT record: one scan per query
                               group).  Logical key positions; entries outside the keys that get
                               a certificate (negative, past the query, or inside the seed prefix
                               or window) and repeats are ignored, -1 may pad a row.  Queries
                               scored together (up to 4 consecutive queries of a sequence) share
                               the union of their rows, which keeps every seed visible to each of
                               them.  Any content leaves the selected set unchanged; keys that
                               score high raise tau and so the pruning */
  int32_t seed_count;       /* entries per row of seed_idx, 0..4096 (0 = none, the default) */
  int32_t reserved;         /* set to 0 */
} dosa_config;

/* Device-resident counters, accumulated (not reset) by each call that gets a
 * non-NULL pointer.  Pairs are causal (query, visible key) pairs. */
typedef struct {
  uint64_t pairs_total;        /* all visible pairs */
  uint64_t pairs_seed;         /* pairs scored exactly in the seed pass */
  uint64_t pairs_bounded;      /* pairs given a certificate (non-seed) */
  uint64_t pairs_survived;     /* bounded pairs whose certificate reached tau */
  uint64_t pairs_scored;       /* pairs scored with all heads after the seed (incl. tile union) */
  uint64_t candidates_written; /* entries appended to candidate buffers */
  uint64_t reselects;          /* in-kernel buffer re-selections */
  uint64_t groups_skipped;     /* query groups whose certificate could prune nothing */
  uint64_t pairs_scored_list;  /* the part of pairs_scored scored from compacted survivor lists */
  uint64_t keys_streamed;      /* key rows the bound pass read (once per query tile or group that
                                  streamed them; skipped groups read none) */
  uint64_t calls_unpruned;     /* dosa_indexer_topk calls scored densely: the certificate could
                                  prune no query the probe planned (the call's last query tile, or
                                  every group of a decode-like call) */
  uint64_t key_blocks_skipped; /* 64-key tiles the bound pass never loaded: the key-block bound
                                  (centre, radius and largest norm of the block's keys) was below
                                  tau for every query of the query tile that needed them */
} dosa_stats;

/* Fill *cfg with the defaults for a given topk. */
int dosa_default_config(int32_t topk, dosa_config* cfg);

/* Bytes of device workspace the call with these shapes needs. q_lens/kv_lens
 * are HOST arrays.  paged != 0 if a page table will be passed.  cfg NULL =
 * defaults.  dense != 0 sizes for dsa_indexer_topk, 0 for dosa_indexer_topk.
 * Returns 0 for invalid arguments. */
size_t dosa_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens,
                           int32_t H, int32_t d, int32_t topk, int32_t q_dtype, int32_t k_dtype,
                           int32_t paged, int32_t dense, const dosa_config* cfg);

/* DoSA path: certificate-pruned exact Top-K.  stats: DEVICE pointer or NULL. */
int dosa_indexer_topk(const void* q, int32_t q_dtype, const float* q_scale, const float* w,
                      const void* k, int32_t k_dtype, const float* k_scale,
                      const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                      const int32_t* page_table, int32_t page_size, int32_t max_pages,
                      int32_t H, int32_t d, int32_t topk,
                      int32_t* out_idx, float* out_score,
                      void* workspace, size_t workspace_bytes,
                      const dosa_config* cfg, dosa_stats* stats, void* stream);

/* Dense path: every visible key scored with all heads, streaming exact Top-K.
 * Of cfg (NULL = defaults) it uses buffer_cap, key_splits and DOSA_SORTED. */
int dsa_indexer_topk(const void* q, int32_t q_dtype, const float* q_scale, const float* w,
                     const void* k, int32_t k_dtype, const float* k_scale,
                     const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                     const int32_t* page_table, int32_t page_size, int32_t max_pages,
                     int32_t H, int32_t d, int32_t topk,
                     int32_t* out_idx, float* out_score,
                     void* workspace, size_t workspace_bytes,
                     const dosa_config* cfg, dosa_stats* stats, void* stream);

/* dosa_indexer_topk without a workspace argument, for callers that cannot
 * allocate device memory (serving loops or harnesses that forbid allocation):
 * the call allocates nothing and runs in a scratch array the library holds
 * in device memory, DOSA_NOALLOC_SCRATCH_BYTES per GPU, reserved when the
 * library's code is loaded on that GPU and kept until the process ends.  The
 * GPU is the device current on the calling thread (the one `stream` belongs
 * to).  A call whose workspace would exceed the scratch size
 * (dosa_workspace_size with dense = 0) returns DOSA_ERR_UNSUPPORTED and
 * enqueues nothing.  Every call on one GPU shares that GPU's scratch: calls
 * that overlap on the device (concurrent streams, or other threads) race and
 * must be serialised by the caller; consecutive calls on one stream are safe,
 * and no state carries over from one call to the next.  Arguments, results and
 * errors otherwise as dosa_indexer_topk. */
#define DOSA_NOALLOC_SCRATCH_BYTES (128u << 20)
int dosa_indexer_topk_noalloc(const void* q, int32_t q_dtype, const float* q_scale, const float* w,
                              const void* k, int32_t k_dtype, const float* k_scale,
                              const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                              const int32_t* page_table, int32_t page_size, int32_t max_pages,
                              int32_t H, int32_t d, int32_t topk,
                              int32_t* out_idx, float* out_score,
                              const dosa_config* cfg, dosa_stats* stats, void* stream);

/* ---------------------------------------------------------------------------
 * Attention next to the indexer: a prompt's causal attention, a paged cache of
 * keys and values in 4 bits with the attention that reads it (every visible
 * key, or the keys the indexer selected), the attention weight each cached key
 * received, and the eviction of the keys that received least.
 *
 * Common to all of them.  Hq query heads share Hkv key/value heads, query head
 * h reads kv head h / (Hq / Hkv).  Queries of a batch are packed as above;
 * query i of sequence b sits at position kv_lens[b] - q_lens[b] + i and sees
 * the keys at positions 0..position.  Packed operands are [tokens, heads, d]
 * with the elements of a token together and a stride in ELEMENTS from one
 * token to the next (a slice of a fused projection needs no copy); their
 * first row and their stride must be 16-byte aligned.  Pointers are DEVICE
 * pointers on the device current on the calling thread; lengths are HOST
 * int32 [batch] and travel as kernel arguments, so a captured graph keeps the
 * lengths it was captured with.  Sequences with q_len = 0 are skipped.
 * Inputs must be finite, and so must what fp32 makes of them: a row's sums of
 * |q_e k_e| stay below 2^127, as they are and times scale, and its sum of |v|
 * over the keys below 2^119 (outputs are divided by the softmax sum last, and
 * weights before that reach 2^8).  Scores, maxima, sums and outputs accumulate
 * in fp32.  The calls allocate nothing, copy nothing to the device and wait for
 * nothing; they may be captured.  What a call writes overlaps nothing else it
 * is given, unless said.  Calls that share a workspace must be ordered (one
 * stream, or graphs replayed one after the other).  Results do not change from
 * run to run.
 *
 * Supported: d in {64, 128}; Hkv <= 128, Hq <= 1024, Hq a multiple of Hkv;
 * types DOSA_F32 and DOSA_BF16; at most 2^31 - 2^16 tokens in a batch and slots
 * in a cache, 2^30 queries times group heads in a sequence; token strides up
 * to 2^23 elements.  scale is positive, not subnormal, and scale * log2(e)
 * finite in fp32 (scale up to 2.3e38).  A launch has less than 2^32 threads: a
 * call that would need more in one (such as 2^26 queries times kv heads over
 * selected keys, 2^31 rows of a bf16 prompt times kv heads, 2^28 tokens appended
 * to a sequence, 2^27 keys moved in one) is refused, to be split.
 *
 * The *_workspace_size functions return the bytes a call with these arguments
 * needs (over the cache: with queries of either type), and 0 for arguments that
 * a call (of either type) would refuse, the limit of a launch aside.
 */

/* Causal attention of packed sequences over contiguous keys and values.
 *   q   [total_q, Hq, d], k and v [total_k, Hkv, d] of dtype; sequence b's keys
 *       at rows sum(kv_lens[0..b-1]) + position (as in the indexer), so whole
 *       prompts (q_len = kv_len), later chunks of one and single tokens mix
 *   out [total_q, Hq, d] of dtype:
 *       out = sum_j w_j v_j,  w = softmax_j(scale * q . k_j)
 *   lse [total_q, Hq] fp32 or NULL: ln sum_j exp(scale * q . k_j)
 * With bf16 the softmax weights are rounded to bf16 for their product with v. */
size_t dsa_prompt_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens,
                                 int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype);
int dsa_prompt_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, int32_t dtype,
                         const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                         int32_t Hq, int32_t Hkv, int32_t d, float scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* A paged cache of keys and values in 4 bits (OCP microscaling FP4).
 *   codes  [num_pages, page_size, Hkv, d/2] bytes: element 2i in the low,
 *          2i+1 in the high nibble of byte i, each an E2M1 code (sign, two
 *          exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6)
 *   scales [num_pages, page_size, Hkv, d/32] bytes: byte e scales 32
 *          consecutive elements by 2^(e-127), e in 0..254
 * Codes must be 16-byte, scales 4-byte aligned.  Position j of sequence b is
 * in page page_table[b*max_pages + j/page_size], slot j%page_size, as in the
 * indexer; page_size is a multiple of 16 (multiples of 64 are read faster) and
 * max_pages * page_size covers every kv_len.  A table entry outside
 * 0..num_pages-1 names no page: its keys are not written and not seen (they
 * read back as zeros).  Slots past a sequence's kv_len may hold anything.
 * Sequences may share pages they only read (dsa_cache_read,
 * dsa_cache_attention); a call that writes to a page (append, weights,
 * eviction) must find it once, in one sequence. */
typedef struct {
  void* k_codes;
  void* k_scales;
  void* v_codes;
  void* v_scales;
  const int32_t* page_table;   /* DEVICE [batch, max_pages] */
  int32_t num_pages, page_size, max_pages;
  int32_t Hkv, d;
  int32_t reserved;            /* set to 0 */
} dsa_cache;

/* Quantise the q_lens[b] newest tokens of each sequence into the cache: token i
 * of sequence b goes to position kv_lens[b] - q_lens[b] + i.  k, v
 * [total_q, Hkv, d] of dtype.  A block of 32 elements takes the smallest scale
 * 2^(e-127), e in 1..254, for which every element is below 7 scales in
 * magnitude, and each element the nearest code, ties to the even one: no
 * element is off by more than half a step.  Magnitudes must stay below 2^127.
 * pos (DEVICE [num_pages, page_size] int32, or NULL): the token's place in the
 * text, seen_lens[b] - q_lens[b] + i, is written to its slot; seen_lens (HOST
 * [batch], >= kv_lens, NULL = kv_lens) counts the tokens of the text so far,
 * evicted ones included. */
int dsa_cache_append(const dsa_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                     int32_t dtype, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                     int32_t* pos, const int32_t* seen_lens, void* stream);

/* Read the q_lens[b] newest tokens of each sequence back: k, v
 * [total_q, Hkv, d] of dtype (exact in both types). */
int dsa_cache_read(const dsa_cache* cache, void* k, int64_t k_stride, void* v, int64_t v_stride,
                   int32_t dtype, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                   void* stream);

/* Attention over the cache, the call's own tokens included (append first).
 *   idx  NULL: every visible key.  Else DEVICE [total_q, topk] int32, the keys
 *        query row t reads (dsa_indexer_topk's out_idx): logical positions in
 *        any order; entries that are negative or past the query are skipped, a
 *        position listed twice counts twice.  topk = 0 without idx, else
 *        1..2^20
 *   out, lse as dsa_prompt_attention, of q_dtype; a row that sees no key gets
 *        zeros and -inf
 * bf16 queries: softmax weights are rounded to bf16 for their product with v.
 * fp32 queries: fp32 products throughout. */
size_t dsa_cache_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens,
                                int32_t Hq, int32_t Hkv, int32_t d, int32_t topk);
int dsa_cache_attention(const dsa_cache* cache, const void* q, int64_t q_stride, int32_t q_dtype,
                        const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, int32_t Hq,
                        const int32_t* idx, int32_t topk, float scale,
                        void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Add up the attention weight each cached key received from the call's
 * queries, over all query heads:
 *   acc_out[slot] = old + sum exp(scale * q . k - lse)
 * with the lse a dsa_cache_attention call without idx returned for these
 * queries.  old is acc[slot] for keys before the call's own tokens, 0 for the
 * call's own tokens and everywhere if acc is NULL.  acc, acc_out: DEVICE
 * [num_pages, page_size] fp32, may be the same.  Every visible slot of a
 * sequence with queries is written, no other.  A query whose lse is -inf adds
 * nothing. */
size_t dsa_weights_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens,
                                  int32_t Hq, int32_t Hkv, int32_t d);
int dsa_cache_weights(const dsa_cache* cache, const void* q, int64_t q_stride, int32_t q_dtype, const float* lse,
                      const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, int32_t Hq, float scale,
                      const float* acc, float* acc_out, void* workspace, size_t workspace_bytes, void* stream);

/* A per-slot array of a paged cache, [num_pages, page_size] rows of row_bytes
 * (the 4-bit codes and scales, the indexer's keys, acc, pos, ...). */
typedef struct {
  const void* src;
  void* dst;            /* == src: the rows that change place are copied within it;
                           else every kept row is copied to it */
  int64_t row_bytes;    /* 1..2^20 */
} dsa_evict_array;

/* Keep new_lens[b] of the kv_lens[b] keys of each sequence: those of largest
 * acc, ties to the lower index, with the first `prefix` and the latest
 * `window` tokens of the text always among them (min(prefix + window, kv_len)
 * <= new_len).  pos [num_pages, page_size] gives each key's place in the text
 * and seen_lens (HOST, >= kv_lens, NULL = kv_lens) the tokens of the text so
 * far; without pos a key's place is its index.  Kept keys at indices below
 * new_len stay; the n-th kept key behind them moves to the n-th freed index in
 * front.  An index in front of new_len whose table entry names no page counts
 * as a key that stays: nothing moves to it, and one key fewer is kept; with so
 * few places left that protected keys do not all fit, the lowest indices among
 * them stay.  Keys are addressed by index through page_table; attention does not
 * depend on their order.  out_src [batch, out_stride] int32: the index each
 * key 0..new_len-1 came from, -1 behind.  arrays (HOST, up to 16) are moved
 * accordingly; an array's dst may be its own src and otherwise overlaps
 * nothing the call reads or writes.  Slots from new_len on keep what they
 * held. */
size_t dsa_evict_workspace_size(int32_t batch, const int32_t* kv_lens, const int32_t* new_lens);
int dsa_cache_evict(const float* acc, const int32_t* pos, const int32_t* page_table,
                    int32_t page_size, int32_t max_pages, int32_t num_pages,
                    const int32_t* kv_lens, const int32_t* new_lens, const int32_t* seen_lens, int32_t batch,
                    int32_t prefix, int32_t window, const dsa_evict_array* arrays, int32_t n_arrays,
                    int32_t* out_src, int32_t out_stride, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Paged keys and values in 16 or 32 bits: page tables and slot maps from the
 * sequences' lengths, the write of new rows, attention of the new tokens over
 * the pages, and block attention: a few blocks per query and kv head, chosen
 * by a cheap score on summaries of the blocks, and attention over their keys.
 * What is common to the calls above holds here too (packed operands, host
 * lengths, page tables, streams, workspaces, sums in fp32).
 */

/* Page tables and slot maps.  Sequence b grows by q_lens[b] tokens to
 * kv_lens[b]; the pages that it needs beyond the ceil((kv_len - q_len) /
 * page_size) that it has are taken from the end of the free list, in the order
 * of the sequences and their pages.
 *   page_table [batch, max_pages] int32: entries of the new pages are written,
 *              no others
 *   free_pages [num_pages] int32: its first *free_count entries are pages that
 *              nobody holds; not written
 *   free_count HOST: pages left, updated by the call.  Fewer than needed:
 *              DOSA_ERR_INVALID_ARG, and nothing changes
 *   slots      [total_q] int32 or NULL: the pool slot of each new token, page *
 *              page_size + place in the page, -1 where the page is none of
 *              0..num_pages-1 (rows the user writes, such as the indexer's keys)
 *   positions  [total_q] int32 or NULL: its position, kv_len - q_len + i
 * Counts are host numbers like lengths: a captured graph keeps them. */
int dsa_pages_assign(int32_t* page_table, int32_t max_pages, int32_t page_size, int32_t num_pages,
                     const int32_t* free_pages, int32_t* free_count, const int32_t* q_lens, const int32_t* kv_lens,
                     int32_t batch, int32_t* slots, int32_t* positions, void* stream);

/* The pages behind the first ceil(new_len / page_size) of each sequence go back
 * to the end of the free list, the last page first, and their table entries
 * become -1 (0 <= new_len <= kv_len; a finished sequence's new_len is 0).  A
 * page that sequences share must be given back once.  What an entry holds is
 * given back as it is, a number that names no page too. */
int dsa_pages_release(int32_t* page_table, int32_t max_pages, int32_t page_size, int32_t num_pages, int32_t* free_pages,
                      int32_t* free_count, const int32_t* new_lens, const int32_t* kv_lens, int32_t batch, void* stream);

/* Keys and values in pages, k and v [num_pages, page_size, Hkv, d] of dtype
 * (DOSA_F32, DOSA_BF16), 16-byte aligned; addressed as dsa_cache is, and with
 * the same rules for table entries that name no page, slots past a kv_len, and
 * pages that sequences share. */
typedef struct {
  void* k;
  void* v;
  const int32_t* page_table;   /* DEVICE [batch, max_pages] */
  int32_t dtype;
  int32_t num_pages, page_size, max_pages;
  int32_t Hkv, d;
} dsa_pages;

/* Summaries of blocks of `block` consecutive positions (16, 32, 64 or 128; it
 * divides page_size).  A block's summary is the mean of its keys in 8 bits:
 *   codes  [num_pages, page_size / block, Hkv, d] integers -127..127, 16-byte
 *          aligned
 *   scales [num_pages, page_size / block, Hkv] bytes: byte e scales a row by
 *          2^(e-127), the smallest e in 1..254 for which every element of the
 *          mean is below 127.5 scales in magnitude; codes are rounded to the
 *          nearest, ties to even.  The mean is summed in 64 bits.
 * An infinite element of a mean counts as fp32's largest number of its sign, one
 * that is no number as 0; so do elements of dsa_block_select's queries. */
typedef struct {
  int8_t* codes;
  uint8_t* scales;
  int32_t num_pages, page_size, block;
  int32_t Hkv, d;
  int32_t reserved;            /* set to 0 */
} dsa_blocks;

/* Write the q_lens[b] newest tokens of each sequence, k, v [total_q, Hkv, d] of
 * the pages' dtype, into their slots, bit for bit.  blocks (of the same pages)
 * or NULL: the summaries of the blocks that these tokens make complete are
 * written too, earlier keys of theirs read from the pages.  With blocks and k =
 * v = NULL only summaries are written, all keys read from the pages: of every
 * block of a sequence with q_len = kv_len, for instance after an eviction (which
 * moves keys between blocks and leaves the summaries as they were). */
int dsa_pages_append(const dsa_pages* pages, const dsa_blocks* blocks, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, void* stream);

/* Attention of the q_lens[b] newest tokens over the pages, themselves included
 * (append first): chunks of prompts and single tokens mix.  q, out [total_q, Hq,
 * d] of the pages' dtype; out, lse as dsa_cache_attention.  bf16: for their
 * product with v the softmax weights of a sequence of few rows (up to 16 queries
 * times group heads) are two bf16 terms, whatever else is in the call; those of
 * other sequences are rounded to bf16.  A page that the table does not name is
 * not seen.  q and what the slots below kv_len hold must be finite: a number
 * that is not may reach every query of the sequence. */
size_t dsa_pages_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                                int32_t d, int32_t dtype);
int dsa_pages_attention(const dsa_pages* pages, const void* q, int64_t q_stride, const int32_t* q_lens,
                        const int32_t* kv_lens, int32_t batch, int32_t Hq, float scale, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Choose topn blocks for each query and kv head.  A query in block o (its
 * position / block) gets the first `sinks` blocks, the latest `local` up to and
 * with o, and of the others in front of them those of largest score, ties to the
 * lower index; all of them where there are no more than topn.
 *   idx   [total_q, Hkv, topn] int32: ascending block indices, -1 behind
 *   score of block j for the group's query heads h:
 *         2^(e_j - 142) * max_h 2^max(f_h - f, -100) * (a_h . c_j)
 *         with c_j, e_j the block's codes and scale byte, a_h the codes of query
 *         head h rounded as a summary with scale 2^f_h (f_h in -126..127), f =
 *         max_h f_h, rounded to fp32 once.  All but that rounding, which only
 *         subnormal results need, is exact: the choice does not depend on how
 *         sums are ordered.  A block whose table entry names no page scores -inf.
 * 0 <= sinks, 1 <= local, sinks + local <= topn <= 4096; at most 32768 blocks in
 * a sequence.  q [total_q, Hq, d] of q_dtype.  The summaries of the blocks in
 * front of o are read, the keys are not. */
int dsa_block_select(const dsa_blocks* blocks, const int32_t* page_table, int32_t max_pages, const void* q,
                     int64_t q_stride, int32_t q_dtype, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                     int32_t Hq, int32_t sinks, int32_t local, int32_t* idx, int32_t topn, void* stream);

/* Attention over listed blocks: query row t of kv head h reads the keys of the
 * blocks idx[t, h, 0..topn-1] that are not behind its position.  Entries that
 * are negative or behind the query's own block are skipped, a block listed twice
 * counts twice.  Neighbouring queries whose lists ascend read the blocks that
 * they have in common once.  topn * block <= 2^20.  bf16: softmax weights are two
 * bf16 terms for sequences of up to 64 rows (queries times group heads) in groups
 * of up to 16 heads, else rounded to bf16.  Workspace: bf16 sequences of more than
 * 64 rows take, for each unit of eight tiles of 16 rows (a tile holds up to eight
 * queries, or a part of one query's heads), 16 bytes for each entry of the lists
 * of the unit's queries, as many as a unit may hold, and 128 bytes; partial
 * results come on top where few units are cut into ranges.  Otherwise as
 * dsa_pages_attention. */
size_t dsa_block_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                                int32_t d, int32_t dtype, int32_t block, int32_t topn);
int dsa_block_attention(const dsa_pages* pages, const void* q, int64_t q_stride, const int32_t* q_lens,
                        const int32_t* kv_lens, int32_t batch, int32_t Hq, const int32_t* idx, int32_t topn,
                        int32_t block, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Per-pass timing (tracing for benchmarks).  Between dosa_profile_begin()
 * and dosa_profile_end(), every kernel the calling thread enqueues through
 * this library is bracketed by two HIP events recorded on the kernel's own
 * stream.  dosa_profile_end() waits for those events, writes up to
 * max_entries per-pass totals to out (HOST array) and returns the number of
 * entries written, or a negative status.  Off by default; profiling creates
 * HIP event objects (no device memory) and reuses them across sessions.
 * Pass names: prep, key_norms, score_seed, select_seed, plan, bound, compact,
 * score_survivor_tiles, score_survivor_lists, score_dense, select_final,
 * prompt_attention, cache_attention, attention_join, cache_append,
 * cache_read, cache_weights, weights_join, evict_select, evict_move, pages_assign,
 * pages_release, pages_append, pages_attention, block_select, block_attention. */
typedef struct {
  const char* name;   /* static string */
  int32_t launches;
  double total_ms;    /* sum of the launches' event-to-event durations */
} dosa_kernel_time;

int dosa_profile_begin(void);
int dosa_profile_end(dosa_kernel_time* out, int32_t max_entries);

/* Human-readable text for a status code (static storage; for DOSA_ERR_HIP it
 * names the failing HIP call of the most recent error on this thread). */
const char* dosa_status_string(int status);

/* Library version string. */
const char* dosa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DOSA_INDEXER_H_ */
