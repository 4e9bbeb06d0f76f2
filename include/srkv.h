/*
 * srkv.h -- C ABI of libsrkv: block-sparse retrieval decode attention over a paged
 * KV cache, for one GB300 GPU (sm_103a).
 *
 * The method (openGauss 7.0.0 DataVec, "KV Cache Query-Based Computation Inference
 * Acceleration"):
 *   - "Feature Description": at prefill, one representation vector is extracted for
 *     every KV block;
 *   - "Overall Solution": the cache of a sequence is split into initial_tokens, the
 *     sliding_window and the offload_tokens between them; at each decode step the
 *     current query is scored by inner product against the representation vector of
 *     every offload block, the topK blocks are kept, and attention runs over the
 *     initial tokens, the kept blocks and the window together;
 *   - "Configuration Parameters": INIT_TOKENS_NUM (1024), LOCAL_TOKENS_NUM (7192),
 *     TOPK_PERCENT (0.2), block size 128, DENSE_BOUNDARY (32K: a prompt shorter than
 *     this is attended densely).
 * Attention itself is softmax(q K^T / sqrt(d)) V (rkmt.cn ATB KV-cache reuse article,
 * §1.1), read through a page table of physical pages (same article, §2.2); a group of
 * query heads shares one K/V head (KV-cache survey "大模型推理百倍加速之KV cache篇",
 * section "Share--KV cache共享").
 *
 * Definitions used by every entry point (S = block_size = 128 tokens per page):
 *   L      = seq_lens[r], the tokens in request r's cache, the current token included;
 *   W      = L - local_tokens, the first token of the sliding window;
 *   candidate blocks of r = logical blocks b whose tokens [bS, bS+S) meet [init_tokens, W);
 *   rep[p][h][:] = fp32 mean of the keys of physical page p, kv head h, over its valid
 *            tokens (the representation vector);
 *   score of block b for (r, h) = (sum of the query vectors of h's group) . rep[bt[r][b]][h];
 *   k = min(n, ceil(topk_percent * n - 1e-9)) of n candidates (0 if n = 0), or n when
 *       prompt_lens[r] < dense_boundary;
 *   selection = the k candidates of highest score, ties to the lower block index;
 *   attended tokens = [0, init_tokens) u (selected blocks n [init_tokens, W)) u [W, L),
 *       as a set; out = softmax over them of q.K/sqrt(d), times V; L = 0 gives 0.
 *
 * Layouts (all row-major, all device memory unless stated):
 *   q, out          [B][Hq][d]        dtype of the config (bf16 or fp32)
 *   k_cache,v_cache [P][Hkv][S][d]    dtype of the config; one (page, kv head) slab of
 *                                     S*d elements is contiguous
 *   reps            [P][Hkv][d]       fp32
 *   block_table     [B][max_blocks]   int32 physical page of logical block b; entries for
 *                                     b >= ceil(L/S) are never read
 *   seq_lens, prompt_lens [B]         int32
 *   sel             [B][Hkv][kmax]    int32 selected logical blocks, ascending
 *   nsel            [B][Hkv]          int32
 * Ownership: the caller owns every buffer.  The library allocates nothing, frees
 * nothing and synchronises only in srkv_retrieval_decode_host (which returns its output in
 * host memory); every other call is asynchronous on `stream` (a
 * cudaStream_t; NULL is the legacy default stream) and returns after launching.
 * Errors: the return value reports host-side argument checks and launch failures.
 * Problems only visible on the device (a page id outside [0, num_pages), a sequence
 * longer than max_blocks*S, a malformed selection, a bounded wait that ran out) make
 * the kernels skip the offending work, never fault, and set SRKV_EFLAG_* bits in the
 * optional device word `error_flags` (may be NULL; the caller clears it).
 * No C++ exception crosses this interface.
 */
#ifndef SRKV_H
#define SRKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* srkv_stream; /* identical to cudaStream_t */

typedef enum {
  SRKV_OK = 0,
  SRKV_ERR_INVALID_ARG = 1, /* null pointer, bad size, bad alignment, bad config value */
  SRKV_ERR_UNSUPPORTED = 2, /* a valid configuration that this build does not implement */
  SRKV_ERR_WORKSPACE = 3,   /* workspace missing or smaller than srkv_decode_workspace_size */
  SRKV_ERR_CUDA = 4         /* a CUDA call or kernel launch failed */
} srkv_status;

typedef enum { SRKV_BF16 = 0, SRKV_F32 = 1 } srkv_dtype;

/* Device-side error bits, OR-ed into *error_flags. */
#define SRKV_EFLAG_PAGE_RANGE 1u /* a block-table entry outside [0, num_pages) was skipped */
#define SRKV_EFLAG_SEQ_LEN 2u    /* seq_len < 0 or > max_blocks*S; clamped into range */
#define SRKV_EFLAG_SELECTION 4u  /* nsel outside [0, kmax], or a sel entry that is not a
                                    candidate or not ascending; such entries were skipped */
#define SRKV_EFLAG_TIMEOUT 8u    /* a bounded on-chip wait ran out; the kernel returned early */
#define SRKV_EFLAG_PREFIX 16u    /* a request maps a block of the declared shared prefix to
                                    another page than the batch's other requests (the
                                    shared-prefix calls read one page for all of them) */
#define SRKV_EFLAG_CHUNK 32u     /* chunk_offsets go down or leave [0, total_tokens], or a chunk
                                    is longer than its sequence (chunk calls) */

/* Configuration: the method's knobs ("Configuration Parameters") and the head layout. */
typedef struct {
  int32_t num_q_heads;    /* Hq, a multiple of num_kv_heads */
  int32_t num_kv_heads;   /* Hkv */
  int32_t head_dim;       /* d: 64 or 128 */
  int32_t block_size;     /* S: must be 128 (the pages' recommended block size) */
  int32_t init_tokens;    /* INIT_TOKENS_NUM, >= 0, default 1024 */
  int32_t local_tokens;   /* LOCAL_TOKENS_NUM, >= 0, default 7192 */
  double topk_percent;    /* TOPK_PERCENT in [0, 1], default 0.2 */
  int32_t dense_boundary; /* DENSE_BOUNDARY, >= 0, default 32768; 0 disables dense mode */
  int32_t dtype;          /* srkv_dtype of q, caches and out */
} srkv_config;

/* Fills the pages' defaults: Hq 32, Hkv 8, d 128, S 128, 1024 / 7192 / 0.2 / 32768, bf16. */
void srkv_default_config(srkv_config* cfg);

/* Human-readable name of a status; never NULL. */
const char* srkv_status_string(srkv_status status);

/* k for n candidates at ratio p (definition above); 0 for n <= 0. */
int64_t srkv_topk_count(int64_t n_candidates, double topk_percent);

/* Number of candidate blocks of a sequence of seq_len tokens under cfg; 0 if cfg is NULL. */
int64_t srkv_num_candidates(const srkv_config* cfg, int64_t seq_len);

/* The sel capacity (kmax) that srkv_score_topk needs for any request of at most
 * max_blocks*S tokens: all candidates when dense mode can occur, else k of them. */
int32_t srkv_kmax_bound(const srkv_config* cfg, int32_t max_blocks);

/*
 * Representation vectors ("Feature Description": extracted block by block at prefill).
 * For i < n_pages: reps[page_ids[i]][h][:] = mean over t < page_valid_tokens[i] of
 * k_cache[page_ids[i]][h][t][:], accumulated in fp32, for every kv head h.  Pages not
 * listed are left untouched.  page_valid_tokens[i] = 0 writes zeros.
 *   k_cache: [num_pages][Hkv][S][d], 16-byte aligned.   reps: [num_pages][Hkv][d] fp32.
 *   page_ids, page_valid_tokens: device int32 [n_pages]; an id outside [0, num_pages) or a
 *   count outside [0, S] is skipped and flagged (SRKV_EFLAG_PAGE_RANGE).
 */
srkv_status srkv_build_block_reps(const srkv_config* cfg, const void* k_cache,
                                  int64_t num_pages, const int32_t* page_ids,
                                  const int32_t* page_valid_tokens, int32_t n_pages,
                                  float* reps, int32_t* error_flags, srkv_stream stream);

/*
 * Decode-time maintenance of the cache and of the vector store (openGauss page, "Feature
 * Description": the representation vectors are extracted block by block, and "Overall
 * Solution": decode keeps adding tokens to the cache).  For every request r and kv head h,
 * the new token's key and value k_new[r][h][:], v_new[r][h][:] are written at position
 * L = seq_lens[r] of the request, i.e. row L % S of page block_table[r][L / S], and that
 * page's representation vector reps[page][h][:] is recomputed over its rows [0, L % S] -- the
 * same value srkv_build_block_reps gives for the page with L % S + 1 valid tokens.
 *   k_new, v_new: [B][Hkv][d] in the cache dtype, 16-byte aligned; k_cache, v_cache,
 *   num_pages, block_table, max_blocks, reps: as for the other calls (written in place).
 *   seq_lens: device int32 [B], read only: the caller advances the lengths (seq_lens[r] += 1)
 *   after the call, and must give request r a page of its own at block L / S (a page shared
 *   with other requests would change for them too).
 *   A length outside [0, max_blocks * S) (SRKV_EFLAG_SEQ_LEN) or a page id outside
 *   [0, num_pages) (SRKV_EFLAG_PAGE_RANGE) skips that request and is flagged.
 * Asynchronous on `stream`; one kernel.
 */
srkv_status srkv_append_kv(const srkv_config* cfg, const void* k_new, const void* v_new,
                           void* k_cache, void* v_cache, int64_t num_pages,
                           const int32_t* block_table, int32_t max_blocks,
                           const int32_t* seq_lens, int32_t batch, float* reps,
                           int32_t* error_flags, srkv_stream stream);

/*
 * A ragged chunk of new tokens appended to the cache, rotated to their positions on the way: a
 * prompt or a piece of one, one token of each request at decode, or both in one batch (the page
 * vectors of openGauss's "Feature Description" stay current, as with srkv_append_kv; the pages name no
 * rotation, whose place in a serving step is between the projections and the cache).  Request r
 * brings rows [chunk_offsets[r], chunk_offsets[r + 1]) of the packed inputs, n_r of them; row i of
 * them stands at position p = seq_lens[r] + i.
 *   rotation: for j < rope_dim / 2, with a = p * rope_freqs[j] (radians), the pair (x, y) of elements
 *     (j, j + rope_dim / 2), or (2j, 2j + 1) if `interleaved`, becomes (x cos a - y sin a,
 *     y cos a + x sin a); elements from rope_dim on stay.  The angle is reduced to a turn without
 *     rounding whatever the position, sine, cosine and products are fp32, and the result is rounded
 *     once to the cache dtype.
 *   q_out[row][j][:] = rotated q[row][j]           (q and q_out both NULL: no queries)
 *   K row p % S of page block_table[r][p / S]      = rotated k_new[row][h]
 *   V row of the same place                        = v_new[row][h]
 *   reps of every page written = mean of its keys, as held, over its rows up to the chunk's last one:
 *     the value that srkv_build_block_reps gives for that many valid tokens.
 *   q: [total_tokens][Hq][d], k_new, v_new: [total_tokens][Hkv][d] in the cache dtype, tokens q_stride,
 *   k_stride, v_stride elements apart (the parts of one fused projection, for instance; multiples of 16
 *   bytes, at least one token's heads); q_out: [total_tokens][Hq][d], q itself where q_stride = Hq d, else
 *   apart from q, k_new and v_new (SRKV_ERR_INVALID_ARG where it lies between their first and last
 *   element); all 16-byte aligned.  rope_freqs: device double [rope_dim / 2], of magnitudes below 2^32, of any sign;
 *   rope_dim: even, 0 to d, 0 leaves out the rotation; a multiple of 16, else SRKV_ERR_UNSUPPORTED.  chunk_offsets: device int32
 *   [batch + 1], from 0 or more up to total_tokens or less, not decreasing; n_r = 0 is allowed, and rows
 *   of the packed tensors outside every request are left alone.  seq_lens: the lengths before the
 *   chunk, read only: the caller advances them (seq_lens[r] += n_r), and gives every request pages of its own
 *   for the tokens written.
 *   A request whose offsets are wrong (SRKV_EFLAG_CHUNK) or whose tokens do not all fit in
 *   [0, max_blocks * S) (SRKV_EFLAG_SEQ_LEN) is skipped, a page id outside [0, num_pages) skips that page
 *   (SRKV_EFLAG_PAGE_RANGE; queries are rotated all the same); all are flagged.  Where offsets go down,
 *   other requests' rows and pages, too, are written as described or left as they were (a row's request is searched for,
 *   as offsets that do not go down allow).
 * Asynchronous on `stream`; one kernel.
 */
srkv_status srkv_append_kv_rope(const srkv_config* cfg, const void* q, int64_t q_stride,
                                const void* k_new, int64_t k_stride, const void* v_new,
                                int64_t v_stride, const int32_t* chunk_offsets,
                                int32_t total_tokens, const double* rope_freqs, int32_t rope_dim,
                                int32_t interleaved, void* q_out, void* k_cache, void* v_cache,
                                int64_t num_pages, const int32_t* block_table, int32_t max_blocks,
                                const int32_t* seq_lens, int32_t batch, float* reps,
                                int32_t* error_flags, srkv_stream stream);

/*
 * Compressed pages (KV-cache survey "大模型推理百倍加速之KV cache篇": quantising the cache is
 * one of the ways to shrink it).  Writes the listed pages of a bf16 cache as E4M3 codes (the
 * 8-bit floating point format "E4M3" of the OCP 8-bit floating point specification: 4
 * exponent bits, 3 mantissa bits, largest finite value 448) with one fp32 scale per
 * (page, kv head, token) row:
 *   scale = max over the row of |x| / 448   (1 for an all-zero row),
 *   code  = E4M3(x / scale), the quotient in fp32, rounded to nearest, ties to even,
 *           finite values past 448 saturated,
 * so a value is code x scale.  Per row rather than per page, so that a later token needs no
 * re-quantisation of its page.
 *   cfg->dtype must be SRKV_BF16 (the source); k_cache, v_cache: [num_pages][Hkv][S][d] bf16;
 *   k_fp8, v_fp8: [num_pages][Hkv][S][d] bytes; k_scale, v_scale: [num_pages][Hkv][S] fp32;
 *   every pointer 16-byte aligned.  Page page_ids[i] of the source is written to the same
 *   page of the destination; other pages are untouched.  An id outside [0, num_pages) is
 *   skipped and flags SRKV_EFLAG_PAGE_RANGE.
 */
srkv_status srkv_quantize_kv_fp8(const srkv_config* cfg, const void* k_cache,
                                 const void* v_cache, int64_t num_pages,
                                 const int32_t* page_ids, int32_t n_pages, void* k_fp8,
                                 void* v_fp8, float* k_scale, float* v_scale,
                                 int32_t* error_flags, srkv_stream stream);

/*
 * 4-bit pages (the same survey's quantisation of the cache, at half the bits of E4M3).  A 4-bit cache is
 * one buffer kv_int4: [num_pages][Hkv][srkv_kv_int4_slab_bytes(cfg)] bytes, 16-byte aligned; the
 * slab of a (page, kv head) holds its 128 keys and values.  A row x (one token's d values) is held as
 *   lo = min x (bf16),  scale = (max x - lo) / 15 rounded up to bf16 (the bf16 below that where
 *          lo + 15 scale would round past bf16's largest value),
 *   code = the integer in 0 .. 15 nearest to (x - lo) / scale, ties to even (difference and quotient in
 *          fp32); 0 if the scale is below 2^-126 (a row whose values are all equal, or nearly zero),
 * and stands for lo + code * scale.  A row with an infinity or a NaN, or whose range passes fp32, gets
 * scale = lo = NaN and reads back as NaN.  The 128 d + 1024 bytes of a slab, in order (words are 32 bits;
 * code j of a word at bit 4 (j / 2) + 16 (j mod 2)):
 *   keys' codes   [128][d / 8] words: elements 8i .. 8i + 7 of token t in word (t, i);
 *   values' codes [4][d / 4][4][4] words: element 4c + e of tokens 32w + 8t .. 32w + 8t + 7 in word
 *                 (w, c, t, e);
 *   keys' rows, then values' rows, [128] words each: scale (low half) and lo (high half).
 */

/* Bytes of one (page, kv head) slab: 128 d + 1024; 0 if cfg is invalid. */
size_t srkv_kv_int4_slab_bytes(const srkv_config* cfg);

/*
 * Compresses listed pages: page page_ids[i] of the bf16 caches, all 128 rows of it, into page
 * int4_page_ids[i] of kv_int4 (NULL: page_ids[i]); other pages are untouched.  The two caches may
 * have different numbers of pages, so that a small bf16 pool can feed a large 4-bit one.
 *   cfg->dtype must be SRKV_BF16 (else SRKV_ERR_UNSUPPORTED); k_cache, v_cache: [num_pages][Hkv][S][d]
 *   bf16, 16-byte aligned; num_int4_pages: pages of kv_int4; the ids: device int32 [n_pages].
 *   An id outside its cache skips that entry and flags SRKV_EFLAG_PAGE_RANGE.  A destination listed
 *   twice with different sources ends up with a mix of them.  Asynchronous; one kernel.
 */
srkv_status srkv_quantize_kv_int4(const srkv_config* cfg, const void* k_cache,
                                  const void* v_cache, int64_t num_pages,
                                  const int32_t* page_ids, int32_t n_pages, void* kv_int4,
                                  int64_t num_int4_pages, const int32_t* int4_page_ids,
                                  int32_t* error_flags, srkv_stream stream);

/*
 * Reads listed pages back: page int4_page_ids[i] of kv_int4 into page page_ids[i] of the bf16
 * caches (NULL: int4_page_ids[i]), as lo + code * scale rounded once to bf16, all 128 rows.  For what
 * takes full-precision pages (the shared-prefix calls, a later prefill chunk).  Arguments and errors
 * as for srkv_quantize_kv_int4.
 */
srkv_status srkv_dequantize_kv_int4(const srkv_config* cfg, const void* kv_int4,
                                    int64_t num_int4_pages, const int32_t* int4_page_ids,
                                    int32_t n_pages, void* k_cache, void* v_cache,
                                    int64_t num_pages, const int32_t* page_ids,
                                    int32_t* error_flags, srkv_stream stream);

/*
 * srkv_append_kv into a 4-bit cache: for every request r and kv head h the new token's key and value
 * (bf16) are quantised and written as row L % S of page block_table[r][L / S], L = seq_lens[r], and
 * the page's representation vector becomes the fp32 mean of its keys as held, lo + code * scale over
 * rows [0, L % S].  (The vectors of pages compressed by srkv_quantize_kv_int4 are the caller's, from
 * srkv_build_block_reps on the bf16 keys.)  The page's other rows keep their codes.  A token written
 * again, or written over after the length was set back, gives the same cache and vector as a
 * first write.  cfg->dtype must be SRKV_BF16 (else SRKV_ERR_UNSUPPORTED).  Other arguments, the page
 * of its own that each request needs at block L / S, and errors: srkv_append_kv.
 */
srkv_status srkv_append_kv_int4(const srkv_config* cfg, const void* k_new, const void* v_new,
                                void* kv_int4, int64_t num_pages, const int32_t* block_table,
                                int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                float* reps, int32_t* error_flags, srkv_stream stream);

/*
 * Scoring and top-k ("Overall Solution": inner product of the current query with each
 * representation vector, keep the topK closest).  For every request r and kv head h:
 * sel[r][h][0..nsel[r][h]) = the selected candidate blocks of (r, h), ascending; dense
 * requests (prompt_lens[r] < dense_boundary) select every candidate.
 *   q: [B][Hq][d] (cfg dtype, 16-byte aligned); reps: [num_pages][Hkv][d] fp32 as written
 *   by srkv_build_block_reps for every page a candidate block maps to;
 *   prompt_lens may be NULL (then prompt = seq_len);
 *   kmax >= srkv_kmax_bound(cfg, max_blocks), else SRKV_ERR_INVALID_ARG;
 *   max_blocks <= 25600 (3 276 800 tokens: the key and page of every candidate are held
 *   on chip while a unit is selected), else SRKV_ERR_UNSUPPORTED.
 * The selection is a function of the inputs alone: bitwise the same on every call.
 */
srkv_status srkv_score_topk(const srkv_config* cfg, const void* q, const float* reps,
                            int64_t num_pages, const int32_t* block_table, int32_t max_blocks,
                            const int32_t* seq_lens, const int32_t* prompt_lens, int32_t batch,
                            int32_t* sel, int32_t kmax, int32_t* nsel, int32_t* error_flags,
                            srkv_stream stream);

/* Bytes of device workspace srkv_sparse_paged_decode needs for `batch` requests on the
 * current device; 0 if cfg is invalid. */
size_t srkv_decode_workspace_size(const srkv_config* cfg, int32_t batch);

/*
 * Sparse paged decode attention ("Overall Solution": the kept blocks are concatenated
 * with the initial and window KV and take part in attention; flash-decoding split and
 * merge as in the survey's "Share--KV cache共享" section).  For every request r and query
 * head j of kv head h = j / G:
 *   out[r][j][:] = softmax over the attended tokens of q[r][j].K_t / sqrt(d), times V_t,
 * with the attended set built from sel/nsel (as written by srkv_score_topk, or any
 * ascending list of candidate blocks).  Accumulation is fp32; out has the cfg dtype.
 *   k_cache, v_cache: [num_pages][Hkv][S][d], 16-byte aligned;
 *   workspace: >= srkv_decode_workspace_size(cfg, batch) bytes, 256-byte aligned, contents
 *   need not be initialised; it is scratch owned by this call until the stream reaches
 *   the end of the call.
 */
srkv_status srkv_sparse_paged_decode(const srkv_config* cfg, const void* q, const void* k_cache,
                                     const void* v_cache, int64_t num_pages,
                                     const int32_t* block_table, int32_t max_blocks,
                                     const int32_t* seq_lens, int32_t batch,
                                     const int32_t* sel, int32_t kmax, const int32_t* nsel,
                                     void* out, void* workspace, size_t workspace_bytes,
                                     int32_t* error_flags, srkv_stream stream);

/*
 * One whole decode step: the result of srkv_score_topk followed by srkv_sparse_paged_decode
 * on the same stream, with the selection written to the caller's sel/nsel buffers (openGauss
 * page, "Overall Solution": score, keep the topK blocks, attend them with the initial tokens
 * and the window).  Arguments as for those two calls; prompt_lens may be NULL (the prompt
 * is then the sequence length).
 *   How: a batch small enough for one thread-block cluster per (request, kv head) unit to be
 *   resident (at most 15 units with clusters of 8 to 16 CTAs, or, for bf16 pages with d 128
 *   and a top-k ratio <= 0.3, at most 36 units with clusters of 4 to 7; the largest cluster
 *   size whose clusters are all resident is taken; <= 1024 candidate blocks per request,
 *   bf16, d 64 or 128, group <= 8) runs as one kernel; otherwise the scoring
 *   kernel, the split decode (which
 *   streams the initial and window pages while the scoring runs) and the combine.  The first
 *   call for a configuration on a device queries the device (cluster residency); make it
 *   before any stream capture.  max_blocks <= 25600 as for srkv_score_topk.
 *   Reproducibility: sel and nsel are bitwise the same on every call.  On the three-kernel
 *   path (and in srkv_sparse_paged_decode) out is too.  On the one-kernel path each
 *   streaming CTA of a unit's cluster gets its first 16 kept blocks assigned by the
 *   selection (round robin); out is bitwise the same on every call when no unit keeps more
 *   than 16 blocks per streaming CTA (with clusters of 12 CTAs, 11 streaming: up to 176 kept
 *   blocks); beyond that the CTAs take the remaining kept blocks from a shared pool as their
 *   pages arrive, the partial sums split at pages that vary from call to call, and out may
 *   differ in its last bits.
 */
srkv_status srkv_retrieval_decode(const srkv_config* cfg, const void* q, const void* k_cache,
                                  const void* v_cache, const float* reps, int64_t num_pages,
                                  const int32_t* block_table, int32_t max_blocks,
                                  const int32_t* seq_lens, const int32_t* prompt_lens,
                                  int32_t batch, int32_t* sel, int32_t kmax, int32_t* nsel,
                                  void* out, void* workspace, size_t workspace_bytes,
                                  int32_t* error_flags, srkv_stream stream);

/*
 * srkv_retrieval_decode with host buffers for the per-step inputs and the output, as a
 * serving loop on the host calls it: q_host ([batch][Hq][d] in the cfg dtype), seq_lens_host
 * and prompt_lens_host ([batch] int32; prompt_lens_host may be NULL) are copied into
 * `staging`, the decode runs on them, out is copied into out_host ([batch][Hq][d] in the cfg
 * dtype), and the call returns once out_host holds it (it synchronises `stream`).  Host
 * buffers in page-locked memory copy asynchronously; pageable ones work too, more slowly.
 *   staging: device memory of at least srkv_host_staging_size(cfg, batch) bytes, 256-byte
 *     aligned, owned by the caller; its contents on entry do not matter.  It holds q, then
 *     seq_lens, then prompt_lens, each at a 256-byte boundary; host inputs that sit in one
 *     buffer at those same offsets go in one copy, others in one copy each.
 *   Every other argument, its layout and its errors: srkv_retrieval_decode (out is still a
 *   device buffer, the one the decode writes).  SRKV_ERR_INVALID_ARG for a NULL host
 *   pointer or staging, a small or unaligned staging; SRKV_ERR_CUDA if a copy or the
 *   synchronisation fails (out_host is then undefined).
 */
size_t srkv_host_staging_size(const srkv_config* cfg, int32_t batch);
srkv_status srkv_retrieval_decode_host(const srkv_config* cfg, const void* q_host,
                                       const int32_t* seq_lens_host,
                                       const int32_t* prompt_lens_host, void* out_host,
                                       void* staging, size_t staging_bytes,
                                       const void* k_cache, const void* v_cache,
                                       const float* reps, int64_t num_pages,
                                       const int32_t* block_table, int32_t max_blocks,
                                       int32_t batch, int32_t* sel, int32_t kmax, int32_t* nsel,
                                       void* out, void* workspace, size_t workspace_bytes,
                                       int32_t* error_flags, srkv_stream stream);

/*
 * srkv_retrieval_decode with an offload tier (openGauss page, "Overall Solution" and
 * "Feature Description": KV blocks past the offload boundary live off the accelerator's
 * memory, their representation vectors stay resident, and only the topK blocks the query
 * selects are fetched each step).  Page ids in [0, num_pages) name pages of the device pool
 * k_cache/v_cache; ids in [num_pages, num_pages + num_host_pages) name page
 * (id - num_pages) of a second pool k_host/v_host with the same [page][Hkv][S][d] layout.
 * The decode reads host pages in place, over the chip-to-chip link, straight into the shared
 * memory stages the device pages go through (no staging copy in HBM); which pages live where
 * is the caller's choice (typically the candidate blocks go to the host pool and the initial
 * and window pages stay on the device).  Results equal srkv_retrieval_decode's on the same
 * page contents.
 *   k_host, v_host: pinned (page-locked, e.g. cudaHostAlloc) or managed host memory, or
 *     device memory; 16-byte aligned; pageable memory is rejected (SRKV_ERR_INVALID_ARG).
 *     May be NULL when num_host_pages = 0 (the call is then srkv_retrieval_decode).
 *   reps: [num_pages + num_host_pages][Hkv][d] fp32 in device memory (computed while the
 *     pages were on the device, e.g. by srkv_build_block_reps before they are moved).
 *   A host pool needs the tensor-core decode (bf16, d 64 or 128, group <= 8), else
 *     SRKV_ERR_UNSUPPORTED.  Other arguments, ownership and errors: srkv_retrieval_decode.
 *     The host pool must not be written while the call runs.
 */
srkv_status srkv_retrieval_decode_tiered(const srkv_config* cfg, const void* q,
                                         const void* k_cache, const void* v_cache,
                                         int64_t num_pages, const void* k_host,
                                         const void* v_host, int64_t num_host_pages,
                                         const float* reps, const int32_t* block_table,
                                         int32_t max_blocks, const int32_t* seq_lens,
                                         const int32_t* prompt_lens, int32_t batch, int32_t* sel,
                                         int32_t kmax, int32_t* nsel, void* out, void* workspace,
                                         size_t workspace_bytes, int32_t* error_flags,
                                         srkv_stream stream);

/*
 * srkv_retrieval_decode over compressed pages (srkv_quantize_kv_fp8): the attended K and V
 * values are code x scale of the E4M3 caches, widened to fp16 (exactly) for the tensor-core
 * products, with fp32 accumulation as in the bf16 decode.  The selection comes from `reps`,
 * the representation vectors of the full-precision keys (built by srkv_build_block_reps
 * before the pages are compressed), so it is the selection the bf16 call makes.
 *   cfg->dtype = SRKV_BF16 (the query and the output), head_dim 128, group <= 8, else
 *   SRKV_ERR_UNSUPPORTED.  k_fp8, v_fp8: [num_pages][Hkv][S][d] bytes; k_scale, v_scale:
 *   [num_pages][Hkv][S] fp32; all 16-byte aligned.  Other arguments, ownership, paths (one
 *   kernel for small batches, else three) and errors: srkv_retrieval_decode.
 */
srkv_status srkv_retrieval_decode_fp8(const srkv_config* cfg, const void* q, const void* k_fp8,
                                      const void* v_fp8, const float* k_scale,
                                      const float* v_scale, const float* reps,
                                      int64_t num_pages, const int32_t* block_table,
                                      int32_t max_blocks, const int32_t* seq_lens,
                                      const int32_t* prompt_lens, int32_t batch, int32_t* sel,
                                      int32_t kmax, int32_t* nsel, void* out, void* workspace,
                                      size_t workspace_bytes, int32_t* error_flags,
                                      srkv_stream stream);

/*
 * srkv_retrieval_decode over a 4-bit cache (srkv_quantize_kv_int4, srkv_append_kv_int4): the attended K and
 * V values are lo + code * scale.  Both products take the codes as fp16 operands with fp32
 * accumulation; the query enters as fp16 times a power of two for each head (exact down
 * to 2^-25 of the head's largest magnitude), each softmax weight times its row's V scale as fp16 (11 bits
 * down to 2^-20 of the largest such product of the head's tokens that a warp has met, to half a step of
 * 2^-31 of it below), the scales and minima in fp32.
 *   Magnitudes: fp32 holds the logits and their parts (|lo| times the query's sum, scale times the query) and the
 *   sums of up to 2^8 times the values over the attended tokens.  So |q| below 2^101, the largest |q| times a
 *   row's K scale or minimum below 2^117, |V| below 2^98 (and V scales below 2^-100 lose bits).
 *   The selection comes from `reps`, as in the other calls.
 *   cfg->dtype = SRKV_BF16 (the query and the output), group <= 8, else SRKV_ERR_UNSUPPORTED;
 *   head_dim 64 or 128.  kv_int4: [num_pages][Hkv][srkv_kv_int4_slab_bytes(cfg)].  A NaN row that is
 *   attended makes the outputs that attend it NaN; rows that are not attended never do.  Other
 *   arguments, ownership, errors and reproducibility: srkv_retrieval_decode; the one-kernel path
 *   takes up to 15 units, and assigns 32 kept blocks to each streaming CTA with the selection.
 */
srkv_status srkv_retrieval_decode_int4(const srkv_config* cfg, const void* q, const void* kv_int4,
                                       const float* reps, int64_t num_pages,
                                       const int32_t* block_table, int32_t max_blocks,
                                       const int32_t* seq_lens, const int32_t* prompt_lens,
                                       int32_t batch, int32_t* sel, int32_t kmax, int32_t* nsel,
                                       void* out, void* workspace, size_t workspace_bytes,
                                       int32_t* error_flags, srkv_stream stream);

/*
 * Shared-prefix decode (KV-cache survey "大模型推理百倍加速之KV cache篇", section "Share--KV
 * cache共享": FlashInfer's cascade inference and Hydragen attend a prefix shared by a batch's
 * requests once, as a matrix-matrix product over all their queries, and merge it with each
 * request's own part like Flash-Decoding partials; the ATB reuse article, §2.1 and §3.3, keeps
 * such prefix pages once and references them from every request).  The results are those of
 * srkv_sparse_paged_decode / srkv_retrieval_decode on the same inputs: only the way the work
 * is split changes.  The first prefix_blocks logical blocks of EVERY request must map to the
 * same physical pages (block_table[r][b] == block_table[0][b] for b < prefix_blocks); the
 * whole pages of that prefix a request's length covers are attended for all requests at once,
 * one (page, kv head) slab read per group of up to 128 query rows, with each request's own
 * rows of it (initial tokens, window, its selected blocks) masked in; the rest of each request
 * goes through the split decode.  A request whose table breaks the contract inside its
 * prefix flags SRKV_EFLAG_PREFIX (its result is then not the definition's).
 *   prefix_blocks: 0 <= prefix_blocks <= max_blocks, at most 2048 (else
 *     SRKV_ERR_UNSUPPORTED); 0 gives the plain call.
 *   cfg: bf16, head_dim 128, group 1, 2, 4 or 8 (else SRKV_ERR_UNSUPPORTED).
 *   workspace: >= srkv_prefix_decode_workspace_size(cfg, batch) bytes, 256-byte aligned.
 *   Other arguments, ownership and errors: srkv_sparse_paged_decode / srkv_retrieval_decode.
 *   Both calls always take the kernels of the split path (no one-kernel path); their output
 *   is bitwise the same on every call.
 */
size_t srkv_prefix_decode_workspace_size(const srkv_config* cfg, int32_t batch);

srkv_status srkv_sparse_paged_decode_prefix(const srkv_config* cfg, const void* q,
                                            const void* k_cache, const void* v_cache,
                                            int64_t num_pages, const int32_t* block_table,
                                            int32_t max_blocks, const int32_t* seq_lens,
                                            int32_t batch, int32_t prefix_blocks,
                                            const int32_t* sel, int32_t kmax,
                                            const int32_t* nsel, void* out, void* workspace,
                                            size_t workspace_bytes, int32_t* error_flags,
                                            srkv_stream stream);

srkv_status srkv_retrieval_decode_prefix(const srkv_config* cfg, const void* q,
                                         const void* k_cache, const void* v_cache,
                                         const float* reps, int64_t num_pages,
                                         const int32_t* block_table, int32_t max_blocks,
                                         const int32_t* seq_lens, const int32_t* prompt_lens,
                                         int32_t batch, int32_t prefix_blocks, int32_t* sel,
                                         int32_t kmax, int32_t* nsel, void* out, void* workspace,
                                         size_t workspace_bytes, int32_t* error_flags,
                                         srkv_stream stream);

/*
 * Attention of a ragged chunk of new tokens over the paged cache that already holds them (what comes
 * between srkv_append_kv_rope and the first decode step: a prompt, a later piece of one, or, with one
 * token a request, a decode step that leaves no block out).  Request r brings the query rows
 * [chunk_offsets[r], chunk_offsets[r + 1]), n_r of them; with L = seq_lens[r], the new tokens counted,
 * row i stands at position p = L - n_r + i, and
 *   srkv_chunk_attention:         attends the tokens t <= p;
 *   srkv_chunk_attention_window:  those of them with t < init_tokens or t > p - local_tokens: the first
 *     tokens and the window of the position (survey "大模型推理百倍加速之KV
 *     cache篇": sinks and a sliding window), as the decode calls see them without a kept block.
 * out[row][j][:] = softmax over those tokens of q[row][j].K_t / sqrt(d), times V_t; a row that attends
 * nothing, or whose logits are all -infinity, gives 0, whatever its values.  Else an attended value that is not
 * finite makes its element of the row infinite or NaN, however small its weight (a weight that fp32 does not hold
 * may turn an infinity into a NaN).  A row depends on no token that it does not attend,
 * whatever that token's key and value hold (NaN and infinities too), nor on anything behind L.  Logits,
 * maxima, sums and outputs are held in fp32.  With bf16 the softmax weights, up to 2^8 each as they are held,
 * are rounded to bf16 for the product with V (by up to 2^-8 of each), so 2^8 times the sum of the attended
 * values' magnitudes has to stay in fp32; with fp32 nothing is rounded below fp32.
 *   q: [total_tokens][Hq][d], tokens q_stride elements apart (a multiple of 16 bytes, at least Hq d);
 *   out: [total_tokens][Hq][d], apart from q (SRKV_ERR_INVALID_ARG where it lies between q's first and last
 *   element); both 16-byte aligned.  Rows outside every request are left as they were.
 *   chunk_offsets: as for srkv_append_kv_rope.  Any group size Hq / Hkv.
 *   workspace: >= srkv_chunk_workspace_size(cfg, total_tokens, batch) bytes, 256-byte aligned; its
 *   contents on entry do not matter; it is scratch of this call until the stream reaches its end, so
 *   calls that may overlap (streams, captured graphs) take one each.
 *   A request whose offsets are wrong is skipped (where offsets go down, a row that two requests claim is either's,
 *   and requests may be skipped that ask for more rows in all than there are); of a chunk longer than its sequence
 *   the first rows attend nothing; all flag SRKV_EFLAG_CHUNK.  A length outside [0, max_blocks * S] is clamped into it
 *   (SRKV_EFLAG_SEQ_LEN).  The tokens of a page whose id is outside [0, num_pages) are left out
 *   (SRKV_EFLAG_PAGE_RANGE).
 *   The output is a function of the inputs alone: bitwise the same on every call.
 * Asynchronous on `stream`; three kernels.
 */
size_t srkv_chunk_workspace_size(const srkv_config* cfg, int32_t total_tokens, int32_t batch);

srkv_status srkv_chunk_attention(const srkv_config* cfg, const void* q, int64_t q_stride,
                                 const void* k_cache, const void* v_cache, int64_t num_pages,
                                 const int32_t* block_table, int32_t max_blocks,
                                 const int32_t* chunk_offsets, int32_t total_tokens,
                                 const int32_t* seq_lens, int32_t batch, void* out,
                                 void* workspace, size_t workspace_bytes, int32_t* error_flags,
                                 srkv_stream stream);

srkv_status srkv_chunk_attention_window(const srkv_config* cfg, const void* q, int64_t q_stride,
                                        const void* k_cache, const void* v_cache,
                                        int64_t num_pages, const int32_t* block_table,
                                        int32_t max_blocks, const int32_t* chunk_offsets,
                                        int32_t total_tokens, const int32_t* seq_lens,
                                        int32_t batch, void* out, void* workspace,
                                        size_t workspace_bytes, int32_t* error_flags,
                                        srkv_stream stream);

/*
 * Number of kernels one srkv_retrieval_decode call with these arguments launches on the
 * current device (1 for the one-kernel small-batch path, else 3); 0 if cfg is invalid.
 * Host only; queries the device like the first call does.
 */
int32_t srkv_retrieval_decode_launches(const srkv_config* cfg, int32_t batch, int32_t max_blocks);

/*
 * For callers that cannot allocate device memory: srkv_sparse_paged_decode without a
 * workspace argument.  (The method's pages have no counterpart of this; it is a service of
 * this library.)  Some callers cannot call cudaMalloc on the decode path: code running under
 * stream capture for a CUDA graph (plain cudaMalloc is not a capturable operation), serving
 * loops that forbid allocator calls so that every step costs the same, plugins handed only
 * their input and output buffers by a host framework that owns all device memory, and
 * processes whose device memory is fully reserved up front.  They pass only inputs and
 * outputs; the scratch space is a file-scope device array of SRKV_NOALLOC_WORKSPACE_BYTES
 * in this library, which every GPU that loads the library holds until the process exits.
 *   - Arguments, layouts and results are those of srkv_sparse_paged_decode.
 *   - A batch whose decode needs more scratch than SRKV_NOALLOC_WORKSPACE_BYTES
 *     (srkv_decode_workspace_size) is rejected with SRKV_ERR_WORKSPACE before any launch.
 *   - The first call on a device looks up the array's device address (with that device
 *     current) and keeps it for the current CUDA context; a call made in another context of
 *     the device (one the caller created, or the primary context brought up again after
 *     cudaDeviceReset) looks it up again.  Make the first call in each context before any
 *     stream capture.
 *   - Every call on a device shares the one array, and each call leaves its contents behind
 *     (nothing in it needs to start at zero: a call writes every value it reads).  Calls
 *     whose kernels overlap on the GPU (on different streams, without ordering between
 *     them) race on it: order them.
 *   - No allocation, free or allocating library routine is called.
 */
#define SRKV_NOALLOC_WORKSPACE_BYTES ((size_t)16 << 20)

srkv_status srkv_sparse_paged_decode_noalloc(const srkv_config* cfg, const void* q,
                                             const void* k_cache, const void* v_cache,
                                             int64_t num_pages, const int32_t* block_table,
                                             int32_t max_blocks, const int32_t* seq_lens,
                                             int32_t batch, const int32_t* sel, int32_t kmax,
                                             const int32_t* nsel, void* out,
                                             int32_t* error_flags, srkv_stream stream);

/*
 * Self-test of the bounded on-chip waits (no counterpart on the pages; a service of this
 * library).  Every wait of the decode kernels gives up after a limit of 2 s, sets
 * SRKV_EFLAG_TIMEOUT and lets its kernel finish instead of hanging.  This call launches one
 * kernel (a cluster of 2 CTAs) whose waits, one on a CTA-scope and one on a cluster-scope
 * mbarrier, have no arrival at all: both run to their limit, OR SRKV_EFLAG_TIMEOUT into
 * *error_flags (device memory) and return, about 4 s after the kernel starts.  Nothing else
 * is read or written, nothing faults, and the context stays usable.
 */
srkv_status srkv_selftest_wait_timeout(int32_t* error_flags, srkv_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SRKV_H */
