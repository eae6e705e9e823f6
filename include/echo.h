/*
 * echo.h — C ABI of the MI355X (gfx950) DSA-indexer + top-k + pool-residency decode step.
 *
 * What the library computes follows the ECHO review page ("OSDI'26 | ECHO：稀疏 attention
 * 省了算力，却把 HBM 撑爆了"):
 *   §2    the lightning-indexer score of a cached token s for query t is the sum over the
 *         64 indexer heads of w[h,t] * ReLU(q[h,t] . k[s]) (d = 128, FP8 q/k, one key per
 *         token shared by all heads), followed by an exact top-k;
 *   §5.1  the pool metadata (free bitmap, per-slot eviction priority, fixed-length result
 *         buffer, the two slot<->host maps with an infinity sentinel);
 *   §5.2  the in-graph allocate / free / recall operations, with the recall copying rows
 *         straight out of host memory from a GPU kernel;
 *   §6.1  threshold prefetch during scoring, made lossless by the guaranteed recall;
 *   §6.3  the indexer kernel whose threshold test feeds a queue that a copy stage in the same
 *         kernel drains from host memory.
 *
 * Conventions for every entry point
 *   - Pointers are DEVICE pointers unless marked [host].  The caller owns every buffer and
 *     stream; no entry point allocates device memory, frees it, or synchronises, except
 *     echo_recall in ECHO_RECALL_MEMCPY mode and the echo_graph_* / echo_host_* helpers,
 *     which say so.  Everything else only enqueues work on the given stream(s), so it can be
 *     captured into a hipGraph.
 *   - Streams are hipStream_t passed as void* (NULL = the null stream).
 *   - FP8 = OCP E4M3FN bytes.  H = 64 heads and D = 128 are fixed.
 *   - Return codes: ECHO_OK, or a negative ECHO_E* code when an argument is rejected on the
 *     host (nothing is enqueued then) or a launch fails; echo_last_error() gives the text
 *     (thread-local).  Failures that depend on device data (pool exhausted, bad host index,
 *     duplicate host index) never trap: they OR bits into the pool's device status word.
 *   - "inf" in the pool maps is INT32_MAX (ECHO_INF).
 */
#ifndef ECHO_H
#define ECHO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ECHO_H_INDEX 64
#define ECHO_D_INDEX 128
#define ECHO_ROW_ELEMS 576 /* MLA latent row: 512 compressed + 64 RoPE values (bf16 bits) */
#define ECHO_VALUE_ELEMS 512 /* its compressed values: what attention sums */
#define ECHO_INF 0x7FFFFFFF
#define ECHO_MAX_TOPK 4096
#define ECHO_FUSED_MAX_RANGE 8192      /* tokens per range of the fused prefetch, at most */
#define ECHO_FUSED_MAX_PER_RANGE 128   /* rows one range of the fused prefetch moves, at most */

/* Prefetch modes (echo_decode_args.prefetch). */
enum {
  ECHO_PREFETCH_OFF = 0,
  ECHO_PREFETCH_RANGED = 1, /* scoring split into n_chunks launches; each also gathers the
                               candidates of the range before it */
  ECHO_PREFETCH_FUSED = 2   /* one launch: scoring waves and a host-gather wave per workgroup
                               (echo_index_scores_fused) */
};

enum {
  ECHO_OK = 0,
  ECHO_EINVAL = -1,      /* bad argument or shape; nothing enqueued */
  ECHO_EUNSUPPORTED = -2,/* outside the supported range; nothing enqueued */
  ECHO_EHIP = -3,        /* a HIP call or kernel launch failed */
  ECHO_EWORKSPACE = -4   /* workspace smaller than the matching *_workspace_bytes() */
};

/* Sticky device status bits (pool->status). */
enum {
  ECHO_ST_EXHAUSTED = 1, /* the misses need more slots than free + evictable; pool untouched */
  ECHO_ST_BAD_HOST = 2,  /* a selected token maps to a host index outside [0, n_host); pool untouched */
  ECHO_ST_DUP_HOST = 4,  /* two selected misses share a host index (caller precondition broken);
                            pool state afterwards is unspecified */
  ECHO_ST_CACHE_FULL = 8,/* echo_decode_append: a request's key range is full; its token was not
                            appended */
  ECHO_ST_NO_PAGES = 16, /* echo_page_step: the step needs more pages than are free, or the stack of
                            free pages does not fit its pool; nothing was handed out */
  ECHO_ST_BAD_LEN = 32   /* echo_page_step: a negative length, one behind the page table's width, or
                            more new tokens than the maps hold; nothing was handed out */
};

/* Types of floating-point tensors. */
enum { ECHO_BF16 = 0, ECHO_FP16 = 1, ECHO_FP32 = 2 };

/* Norms of query and key heads (echo_qk_args). */
enum {
  ECHO_NORM_NONE = 0,
  ECHO_NORM_RMS = 1,   /* x / sqrt(mean(x^2) + eps) * weight + bias */
  ECHO_NORM_LAYER = 2  /* (x - mean) / sqrt(mean((x - mean)^2) + eps) * weight + bias */
};

/* Recall modes for echo_recall. */
enum {
  ECHO_RECALL_GATHER = 0, /* GPU kernel reads mapped pinned host memory; graph-capturable */
  ECHO_RECALL_MEMCPY = 1  /* host reads the miss list (synchronises the stream) and issues one
                             hipMemcpyAsync per row; NOT graph-capturable */
};

/*
 * GPU pool of one layer plus its host backup (§5.1).  All members are device pointers the
 * caller allocated; sizes: gpu_free/gpu_priority/gpu_to_host/indices_buf [n_gpu],
 * host_to_gpu [n_host], gpu_kv [n_gpu * 576], host_kv [n_host * 576], status [1].
 *   gpu_free      1 = slot free, 0 = occupied (GPUTokenFree)
 *   gpu_priority  eviction priority, lowest evicted first, -1 for a free slot (GPUTokenPriority)
 *   gpu_to_host   host index held by the slot, ECHO_INF when empty (GPUTokenToHost)
 *   host_to_gpu   slot holding the host index, ECHO_INF when not resident (HostTokenToGPU)
 *   indices_buf   fixed-length result list: slot given to the i-th miss, -1 after the last
 *                 (GPUIndicesBuffer); see echo_pool_lookup_alloc for how far it is written
 *   gpu_kv        latent rows of the slots, bf16 bits, 1152 bytes per row
 *   host_kv       the host backup: a DEVICE-ACCESSIBLE pointer to pinned, mapped host
 *                 memory (echo_host_alloc gives one), read by GPU kernels over the host link
 *   status        sticky ECHO_ST_* bits; cleared only by echo_pool_init / echo_status_clear
 */
typedef struct {
  int32_t n_gpu;
  int32_t n_host;
  uint8_t *gpu_free;
  int32_t *gpu_priority;
  int32_t *gpu_to_host;
  int32_t *host_to_gpu;
  int32_t *indices_buf;
  uint16_t *gpu_kv;
  const uint16_t *host_kv;
  int32_t *status;
} echo_pool;

/* Bytes of pool metadata: 4*n_host + 13*n_gpu (§5.1). */
size_t echo_pool_metadata_bytes(int32_t n_host, int32_t n_gpu);

/* Resets a pool to empty: free = 1, priority = -1, both maps = ECHO_INF, indices_buf = -1,
 * status = 0.  Rows are left as they are.  Enqueued on `stream`. */
int echo_pool_init(echo_pool *pool, void *stream);

/* Sets *status = 0 (enqueued). */
int echo_status_clear(int32_t *status, void *stream);

/*
 * Decode indexer scores (§2).  For every query (request) r in [0, n_q) and key s in
 * [0, key_len[r]):
 *     scores[r*ld + s] = sum_h w[r*64 + h] * ReLU(scale(s) * (q[r,h,:] . k[key_begin[r] + s, :]))
 * with scale(s) = k_scale[key_begin[r] + s] when k_scale != NULL, else 1 (k_scale dequantises
 * the FP8 key; the library applies it after the head sum, which is equal in exact arithmetic
 * because scale > 0).  Products are exact, sums are fp32.
 *   q        [n_q, 64, 128] FP8 bytes     w       [n_q, 64] fp32
 *   k        [n_k, 128] FP8 bytes, 128-byte rows; request r owns rows key_begin[r] .. +key_len[r]
 *   k_scale  [n_k] fp32 > 0, or NULL
 *   key_begin [n_q] int64, key_len [n_q] int32 (0 <= key_len[r] <= max_key_len)
 *   scores   [n_q, ld] fp32, ld >= max_key_len; entries s >= key_len[r] are not written.
 * Errors: EINVAL for n_q < 0, max_key_len < 0, ld < max_key_len or NULL pointers.
 * Device-side lengths above max_key_len are clamped to max_key_len (never read out of range).
 */
int echo_index_scores(const uint8_t *q, const float *w, const uint8_t *k, const float *k_scale,
                      const int64_t *key_begin, const int32_t *key_len, int32_t n_q,
                      int32_t max_key_len, float *scores, int64_t ld, void *stream);

/*
 * echo_index_scores over a paged key cache (§5.1: per-layer caches in fixed-size pages): the key
 * (and key scale) of token s of request r is row page_table[r * max_pages + s / page_size] *
 * page_size + s % page_size of k_pages (k_scale_pages; NULL = scale 1).  Same scores as
 * echo_index_scores over the same keys laid out contiguously.  page_size is a power of two in
 * [16, 65536]; max_pages * page_size >= max_key_len.  Errors as echo_index_scores, EINVAL for a
 * NULL page table or too few pages, EUNSUPPORTED for a bad page size.
 */
int echo_index_scores_paged(const uint8_t *q, const float *w, const uint8_t *k_pages,
                            const float *k_scale_pages, const int32_t *page_table,
                            int32_t page_size, int32_t max_pages, const int32_t *key_len,
                            int32_t n_q, int32_t max_key_len, float *scores, int64_t ld,
                            void *stream);

/*
 * echo_index_scores plus, in the same launch, the first radix pass of the exact top-k (§2):
 * hist[r*2048 + b] += the number of tokens s < key_len[r] of request r whose score's order key
 * has top 11 bits b, where the order key is ~key(score) and key(x) maps a float to uint32 in
 * increasing order (-0 counted as +0): bin 0 holds the highest scores.  hist [n_q, 2048] is
 * accumulated (zero it first).  The decode step's scoring launch is this one.  Errors as
 * echo_index_scores, and EINVAL for a NULL hist.
 */
int echo_index_scores_hist(const uint8_t *q, const float *w, const uint8_t *k,
                           const float *k_scale, const int64_t *key_begin, const int32_t *key_len,
                           int32_t n_q, int32_t max_key_len, float *scores, int64_t ld,
                           uint32_t *hist, void *stream);

/*
 * Threshold prefetch fused into scoring (§6.1).  Scores tokens [tok_lo, tok_hi) of every
 * request exactly as echo_index_scores does, and in addition lists scored tokens s with
 * score > theta[r] whose host index h = req_to_host[key_begin[r] + s] lies in [0, n_host) and is
 * not resident (host_to_gpu[h] == ECHO_INF) in this call's list cand[r*cap + j],
 * j < cand_cnt[r].  Every such token counts in the step-wide per-request counter total_cnt[r]
 * (the demand); listed tokens are bounded by cap_r = min(cap, ceil(key_len[r] / cap_div)) over
 * the step (the page's global prefetch counter, bounded in proportion to the context length).
 * Each workgroup (a run of at most 4096 tokens of one request) collects its qualifying tokens
 * (at most 1024 of them for listing; any further ones are counted only) and, at its end, adds
 * their number to total_cnt[r] and lists as many as cap_r still allows, reserving places in
 * the list with an atomic add on cand_cnt[r] and giving back those past the cap (so cand_cnt[r]
 * may run past the count while the call runs; after it, it is the number listed).  Which
 * qualifying tokens are listed, and in which order, depends on timing; the scores never do.  Because each call has its own list, a
 * consumer that waits for this call sees a complete list (echo_prefetch_gather).
 *   theta [n_q] fp32; req_to_host [n_k] int32; host_to_gpu [n_host]; cand [n_q, cap] int32;
 *   cand_cnt [n_q] (zeroed by the caller before this call); total_cnt [n_q] (zeroed once per
 *   step).
 */
int echo_index_scores_prefetch(const uint8_t *q, const float *w, const uint8_t *k,
                               const float *k_scale, const int64_t *key_begin,
                               const int32_t *key_len, int32_t n_q, int32_t max_key_len,
                               int32_t tok_lo, int32_t tok_hi, float *scores, int64_t ld,
                               const float *theta, const int32_t *req_to_host,
                               const int32_t *host_to_gpu, int32_t n_host, int32_t *cand,
                               int32_t *cand_cnt, int32_t *total_cnt, int32_t cap,
                               int32_t cap_div, void *stream);

/*
 * Scoring and threshold prefetch in one kernel (§6.3, with the §6.1 threshold and the §5.2
 * allocate and zero-copy row reads).  Scores every request exactly as echo_index_scores does
 * (same values), and moves rows of tokens scoring above theta[r] into free GPU slots while the
 * later keys are still being scored.
 *   Ranges.  Request r's tokens are cut into ranges of `range` tokens (one workgroup each;
 *   range = 0 picks one; else a multiple of 128 in [128, ECHO_FUSED_MAX_RANGE]).
 *   Which rows.  The tokens s with score > theta[r] (fp32, strict; NaN never passes) whose host
 *   index h = req_to_host[key_begin[r] + s] is in [0, n_host) and not resident
 *   (host_to_gpu[h] == ECHO_INF when the call starts) qualify.  Each range asks for places for
 *   its first ECHO_FUSED_MAX_PER_RANGE qualifying tokens in token order (its candidates).
 *   Cap and places.  Request r may move c_r = min(cap, ceil(key_len[r] / cap_div), n_gpu) rows,
 *   scaled to floor(c_r * F / C) when the caps add up to C > F, the pool's free slots at the
 *   start.  Those free slots, ascending, form a list; request r owns c_r entries of it, after
 *   those of requests < r.  Its ranges claim them first come, first served (one counter per
 *   request): min(#candidates, c_r) rows move, each range's a token-order prefix of its
 *   candidates in ascending slots, into the request's first entries.  So when a request's
 *   candidates fit its cap, all of them move; which of the request's slots each one gets
 *   depends on timing.
 *   Each moved token: free = 0, gpu_to_host = h, host_to_gpu[h] = slot, priority 0, and its
 *   row copied from host_kv.  Nothing is evicted; nothing moves when the status word is
 *   nonzero.
 *   Outputs: *n_prefetched = rows moved; *demand (or NULL) = qualifying tokens, before caps.
 *   Workspace: echo_fused_workspace_bytes(n_q, pool->n_gpu) bytes.  Host indices are unique
 *   across requests (caller precondition).
 * Errors: EINVAL for negative sizes, ld < max_key_len, cap < 0, cap_div < 1, NULL pointers or
 * an incomplete pool; EUNSUPPORTED for n_q > 65535, max_key_len or n_gpu above 2^22, or a bad
 * range; EWORKSPACE for a short workspace.
 */
size_t echo_fused_workspace_bytes(int32_t n_q, int32_t n_gpu);
int echo_index_scores_fused(const uint8_t *q, const float *w, const uint8_t *k,
                            const float *k_scale, const int64_t *key_begin,
                            const int32_t *key_len, int32_t n_q, int32_t max_key_len,
                            float *scores, int64_t ld, const float *theta,
                            const int32_t *req_to_host, const echo_pool *pool, int32_t cap,
                            int32_t cap_div, int32_t range, int32_t *n_prefetched,
                            int32_t *demand, void *ws, size_t ws_bytes, void *stream);

/*
 * Per-request prefetch threshold: theta[r] = the nearest-rank `percentile` of the scores of
 * request r at the n_sample positions floor(i * L_r / n_sample), i < n_sample, with
 * L_r = min(key_len[r], max_key_len) (the stand-in for the page's per-layer EMA prediction of
 * the k-th score, §6.1, on a single step with no history).  theta[r] = +inf when L_r <= 0.
 * n_sample must be a power of two in [64, 4096].  Computes the sampled scores itself from q, w,
 * k, k_scale (as echo_index_scores does).  Errors: EINVAL for negative n_q or max_key_len, a
 * percentile outside (0, 100] or NULL pointers; EUNSUPPORTED for n_sample outside the range or
 * n_q > 65535.
 */
int echo_prefetch_threshold(const uint8_t *q, const float *w, const uint8_t *k,
                            const float *k_scale, const int64_t *key_begin,
                            const int32_t *key_len, int32_t n_q, int32_t max_key_len,
                            int32_t n_sample, float percentile, float *theta, void *stream);

/*
 * Prefill (causal) indexer scores (§3.4: quadratic in the context).  Query rows t in
 * [0, n_q) sit at absolute positions q_pos0 + t and see keys s in [0, min(n_k, q_pos0+t+1)):
 *     scores[t*ld + s] = sum_h w[t*64+h] * ReLU(q[t,h,:] . k[s,:])
 *   q [n_q, 64, 128] FP8; w [n_q, 64] fp32; k [n_k, 128] FP8; scores [n_q, ld] fp32,
 *   ld >= n_k; entries past a row's causal length are not written.
 */
int echo_index_scores_prefill(const uint8_t *q, const float *w, const uint8_t *k, int32_t n_q,
                              int32_t n_k, int32_t q_pos0, float *scores, int64_t ld,
                              void *stream);

/*
 * Exact top-k per row (§2).  Row r holds len[r] scores at scores[r*ld ...].  Selects the
 * min(k, len[r]) highest scores; ties go to the lower index; -0.0 equals +0.0.  Writes
 * idx[r*k + j], the selected token indices in ascending order, -1 padded to k.
 * NaN scores are outside the contract.  1 <= k <= ECHO_MAX_TOPK.
 *   ws: device workspace of at least echo_topk_workspace_bytes(n_rows, max_len) bytes.
 * len[r] above max_len is clamped to max_len.
 */
size_t echo_topk_workspace_bytes(int32_t n_rows, int32_t max_len);
int echo_topk(const float *scores, int64_t ld, const int32_t *len, int32_t n_rows,
              int32_t max_len, int32_t k, int32_t *idx, void *ws, size_t ws_bytes,
              void *stream);

/*
 * Approximate top-k subset per row for the inter-query prefetch of a chunked prefill (§6.2).
 * Every score of row r (scores[r*ld + s], s < len[r]) is shifted, x = fl32(score - shift), and
 * mapped by the top 8 bits of its order key (sign-flipped, -0 as +0) to one of 256 bins.  The
 * highest bins whose total stays <= k are taken whole and the next bin down is the threshold
 * bin.  subset[r*k + j] lists the tokens of the taken bins in ascending order, -1 padded to k;
 * subset_cnt[r] is their number (<= k, and > k - the threshold bin's size when there is one);
 * thr_cnt[r] (optional) is the threshold bin's size (0 when every bin fits).  The subset lies
 * inside the row's exact top-k.  shift [1] is a device float, the prediction of the k-th score
 * (NULL or NaN = 0: no prediction yet).  len[r] above max_len is clamped; ld >= max_len.
 * 1 <= k <= ECHO_MAX_TOPK.  ECHO_EINVAL for negative sizes, ld < max_len or NULL pointers
 * (thr_cnt and shift may be NULL); ECHO_EUNSUPPORTED for k outside the range.
 */
int echo_topk_subset(const float *scores, int64_t ld, const int32_t *len, int32_t n_rows,
                     int32_t max_len, int32_t k, const float *shift, int32_t *subset,
                     int32_t *subset_cnt, int32_t *thr_cnt, void *stream);

/*
 * Union of index lists (§6.2: a query block's prefetch set is the union of its rows' subsets, and
 * its guaranteed recall covers the union of its rows' exact top-k).  Entries of idx [n_rows, k]
 * in [0, n_keys) are collected (others, -1 included, are ignored) and listed in ascending order
 * in segments of 4096 consecutive keys: out[s*4096 + j] for the union's keys in
 * [4096 s, 4096 s + 4096), -1 padded; out_cnt[s] their number; n_seg = ceil(n_keys / 4096)
 * (1 when n_keys = 0).  The segments are 4096-wide selection rows with key_begin 0 for
 * echo_pool_lookup_alloc (k = 4096) and candidate rows for echo_prefetch_gather (cap = 4096).
 * ws: echo_union_workspace_bytes(n_keys) bytes (a bitmap, cleared by the call).  ECHO_EINVAL
 * for negative sizes or NULL pointers, ECHO_EWORKSPACE for a short workspace,
 * ECHO_EUNSUPPORTED above 2^30 keys.
 */
size_t echo_union_workspace_bytes(int32_t n_keys);
int echo_union_rows(const int32_t *idx, int32_t n_rows, int32_t k, int32_t n_keys, int32_t *out,
                    int32_t *out_cnt, void *ws, size_t ws_bytes, void *stream);

/*
 * k-th score and its EMA (§6.1, §6.2): for each row r, kth[r] = the smallest score among the
 * selected tokens idx[r*k + j] >= 0 (NaN when there is none), and theta[r] = kth[r] if theta[r]
 * is NaN, else fmaf(alpha, theta[r], (1 - alpha) * kth[r]); a row with no selection keeps theta.
 * Either output may be NULL (not both).  0 <= alpha <= 1.
 */
int echo_threshold_ema(const float *scores, int64_t ld, const int32_t *idx, int32_t n_rows,
                       int32_t k, float alpha, float *theta, float *kth, void *stream);

/*
 * Residency lookup + eviction + allocation for the selected tokens (§5.2 free/allocate and
 * the lookup half of recall), without the row copy.  For the entries idx[r*k + j] >= 0 taken
 * in (r, j) order: h = req_to_host[key_begin[r] + idx]; hit iff host_to_gpu[h] != ECHO_INF.
 *   - every hit slot is protected for this call (a bitmap in the workspace);
 *   - need = max(0, n_miss - #free); the `need` unprotected occupied slots with the smallest
 *     (priority, slot index) are evicted: free = 1, priority = -1, both maps = ECHO_INF; their
 *     rows are not touched (the host holds the backup);
 *   - the i-th miss gets the i-th free slot in ascending slot order: free = 0, maps set,
 *     priority = step_id; miss_host[i] = h, miss_slot[i] = slot, indices_buf[i] = slot;
 *     miss_host/miss_slot entries past n_miss and indices_buf entries [n_miss,
 *     min(n_gpu, n_rows*k)) are -1;
 *   - every selected slot's priority = step_id; topk_slot[r*k + j] = its slot (-1 where
 *     idx is -1); *n_miss = number of misses.
 * req_to_host has n_k entries; a token index key_begin[r] + idx outside [0, n_k), a host index
 * outside [0, n_host) or a HostTokenToGPU entry outside [0, n_gpu) sets ECHO_ST_BAD_HOST.
 * On ECHO_ST_EXHAUSTED or ECHO_ST_BAD_HOST the pool is left untouched and topk_slot,
 * miss_*, n_miss are unspecified.  Rows of missed tokens still have to be copied by
 * echo_recall.  step_id must exceed every priority already in the pool for the policy to be
 * least-recently-selected-first (not checked).  1 <= k <= ECHO_MAX_TOPK; n_gpu <= 2^22.
 *   ws: device workspace of at least echo_pool_workspace_bytes(n_rows, k, pool->n_gpu).
 */
size_t echo_pool_workspace_bytes(int32_t n_rows, int32_t k, int32_t n_gpu);
int echo_pool_lookup_alloc(const echo_pool *pool, const int32_t *idx, const int64_t *key_begin,
                           const int32_t *req_to_host, int64_t n_k, int32_t n_rows, int32_t k,
                           int32_t step_id, int32_t *topk_slot, int32_t *miss_host,
                           int32_t *miss_slot, int32_t *n_miss, void *ws, size_t ws_bytes,
                           void *stream);

/*
 * echo_pool_lookup_alloc without a workspace argument, for callers that cannot allocate
 * (code under hipGraph capture, tight serving loops, harnesses that forbid hipMalloc).  Same
 * arguments, results and errors as echo_pool_lookup_alloc; its workspace is a fixed device array
 * of ECHO_STATIC_SCRATCH_BYTES inside the library, one per GPU, held until the process ends.
 * Sizes whose echo_pool_workspace_bytes(n_rows, k, pool->n_gpu) exceeds that are rejected with
 * ECHO_EUNSUPPORTED (nothing enqueued).  Allocates nothing; launch on a stream of the current
 * device.  Every call on one GPU shares that GPU's array: calls that overlap in time on one GPU
 * (other streams, other threads) race and give undefined results.  Each call clears what must
 * start at zero itself.
 */
#define ECHO_STATIC_SCRATCH_BYTES (16u << 20)
int echo_pool_lookup_alloc_static(const echo_pool *pool, const int32_t *idx,
                                  const int64_t *key_begin, const int32_t *req_to_host, int64_t n_k,
                                  int32_t n_rows, int32_t k, int32_t step_id, int32_t *topk_slot,
                                  int32_t *miss_host, int32_t *miss_slot, int32_t *n_miss,
                                  void *stream);

/*
 * Recall (§5.2): gpu_kv[miss_slot[i]] = host_kv[miss_host[i]] bitwise (1152 bytes) for
 * i < *n_miss (n_miss is read on the device; max_miss bounds it).
 *   ECHO_RECALL_GATHER: one kernel reads the rows straight from mapped pinned host memory.
 *   ECHO_RECALL_MEMCPY: synchronises `stream`, reads n_miss and the lists to the host and
 *     issues one hipMemcpyAsync (host -> device) per row on `stream`; returns after enqueueing.
 * Skipped entirely when the pool status word is nonzero.  ECHO_EINVAL for a pool with a
 * NULL gpu_kv, host_kv, host_to_gpu or status, or with n_gpu or n_host below 1.
 */
int echo_recall(const echo_pool *pool, const int32_t *miss_host, const int32_t *miss_slot,
                const int32_t *n_miss, int32_t max_miss, int32_t mode, void *stream);

/*
 * Prefetch side of the overlap (§6.1 with the §5.2 allocate and UVM copy).
 * echo_prefetch_begin lists the pool's free slots (in no particular order) into free_list
 * [n_gpu] and sets free_count[0] = their number, free_count[1] = 0 (taken so far).
 * echo_prefetch_gather takes the candidates of one echo_index_scores_prefetch call (cand,
 * cand_cnt), gives each a slot from free_list (counter free_count[1]; never evicts: candidates
 * beyond the free slots are dropped), sets both maps, gives the slot priority 0 (first to go
 * when space is short later), copies the row from host memory, and adds the number of rows it
 * moved to *n_prefetched.  Skipped when the pool status word is nonzero.  Both reject a pool
 * with NULL members it uses or n_gpu (n_host) below 1 with ECHO_EINVAL.
 */
int echo_prefetch_begin(const echo_pool *pool, int32_t *free_list, int32_t *free_count,
                        void *stream);
int echo_prefetch_gather(const echo_pool *pool, const int64_t *key_begin,
                         const int32_t *req_to_host, const int32_t *cand,
                         const int32_t *cand_cnt, int32_t n_q, int32_t cap,
                         const int32_t *free_list, int32_t *free_count, int32_t *n_prefetched,
                         void *stream);

/*
 * The whole decode step (§4): scores -> [threshold prefetch] -> exact top-k -> lookup /
 * evict / allocate -> recall -> priorities.  Pure enqueue on `main_stream`, so the call can be
 * captured into one hipGraph (echo_graph_capture_decode).  Work that overlaps the critical
 * path (the pool's priority histogram, prefetch gathers, reading missed rows from host memory
 * into a staging area of the workspace) rides along as extra workgroups of the same launches.
 * Prefetch (§6.1): ECHO_PREFETCH_RANGED scores in n_chunks launches, each of which also gathers
 * the candidates of the range before it (which candidates win the cap depends on timing);
 * ECHO_PREFETCH_FUSED scores in one launch with a host-gather wave per workgroup, with the
 * rows and slots of echo_index_scores_fused (§6.3).  Either way the
 * threshold is theta_ema when given, else the sample percentile, and the selection and the
 * selected rows are those of the step without prefetch.  With prefetch on, the rest of the
 * pool is not reproducible from run to run: which unselected candidates move, the free slot
 * each takes, and so the slots the guaranteed recall then finds free and the contents of
 * topk_slot / miss_slot / indices_buf, depend on the order in which workgroups finish.  The
 * pool invariants (maps a bijection, every resident row equal to its host row) always hold.
 * `side_stream` is reserved and ignored (pass NULL or main_stream).  Workspace:
 * echo_decode_workspace_bytes(a, pool->n_gpu) bytes (it includes n_rows * topk staged rows of
 * ECHO_ROW_ELEMS bf16 values).
 */
typedef struct {
  const uint8_t *q;          /* [n_rows, 64, 128] FP8 */
  const float *w;            /* [n_rows, 64] */
  const uint8_t *k;          /* [n_k, 128] FP8 */
  const float *k_scale;      /* [n_k] or NULL */
  const int64_t *key_begin;  /* [n_rows] */
  const int32_t *key_len;    /* [n_rows] */
  const int32_t *req_to_host;/* [n_k] host index of every cached token */
  int32_t n_rows;
  int32_t max_key_len;
  int32_t topk;
  int32_t step_id;
  /* prefetch: ECHO_PREFETCH_OFF, _RANGED or _FUSED */
  int32_t prefetch;
  int32_t n_chunks;          /* RANGED: scoring split into this many token ranges (1..16); ranges
                                0..c together list at most floor(cap_r (c+1) / n) of a request's
                                cap (a share left unused passes on), so the gathers spread over
                                the later launches */
  int32_t n_sample;          /* threshold sample size (power of two, 64..4096) */
  float percentile;          /* threshold percentile, e.g. 95 */
  int32_t cap;               /* per-request candidate cap bound */
  int32_t cap_div;           /* cap_r = min(cap, ceil(L_r / cap_div)) */
  /* EMA threshold (§6.1; off when theta_ema == NULL).  theta_ema [n_rows] is the caller's
     per-request estimate of the k-th largest score, kept from step to step.  With prefetch on
     it replaces the sample percentile as the threshold (NaN = no estimate yet: nothing is
     prefetched).  At the end of the step it is updated from this step's k-th score kth (the
     smallest selected score): theta = kth if theta is NaN, else
     fmaf(ema_alpha, theta, (1 - ema_alpha) * kth); a request with no selection keeps it. */
  float *theta_ema;
  float ema_alpha;           /* the page uses 0.5 */
  /* [1] or NULL: when given, the step stamp is read on the device from *step_dev instead of
     step_id, so that one captured graph can serve every step (echo_step_advance moves it on) */
  const int32_t *step_dev;
  /* Free slots the guaranteed recall leaves after its allocation, as room for the next step's
     prefetch (which only takes free slots): it evicts further down the same (priority, slot)
     order until reserve_free slots stay free, as far as unprotected slots allow.  0 = evict
     only what the misses need.  0 <= reserve_free <= n_gpu. */
  int32_t reserve_free;
  /* FUSED: tokens per range (0 = the library picks; else as echo_index_scores_fused) */
  int32_t pf_range;
  /* Paged indexer-K cache (§5.1: the caches are kept per layer in fixed-size pages; NULL = the
     contiguous layout).  With a page table, token s of request r has its key at row
     k_page_table[r * k_max_pages + s / k_page_size] * k_page_size + s % k_page_size of k (and
     k_scale); key_begin then only offsets req_to_host.  k_page_size is a power of two in
     [16, 65536], k_max_pages * k_page_size >= max_key_len.  Not with ECHO_PREFETCH_FUSED
     (EUNSUPPORTED). */
  const int32_t *k_page_table;
  int32_t k_page_size;
  int32_t k_max_pages;
} echo_decode_args;

typedef struct {             /* device outputs of one step */
  float *scores;             /* [n_rows, max_key_len] */
  int32_t *topk_idx;         /* [n_rows, topk] */
  int32_t *topk_slot;        /* [n_rows, topk] */
  int32_t *miss_host;        /* [n_rows * topk] */
  int32_t *miss_slot;        /* [n_rows * topk] */
  int32_t *counters;         /* [8]: 0 n_miss (guaranteed recall), 1 prefetch demand (tokens
                                above threshold and not resident, summed over requests),
                                2 rows prefetched, 3..7 reserved (zero) */
  float *kth;                /* [n_rows] or NULL: smallest selected score per request (the k-th
                                largest when key_len >= topk; NaN when nothing is selected) */
} echo_decode_out;

size_t echo_decode_workspace_bytes(const echo_decode_args *a, int32_t n_gpu);
int echo_decode_select(const echo_decode_args *a, const echo_pool *pool,
                       const echo_decode_out *out, void *ws, size_t ws_bytes, void *main_stream,
                       void *side_stream);

/*
 * One new token per request, before its query is scored (§2: a token's latent row is backed up
 * to host memory when it is generated, so eviction never moves data; §5.2: allocate serves
 * newly generated KV as well as recalled tokens).  For every request r with
 * p = key_len[r] < capacity and key_begin[r] + p < n_k:
 *   k[key_begin[r] + p] = new_k[r] (128 FP8 bytes); k_scale[...] = new_scale[r] when given;
 *   req_to_host[key_begin[r] + p] = new_host[r]; key_len[r] = p + 1 (on the device);
 *   host_kv_w[new_host[r]] = new_kv[r] (576 bf16 values written through the host link);
 * a request at capacity appends nothing and sets ECHO_ST_CACHE_FULL.  Then the appended tokens,
 * in request order, get GPU slots exactly as misses of echo_pool_lookup_alloc with k = 1
 * (nothing protected, eviction of the lowest (priority, slot) when no slot is free, priority
 * step_id), and their rows are copied from new_kv into those slots.  new_slot[r] receives the
 * slot (-1 for a request that appended nothing); it is unspecified when the pool status word
 * is nonzero afterwards.  new_host[r] must lie in [0, n_host), be distinct and not be resident
 * (ECHO_ST_BAD_HOST / ECHO_ST_DUP_HOST otherwise; the pool is then left untouched, the key
 * cache and host rows are still written).  Pure enqueue on `stream`; workspace:
 * echo_append_workspace_bytes(n_rows, pool->n_gpu).  Argument errors (nothing enqueued):
 * ECHO_EINVAL for NULL inputs, an incomplete pool, capacity or n_k below 1, or k_scale and
 * new_scale not both given or both NULL; ECHO_EUNSUPPORTED for n_rows outside [1, 65535] or more
 * than 2^22 GPU slots; ECHO_EWORKSPACE for a short workspace.
 */
typedef struct {
  int32_t n_rows;
  int32_t capacity;          /* key rows reserved per request (key_len never exceeds it) */
  int64_t n_k;               /* rows of k, k_scale and req_to_host */
  const uint8_t *new_k;      /* [n_rows, 128] FP8 */
  const float *new_scale;    /* [n_rows], or NULL when k_scale is NULL */
  const uint16_t *new_kv;    /* [n_rows, 576] bf16 bits, device memory */
  const int32_t *new_host;   /* [n_rows] host row of each new token */
  uint8_t *k;                /* [n_k, 128] the indexer K cache */
  float *k_scale;            /* [n_k] or NULL */
  const int64_t *key_begin;  /* [n_rows] */
  int32_t *key_len;          /* [n_rows], incremented */
  int32_t *req_to_host;      /* [n_k] */
  uint16_t *host_kv_w;       /* WRITABLE device-mapped pointer to the pool's host backup
                                (the same memory as echo_pool.host_kv) */
  int32_t step_id;
  const int32_t *step_dev;   /* [1] or NULL: the step stamp read on the device (as in
                                echo_decode_args) */
} echo_append_args;
size_t echo_append_workspace_bytes(int32_t n_rows, int32_t n_gpu);
int echo_decode_append(const echo_append_args *a, const echo_pool *pool, int32_t *new_slot,
                       void *ws, size_t ws_bytes, void *stream);

/* *step_dev += 1, enqueued on `stream` (one thread).  With the stamp on the device, a captured
 * sequence echo_step_advance -> echo_decode_append -> echo_decode_select is one whole decode
 * step that can be replayed for every step (the caller refreshes the step's query and new
 * tokens in the same device buffers between replays).  ECHO_EINVAL for NULL. */
int echo_step_advance(int32_t *step_dev, void *stream);

/* Graph helpers (host side; they create HIP objects).  Capture one echo_decode_select into a
 * hipGraph on `main_stream`, instantiate it, and replay it.  The graph
 * reads and writes the buffers that were passed at capture time. */
typedef struct echo_graph_s *echo_graph;
int echo_graph_capture_decode(const echo_decode_args *a, const echo_pool *pool,
                              const echo_decode_out *out, void *ws, size_t ws_bytes,
                              void *main_stream, void *side_stream, echo_graph *graph);
int echo_graph_launch(echo_graph graph, void *stream);
int echo_graph_destroy(echo_graph graph);

/* Capture of any sequence of echo_* calls enqueued on `stream` between the two calls (host side;
 * they create HIP objects): echo_graph_begin starts a stream capture, echo_graph_end ends it and
 * instantiates the graph (launch with echo_graph_launch, free with echo_graph_destroy).  Calls
 * that synchronise (echo_recall in ECHO_RECALL_MEMCPY mode) cannot be captured.  A failed
 * echo_graph_end leaves *graph NULL and the stream no longer capturing. */
int echo_graph_begin(void *stream);
int echo_graph_end(void *stream, echo_graph *graph);

/* Pinned, device-mapped host memory for the host backup (hipHostMalloc, mapped; coherent when
 * `coherent` != 0).  *host receives the host pointer, *dev the device-side pointer to pass as
 * echo_pool.host_kv.  Free with echo_host_free. */
int echo_host_alloc(size_t bytes, int coherent, void **host, void **dev);
int echo_host_free(void *host);

/*
 * What a step needs before its scores: the page maps of a paged key cache, the FP8 products that
 * give the indexer's queries and keys, and their norms, rotation and FP8 form.  In the order of a
 * step: echo_page_step, echo_quant_fp8 and echo_matmul_fp8 (projections), echo_indexer_qk,
 * echo_newest_queries, then echo_index_scores_paged.
 */

/*
 * Advances the page tables of n_rows requests by one step and maps its new tokens, from lengths
 * that are on the GPU.  Pages have page_size tokens (a power of two in [16, 65536]); free pages
 * are a stack, free_list[0 .. *count_in), its top at the end.
 *   1. A request r with done[r] != 0 (done may be NULL: none) gives back its ceil(len_in[r] /
 *      page_size) pages, pushed in (request, page) order, and its length becomes 0.  It may get
 *      new tokens in the same step: a row of the batch taken over by the next request.
 *   2. Each request gets the pages its new_len[r] further tokens need; the i-th new page of the
 *      step in (request, page) order is the i-th from the top of the stack and is entered into
 *      page_table[r].  len_out[r] = length + new_len[r]; *count_out = pages left.
 *   3. New token t of the step (requests in order) gets slot[t] = page * page_size + offset, its
 *      row of the paged cache; row[t] = r (row may be NULL); pos[t] = its position in the request.
 *      All three are -1 for t in [row_begin[n_rows], max_new).  row_begin[r] is request r's first
 *      new token.
 * len_out may be len_in and count_out may be count_in (a step in place); no other arrays may
 * overlap.  Entries of page_table that no page of step 2 takes, and the stack above *count_out
 * except for what step 1 pushed, are left as they were.  A step that cannot be done whole is not
 * done at all: ECHO_ST_NO_PAGES and/or ECHO_ST_BAD_LEN are ORed into *status, lengths and count
 * are copied through, row_begin is 0 and every map entry -1.  A step of no requests (n_rows = 0) copies
 * the count and sets row_begin[0] = 0, whatever max_new is.  The pages in the tables of the
 * requests and on the stack are the caller's: all distinct and in [0, n_pages).
 * Sizes: page_table [n_rows, max_pages], free_list [n_pages], row_begin [n_rows + 1], slot / row /
 * pos [max_new].  Workspace: echo_page_workspace_bytes; two steps that may run at the same time
 * (two graphs, two streams) need one each.  Pure enqueue.  ECHO_EINVAL for negative sizes, NULL
 * pointers and arrays or a workspace not aligned to their types (4 bytes), ECHO_EUNSUPPORTED for other
 * page sizes and for more than 65535 requests, ECHO_EWORKSPACE for a short workspace.  An array of no
 * entries may be NULL.
 */
typedef struct {
  int32_t n_rows;
  int32_t page_size;
  int32_t max_pages;         /* width of page_table */
  int32_t n_pages;           /* pages of the pool */
  int32_t max_new;           /* room of slot, row and pos */
  const int32_t *len_in;     /* [n_rows] */
  const int32_t *new_len;    /* [n_rows] */
  const uint8_t *done;       /* [n_rows] or NULL */
  int32_t *page_table;
  int32_t *free_list;
  const int32_t *count_in;   /* [1] */
  int32_t *len_out;          /* [n_rows] */
  int32_t *count_out;        /* [1] */
  int32_t *row_begin;
  int64_t *slot;
  int32_t *row;              /* or NULL */
  int32_t *pos;
  int32_t *status;           /* [1], sticky */
} echo_page_args;
size_t echo_page_workspace_bytes(int32_t n_rows, int32_t max_new);
int echo_page_step(const echo_page_args *a, void *ws, size_t ws_bytes, void *stream);

/*
 * FP8 codes of a matrix, with one scale per row and block of 128 columns (the last block may be
 * short): scale = max(largest |x| of the block / 448, 2^-126), y = the fp32 quotient x / scale rounded to
 * the nearest E4M3FN number (ties to even).  x has type x_type and row stride ldx, y row stride ldy (both in elements);
 * scale[r * scale_row + b * scale_blk].  What the codes of a block with a NaN or an infinity
 * stand for is NaN.  x and scale are aligned to their types, y to nothing; rows of x on 16 bytes
 * and of y on 8 are fastest.  ECHO_EINVAL for negative sizes, NULL pointers, an unknown type and
 * strides that make rows or scales overlap; ECHO_EUNSUPPORTED above 2^30 columns or from 2^30 blocks on.
 * No rows or columns: ECHO_OK.
 */
int echo_quant_fp8(const void *x, int32_t x_type, int64_t n_rows, int32_t n_cols, int64_t ldx, uint8_t *y,
                   int64_t ldy, float *scale, int64_t scale_row, int64_t scale_blk, void *stream);

/*
 * Product of two FP8 matrices with fp32 scales in blocks of 128:
 *   c[i][j] = sum over blocks t of a_scale(i, t) * b_scale(j / 128, t) *
 *             (sum over p in block t, p < k, of a[i][p] * b[j][p])
 * a [m, k] are activations with a scale per row and 128 columns, a_scale(i, t) =
 * a_scale[i * as_row + t * as_blk]; b [n, k] are weights with a scale per 128 rows and 128 columns,
 * b_scale[(j / 128) * bs_row + t * bs_blk].  The two scales are multiplied first, in fp32, so their
 * product has to be a normal fp32 number.  Sums are kept in fp32 and rounded once to c's type
 * c_type (ECHO_BF16, ECHO_FP16 or ECHO_FP32); c[i * ldc + j].  Products are exact for ECHO_FP32
 * and for few outputs (up to 32 rows, or at most 256 tiles of 32 x 32: echo_matmul_fp8_form says
 * "few"); other 16-bit results come from the FP8 matrix core, which cuts
 * each product at 2^-13 of the largest of its eight neighbours in k (about 1.6e-5 of a sum of
 * normally distributed terms, against the result's own 2^-9 or 2^-12).  The kernel and with it the order
 * of a sum go by m, n, k and the type, so a row's result may differ in its last bits with the number
 * of rows beside it; for the same sizes it is the same bits always: no atomics, no workspace.  a, b, lda
 * and ldb are multiples of 16 and every row, the last too, is readable up to k rounded up to 16; what
 * stands behind k is ignored.  c must not overlap an input.  m = 0 or n = 0: ECHO_OK; k = 0 writes zeros.
 * ECHO_EINVAL for negative
 * sizes, NULL pointers, an unknown type, lda or ldb below k, ldc below n, c not aligned to its type;
 * ECHO_EUNSUPPORTED for other alignments, lda, ldb or as_row above 2^22, negative scale strides, and
 * sizes beyond a launch (m or n above 2^26, 2^24 output tiles of 128 x 128).
 */
int echo_matmul_fp8(const uint8_t *a, int64_t lda, const float *a_scale, int64_t as_row, int64_t as_blk,
                    const uint8_t *b, int64_t ldb, const float *b_scale, int64_t bs_row, int64_t bs_blk, int32_t m,
                    int32_t n, int32_t k, void *c, int64_t ldc, int32_t c_type, void *stream);

/* The kernel that a product of these sizes takes, as text: "few ..." (exact for every type), "split ..."
 * or "tile ..." with the outputs of a workgroup; "" for no outputs.  For profiles and tests. */
const char *echo_matmul_fp8_form(int32_t m, int32_t n, int32_t k, int32_t c_type);

/*
 * Norms of n_q_heads query heads and n_k_heads key heads of n_tok tokens, and the rotation of
 * rot_dim values of each head from rot_begin on by the token's angles, in one pass.  Row pos[t] of
 * cos_sin [n_pos, rot_dim] holds the cosines of the rot_dim / 2 angles and then their sines.  The
 * pair of angle i is (rot_begin + i, rot_begin + rot_dim / 2 + i), or with interleaved != 0
 * (rot_begin + 2 i, rot_begin + 2 i + 1): (u, v) becomes (u cos - v sin, v cos + u sin).  Values
 * are computed in fp32 and rounded once.  q and k are [n_tok, heads, head_dim] of type `type`
 * with strides in elements; weights and biases are fp32 [head_dim] or NULL (1 and 0), not read
 * without a norm.  A token
 * whose pos is outside [0, n_pos) is padding: nothing of it is written.  head_dim is a multiple of 8
 * up to 256, rot_dim (0: none, cos_sin may be NULL) a multiple of 16, rot_begin of 8; pointers and
 * strides of q, k, cos_sin, weights and outputs are multiples of 16 bytes; anything else is
 * ECHO_EUNSUPPORTED, as are more than 2^31 - 2^16 query or key heads and more than a launch holds (2^26
 * waves: 2^30 heads of 72 to 128 values, twice as many of half that size, half as many of twice).
 * ECHO_EINVAL for negative sizes,
 * NULL pointers (where there is something to read or write), an unknown type or norm, a rotated part
 * behind the head's end, eps below 0 or NaN.
 */
typedef struct {
  int32_t n_tok, n_q_heads, n_k_heads, head_dim;
  int32_t type;
  int32_t q_norm, k_norm;    /* ECHO_NORM_* */
  int32_t rot_begin, rot_dim, interleaved, n_pos;
  float eps;
  const void *q, *k;
  int64_t q_tok_stride, q_head_stride, k_tok_stride, k_head_stride;
  const float *q_weight, *q_bias, *k_weight, *k_bias;
  const int32_t *pos;        /* [n_tok] */
  const float *cos_sin;
} echo_qk_args;

/* q_out and k_out have the inputs' type; each may be its input (same strides) but overlap nothing
 * else, nor may their heads overlap (ECHO_EINVAL). */
int echo_qk_norm_rope(const echo_qk_args *a, void *q_out, int64_t qo_tok_stride, int64_t qo_head_stride,
                      void *k_out, int64_t ko_tok_stride, int64_t ko_head_stride, void *stream);

/*
 * The same for the indexer (head_dim = 128, at most one key head), ending in what
 * echo_index_scores_paged reads: q8 [n_tok, n_q_heads, 128] FP8 queries, each head quantised with a
 * scale of its own as in echo_quant_fp8 and the scale folded into the head's weight, w_out[t][h] =
 * w[t][h] * scale(t, h) * w_mul (w has token stride w_tok_stride); and the token's key as FP8 row
 * k_cache[slot[t]] with k_scale[slot[t]].  A token whose slot is outside [0, n_slots) writes no key
 * (its query is written); the slots of a call are distinct.  q8 and k_cache are 8-byte aligned.
 */
int echo_indexer_qk(const echo_qk_args *a, const float *w, int64_t w_tok_stride, float w_mul, uint8_t *q8,
                    float *w_out, uint8_t *k_cache, float *k_scale, const int64_t *slot, int64_t n_slots,
                    void *stream);

/*
 * The queries to score after a step, one per request: where echo_page_step gave request r new tokens
 * (row_begin[r] < row_begin[r + 1]), its newest one's query and folded weights, rows
 * row_begin[r + 1] - 1 of q8 [n_tok, n_q_heads, 128] and w [n_tok, n_q_heads], go to rows r of q_out
 * and w_out, and len_out[r] = len[r], its keys.  A request without new tokens (padding, a finished one,
 * every one of a refused step) has no query: len_out[r] = 0 and its rows of q_out and w_out are left as
 * they were.  So is one whose rows are not within [0, n_tok].  Outputs overlap no input; q8 and q_out
 * are 8-byte aligned.  Pure enqueue; ECHO_EINVAL for negative sizes, NULL pointers and others not aligned
 * to their types, ECHO_EUNSUPPORTED for more than 65535 requests.
 */
int echo_newest_queries(const uint8_t *q8, const float *w, const int32_t *row_begin, const int32_t *len,
                        int32_t n_rows, int32_t n_tok, int32_t n_q_heads, uint8_t *q_out, float *w_out,
                        int32_t *len_out, void *stream);

/*
 * Behind the selection: attention over the latent rows that were selected, over blocks of a paged
 * cache or over a shared prefix, and the weight each token got there as the pool's eviction order.
 * A latent row (ECHO_ROW_ELEMS values) is one token's key for every head, its first ECHO_VALUE_ELEMS
 * values are the token's value.  In the order of a step: echo_decode_select (topk_slot, rows in
 * gpu_kv) or echo_topk / echo_block_topk (positions or blocks of a paged cache),
 * echo_sparse_attention, echo_attention_weights, echo_pool_weigh.
 */

/*
 * The k blocks of `block` consecutive tokens that each row's scores select: block b < ceil(len[r] /
 * block) scores the largest of scores[r * ld + t] over its tokens t < len[r]; the first n_first and the
 * last n_last blocks of the row score +infinity.  Then as echo_topk over the blocks: the highest k, ties
 * to the lower block, written to idx[r * k ..] in ascending order, -1 padded.  len[r] above max_len
 * is clamped, below 0 is 0.  NaN scores are outside the contract.  block is a power of two in [16, 65536],
 * 1 <= k <= ECHO_MAX_TOPK, ld >= max_len.  Workspace: echo_block_topk_workspace_bytes; calls that may run
 * at the same time need one each.  Pure enqueue.  ECHO_EINVAL for negative sizes, ld < max_len, NULL
 * pointers and arrays not aligned to their types; ECHO_EUNSUPPORTED for other blocks or k and for more than
 * a launch holds (2^22 rows, 2^26 waves of 1024 tokens or, where larger, a block); ECHO_EWORKSPACE.
 */
size_t echo_block_topk_workspace_bytes(int32_t n_rows, int32_t max_len, int32_t block);
int echo_block_topk(const float *scores, int64_t ld, const int32_t *len, int32_t n_rows, int32_t max_len, int32_t block,
                    int32_t n_first, int32_t n_last, int32_t k, int32_t *idx, void *ws, size_t ws_bytes, void *stream);

/*
 * Queries of n_rows tokens and the cache rows each of them attends to.  Row r lists entries idx[r *
 * idx_stride + i], i < k, each of them `block` (a power of two, 1 to 65536) consecutive positions
 * from entry * block on; a negative entry lists nothing, and an entry listed twice counts twice.  A position at or behind
 * len[r] (len may be NULL: none) is passed over.  Position p is row p of the cache, or, with page_size
 * != 0, row page_table[t * max_pages + p / page_size] * page_size + p % page_size with t = req[r] (req
 * may be NULL: r), page_size a power of two in [16, 65536].  A position whose page lies behind
 * max_pages, a t outside [0, n_tables) and a row outside [0, n_kv) are passed over too: nothing
 * outside the arrays is read, and nothing of a row that is passed over gets into a result, NaN or not.
 */
typedef struct {
  int32_t n_rows, n_heads;   /* up to 2^22 rows, 1024 heads */
  int32_t type;              /* ECHO_BF16 or ECHO_FP16: q, kv and the output */
  float scale;               /* of the scores; |scale| <= 1e38 */
  const void *q;             /* [n_rows, n_heads, 576], strides in elements */
  int64_t q_row_stride, q_head_stride;
  const void *kv;            /* [n_kv, 576] */
  int64_t kv_stride;
  int32_t n_kv;
  int32_t k, block;
  const int32_t *idx;
  int64_t idx_stride;
  const int32_t *len;        /* [n_rows] or NULL */
  const int32_t *page_table; /* [n_tables, max_pages], with page_size != 0 */
  int32_t page_size, max_pages, n_tables;
  const int32_t *req;        /* [n_rows] or NULL */
} echo_latent_args;

/*
 * out[r][h] = sum over row r's tokens t of p_t * kv[t][0 .. 512), p = softmax of the scores scale *
 * (q[r][h] . kv[t]); lse[r * n_heads + h] = log sum exp of the scores (natural, lse may be NULL).  A
 * row without a token gives zeros and -infinity.  Products are exact in fp32; scores, maxima and sums
 * are fp32; the weights are rounded to the type for the second product (half a step each), the result
 * once.  Scores behind fp32's range, and infinities or NaN in rows that are attended to, give what the formula gives
 * in fp32.  The same call gives the same bits always (no atomics); how a row's tokens are cut into
 * chunks, and with it the last bits, goes by n_rows, n_heads and k * block.  q, kv and out and their
 * strides are multiples of 16 bytes; out's heads overlap nothing.  Workspace:
 * echo_sparse_attention_workspace_bytes with n_tok = k * block (0 where no row is cut); calls that
 * may run at the same time need one each.  Pure enqueue.  ECHO_EINVAL for negative sizes, NULL
 * pointers, other types, overlapping heads of out, arrays not aligned to their types; ECHO_EUNSUPPORTED
 * for alignments, blocks, page sizes and sizes outside these limits (k * block up to 2^28, kv_stride up to 2^30, 2^23 workgroups);
 * ECHO_EWORKSPACE.  No rows or heads: ECHO_OK.
 */
size_t echo_sparse_attention_workspace_bytes(int32_t n_rows, int32_t n_heads, int32_t n_tok);
int echo_sparse_attention(const echo_latent_args *a, void *out, int64_t out_row_stride, int64_t out_head_stride, float *lse,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * Attention of a batch whose requests share prefixes: rows [group_begin[g], group_begin[g + 1]) attend
 * to the first prefix_len[g] positions of row g of prefix_table and then to the first own_len[r]
 * positions of row r of own_table, as one softmax; a row in no group has its own tokens only.
 * A prefix is read once for up to 64 heads of all the rows in its group.  Both tables go into the same cache, in
 * pages of page_size tokens.  group_begin is ascending in [0, n_rows] (other values: rows of
 * unspecified content, nothing read or written elsewhere).  Lengths above max_prefix and max_own are
 * clamped, below 0 are 0; what lies outside tables or cache is passed over, as above.  Results, errors,
 * alignments and workspace as echo_sparse_attention; ECHO_EUNSUPPORTED for more than 65536 groups too.
 */
typedef struct {
  int32_t n_rows, n_heads, type;
  float scale;
  const void *q;             /* [n_rows, n_heads, 576] */
  int64_t q_row_stride, q_head_stride;
  const void *kv;            /* [n_kv, 576] */
  int64_t kv_stride;
  int32_t n_kv, page_size;
  int32_t n_groups, max_prefix, prefix_pages, max_own, own_pages;
  const int32_t *group_begin;   /* [n_groups + 1] */
  const int32_t *prefix_len;    /* [n_groups] */
  const int32_t *prefix_table;  /* [n_groups, prefix_pages] */
  const int32_t *own_len;       /* [n_rows] */
  const int32_t *own_table;     /* [n_rows, own_pages] */
} echo_prefix_args;
size_t echo_prefix_attention_workspace_bytes(int32_t n_rows, int32_t n_heads, int32_t n_groups, int32_t max_prefix,
                                             int32_t max_own);
int echo_prefix_attention(const echo_prefix_args *a, void *out, int64_t out_row_stride, int64_t out_head_stride, float *lse,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * What each listed token got from all heads of its row in an attention that gave lse [n_rows, n_heads]:
 * w[r * w_stride + i] = sum over h of exp(scale * (q[r][h] . kv[t]) - lse[r][h]) for token i < k * block
 * of row r's list, 0 where a token is passed over.  fp32 throughout.  Limits and errors as
 * echo_sparse_attention, ECHO_EINVAL for no heads and for rows of w that overlap.
 */
int echo_attention_weights(const echo_latent_args *a, const float *lse, float *w, int64_t w_stride, void *stream);

/*
 * Eviction by accumulated attention weight.  mass [n_gpu] holds each pool slot's weight so far:
 *     mass[s] = decay * (fresh ? 0 : mass[s]) + the sum of w[i] over the entries with slot[i] = s,
 * where a slot is fresh if fresh [n_fresh] lists it (the step's miss_slot: it holds another token now), and
 * gpu_priority[s] = the bits of mass[s] as an integer, which keep its order, so that the pool step
 * (echo_pool_lookup_alloc, echo_decode_select) evicts the unprotected slots of the smallest
 * accumulated weight first, ties to the lower slot.  Free slots get mass 0 and priority -1.  Entries and
 * fresh slots outside [0, n_gpu) (-1: padding) are passed over.  A slot's weights are added up in
 * units of 2^-32, each clamped to [0, 1024] (NaN: 0), so their order does not matter, and a slot may be listed
 * any number of times; the sum is rounded to fp32 and added to the product in fp32.  A mass below 0 or
 * NaN counts as 0.  0 <= decay <= 1.  Up to 2^22 slots, 2^21 entries and 2^21 fresh slots
 * (ECHO_EUNSUPPORTED).  Workspace: echo_pool_weigh_workspace_bytes, 8-byte aligned; calls that
 * may run at the same time need one each.  Pure enqueue.  ECHO_EINVAL for negative sizes, NULL pointers,
 * decay outside its range, arrays not aligned to their types; ECHO_EWORKSPACE.  The arrays overlap nothing.
 */
size_t echo_pool_weigh_workspace_bytes(int32_t n_gpu);
int echo_pool_weigh(const uint8_t *gpu_free, int32_t *gpu_priority, float *mass, int32_t n_gpu, const int32_t *slot, const float *w,
                    int64_t n_entries, const int32_t *fresh, int64_t n_fresh, float decay, void *ws, size_t ws_bytes, void *stream);

/* Text of the last error on this thread ("" if none). */
const char *echo_last_error(void);

/* Library version string. */
const char *echo_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ECHO_H */
