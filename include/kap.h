/*
 * kap.h - C ABI of the selected-KV sparse decode hot path (GB300, sm_103a).
 *
 * The operations follow the runtime access plan A = (U, M, pos, rho_access, rho_verify) of
 * "KAP: Bridging the Knowledge Selection-Runtime Consumption Gap in LLM Systems" (the arXiv paper and
 * its agifrontier.github.io tutorial, section on the runtime access plan):
 *   U           - units: KV pages (16 tokens) or token spans,
 *   M           - page map: block table from logical page to physical page, plus lengths,
 *   pos         - logical positions, kept on both the proposal and the verification path,
 *   rho_access  - sparse-access policy: the A<a>R<r>K<k> split of the KRI page (knlp.io, "The A<a>R<r>K<k> tag"),
 *   rho_verify  - verification policy: the short causal query window of the full-context verifier.
 *
 * Conventions shared by every entry point
 *   - Every pointer argument named *_dev, and every pointer inside the structs below, is DEVICE memory owned by
 *     the caller. The library never allocates, frees or synchronises on these calls; all launches go to `stream`
 *     (NULL = the legacy default stream), so the calls that take their workspace from the caller can be captured
 *     in a CUDA graph.
 *   - KV pool layout: K and V are separate arrays [num_pages][num_kv_heads][16][head_dim] of the pool dtype.
 *     One (page, head) chunk is 16*head_dim*elem bytes and contiguous.
 *   - Query head hq reads KV head hq / (num_q_heads / num_kv_heads) (grouped-query attention).
 *   - Attention logits are (q . k) / sqrt(head_dim); lse is the natural-log log-sum-exp of those logits (fp32).
 *   - K in the pool is post-RoPE; queries passed to attention are post-RoPE at their logical positions.
 *   - Errors are returned as kap_status; nothing is thrown across the ABI. Host-side argument checks always run.
 *     Kernels that meet an inconsistent device-side value (a page id outside the pool, a selection larger than its
 *     capacity) skip that access and record a code readable with kap_device_error().
 */
#ifndef KAP_H
#define KAP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st *kap_stream; /* same type as cudaStream_t */

typedef enum {
  KAP_OK = 0,
  KAP_FALLBACK_FULL = 1,   /* plan infeasible for selected access: use full-context attention (KAP paper, fallback) */
  KAP_EINVAL = -1,         /* a NULL pointer, a negative size, or an out-of-range scalar */
  KAP_ESHAPE = -2,         /* shapes that are inconsistent with one another */
  KAP_ECAPACITY = -3,      /* a caller buffer (capacity, workspace) is too small */
  KAP_ECUDA = -4,          /* a CUDA runtime call failed; see kap_last_cuda_error() */
  KAP_EUNSUPPORTED = -5    /* a shape this build has no kernel for (head_dim, group size, dtype) */
} kap_status;

typedef enum { KAP_BF16 = 0, KAP_F32 = 1 } kap_dtype;

/* Paged KV pool. All pointers are device memory owned by the caller. */
typedef struct {
  int32_t num_pages;    /* physical pages in the pool */
  int32_t page_size;    /* tokens per page; must be 16 */
  int32_t num_kv_heads; /* Hkv */
  int32_t num_q_heads;  /* Hq, a multiple of Hkv; G = Hq / Hkv in 1..8 */
  int32_t head_dim;     /* d: 64 or 128 */
  int32_t dtype;        /* kap_dtype of K, V, queries and attention outputs */
  void *k_pages;        /* [num_pages][Hkv][16][d] post-RoPE keys */
  void *v_pages;        /* [num_pages][Hkv][16][d] values */
  float *k_summary;     /* [num_pages][Hkv][d] fp32 block-mean keys (K-summary cache); may be NULL if unused */
} kap_kv_pool;

/* A pool with packed pages beside its 16-bit ones. Physical page ids below pool.num_pages name 16-bit pages (bf16),
 * ids num_pages + j name packed page j, so one block table or view mixes both and every call that only moves ids
 * (views, slot mappings, kap_extend_tables) takes it as it is; pages are given back by kind (kap_release_tables_packed). A packed page holds K and V in 4 bits: for nb = head_dim / 64
 * blocks of 64 dims, the chunk of one (page, KV head) is
 *   K codes [nb][16 tokens][32 bytes], V codes alike, K params [nb][16][2] bf16, V params alike,
 * kap_packed_chunk_bytes(head_dim) = 1152 * nb bytes. Byte b of a token's block holds dim 2b in its low and dim 2b + 1
 * in its high four bits; params are (scale, lowest value) and code c stands for lowest + scale * c. */
typedef struct {
  kap_kv_pool pool;   /* the 16-bit pages; dtype must be KAP_BF16. k_summary, when given, has
                         num_pages + num_packed rows, one per physical page id */
  int32_t num_packed; /* packed pages (0 or more) */
  void *packed;       /* [num_packed][Hkv][kap_packed_chunk_bytes(head_dim)], 16-byte aligned */
} kap_packed_pool;

/* Page map M and lengths. Logical page j of request r covers positions 16j .. 16j+15. */
typedef struct {
  int32_t num_seqs;           /* R */
  int32_t max_pages;          /* row stride of block_table */
  const int32_t *block_table; /* [R][max_pages] physical page of each logical page */
  const int32_t *ctx_len;     /* [R] prompt tokens: positions < ctx_len are the selectable prompt */
  const int32_t *seq_len;     /* [R] tokens present (prompt + generated); a decode query sits at seq_len-1 */
} kap_page_map;

/* rho_access: the A<a>R<r>K<k> split. Prompt pages [0,a) and the last r prompt pages are pinned; k more pages
 * are chosen from the middle by score (ties to the lower page id). */
typedef struct {
  int32_t anchor, recent, topk;  /* a, r, k used for every request when per_seq_ark is NULL */
  int32_t per_kv_head;           /* 1: one selection per KV head; 0: one selection shared by all heads */
  int32_t cap;                   /* capacity of one selection row (entries) */
  const int32_t *per_seq_ark;    /* optional device [R][3] = (a, r, k) per request; overrides the scalars */
} kap_access_policy;

/* Compact selected-KV view, written by kap_compile_view and read by kap_attn_propose.
 * Row (r, v) with v < rows_per_seq lists the visible pages of request r for KV head v (or for all heads when
 * rows_per_seq == 1): first the n_selected selected prompt pages in ascending logical order (the order in which
 * they are accessed), then the tail pages holding positions >= ctx_len, up to the horizon given at compile time. */
typedef struct {
  int32_t rows_per_seq;   /* Hkv (per-head views) or 1 (one view shared by all heads) */
  int32_t cap;            /* entries per row */
  int32_t *block_table;   /* [R][rows_per_seq][cap] physical page of each entry */
  int32_t *logical_page;  /* [R][rows_per_seq][cap] logical page of each entry (keeps logical positions) */
  int32_t *n_entries;     /* [R][rows_per_seq] entries in use */
  int32_t *n_selected;    /* [R][rows_per_seq] leading entries that are selected prompt pages */
  /* Read by kap_attn_propose and kap_append_propose only; ignored (and left unchanged) by the calls that write a
   * view. Nonzero is the caller's promise that this view, the page map, the prompt tokens of the pool
   * (positions < ctx_len) and the rotary frequencies were last written before the kernel launched just ahead of
   * the call on the same stream. The call may then read them, and start streaming the selected prompt pages, while that kernel is
   * still finishing; it waits for it before reading anything else or writing anything. Zero: the call waits for
   * the previous kernel before its first memory access. The promise does not hold for a call that directly
   * follows the kernel that wrote the view. */
  int32_t settled;
} kap_view;

/* rho_verify: the verification window. Request r owns query rows q_offsets[r] .. q_offsets[r+1]-1; row i of
 * request r sits at logical position q_start_pos[r] + i and sees every position <= its own (full context,
 * causal among the candidates). */
typedef struct {
  int32_t max_q;              /* upper bound on q_offsets[r+1]-q_offsets[r]; G*max_q <= 64 */
  int32_t total_q;            /* q_offsets[R] */
  const int32_t *q_offsets;   /* [R+1] */
  const int32_t *q_start_pos; /* [R] */
} kap_verify_policy;

/* Requests that share a prefix: group g owns the requests group_offsets[g] .. group_offsets[g+1]-1, whose block_table
 * rows begin with the same prefix_pages[g] physical pages. group_offsets rises from 0 to num_seqs. */
typedef struct {
  int32_t num_groups;           /* 0: nothing is shared */
  const int32_t *group_offsets; /* [num_groups+1] */
  const int32_t *prefix_pages;  /* [num_groups] */
} kap_prefix_groups;

/* ---------------------------------------------------------------------------------------------------------
 * K-summary cache. EarlySelectKV page (routing over a K-summary cache) and the KRI page's KRI-Q row
 * (block-mean K). For every request r and prompt page j < ceil(ctx_len[r]/16), with n = min(16, ctx_len-16j)
 * valid tokens: k_summary[page][h][i] = (sum over t < n of K[page][h][t][i], fp32, t ascending) / n.
 * Requires pool->k_summary. Pages shared between requests must agree on n. */
kap_status kap_build_summaries(const kap_kv_pool *pool, const kap_page_map *map, kap_stream stream);

/* Refresh of the K summaries of listed pages: for each i < num_listed, the physical page pages_dev[i] with
 * n = n_valid_dev[i] valid tokens (1 <= n <= 16) gets k_summary[page][h][:] = (sum over t < n of K[page][h][t][:],
 * fp32, t ascending) / n, the same arithmetic as kap_build_summaries, so a refreshed page equals a full rebuild bit
 * for bit. EarlySelectKV page: routing scores pages against a K-summary cache held beside the KV pool; the page
 * does not say when that cache is updated. Here it changes only when committed tokens enter the prompt (ctx_len
 * grows): list the partial last prompt page and any new prompt pages; a full rebuild would re-read every prompt
 * page. Appends of generated tokens need no refresh, since summaries cover prompt tokens only. Listed pages must be
 * distinct (two CTAs would write one summary).
 *   pages_dev, n_valid_dev [num_listed] int32, device.
 * Errors: KAP_EINVAL for a null pointer or num_listed < 0; the pool checks of kap_build_summaries. A page outside the
 * pool or a count outside [1, 16] is skipped on the device and reported through kap_device_error. */
kap_status kap_refresh_summaries(const kap_kv_pool *pool, const int32_t *pages_dev, const int32_t *n_valid_dev,
                                 int32_t num_listed, kap_stream stream);

/* Page scoring and A/R/K top-K. KRI page (KRI-Q row; A<a>R<r>K<k> tag and its 128-block example) and
 * EarlySelectKV page (routing ranks pages by their K summaries, possibly against a proxy query).
 *   q_dev     [R][Hq][d] pool dtype: the routing query (the real query or a proxy).
 *   qbar[h]   = sum over g < G of q[h*G+g] (fp32, g ascending).
 *   score     = dot(qbar[h], k_summary[page][h]) in the fixed 32-lane order: lane l accumulates fmaf over
 *               i = l, l+32, ...; then lanes are combined by xor-butterfly 16, 8, 4, 2, 1 (a + b).
 *               Shared selection (per_kv_head = 0): score = sum over h ascending of the per-head scores.
 *   sel_ids   [R][rows][cap] out: selected prompt pages ascending; rows = Hkv or 1.
 *   n_sel     [R][rows] out: count = min(N, a + r + k) with N = ceil(ctx_len/16).
 *   workspace >= kap_score_workspace_size(...) bytes of device memory. On completion it holds the page scores,
 *             fp32 [R][rows][max_pages] from its first byte: entry (r, v, j) for j < N is the score above, entries
 *             at or past N are unspecified.
 * Errors: KAP_EINVAL for a null or misaligned pointer or a negative a, r or k; KAP_ECAPACITY for a workspace or a
 * cap too small; KAP_EUNSUPPORTED when R * rows > 65535 or the top-K row (4 bytes per page) exceeds 200 KiB. */
kap_status kap_score_topk(const kap_kv_pool *pool, const kap_page_map *map, const void *q_dev,
                          const kap_access_policy *policy, int32_t *sel_ids, int32_t *n_sel,
                          void *workspace, size_t workspace_bytes, kap_stream stream);
size_t kap_score_workspace_size(int32_t num_seqs, int32_t rows_per_seq, int32_t max_pages);

/* Page scoring, A/R/K top-K and view compilation in one call: the same outputs as kap_score_topk followed by
 * kap_compile_view(map, sel_ids, n_sel, rows, policy->cap, horizon_tokens, view, fallback_dev, s_max, slot_out,
 * pos_out), where rows = Hkv (per_kv_head) or 1. The top-K kernel compiles each row's view right after selecting
 * it, which saves the view kernel's launch and its reload of the selection. Needs map->seq_len; view->rows_per_seq
 * must equal rows and view->cap >= policy->cap + ceil(horizon_tokens/16) + 1. */
kap_status kap_score_topk_view(const kap_kv_pool *pool, const kap_page_map *map, const void *q_dev,
                               const kap_access_policy *policy, int32_t *sel_ids, int32_t *n_sel, void *workspace,
                               size_t workspace_bytes, int32_t horizon_tokens, const kap_view *view,
                               int32_t *fallback_dev, float s_max, int64_t *slot_out, int32_t *pos_out,
                               kap_stream stream);

/* External-prior selection. KRI page, prior schema and connector: a baked prior block_affinities[L][H][N] per
 * request prefix is mean-pooled across layers and heads and the top-K is taken per request (one selection row
 * shared by all heads), here under the A<a>R<r>K<k> split of `policy`, whose per_kv_head must be 0.
 *   affinities_dev [R][L][H][max_pages] fp32: the prior's block scores of each request; columns at or past
 *                  ceil(ctx_len/16) are ignored. L * H <= 2048.
 *   pooled score   = (sum over rows i = l*H + h, in chunks of 32 consecutive rows each summed from 0 with i
 *                    ascending, the chunk sums added in ascending order, all in fp32) / (L*H), one rounding.
 *                    The page states no order; this one is fixed so that selections reproduce bit for bit.
 *   sel_ids [R][1][policy->cap] out, ascending; n_sel [R][1] out (same rule and ties as kap_score_topk).
 *   workspace >= kap_score_workspace_size(R, 1, max_pages) bytes (the pooled scores).
 * Errors: KAP_EINVAL for a null pointer, L or H < 1, L*H > 2048 or per_kv_head != 0; KAP_ECAPACITY for a cap or
 * workspace that is too small. Follow with kap_compile_view (sel_rows_per_seq = 1) for the compact view. */
kap_status kap_prior_topk(const kap_page_map *map, const float *affinities_dev, int32_t num_layers,
                          int32_t num_heads, const kap_access_policy *policy, int32_t *sel_ids, int32_t *n_sel,
                          void *workspace, size_t workspace_bytes, kap_stream stream);

/* Materialised compact workspace. KAP paper, compiler (the selected spans are resolved to KV pages and materialised
 * as a compact physical view that keeps logical positions) and fallback (full-context access when the plan exceeds
 * the compact workspace). Request r owns the ws_pages_per_seq pool pages from ws_first_page + r * ws_pages_per_seq,
 * pages that no block table or view may reference otherwise (e.g. pages reserved at the end of the pool).
 * For every row (r, v) of `view`, selected entry i is copied to workspace page i of request r when all its tokens
 * are prompt tokens (16 * (logical page + 1) <= map->ctx_len[r]): K and V of head v for a per-head view
 * (rows_per_seq = Hkv), of every head for a shared view (rows_per_seq = 1). A selected page that also holds
 * positions >= ctx_len keeps its own page: generated tokens are written into it through the full table later.
 * out_view gets the row with the copied entries pointing at the workspace; tail entries, logical pages and counts
 * are copied unchanged. out_view may be `view` itself (rewritten in place); its cap >= view->cap.
 * A row whose n_selected exceeds ws_pages_per_seq is copied unchanged (attention over it stays correct, reading the
 * pool's own pages) and sets fallback_dev[r] = 1 when fallback_dev is given; the call never clears a flag.
 * Proposal attention over out_view equals attention over `view` bit for bit.
 * Errors: KAP_EINVAL for null pointers or sizes < 1; KAP_ESHAPE when rows_per_seq is neither 1 nor Hkv or the two
 * views differ in it; KAP_ECAPACITY when the workspace pages run past the pool or out_view->cap < view->cap. */
kap_status kap_materialize_view(const kap_kv_pool *pool, const kap_page_map *map, const kap_view *view,
                                int32_t ws_first_page, int32_t ws_pages_per_seq, const kap_view *out_view,
                                int32_t *fallback_dev, kap_stream stream);

/* Tolerant acceptance and commit of verify windows. KAP paper, verifier: the window is the verifier-approved carry
 * token followed by the k proposals; a proposal is accepted when it lies within the target's top-n candidates under
 * the full context (the Top-3 rule: top_n = 3; top_n = 1 is greedy exact match); m counts the proposals accepted
 * consecutively from the start; the same transition emits the next carry and advances the committed state.
 *   logits_dev         [total_rows][vocab] of logits_dtype (KAP_BF16 or KAP_F32): row j is the verifier's prediction
 *                      after window token j (the verify attention's window rows, through the model's head).
 *   window_offsets_dev [num_seqs+1] int32: request r owns rows [off[r], off[r+1]); every window holds 1 to 32 rows
 *                      and off[num_seqs] = total_rows (rows past 32 are not judged and set device error bit 4).
 *   tokens_dev         [total_rows] int32: the window's tokens; row off[r] is the carry, the rest are proposals.
 *   Rank order of a row: logit descending, lower token id first, NaN last. Proposal j passes when fewer than top_n
 *   tokens of row j - 1 come before it; a token outside [0, vocab) fails.
 *   accepted_out [num_seqs] = m; carry_out [num_seqs] = the first token of row m (the next carry);
 *   seq_len_out [num_seqs] (may be NULL, may alias a page map's seq_len) = start_pos[r] + 1 + m, the committed length:
 *   the carry at start_pos[r] and the accepted proposals after it, whose KV the window append already wrote.
 *   workspace >= kap_accept_workspace_size(num_seqs, total_rows, vocab) bytes, zeroed once before the first call
 *   (the call leaves its counters at zero).
 * Errors: KAP_EINVAL for null pointers, vocab or top_n < 1, total_rows < num_seqs; KAP_EUNSUPPORTED for another
 * dtype or more than 65535 rows; KAP_ECAPACITY for a small workspace. */
kap_status kap_accept_commit(const void *logits_dev, int32_t logits_dtype, int32_t vocab, int32_t num_seqs,
                             int32_t total_rows, const int32_t *window_offsets_dev, const int32_t *tokens_dev,
                             const int32_t *start_pos_dev, int32_t top_n, int32_t *accepted_out,
                             int32_t *carry_out, int32_t *seq_len_out, void *workspace, size_t workspace_bytes,
                             kap_stream stream);
size_t kap_accept_workspace_size(int32_t num_seqs, int32_t total_rows, int32_t vocab);

/* Span selection. KAP paper, compiler stage 3 (selected spans resolved to KV pages): a prompt page is kept when
 * any token of a selected span falls in it; pinned anchor/recent pages (policy a, r) are added. One row per
 * request (shared by all heads).
 *   spans_dev        [S][2] int32 (first token, length); span_offsets_dev [R+1] splits them by request.
 *   sel_ids          [R][1][policy->cap] out, ascending; n_sel [R][1] out. */
kap_status kap_select_spans(const kap_page_map *map, const int32_t *spans_dev, const int32_t *span_offsets_dev,
                            const kap_access_policy *policy, int32_t *sel_ids, int32_t *n_sel, kap_stream stream);

/* View compilation. KAP paper, compiler stage 3 and "selected-KV view" (selected pages compacted in access
 * order, logical positions preserved through block tables). For each row: entries 0..n_sel-1 are the selected
 * pages (block_table[i] = map->block_table[r][sel[i]], logical_page[i] = sel[i]); then tail pages: every page
 * j >= floor(ctx_len/16) with 16j < seq_len + horizon_tokens that is not already selected.
 *   sel_rows_per_seq/sel_cap give the layout of sel_ids; view->rows_per_seq must equal sel_rows_per_seq.
 *   fallback_dev     optional [R] out: 1 when request r's retained prompt fraction n_sel/N exceeds s_max,
 *                    else 0 (KAP paper, fallback: the plan keeps too large a share of the KV).
 *   slot_out/pos_out optional [R][horizon_tokens] out: the slot mapping of the tokens the cycle will append,
 *                    at positions seq_len[r] + i (same rule as kap_slot_mapping); NULL to skip.
 * Returns KAP_ECAPACITY when view->cap < sel_cap + ceil(horizon/16) + 1. */
kap_status kap_compile_view(const kap_page_map *map, const int32_t *sel_ids, const int32_t *n_sel,
                            int32_t sel_rows_per_seq, int32_t sel_cap, int32_t horizon_tokens,
                            const kap_view *view, int32_t *fallback_dev, float s_max, int64_t *slot_out,
                            int32_t *pos_out, kap_stream stream);

/* Slot mapping. KAP paper, selected-KV view (each newly scheduled token is sent to its physical KV slot).
 * Request r owns tokens tok_offsets[r] .. tok_offsets[r+1]-1; token j sits at pos = start_pos[r] + (j -
 * tok_offsets[r]) and slot = block_table[r][pos/16]*16 + pos%16 (-1 when the page is outside the table or
 * negative). Writes slot_out[j] and pos_out[j]. */
kap_status kap_slot_mapping(const kap_page_map *map, const int32_t *tok_offsets_dev, const int32_t *start_pos_dev,
                            int32_t num_tokens, int64_t *slot_out, int32_t *pos_out, kap_stream stream);

/* RoPE inverse frequencies. KAP paper, selected-KV view: the proposal and the verifier keep the same logical
 * positions, so every call that rotates (kap_append_kv, kap_append_propose) takes the one table this fills.
 * Writes inv_freq_host[i] = theta^(-2i/d) for 0 <= i < d/2, formed in double precision and rounded once to fp32,
 * into HOST memory of d/2 floats owned by the caller (who copies it to the device). No device work, no stream.
 * Returns KAP_EINVAL for a NULL pointer, d <= 0, odd d, or theta not finite and > 0. */
kap_status kap_rope_inv_freq(int32_t head_dim, double theta, float *inv_freq_host);

/* KV append with RoPE. KAP paper, executor (proposal KV written through the slot mapping; the verifier advances
 * the full-context KV state). For token t (0 <= t < T) with p = pos[t*tok_stride], s = slots[t*tok_stride]:
 * when s >= 0, K[s] = RoPE(k_new[t], p), V[s] = v_new[t] (fp32 math, round-to-nearest into the pool dtype);
 * when q_inout is not NULL, q_inout[t] = RoPE(q_inout[t], p) in place.
 * RoPE: pairs (i, i + d/2), angle = (float)p * inv_freq[i] (fp32), x' = x*cos - y*sin, y' = x*sin + y*cos.
 *   k_new, v_new [T][Hkv][d], q_inout [T][Hq][d] in the pool dtype; inv_freq_dev [d/2] fp32. */
kap_status kap_append_kv(const kap_kv_pool *pool, const void *k_new, const void *v_new, void *q_inout,
                         const int32_t *pos_dev, const int64_t *slots_dev, int32_t num_tokens, int32_t tok_stride,
                         const float *inv_freq_dev, kap_stream stream);

/* Which position axis turns each rotary pair: the table that kap_append_kv_norm takes for positions of several axes
 * (time, height and width of images and video). Pair i of d/2 gets axis_host[i] in [0, num_axes).
 *   interleaved 0: the first sections[0] pairs turn by axis 0, the next sections[1] by axis 1, and so on;
 *   interleaved 1: pair i turns by axis i % num_axes where that axis a > 0 has i < num_axes * sections[a], else by axis 0.
 * Writes HOST memory of d/2 entries owned by the caller. KAP_EINVAL for a NULL pointer, d <= 0 or odd, num_axes outside
 * 1..8, a negative section, sections that do not add up to d/2 or that the interleaving does not give. */
kap_status kap_rope_freq_axis(int32_t head_dim, const int32_t *sections_host, int32_t num_axes, int32_t interleaved,
                              int32_t *axis_host);

/* KV append of a model that normalises its queries and keys, or whose positions have several axes. The paper's models are
 * of both kinds (KAP paper, setup); its executor's append is otherwise that of kap_append_kv. For token t with
 * slot s = slots[t*tok_stride], all in fp32 with one rounding into the pool dtype at the end:
 *   y = x * (mean of x^2 over the head's d dims + eps)^(-1/2) * weight   (y = x where the weight is NULL)
 *   pairs (i, i + d/2) of y turn by pos[axis(i)*axis_stride + t*tok_stride] * inv_freq[i], axis(i) = freq_axis[i]
 *   (0 where freq_axis is NULL; a pair whose axis lies outside [0, num_axes) keeps its y)
 * for the rows of k_new into K[s] and of q into q_out; v_new goes to V[s] unchanged. With s < 0 the token's K and V are
 * not written (q_out is). The angle is not rounded to fp32 before its sine and cosine, as kap_append_kv and
 * kap_append_propose do: at position 131072 theirs may be off by 1/128 rad. The keys of one cache are to be written by
 * calls of one kind. The mean of squares is formed in fp32: it takes |x| up to 2^60.
 *   Rows: token t's heads start t*stride elements after the pointer and are contiguous [heads][d], so the parts of one
 *   fused projection are taken as they are. Pointers 16-byte aligned, strides multiples of 16 bytes and at least
 *   heads*d. q may be NULL (then q_out is not used); q_out may be q with the same stride (in place) and must not overlap an
 *   input otherwise. Slots >= 0 must be distinct.
 * Errors: KAP_EINVAL for null or misaligned pointers, sizes or strides out of range, eps < 0 or not finite, num_axes
 * outside 1..8. A slot past the pool is skipped and sets device error bit 1. */
typedef struct {
  const void *k_new, *v_new;  /* [T][Hkv][d] pool dtype */
  const void *q;              /* [T][Hq][d], or NULL */
  void *q_out;                /* [T][Hq][d] */
  int64_t k_stride, v_stride, q_stride, q_out_stride; /* elements between tokens */
  const float *q_weight, *k_weight; /* [d] fp32, or NULL: not normalised */
  float eps;
  int32_t num_axes;
  const int32_t *pos;         /* [num_axes][axis_stride] */
  int64_t axis_stride;
  const int32_t *freq_axis;   /* [d/2], or NULL */
  const int64_t *slots;
  const float *inv_freq;      /* [d/2] */
  int32_t num_tokens, tok_stride;
} kap_norm_append;
kap_status kap_append_kv_norm(const kap_kv_pool *pool, const kap_norm_append *args, kap_stream stream);

/* Selected-KV proposal attention, q = 1 per request. KAP paper, executor (proposal: a decode-like step with
 * q_prop = 1 over the compact view; only prompt-side KV is restricted) and EarlySelectKV (sparse attention with
 * the real query on precomputed page indices).
 * Query of request r, head hq sits at position P = seq_len[r]-1. A token at position p of view entry i is
 * visible when p <= P and (i < n_selected or p >= ctx_len).
 *   q_dev [R][Hq][d], out [R][Hq][d] (pool dtype), lse [R][Hq] fp32.
 *   workspace >= kap_propose_workspace_size(...) bytes, zero-filled once before first use (the kernels leave
 *   their counters at zero again on completion). */
kap_status kap_attn_propose(const kap_kv_pool *pool, const kap_page_map *map, const kap_view *view,
                            const void *q_dev, void *out, float *lse, void *workspace, size_t workspace_bytes,
                            kap_stream stream);
size_t kap_propose_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads, int32_t head_dim);

/* One proposal step with the step token's KV append fused in. KAP paper, executor (a proposal step writes its own
 * token's KV at that token's logical position through the view's slots and attends over the compact view).
 * Same pool, map, view, outputs and workspace as kap_attn_propose; in addition, for every request r:
 *   - the step token sits at position P = seq_len[r] - 1, which must lie on a page of the view (view compiled with
 *     a horizon that covers the step); a request whose P lies on no view page gets no append and sets device error
 *     bit 4;
 *   - k_new, v_new [R][Hkv][d] (pool dtype): the token's key before RoPE and its value. K = RoPE(k_new, P) and
 *     V = v_new are written into the pool at P's slot and take part in this step's attention;
 *   - q_dev [R][Hq][d] holds the step's queries BEFORE RoPE; they are rotated at P inside the call (the buffer is
 *     only read);
 *   - inv_freq_dev [d/2] fp32, as for kap_append_kv.
 * The result equals kap_append_kv at positions seq_len-1 (q rotated) followed by kap_attn_propose: the rotation
 * and its rounding into the pool dtype are the same. */
kap_status kap_append_propose(const kap_kv_pool *pool, const kap_page_map *map, const kap_view *view,
                              const void *q_dev, const void *k_new, const void *v_new, const float *inv_freq_dev,
                              void *out, float *lse, void *workspace, size_t workspace_bytes, kap_stream stream);

/* Full-context verification attention, q = n_q per request, causal among the candidates. KAP paper, verifier
 * (short contiguous query window over the full KV cache, full block table and original positions).
 *   q_dev [total_q][Hq][d], out [total_q][Hq][d] (pool dtype), lse [total_q][Hq] fp32.
 *   workspace >= kap_verify_workspace_size(...) bytes, zero-filled once before first use. */
kap_status kap_attn_verify(const kap_kv_pool *pool, const kap_page_map *map, const kap_verify_policy *vp,
                           const void *q_dev, void *out, float *lse, void *workspace, size_t workspace_bytes,
                           kap_stream stream);
size_t kap_verify_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads, int32_t head_dim,
                                 int32_t max_q);

/* Verification attention of requests that share prefixes: several questions on one document, or several answers to one
 * question (KAP paper: the knowledge that requests share is prompt KV). The same arguments, visibility and outputs as
 * kap_attn_verify (windows of one row are decode), over the whole table, but the pages that a group shares are read once
 * for all its requests, through the row of the group's first request. A group of one request, and a request whose
 * window starts inside its group's shared pages, are taken as sharing nothing. The results are those of kap_attn_verify
 * up to rounding: sums and statistics are fp32; over a bf16 pool probabilities enter the product with the values as bf16
 * (those of kap_attn_verify do so at head_dim 128; at 64 they stay in fp32 there).
 * A token that a row does not see adds nothing to it, whatever its K and V hold. A row that sees no token gets zeros
 * and lse -infinity; rows of q outside the windows (before q_offsets[0], from q_offsets[R] on) leave out and lse as they
 * are. Tokens on a page id outside the pool, or past the table's end, are skipped (device error bit 1).
 *   groups: see kap_prefix_groups; group_offsets that do not rise from 0 to num_seqs, q_offsets that do not rise within
 *   0 .. total_q, and a window on more than 32 pages set device error bit 4 (the results of the requests concerned are then
 *   undefined).
 *   workspace >= kap_shared_workspace_size(R, Hkv, Hq, d, total_q, num_groups) bytes, at any multiple of 16 bytes; it needs
 *   no clearing. Calls that may run at the same time, captured graphs among them, need a workspace each.
 *   total_q == 0: KAP_OK once sizes and groups are checked; outputs, queries, offsets and workspace are not looked at.
 * Errors: those of kap_attn_verify; KAP_EINVAL for num_groups < 0 or null group arrays; KAP_EUNSUPPORTED for more than 2^26
 * table columns, 2^20 groups or 2^31 - 1 query rows (total_q * Hq). */
kap_status kap_attn_verify_shared(const kap_kv_pool *pool, const kap_page_map *map, const kap_verify_policy *vp,
                                  const kap_prefix_groups *groups, const void *q_dev, void *out, float *lse,
                                  void *workspace, size_t workspace_bytes, kap_stream stream);
size_t kap_shared_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads, int32_t head_dim,
                                 int32_t total_q, int32_t num_groups);

/* Proposal attention without a caller workspace, for callers that cannot allocate device memory (a serving host
 * that fixes its device memory budget at start-up and owns the only allocator, a plug-in without access to that
 * allocator, or a loop where an allocation and its implicit device synchronisation are not allowed). The pages have
 * no counterpart to this call: it is a deployment variant of kap_attn_propose with identical arguments and results,
 * minus the workspace.
 *   - Scratch: a fixed array of kap_noalloc_scratch_bytes() = 16 MiB inside the library, present on every GPU that
 *     loads the library until the process exits. Shapes whose kap_propose_workspace_size exceeds it are rejected
 *     with KAP_ECAPACITY.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library routine. Each call clears the scratch's
 *     counters with cudaMemsetAsync on `stream`, then launches the same kernel as kap_attn_propose.
 *   - The first call on a device looks up the scratch's device address (cudaGetSymbolAddress) with that device
 *     current; make that first call before any stream capture. The address is kept for the life of the process:
 *     after a cudaDeviceReset of that device the library must not be called on it again in the same process.
 *   - A failed CUDA call (the address lookup, the clearing of the counters, the launch) returns KAP_ECUDA with its
 *     text in kap_last_cuda_error, as for every other call.
 *   - Every call on a device shares the one scratch array and it keeps the last call's contents: calls that overlap
 *     on the GPU (different streams, no ordering between them) race and give wrong results. */
kap_status kap_attn_propose_noalloc(const kap_kv_pool *pool, const kap_page_map *map, const kap_view *view,
                                    const void *q_dev, void *out, float *lse, kap_stream stream);
size_t kap_noalloc_scratch_bytes(void);

/* ---------------------------------------------------------------------------------------------------------
 * Packed pages. The pages describe caches of 16-bit keys and values only; what they do describe is that decode is bound
 * by the bytes of the KV it reads (KAP paper, cost model), which packing divides by 3.6.
 *
 * Packing: for each i < num_listed, 16-bit page src_pages_dev[i] becomes packed page dst_pages_dev[i] (both physical
 * ids, dst >= pool.num_pages). Every group of 64 dims of one token, KV head and tensor is coded by itself:
 *   lowest = min x;  scale = the least bf16 number that is not below (max x - min x) / 15;
 *   code = (x - lowest) / scale rounded to nearest, ties to even (0 when scale is 0),
 * decided exactly, with no rounding in between. A group that holds an infinity or a NaN reads back as NaN
 * throughout. All 16 token rows are packed, whatever the page's length. When k_summary is
 * given, the source page's summary is copied to the destination's row, so that routing scores stay as they were.
 * Unpacking: packed page src_pages_dev[i] to 16-bit page dst_pages_dev[i]: each element is lowest + scale * code in
 * fp32 (one rounding), then rounded to bf16; the summary is copied back.
 * Source and destination lists have num_listed int32 entries on the device; destinations must be distinct.
 * Errors: KAP_EINVAL for null or misaligned pointers or a negative count; KAP_EUNSUPPORTED for an fp32 pool. An id
 * outside its pool is skipped and sets device error bit 1. */
size_t kap_packed_chunk_bytes(int32_t head_dim);
kap_status kap_pack_pages(const kap_packed_pool *pool, const int32_t *src_pages_dev, const int32_t *dst_pages_dev,
                          int32_t num_listed, kap_stream stream);
kap_status kap_unpack_pages(const kap_packed_pool *pool, const int32_t *src_pages_dev, const int32_t *dst_pages_dev,
                            int32_t num_listed, kap_stream stream);

/* Attention over a pool with packed pages: kap_attn_propose and kap_attn_verify with the same arguments, visibility
 * rules and outputs, over pages of both kinds. Keys and values are those that the codes stand for (lowest + scale *
 * code, not rounded); sums and softmax statistics are fp32, probabilities enter the product with the values as fp16
 * (packed pages) or as two bf16 terms (16-bit pages). Probability times value scale keeps its 11 bits down to
 * 2^-15 of the largest scale met in a row's part (beside scales below 2^-20, 2^-40 of the largest 16-bit value counts as
 * one), and below that an error of 2^-25 of it. Sums are divided by the probabilities' sum at the end: 2^8 times a value
 * for each token has to fit fp32, so values of up to 2^96 in magnitude do at any length. The same goes for a logit's
 * sums, of lowest * sum q and of scale * sum q * code.
 * Every group size G in 1..8 is supported. kap_view.settled is not read. A hidden or skipped token adds nothing,
 * whatever its codes, parameters or 16-bit values hold. A query row that sees no token gets zeros and lse -infinity
 * (and, for the proposal, device error bit 4).
 *   workspace >= kap_packed_workspace_size(R, Hkv, Hq, d, max_q) bytes (max_q = 1 for the proposal), zero-filled once
 *   before first use; the kernels leave its counters at zero. Calls of other sizes may take the same workspace in turn
 *   if it is large enough for each. Calls that may run at the same time, captured graphs among them, need a workspace
 *   each. */
kap_status kap_attn_propose_packed(const kap_packed_pool *pool, const kap_page_map *map, const kap_view *view,
                                   const void *q_dev, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, kap_stream stream);
kap_status kap_attn_verify_packed(const kap_packed_pool *pool, const kap_page_map *map, const kap_verify_policy *vp,
                                  const void *q_dev, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  kap_stream stream);
size_t kap_packed_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads, int32_t head_dim,
                                 int32_t max_q);

/* Log probabilities of given tokens, beside the acceptance of verify windows: how sure the verifier is of each token,
 * which kap_accept_commit reduces to a yes or no. For each row of logits x over the vocabulary, in fp32:
 *   lse = log sum exp x;  logprob_out = x[token] - lse;  entropy_out = -sum p log p with p = exp(x - lse);
 *   rank_out = how many tokens come before the given one (kap_accept_commit's order: logit descending, lower token id
 *   first, NaN last);  top_ids, top_logprobs [rows][top_n] = the first top_n tokens of that order.
 * logits_dev [rows] rows of `vocab` values (KAP_BF16 or KAP_F32), row_stride elements apart, at any element alignment;
 * tokens_dev [rows] int32. entropy_out and rank_out may be NULL; top_ids and top_logprobs are used when top_n > 0.
 * A logit of -infinity has probability 0 and adds nothing. A row with a NaN or +infinity, or with -infinity
 * throughout, has no distribution: its log probabilities and entropy are NaN, ranks and ids hold. A token outside
 * [0, vocab) gets -infinity and rank vocab.
 *   workspace >= kap_logprobs_workspace_size(rows, vocab) bytes, zero-filled once before first use; the call leaves its
 *   counters at zero. Calls of other sizes may take the same workspace in turn if it is large enough for each; calls
 *   that may run at the same time need a workspace each.
 * Errors: KAP_EINVAL for null pointers, rows < 0, vocab < 1, row_stride < vocab, top_n outside [0, min(32, vocab)];
 * KAP_EUNSUPPORTED for another dtype or vocab > 2^24; KAP_ECAPACITY for a small workspace. */
kap_status kap_token_logprobs(const void *logits_dev, int32_t logits_dtype, int32_t vocab, int64_t row_stride,
                              int32_t rows, const int32_t *tokens_dev, int32_t top_n, float *logprob_out,
                              float *entropy_out, int32_t *rank_out, int32_t *top_ids, float *top_logprobs,
                              void *workspace, size_t workspace_bytes, kap_stream stream);
size_t kap_logprobs_workspace_size(int32_t rows, int32_t vocab);

/* Sampling of one token a row from given random numbers: the proposal's and the carry's tokens where decoding is not
 * greedy. Row r has logits x over the vocabulary, the largest m, and settings of its own, each optional (NULL: off):
 *   temperature  T (1 where NULL): weight w = exp((x - m) / T). T that is not above 0 takes the first token.
 *   top_k        keeps the first k of the rank order of kap_accept_commit (logit descending, lower id first); off when
 *                k < 1 or k is not below the number of tokens.
 *   min_p        keeps tokens with w >= min_p; off when not above 0.
 *   top_p        of the tokens that both keep, the shortest run of the rank order whose weight reaches top_p times their
 *                weight; off when not below 1. The first token is always kept.
 *   uniform      u in [0, 1): the token drawn is the first in id order at which the running sum of the kept weights passes
 *                u times their sum. Values outside [0, 1) are taken to its nearest end, NaN to 0.
 * tokens_out [rows]; logprob_out [rows] (may be NULL) = log of the drawn token's share of the kept weight; kept_out [rows]
 * (may be NULL) = how many tokens were kept. Weights are whole numbers of 2^-44 of the largest (fewer bits past 2^18
 * tokens), each right to 2^-37 of itself and a unit: one that rounds to nothing is never drawn. Sums are whole numbers, so a
 * row's result does not depend on the other rows, on their number or on the order of any addition. A logit of -infinity is
 * never kept. A row with a NaN or +infinity, or with -infinity throughout, has no distribution: it gets the first token of
 * the rank order, NaN and 0.
 *   logits_dev [rows] rows of `vocab` values (KAP_BF16 or KAP_F32), row_stride elements apart, at any element alignment;
 *   the others [rows] on the device, fp32 but for top_k (int32). No workspace.
 * Errors: KAP_EINVAL for null pointers, rows < 0, vocab < 1, row_stride < vocab; KAP_EUNSUPPORTED for another dtype,
 * vocab > 2^24 or rows > 2^26. */
kap_status kap_sample_tokens(const void *logits_dev, int32_t logits_dtype, int32_t vocab, int64_t row_stride, int32_t rows,
                             const float *uniform_dev, const float *temperature_dev, const int32_t *top_k_dev,
                             const float *top_p_dev, const float *min_p_dev, int32_t *tokens_out, float *logprob_out,
                             int32_t *kept_out, kap_stream stream);

/* Block tables and slot maps from request lengths. KAP paper, compiler and executor (block tables and slot mappings
 * are plan objects of fixed shape): the tables grow and the slots of a step are found on the device, from the lengths
 * and a stack of free pages (free_pages[0 .. free_count-1], its top last), without a copy to the host.
 *
 * kap_extend_tables: request r holds seq_len[r] tokens on the first ceil(seq_len / 16) entries of its block_table row
 * and takes new_tokens[r] more. Requests are served in order: with need[r] the new pages that r wants, r is granted
 * when need[r] is 0 or the needs of all requests up to and including r fit free_count. A granted request's new entries
 * are written, in page order, from the stack's top down; a request that wants a row longer than max_pages counts as
 * need 0, is not granted and sets device error bit 2.
 *   tok_offsets [R+1] = exclusive sums of new_tokens; token tok_offsets[r] + i sits at pos_out = seq_len[r] + i and, when
 *   r is granted, at slot_out = page * 16 + pos % 16 (-1 when not granted or when its page is negative). Tokens past
 *   max_tokens are not written (device error bit 2); entries of slot_out and pos_out past the last token are left as
 *   they are. seq_len_out[r] = seq_len[r] + new_tokens[r] when granted, else seq_len[r]; granted_out[r] = 1 or 0;
 *   free_count_out = free_count less the pages taken.
 * kap_release_tables: the pages of every request with released[r] != 0 (the first ceil(seq_len / 16) entries of its row)
 * are pushed on the stack in request and then page order; seq_len_out[r] = 0 for these and seq_len[r] for the others;
 * free_count_out = free_count plus the pages pushed. Pages past free_capacity are dropped (device error bit 2). The
 * rows themselves are left as they are. The ids are pushed as they stand, so this call is for tables whose pages are
 * all of one kind: new tokens are written to 16-bit pages, and a packed id on the stack would be granted for them.
 * kap_release_tables_packed: the same over a pool with packed pages. Ids below num_pages are pushed on free_pages, the
 * num_packed ids after them on free_packed (physical ids, as kap_pack_pages takes its destinations), each stack in
 * request and then page order, with a count and a capacity of its own; any other id is dropped (device error bit 1).
 * Output arrays must not alias the inputs (seq_len_out, free_count_out, packed_count_out), nor the stacks and counts of
 * the two kinds one another. A negative length or count counts as 0 and a
 * free_count past free_capacity as free_capacity (device error bits 4 and 2). All arrays are int32 on the device,
 * slot_out is int64. Errors: KAP_EINVAL for null pointers, num_seqs or max_pages < 1, negative capacities or page counts,
 * or aliased outputs. */
kap_status kap_extend_tables(int32_t num_seqs, int32_t max_pages, int32_t *block_table, const int32_t *seq_len,
                             const int32_t *new_tokens, const int32_t *free_pages, int32_t free_capacity,
                             const int32_t *free_count, int32_t *free_count_out, int32_t *tok_offsets,
                             int64_t *slot_out, int32_t *pos_out, int32_t max_tokens, int32_t *seq_len_out,
                             int32_t *granted_out, kap_stream stream);
kap_status kap_release_tables(int32_t num_seqs, int32_t max_pages, const int32_t *block_table,
                              const int32_t *seq_len, const int32_t *released, int32_t *free_pages,
                              int32_t free_capacity, const int32_t *free_count, int32_t *free_count_out,
                              int32_t *seq_len_out, kap_stream stream);
kap_status kap_release_tables_packed(int32_t num_seqs, int32_t max_pages, const int32_t *block_table,
                                     const int32_t *seq_len, const int32_t *released, int32_t num_pages,
                                     int32_t *free_pages, int32_t free_capacity, const int32_t *free_count,
                                     int32_t *free_count_out, int32_t num_packed, int32_t *free_packed,
                                     int32_t packed_capacity, const int32_t *packed_count, int32_t *packed_count_out,
                                     int32_t *seq_len_out, kap_stream stream);

/* Check of the bounded waits. Every wait of a kernel on an mbarrier (a copy landing, a slot freed, an MMA done)
 * gives up after at most about a second, sets bit 8 of the device error word and lets the kernel return, so that a
 * lost arrival cannot hang the GPU. This call runs the same bounded wait, on a barrier that nothing completes and
 * with nothing in flight, for `polls` polls of at most `suspend_ns` each (1 <= polls <= 1024,
 * 1 <= suspend_ns <= 2^20), and writes 1 to *timed_out_dev (device int32) when the wait gave up, 0 otherwise. The
 * pages have no counterpart: this is a diagnostic of the library. KAP_EINVAL for out-of-range arguments. */
kap_status kap_selftest_wait_timeout(uint32_t polls, uint32_t suspend_ns, int32_t *timed_out_dev, kap_stream stream);

/* Diagnostics. */
const char *kap_status_str(kap_status s);
const char *kap_last_cuda_error(void);   /* text of the last CUDA error seen by this thread, "" if none */
/* Reads (with a device synchronisation) and clears the device-side error word of the current device.
 * 0 = no error; otherwise a bit set: 1 page id out of the pool, 2 selection over capacity, 4 bad page length,
 * 8 a bounded wait in a kernel ran out. */
kap_status kap_device_error(int32_t *code_out);

#ifdef __cplusplus
}
#endif
#endif /* KAP_H */
