/*
 * oscar.h -- C ABI of the OSCAR mixed-precision INT2 KV-cache decode library
 * (CUDA, sm_103a).
 *
 * What it implements. OSCAR keeps each request's KV cache as one token pool
 * in three regions, "BF16 sink (64 tokens) | INT2 history | BF16 recent (256
 * tokens)" (news article "超越 TurboQuant，显存压力终于得到缓解！Together AI
 * 最新论文 OSCAR…", section "OSCAR 的设计思路"; MarkTechPost article "Together AI
 * 开源 OSCAR：一种用于长上下文 LLM 服务的注意力感知 2 位 KV 缓存量化系统",
 * section "服务系统：混合精度缓存布局"). History tokens are rotated by
 * R = U H_Had P_br (U from the attention-aware covariances C_Q and C_S,
 * H_Had the Walsh-Hadamard matrix, P_br bit reversal; MarkTechPost article,
 * "OSCAR 有何不同做法"), clipped to per-channel thresholds, quantised to
 * per-token asymmetric INT2 over 64-channel groups and packed 4 codes per
 * byte. Decode attention runs separately over the BF16 and INT2 segments and
 * merges them with an online-softmax (log-sum-exp) merge.
 *
 * Conventions for every call:
 *  - Return value: OSCAR_OK (0) or a negative OSCAR_ERR_* code. Nothing traps
 *    or aborts. Argument errors are detected on the host before any launch.
 *  - Memory: every device buffer is allocated and owned by the caller and
 *    must stay alive until the work enqueued on `stream` has finished. The
 *    library never allocates device memory; it carves the pool and workspace
 *    buffers handed to oscar_cache_create. Host pointers are read before the
 *    call returns.
 *  - Streams: `stream` is a cudaStream_t passed as void*; NULL is the legacy
 *    default stream. All device work of a call is enqueued on that stream, in
 *    order; calls never synchronise except oscar_get_status and
 *    oscar_profile_read.
 *  - Device-side errors (a page id outside the pool, a sequence longer than its
 *    page table allows) set bits in a device status word and the affected
 *    work is skipped; oscar_get_status reports them.
 *  - Threading: a cache handle may be used from one host thread at a time.
 *  - Fixed shape support: head_dim 128, group 64, page_size 64; sink and
 *    recent multiples of page_size; num_q_heads / num_kv_heads in {1,2,4,8}.
 *    Other values return OSCAR_ERR_UNSUPPORTED.
 *
 * Data layouts (all little-endian, row-major, no padding unless stated):
 *  - Per-request page tables are int32 device arrays owned by the caller:
 *      hist_pt [B][max_hist_pages]  INT2 page id of history page i
 *      bf16_pt [B][(sink+recent)/page_size]  BF16 page ids: the sink pages,
 *              then the recent ring pages
 *    Placement of position pos of a request with length L:
 *      pos < sink                        -> bf16_pt[pos / P], row pos % P
 *      pos >= max(sink, L - recent)      -> slot = (pos - sink) % recent,
 *                                           bf16_pt[sink/P + slot/P], row slot % P
 *      otherwise (history)               -> h = pos - sink,
 *                                           hist_pt[h / P], row h % P
 *    Requests may share sink and history pages (prefix caching); recent pages
 *    must be private to one request.
 *  - INT2 page block, one per (page, kv head), 5120 bytes in the default
 *    OSCAR_META_F16 format (the compact OSCAR_META_U8 format is described with
 *    its define below):
 *      [0, 2048)    K codes, row t at 32 t: channel j in byte j/4, bits 2(j%4)
 *      [2048, 4096) V codes, channel-major: channel c's 64 codes in the 16 bytes
 *                   at 2048 + 16 (c ^ ((c >> 4) & 7)); row t in their 32-bit word
 *                   (t >> 1) & 3 at bit 16 (t & 1) + 4 (t >> 4) + 2 ((t >> 3) & 1)
 *      [4096, 4608) K metadata, row t at 4096 + 8 t: fp16 scale0, zero0,
 *                   scale1, zero1 (group g = channels 64g..64g+63)
 *      [4608, 5120) V metadata, same layout
 *    Dequantised value of channel j: zero_g + scale_g * code_j, in the rotated
 *    basis x R.
 *  - BF16 page block, one per (page, kv head), 32768 bytes: K [64][128] bf16
 *    then V [64][128] bf16.
 *  - Per layer, the pool holds the INT2 blocks [num_int2_pages][Hkv], the
 *    BF16 blocks [num_bf16_pages][Hkv] and the rotation parameters; offsets
 *    come from oscar_layer_offsets.
 */
#ifndef OSCAR_H
#define OSCAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes -------------------------------------------------------- */
#define OSCAR_OK                 0
#define OSCAR_ERR_INVALID_ARG   (-1)  /* bad pointer, size, index or layout   */
#define OSCAR_ERR_UNSUPPORTED   (-2)  /* valid but not implemented shape      */
#define OSCAR_ERR_CUDA          (-3)  /* a CUDA runtime call failed           */
#define OSCAR_ERR_DEVICE_STATUS (-4)  /* device status word has error bits    */
#define OSCAR_ERR_TIMEOUT       (-5)  /* a bounded device wait gave up        */
#define OSCAR_ERR_NOT_ORTHOGONAL (-6) /* rotation rejected: max|U^T U - I| > 1e-3 */

/* bits of the device status word (oscar_get_status) */
#define OSCAR_STATUS_BAD_PAGE    1    /* a page id outside [0, pages)         */
#define OSCAR_STATUS_BAD_SEQLEN  2    /* seq_len < 1 or beyond its page table */
#define OSCAR_STATUS_TIMEOUT     4    /* a bounded wait expired               */
#define OSCAR_STATUS_NONFINITE   8    /* a NaN or infinity in an input q, k or v row (or in a
                                         rotated row the writers quantise); the row is still
                                         written: NaN and infinities are clipped like any value */
#define OSCAR_STATUS_SATURATED  16    /* an fp16 scale, range or zero of a history group fell
                                         outside +-65504 and was stored saturated (fp16 and
                                         codebook metadata formats; clip thresholds that keep
                                         every group inside +-65504 rule it out) */

#define OSCAR_STATUS_NO_PAGES   32    /* a free ring holds fewer pages than oscar_build_tables
                                         needs: nothing was changed                          */
#define OSCAR_STATUS_BAD_TREE   64    /* a draft's parent, node index or node count out of range */

/* V handling (MarkTechPost article, "服务系统：混合精度缓存布局": R_V may be
 * absorbed offline into the value/output projections). */
#define OSCAR_V_ABSORBED 0   /* caller's V is already v R_V; output is o R_V  */
#define OSCAR_V_EXPLICIT 1   /* V is raw; write path rotates history V and the
                                merge applies R_V^T to the INT2 partial       */

#define OSCAR_OUT_BF16 0
#define OSCAR_OUT_FP32 1

#define OSCAR_KIND_K 0
#define OSCAR_KIND_V 1

/* decode kernel choice (oscar_set_decode_algo) */
#define OSCAR_DECODE_SIMT 0  /* CUDA-core INT2 decode                          */
#define OSCAR_DECODE_MMA  1  /* tensor-core (mma.sync) INT2 decode             */
#define OSCAR_DECODE_TC   2  /* 5th-generation tensor-core (tcgen05, TMEM) INT2
                                decode: fp16 metadata and up to 4 query heads
                                per kv head; other layouts run OSCAR_DECODE_MMA */

/* INT2 group metadata format (oscar_layout.meta_format). The pages budget the
 * history at 2.25 bits per element (news article "超越 TurboQuant…", section
 * "精度表现": rotation baselines at about 2.25 BPE; 2 bits per code plus 16
 * bits per group of 64) without fixing how the 16 bits are split.
 *  OSCAR_META_F16: per (row, group) an fp16 scale and an fp16 zero (32 bits:
 *    2.5 bits per element, 5120-byte page blocks). The default.
 *  OSCAR_META_U8: per (row, group) two bytes mn8, mx8 (16 bits: 2.25 bits per
 *    element, 4608-byte page blocks): the clipped group's minimum and maximum
 *    rounded down / up to a grid of 255 steps over [-T, T], T the group's
 *    largest clip threshold. With D = fl32(2T / 255) and E = fl32(D / 3),
 *    zero' = fma(mn8, D, -T) and scale' = (mx8 - mn8) * E (float32); codes are
 *    round-to-nearest-even((y - zero') / scale') clamped to [0, 3], 0 where
 *    scale' = 0. Block layout: K codes [0, 2048), V codes [2048, 4096), K
 *    metadata [4096, 4352) at 4 bytes per row (mn8, mx8 of group 0, then of
 *    group 1), V metadata [4352, 4608). */
#define OSCAR_META_F16 0
#define OSCAR_META_U8  1
/* OSCAR_META_CB: the Lloyd-Max codebook variant (news article "超越 TurboQuant…",
 * section "总结与展望": the latest code adds a Lloyd-Max codebook to the
 * attention-aware rotation). The 2-bit code indexes a codebook of 4 levels
 * c_i = k_i / 255 (bytes 0 <= k_0 <= k_1 <= k_2 <= k_3 <= 255, one codebook
 * per (layer, kv head, K / V), set by oscar_set_codebook) on each group's
 * normalised range. Per (row, group) the metadata are fp16 range' =
 * fp16(max - min) and zero' = fp16(min) (RNE, saturating), in the bytes and
 * the 5120-byte block layout of OSCAR_META_F16 (range' in the scale slot).
 * Encoding in float32: t = (y - zero') / range', theta_i = (k_i + k_{i+1}) /
 * 510, code = number of i with t > theta_i (0 where range' = 0). Dequantised
 * value: zero' + range' * k_code / 255. (0, 85, 170, 255) gives the uniform
 * levels. */
#define OSCAR_META_CB  2

typedef struct oscar_layout {
  int num_layers;      /* >= 1                                                */
  int num_kv_heads;    /* Hkv >= 1                                            */
  int num_q_heads;     /* Hq, a multiple of Hkv, Hq/Hkv in {1,2,4,8}          */
  int head_dim;        /* 128                                                 */
  int group;           /* channels per quantisation group, 64                 */
  int page_size;       /* tokens per page, 64                                 */
  int sink;            /* S0, BF16 sink tokens, multiple of page_size (64)    */
  int recent;          /* W, BF16 recent ring, multiple of page_size (256)    */
  int num_int2_pages;  /* INT2 page capacity per layer                        */
  int num_bf16_pages;  /* BF16 page capacity per layer                        */
  int v_mode;          /* OSCAR_V_ABSORBED or OSCAR_V_EXPLICIT                */
  int max_batch;       /* largest B any call will pass                        */
  int max_splits;      /* largest number of history splits per (request, kv head) */
  int meta_format;     /* OSCAR_META_F16 (0) or OSCAR_META_U8 (1), see below   */
} oscar_layout;

typedef struct oscar_cache oscar_cache;

/* Bytes the caller must allocate (device memory, 256-byte aligned) for the
 * pool and the workspace of a layout. Either output pointer may be NULL. */
int oscar_cache_bytes(const oscar_layout* layout, size_t* pool_bytes, size_t* workspace_bytes);

/* Validate `layout` and bind the caller's pool and workspace (device
 * pointers, 256-byte aligned, sizes from oscar_cache_bytes). Allocates only the
 * host-side handle. The pool is not cleared. Errors: INVALID_ARG,
 * UNSUPPORTED, CUDA (device query failed). */
int oscar_cache_create(const oscar_layout* layout, void* pool, void* workspace, oscar_cache** out);

/* Free the host-side handle (not the caller's device buffers). NULL is a no-op. */
int oscar_cache_destroy(oscar_cache* cache);

/* Byte offsets, inside the pool buffer, of a layer's INT2 blocks, BF16 blocks
 * and rotation parameters. */
int oscar_layer_offsets(const oscar_cache* cache, int layer, size_t* int2_off, size_t* bf16_off,
                        size_t* params_off);

/* Load a layer's rotation and clip parameters (MarkTechPost article, "OSCAR
 * 有何不同做法": R_K = U_Q H_Had P_br, R_V = U_S H_Had P_br; "服务系统：混合精度
 * 缓存布局": clipping to calibration-derived percentile thresholds).
 *  U_K, U_V : host float32 [Hkv][128][128], row-major; column c is the c-th
 *             eigenvector (descending eigenvalue). R = U H P_br is applied as
 *             x -> x R to row vectors; H and P_br are never stored.
 *  tau_K, tau_V : host float32 [Hkv][128], clip thresholds in the rotated basis.
 *  U_V may be NULL in V-absorbed mode (then it is not used).
 * Each U is checked on the host: max|U^T U - I| > 1e-3 returns
 * OSCAR_ERR_NOT_ORTHOGONAL and nothing is copied. The copy is enqueued on
 * `stream`. */
int oscar_set_rotation(oscar_cache* cache, int layer, const float* U_K, const float* U_V,
                       const float* tau_K, const float* tau_V, void* stream);

/* Load a layer's codebooks (OSCAR_META_CB layouts; see OSCAR_META_CB).
 *  cb_K, cb_V : host uint8 [Hkv][4], each codebook non-decreasing.
 * oscar_set_rotation resets both to the uniform (0, 85, 170, 255), so call this
 * after it. Errors: INVALID_ARG (null pointer, bad layer, a decreasing
 * codebook), UNSUPPORTED (the layout is not OSCAR_META_CB), CUDA. The copy is
 * enqueued on `stream`. */
int oscar_set_codebook(oscar_cache* cache, int layer, const uint8_t* cb_K, const uint8_t* cb_V, void* stream);

/* Lloyd-Max calibration of one codebook on the host (news article "超越
 * TurboQuant…", section "总结与展望"): from rotated float32 calibration rows
 * x_rot [N][128] (host), clipped to tau [128], every 64-channel group with
 * max > min contributes its values normalised to u = (y - min) / (max - min).
 * Lloyd's iteration from the levels (0, 1/3, 2/3, 1): thresholds at the
 * midpoints, each level the mean of its cell (u <= t_0, t_0 < u <= t_1, ...;
 * an empty cell keeps its level), until no level moves by more than 1e-12 or
 * 1000 iterations; then cb[i] = rint(255 level_i) clamped and sorted.
 * Errors: INVALID_ARG (null pointer, N < 1). */
int oscar_calibrate_codebook(const float* x_rot, int N, const float* tau, uint8_t* cb);

/* Bulk write of B requests' prompt tokens (MarkTechPost article, "服务系统：
 * 混合精度缓存布局", write path: rotate, clip, quantise, pack).
 *  k, v        : device bf16 [total_tokens][Hkv][128], requests concatenated
 *  cu_seqlens  : device int32 [B+1], cu_seqlens[0] = 0, cu_seqlens[B] = total_tokens
 *  total_tokens: host copy of cu_seqlens[B]
 * Request r's token i sits at position i; its final length is
 * L_r = cu_seqlens[r+1] - cu_seqlens[r], which decides sink / history / recent
 * placement as above. In V-absorbed mode V is quantised without rotation. */
int oscar_quantize_prefill(oscar_cache* cache, int layer, int B, const void* k, const void* v,
                           const int32_t* cu_seqlens, int total_tokens, const int32_t* hist_pt,
                           int max_hist_pages, const int32_t* bf16_pt, void* stream);

/* Rows [tokens][heads][128] with free strides (elements, multiples of 8), the channels of a head contiguous; 16-byte
 * aligned. */
typedef struct oscar_heads {
  const void* ptr;
  int64_t token, head;
} oscar_heads;

/* Causal attention of B whole prompts over themselves: token i of a prompt attends to its tokens 0 .. i, in the caller's
 * q, k and v (nothing of the pool is read or written: store the prompt with oscar_quantize_prefill).
 *  q          : bf16 [total_tokens] rows of Hq heads; k, v: of Hkv heads; query head i reads kv head i / (Hq / Hkv)
 *  cu_seqlens : device int32 [B+1], as for oscar_quantize_prefill; tokens before cu_seqlens[0] and from cu_seqlens[B] on
 *               belong to no prompt, and their rows of out and lse stay as they are
 *  out        : device [total_tokens][Hq][128], bf16 or fp32 (out_dtype), 16-byte aligned
 *  lse        : device float32 [total_tokens][Hq] natural-log sum of exp(sm_scale q.k), or NULL; NaN where a logit is NaN or
 *               +infinity
 * Logits, softmax statistics and sums are float32; weights are rounded once to bf16 (2^-8 at most) for the product with
 * v, and the tensor cores' sums truncate (a few 1e-5 of the values' mean at 32K tokens, about 1e-3 at 256K): an fp32 out
 * carries that error too. Bounds out of order or outside [0, total_tokens] are taken within them (BAD_SEQLEN), and rows of
 * such prompts may be left unwritten. A NaN or infinity in k or v reaches no rows but those that attend to it, one in v
 * their results in its own channel alone and no lse, one in q no row but its own; a row of out that is not finite raises
 * NONFINITE. All inputs may come from the kernel just before; calls may overlap. Errors: INVALID_ARG (B or total_tokens < 0,
 * null pointers, strides that are not positive multiples of 8, alignment, out_dtype, sm_scale), UNSUPPORTED (more than
 * 2^31 - 1 tiles, or than 2^24 prompts times kv heads), CUDA. */
int oscar_prompt_attention(oscar_cache* cache, int B, const oscar_heads* q, const oscar_heads* k, const oscar_heads* v,
                           const int32_t* cu_seqlens, int total_tokens, float sm_scale, void* out, int out_dtype,
                           float* lse, void* stream);

/* The same bulk write from the prompt's hidden states, fused with the K and V
 * projections (MarkTechPost article, "服务系统：混合精度缓存布局": the write path
 * runs fused, so K and V are never written out and read back):
 *   K = bf16(x W_k^T), V = bf16(x W_v^T), rounded to nearest even,
 * then placed and quantised exactly as oscar_quantize_prefill does with those K
 * and V.
 *  x        : device bf16 [total_tokens][d_model], requests concatenated as in
 *             cu_seqlens (row-major, 16-byte aligned)
 *  w_k, w_v : device bf16 [Hkv * 128][d_model] (a linear layer's weight: output
 *             row j is kv head j / 128, channel j % 128), 16-byte aligned
 *  d_model  : a multiple of 64
 * The products accumulate in float32 on the tensor cores, then round to bf16.
 * Errors: INVALID_ARG (as oscar_quantize_prefill, d_model <= 0, a pointer not
 * 16-byte aligned), UNSUPPORTED (d_model not a multiple of 64, an odd Hkv,
 * B > 4096), CUDA. */
int oscar_project_quantize_prefill(oscar_cache* cache, int layer, int B, const void* x, int d_model,
                                   const void* w_k, const void* w_v, const int32_t* cu_seqlens,
                                   int total_tokens, const int32_t* hist_pt, int max_hist_pages,
                                   const int32_t* bf16_pt, void* stream);

/* Append one token per request at position seq_lens_before[r] (news article,
 * "OSCAR 的设计思路": a new token enters the recent window; the oldest recent
 * token is rotated / clipped / quantised / packed into the INT2 history).
 *  k, v            : device bf16 [B][Hkv][128]
 *  seq_lens_before : device int32 [B], lengths before this token
 * If seq_lens_before[r] >= sink + recent, the token at position
 * seq_lens_before[r] - recent is demoted to history slot
 * seq_lens_before[r] - recent - sink before its ring slot is overwritten.
 * As in oscar_decode_step, seq_lens_before, the page tables and the pool's
 * rows are read before the wait for the kernel launched just before; only
 * k and v may come from a kernel of the caller's launched just before. */
int oscar_append_kv(oscar_cache* cache, int layer, int B, const void* k, const void* v,
                    const int32_t* seq_lens_before, const int32_t* hist_pt, int max_hist_pages,
                    const int32_t* bf16_pt, void* stream);

/* Decode attention for one query token per request (news article, "OSCAR 的设计
 * 思路": BF16 segment and INT2 segment computed separately, combined by an
 * online-softmax merge).
 *  q        : device bf16 [B][Hq][128], 16-byte aligned; query head i reads kv head i/(Hq/Hkv)
 *  seq_lens : device int32 [B], lengths including the current token (>= 1)
 *  sm_scale : softmax scale (1/sqrt(128) for standard attention)
 *  out      : device [B][Hq][128], bf16 or fp32 per out_dtype. In V-absorbed
 *             mode the output is in the rotated value basis (o R_V).
 *  lse      : device float32 [B][Hq] natural-log sum of exp(sm_scale q.k), or NULL
 * History logits use the rotated query q R_K against the dequantised keys,
 * equal to attending with inverse-rotated keys because R_K is orthogonal. */
int oscar_decode_attention(oscar_cache* cache, int layer, int B, const void* q, const int32_t* seq_lens,
                           const int32_t* hist_pt, int max_hist_pages, const int32_t* bf16_pt,
                           float sm_scale, void* out, int out_dtype, float* lse, void* stream);

/* One decode step of a layer: oscar_append_kv(k, v at position
 * seq_lens_before[r]) followed by oscar_decode_attention(q) over
 * seq_lens_before[r] + 1 tokens, with the same arguments, layouts and
 * results as those two calls, issued as one chain of three launches, each a
 * programmatic dependent of the one before it: one step prologue (per
 * request, kv head and K / V: the demoted row, and for K the query rows, are
 * rotated together on the tensor cores; the demoted row is quantised into
 * the history, the queries become the decode's fragments, the new token goes
 * to its ring slot), the decode kernel and the merge. The decode kernel
 * prefetches history pages the append cannot touch before it waits.
 * Ordering: only q, k and v may be produced by the kernel launched just
 * before this call. The prologue is a programmatic dependent of that kernel:
 * it reads seq_lens_before, the page tables and the pool's BF16 rows before
 * it waits for it. These inputs must be complete when that kernel starts
 * (host copies, or any earlier kernel). Straight after a call of this library
 * that writes page tables or pool rows (the prefills, oscar_build_tables,
 * oscar_commit_draft) on the same stream, also in one capture, the prologue
 * is launched without that overlap, and all of it is seen. */
int oscar_decode_step(oscar_cache* cache, int layer, int B, const void* q, const void* k, const void* v,
                      const int32_t* seq_lens_before, const int32_t* hist_pt, int max_hist_pages,
                      const int32_t* bf16_pt, float sm_scale, void* out, int out_dtype, float* lse, void* stream);

/* Shared-prefix variants (MarkTechPost article "Together AI 开源 OSCAR…",
 * section "服务系统：混合精度缓存布局": the pool stays compatible with paged
 * KV and prefix caching). The caller states that history pages
 * [0, shared_hist_pages) of every request are the same pages: the entries
 * hist_pt[r][0 .. shared_hist_pages) are equal for all r, and every request
 * holds at least that many history pages. The result is the same as the
 * call without the suffix.
 *
 * On the tensor-core path one extra kernel then reads each shared page once
 * per step for all B x Hq / Hkv queries of its kv head, in CTAs of 128 query
 * rows. Each page is expanded once into shared memory and both products run
 * as 128-row tensor-core tiles. The per-request kernel covers only each
 * request's own pages. The CUDA-core path ignores shared_hist_pages.
 *
 * With oscar_decode_step_shared, the token each step demotes must land in
 * the request's own pages, so every request's history must already extend
 * past the shared pages. Error behaviour is as in the plain calls, and
 * 0 <= shared_hist_pages <= max_hist_pages is checked on the host. */
int oscar_decode_attention_shared(oscar_cache* cache, int layer, int B, const void* q, const int32_t* seq_lens,
                                  const int32_t* hist_pt, int max_hist_pages, int shared_hist_pages,
                                  const int32_t* bf16_pt, float sm_scale, void* out, int out_dtype, float* lse,
                                  void* stream);
int oscar_decode_step_shared(oscar_cache* cache, int layer, int B, const void* q, const void* k, const void* v,
                             const int32_t* seq_lens_before, const int32_t* hist_pt, int max_hist_pages,
                             int shared_hist_pages, const int32_t* bf16_pt, float sm_scale, void* out, int out_dtype,
                             float* lse, void* stream);

/* ---- verifying drafted tokens --------------------------------------------- */

/* The steps of a speculative decoder's verify call, all on the device and capturable into a CUDA graph:
 * oscar_tree_layout turns the draft's tree into masks and positions, oscar_rope rotates q and k by them and
 * oscar_tree_attention attends from every drafted node over the cache and the node's drafted ancestors. Drafted tokens
 * are not in the cache and need no pages. Once the accepted counts are known, oscar_build_tables gives the requests
 * the pages of their new lengths and oscar_commit_draft moves the accepted path into the cache. */

#define OSCAR_MAX_DRAFT  256   /* largest T, drafted nodes of a request            */
#define OSCAR_MAX_TABLE_BATCH 4096   /* largest B of oscar_build_tables            */

/* Page tables and token slots of requests that go from old_lens[r] to new_lens[r] tokens. old_lens are the lengths that
 * the last call left: pages once taken go back only when the request is released, and a call that starts from less
 * takes new ones for entries that are filled, whose old pages are then lost to the rings.
 *  old_lens, new_lens : device int32 [B]. new >= old >= 0 grows the request, new = 0 < old releases it.
 *  hist_pt, bf16_pt   : the page tables, as everywhere. Entries of pages that the new length adds are written,
 *                       those of a released request become -1, all others stay.
 *  free_int2, free_bf16 : device int32 [num_int2_pages], [num_bf16_pages]: rings of free page ids
 *  rings_in, rings_out  : device int32 [4]: head and count of the INT2 ring, head and count of the BF16 ring
 *                       (entries head .. head + count - 1 modulo the ring's size are free). Pages are taken at
 *                       the head in (request, page) order and released to the end. rings_out may be rings_in.
 *  cu_tokens          : device int32 [B+1] or NULL: first new token of each request, in request order
 *  slots              : device int32 [max_tokens][4], 16-byte aligned, or NULL: per new token its position, its
 *                       region (0 sink, 1 history, 2 recent), page id and row, once all new tokens are in.
 *                       Rows behind the last new token stay as they are.
 * Pages shared by several requests (prefix caching) have no reference count: do not release them here.
 * Nothing is changed, and a status bit says why, if a length is negative, shrinks to other than 0 or needs more
 * than max_hist_pages pages, or the new tokens exceed max_tokens (BAD_SEQLEN), a ring's head or count is out of
 * range (BAD_PAGE) or a ring is too short (NO_PAGES). One word of the cache's workspace orders the call's CTAs:
 * as for decode, calls on one cache must not overlap. Errors: INVALID_ARG (B < 0, null pointers, slots not 16-byte
 * aligned, max_tokens < 0), UNSUPPORTED (B > OSCAR_MAX_TABLE_BATCH), CUDA. */
int oscar_build_tables(oscar_cache* cache, int B, const int32_t* old_lens, const int32_t* new_lens,
                       int32_t* hist_pt, int max_hist_pages, int32_t* bf16_pt, int32_t* free_int2,
                       int32_t* free_bf16, const int32_t* rings_in, int32_t* rings_out, int32_t* cu_tokens,
                       int32_t* slots, int max_tokens, void* stream);

/* Masks and positions of drafted trees.
 *  parents   : device int32 [B][T]: the parent of node i, below i, or -1 where it follows the last cached token
 *  n_draft   : device int32 [B], nodes of each request (0 .. T), or NULL: T
 *  seq_lens  : device int32 [B], cached tokens
 *  mask      : device uint64 [B][T][(T + 63) / 64]: bit j of node i's words is set when j is i or above it
 *  positions : device int32 [B][T]: seq_lens[r] + the number of drafted nodes above i
 * Nodes from n_draft[r] on, nodes at or below a parent out of range (BAD_TREE), and all nodes of a request whose
 * length is negative or leaves no room for T positions below 2^31 (BAD_SEQLEN) get an empty mask and position -1. The
 * length of a request without nodes is not looked at.
 * Errors: INVALID_ARG (B < 0, T < 1, null pointers, mask not 8-byte aligned), UNSUPPORTED (T > OSCAR_MAX_DRAFT),
 * CUDA. */
int oscar_tree_layout(oscar_cache* cache, int B, int T, const int32_t* parents, const int32_t* n_draft,
                      const int32_t* seq_lens, uint64_t* mask, int32_t* positions, void* stream);

/* Rotary positions. Plan: the frequency of every pair of channels (host).
 *  rotary_dim : rotated channels of a head, even; pair i turns by inv_freq[i] radians per position
 *  base       : inv_freq[i] = base^(-2 i / rotary_dim) before scaling, base > 1
 *  scaling    : OSCAR_ROPE_NONE; OSCAR_ROPE_LINEAR: all frequencies divided by factor; OSCAR_ROPE_NTK: the base
 *               times factor^(rotary_dim / (rotary_dim - 2)) (rotary_dim > 2); OSCAR_ROPE_YARN: pairs that turn
 *               less than beta_slow times in original_length positions are divided by factor, pairs that turn
 *               more than beta_fast times stay, a linear ramp over the pair index between them; *scale becomes
 *               0.1 ln(factor) + 1 (1 for the other kinds)
 *  inv_freq   : host float64 [rotary_dim / 2];  scale : factor of the rotated values
 * oscar_rope_turns turns frequencies (n of them, 0 <= f < 2 pi) into the table oscar_rope reads, 64-bit fractions
 * of a turn per position: integer products keep the angle of any position to 2^-32 turns, and what is rounded to
 * float32 is less than half a turn (2^-26 turns, or 1e-7 radians). Copy it to the device once. Errors: INVALID_ARG. */
#define OSCAR_ROPE_NONE   0
#define OSCAR_ROPE_LINEAR 1
#define OSCAR_ROPE_NTK    2
#define OSCAR_ROPE_YARN   3
int oscar_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double original_length,
                           double beta_fast, double beta_slow, double* inv_freq, float* scale);
int oscar_rope_turns(const double* inv_freq, int n, uint64_t* turns);

#define OSCAR_ROPE_HALF  0    /* pair i: channels i and i + rotary_dim / 2 */
#define OSCAR_ROPE_PAIRS 1    /* pair i: channels 2i and 2i + 1            */
#define OSCAR_DTYPE_BF16 0
#define OSCAR_DTYPE_FP32 1
#define OSCAR_DTYPE_FP16 2

/* [N][heads][head_dim] rows, strides in elements, the channels of a head contiguous. out = in with equal strides
 * works in place; any other overlap is undefined. */
typedef struct oscar_rope_tensor {
  const void* in;
  void* out;
  int64_t in_token, in_head, out_token, out_head;
  int heads;                       /* 0: no such tensor */
} oscar_rope_tensor;

/* Rotate token n's heads of q and k by positions[n] (device int32 [N]):
 *   (a, b) -> scale (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq of the pair,
 * or with -t where inverse is 1: the gradient of the forward rotation. Channels from rotary_dim on are copied.
 * Rows with a negative position are left as they are. q and k have one dtype (OSCAR_DTYPE_*); products in
 * float32, one rounding at the end.
 *  turns : device uint64 [rotary_dim / 2] from oscar_rope_turns, 8-byte aligned
 * Errors: INVALID_ARG (null pointers, N < 0, negative heads or strides, odd or too large rotary_dim, a bad dtype,
 * layout or scale), UNSUPPORTED (head_dim odd or above 512, more than 2^30 heads of q and k together), CUDA. Works without
 * a cache. */
int oscar_rope(const oscar_rope_tensor* q, const oscar_rope_tensor* k, int N, int head_dim, int dtype,
               const int32_t* positions, const uint64_t* turns, int rotary_dim, int layout, float scale, int inverse,
               void* stream);

/* A rotation as the calls below take it. Positions may have several axes (time, height and width of images and video):
 * pair i then turns by its frequency and the token's position on axis axes[i]. */
#define OSCAR_MAX_ROPE_AXES 4
typedef struct oscar_rotary {
  const uint64_t* turns;           /* device [rotary_dim / 2] from oscar_rope_turns, 8-byte aligned                */
  const uint8_t* axes;             /* device [rotary_dim / 2], or NULL: axis 0. Values from num_axes on count as
                                      num_axes - 1                                                                */
  int num_axes;                    /* 1 .. OSCAR_MAX_ROPE_AXES                                                    */
  int rotary_dim, layout;          /* as for oscar_rope                                                           */
  float scale;
} oscar_rotary;

/* oscar_rope with positions on several axes: positions is device int32 [num_axes][N]. A row with a negative position on
 * any axis is left as it is. With one axis the results are oscar_rope's, bit by bit. Errors: as oscar_rope, INVALID_ARG
 * (num_axes out of range). Works without a cache. */
int oscar_rope_axes(const oscar_rope_tensor* q, const oscar_rope_tensor* k, int N, int head_dim, int dtype,
                    const int32_t* positions, const oscar_rotary* rotary, int inverse, void* stream);

/* Root-mean-square norm of every head's row and the rotation of the result, in one pass:
 *   y = Rot(x r w),  r = (mean of x^2 over the head's channels + eps)^-1/2.
 * All channels are normalised, the first rotary_dim of them rotated. Everything is float32 up to one rounding at the
 * end (squares beyond float32's range are the caller's to avoid). q and k, positions and padded rows as for
 * oscar_rope_axes; out = in with equal strides works in place.
 *  q_weight, k_weight : device [head_dim], of the rows' dtype, or NULL: ones;  eps > 0
 * Errors: as oscar_rope_axes, INVALID_ARG (eps, a weight not aligned to its type), UNSUPPORTED (more than 8,192 heads of q
 * or k). Works without a cache. */
typedef struct oscar_head_norm {
  const void *q_weight, *k_weight;
  float eps;
} oscar_head_norm;
int oscar_norm_rope(const oscar_rope_tensor* q, const oscar_rope_tensor* k, int N, int head_dim, int dtype,
                    const int32_t* positions, const oscar_rotary* rotary, const oscar_head_norm* norm, void* stream);

/* Gradient of oscar_norm_rope. q, k: in = the rows that were normalised, out = the gradient by them; grad_q, grad_k: in =
 * the gradient by the results (heads as in q and k; out is not used). With g that gradient: h = Rot^T g, u = h w,
 *   dx = r (u - x r^2 mean(u x)),   dw = sum over tokens and heads of h x r.
 * out may be in, or the gradient that was given, with equal strides. Rows with a negative position are left as they are
 * and add nothing to dw.
 *  dq_weight, dk_weight : device float32 [head_dim], written (not added to), each may be NULL. Sums are taken in an order
 *                         that depends on the sizes, the dtype, the layout and the rows' alignment alone: the same call gives
 *                         the same bits. No rows give zeros.
 *  workspace : device, 16-byte aligned, of oscar_norm_rope_workspace_bytes(head_dim) bytes, not needed (NULL) without
 *              weight gradients; calls that may overlap need one each
 * Errors: as oscar_norm_rope, INVALID_ARG (workspace too small). Works without a cache. */
int oscar_norm_rope_workspace_bytes(int head_dim, size_t* bytes);
int oscar_norm_rope_backward(const oscar_rope_tensor* q, const oscar_rope_tensor* k, const oscar_rope_tensor* grad_q,
                             const oscar_rope_tensor* grad_k, int N, int head_dim, int dtype, const int32_t* positions,
                             const oscar_rotary* rotary, const oscar_head_norm* norm, float* dq_weight, float* dk_weight,
                             void* workspace, size_t workspace_bytes, void* stream);

/* One token per request from the raw projections: q and k are normalised and rotated on the way into the append and the
 * decode, with oscar_norm_rope's formulas and one rounding to bf16.
 *  q, k, v   : device bf16 [B][Hq][128], [B][Hkv][128], [B][Hkv][128], 16-byte aligned; q_row, k_row, v_row: elements
 *              between two requests' rows, multiples of 8 (views of one fused projection)
 *  q_out     : device bf16 [B][Hq][128], 16-byte aligned: the normed and rotated queries; may be q where q_row is Hq * 128
 *  positions : device int32 [num_axes][B], or NULL: seq_lens_before[r] on every axis. A negative one counts as 0
 *              (BAD_SEQLEN).
 *  norm      : NULL: no norm, the rotation alone */
typedef struct oscar_raw_step {
  const void *q, *k, *v;
  int64_t q_row, k_row, v_row;
  void* q_out;
  const int32_t* positions;
  const oscar_rotary* rotary;
  const oscar_head_norm* norm;
} oscar_raw_step;

/* oscar_append_kv of the normed and rotated k and of v; q_out gets the queries for an oscar_decode_attention behind it.
 * q may be NULL (then q_out is not used). All inputs but the cache's rotations may come from the kernel just before, unlike
 * those of oscar_append_kv. A key, value or query that is not finite raises NONFINITE. Errors: as oscar_append_kv and
 * oscar_norm_rope, INVALID_ARG (a missing structure, rows not 16-byte aligned or not a multiple of 8 elements apart,
 * q_out = q with another row, a rotary_dim above 128). */
int oscar_append_kv_rope(oscar_cache* cache, int layer, int B, const oscar_raw_step* raw, const int32_t* seq_lens_before,
                         const int32_t* hist_pt, int max_hist_pages, const int32_t* bf16_pt, void* stream);

/* oscar_decode_step (oscar_decode_step_shared where shared_hist_pages > 0) from raw q, k and v: the same three launches,
 * with the norm and the rotation in the first. The results are those of oscar_append_kv_rope followed by
 * oscar_decode_attention of q_out over seq_lens_before[r] + 1 tokens. */
int oscar_decode_step_rope(oscar_cache* cache, int layer, int B, const oscar_raw_step* raw, const int32_t* seq_lens_before,
                           const int32_t* hist_pt, int max_hist_pages, int shared_hist_pages, const int32_t* bf16_pt,
                           float sm_scale, void* out, int out_dtype, float* lse, void* stream);

/* Attention of drafted nodes over the cache and their drafted ancestors.
 *  q                : device bf16 [B][T][Hq][128]; k_draft, v_draft : device bf16 [B][T][Hkv][128] (not in the cache)
 *  mask             : device uint64 [B][T][(T + 63) / 64]: bit j of row i lets node i attend to drafted node j;
 *                     bits from n_draft[r] on are ignored. Any pattern is allowed (oscar_tree_layout's, a chain, a
 *                     block), also an empty row, which then attends to the cache alone.
 *  n_draft          : device int32 [B] (0 .. T), or NULL: T
 *  seq_lens         : device int32 [B]: cached tokens (>= 0), all visible to every node and read as they are: with a
 *                     full recent window its oldest token is still BF16 here, while oscar_decode_step, which has the
 *                     new token in the cache, moves it to the INT2 history before it attends. Below sink + recent
 *                     tokens a single node is a decode step.
 *  out              : device [B][T][Hq][128], bf16 or fp32 (out_dtype), in the value basis of
 *                     oscar_decode_attention; lse : device float32 [B][T][Hq] or NULL
 *  workspace        : device, 256-byte aligned, of oscar_tree_workspace_bytes(cache, B, T, max_hist_pages) bytes; less
 *                     is accepted and splits the history less, down to two slots of 528 bytes (one more for every
 *                     4,096 history pages beyond the first 4,096) for each query row, where the T Hq / Hkv rows of
 *                     a request and kv head count as a multiple of 8 up to 128 and of 128 above. Slots of more than 512
 *                     history pages (256 where a kv head has more than 128 rows), which only such a workspace makes,
 *                     sum so many products into one accumulator that its truncation shows: up to 1.3e-3 of the values'
 *                     mean at 4,096 pages. Calls that may overlap need a workspace each.
 * Rows of nodes from n_draft[r] on are left as they are. A row that attends to nothing is 0 with lse -inf. A NaN or
 * infinity in a drafted row reaches the rows that attend to it and no others (NONFINITE); one in a row of q makes that
 * row's output and lse NaN and touches no other (NONFINITE).
 * The cache is only read; all inputs but the cache's rotations may come from the kernel just before.
 * q, k_draft, v_draft and out are 16-byte aligned, mask 8-byte. Errors: INVALID_ARG (as
 * oscar_decode_attention, workspace too small), UNSUPPORTED (T > OSCAR_MAX_DRAFT, B > 65535, sink + recent above
 * 130,560 tokens), CUDA. */
int oscar_tree_workspace_bytes(const oscar_cache* cache, int B, int T, int max_hist_pages, size_t* bytes);
int oscar_tree_attention(oscar_cache* cache, int layer, int B, int T, const void* q, const void* k_draft,
                         const void* v_draft, const uint64_t* mask, const int32_t* n_draft, const int32_t* seq_lens,
                         const int32_t* hist_pt, int max_hist_pages, const int32_t* bf16_pt, float sm_scale, void* out,
                         int out_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Append the accepted drafted tokens: for j < n_accept[r], node path[r][j] at position seq_lens_before[r] + j, with
 * the bytes that n_accept[r] calls of oscar_append_kv would leave (each demotes the token that leaves the recent
 * window).
 *  k_draft, v_draft : device bf16 [B][T][Hkv][128], 16-byte aligned
 *  n_accept         : device int32 [B], 0 .. max_accept
 *  path             : device int32 [B][max_accept], or NULL: nodes 0, 1, 2, ... (a ragged append of T tokens)
 *  max_accept       : 1 .. recent; with a path it may exceed T (a node may be named twice)
 * A request with a length or count out of range is left as it is (BAD_SEQLEN); a token whose node (BAD_TREE), page
 * (BAD_PAGE) or history page (BAD_SEQLEN, BAD_PAGE) is out of range is left out. All inputs may come from the kernel
 * just before. Errors: INVALID_ARG (as oscar_append_kv, T < 1, max_accept outside 1 .. recent, path NULL with
 * max_accept > T), CUDA. */
int oscar_commit_draft(oscar_cache* cache, int layer, int B, int T, const void* k_draft, const void* v_draft,
                       const int32_t* seq_lens_before, const int32_t* n_accept, int max_accept, const int32_t* path,
                       const int32_t* hist_pt, int max_hist_pages, const int32_t* bf16_pt, void* stream);

/* Choose the INT2 decode kernel (OSCAR_DECODE_MMA by default). */
int oscar_set_decode_algo(oscar_cache* cache, int algo);

/* Synchronise the device, return the device status word in *code and clear
 * it. Returns OSCAR_ERR_DEVICE_STATUS when *code != 0. */
int oscar_get_status(oscar_cache* cache, int* code);

/* ---- test and debug entry points ----------------------------------------- */

/* Clip, quantise and pack pre-rotated float32 values into history rows,
 * skipping the rotation (for bit-exact checks of the quantiser and packing).
 *  kind   : OSCAR_KIND_K or OSCAR_KIND_V (writes that half of the row)
 *  xrot   : device float32 [N][Hkv][128], already in the rotated basis
 *  page_ids, rows : device int32 [N], INT2 page id and row (0..63) per token */
int oscar_pack_rotated(oscar_cache* cache, int layer, int kind, const float* xrot, const int32_t* page_ids,
                       const int32_t* rows, int N, void* stream);

/* y = x R (kind K: R_K, kind V: R_V) as the write path computes it.
 *  x : device bf16 [N][Hkv][128];  y : device float32 [N][Hkv][128] */
int oscar_rotate(oscar_cache* cache, int layer, int kind, const void* x, float* y, int N, void* stream);

/* ---- BF16 comparison kernel ---------------------------------------------- */

/* Workspace bytes of oscar_bf16_decode. */
int oscar_bf16_decode_workspace_bytes(int max_batch, int num_q_heads, int max_splits, size_t* bytes);

/* Decode attention over a plain all-BF16 paged cache, the baseline OSCAR's
 * speedups are measured against.
 *  kv_pages   : device bf16 [num_pages][Hkv][2][64][128] (K block then V block)
 *  page_table : device int32 [B][max_pages]; position pos -> page_table[pos/64], row pos%64
 *  workspace  : device, oscar_bf16_decode_workspace_bytes(B or more, Hq, max_splits) */
int oscar_bf16_decode(int B, int num_q_heads, int num_kv_heads, const void* kv_pages, int num_pages,
                      const void* q, const int32_t* seq_lens, const int32_t* page_table, int max_pages,
                      float sm_scale, void* out, int out_dtype, float* lse, void* workspace,
                      size_t workspace_bytes, int max_splits, void* stream);

/* ---- offline calibration (host) ------------------------------------------ */

/* Offline calibration of one (layer, kv head) on the host (MarkTechPost
 * article, "OSCAR 有何不同做法"; visual guide step 2):
 *   C_Q = (1/N) sum_n q_n^T q_n over the N calibration queries,
 *   C_S = (1/N) V^T S^T S V with S = row-softmax(sm_scale Q K^T) (no mask),
 *   U_K, U_V = eigenvectors of C_Q, C_S (columns, descending eigenvalue,
 *   each column's largest-magnitude entry positive),
 *   tau_K[j] = c_K-quantile of |K R_K|[:, j], tau_V[j] = c_V-quantile of
 *   |V R_V|[:, j] (linear interpolation between order statistics).
 *  Q, K, V : host float32 [N][128]; outputs host float32 U [128][128], tau [128].
 *  eig_K, eig_V : optional host float64 [128] eigenvalue outputs (may be NULL). */
int oscar_calibrate(const float* Q, const float* K, const float* V, int N, float sm_scale, float c_K,
                    float c_V, float* U_K, float* U_V, float* tau_K, float* tau_V, double* eig_K,
                    double* eig_V);

/* ---- tracing ------------------------------------------------------------- */

/* Start tracing decode calls: while enabled, every oscar_decode_attention and
 * oscar_decode_step records a CUDA event pair on its stream around its
 * history kernel (the fused tensor-core decode kernel, or the CUDA-core
 * history kernel), the dominant launch of the call; at most `capacity` calls
 * are kept. The events separate that kernel from the programmatic overlap
 * with its neighbours, so it is timed alone. Event records can be captured
 * into a CUDA graph; the graph then re-records the same events on every
 * replay. */
int oscar_profile_begin(oscar_cache* cache, int capacity);

/* Stop, synchronise and report the summed device time (ms) of the traced
 * calls and their count. */
int oscar_profile_read(oscar_cache* cache, double* total_ms, int* launches);

/* ---- allocation-free decode ---------------------------------------------- */

#define OSCAR_ERR_TOO_LARGE (-7)  /* the call needs more than the fixed device scratch */

/* Decode attention that allocates nothing. The paper has no counterpart: this
 * entry point exists for callers that cannot call cudaMalloc, such as serving
 * engines whose allocator already owns all device memory and forbids side
 * allocations, and hosts that may not allocate on a latency-critical path
 * (cudaMalloc can synchronise the device and take milliseconds).
 *
 * It computes exactly what oscar_decode_attention computes, with the same
 * arguments, except:
 *  - the cache is given by its layout and pool instead of a handle: `pool` is
 *    the device buffer a cache with this `layout` was created on (rotation and
 *    tokens already written through the other entry points);
 *  - no workspace is used: the scratch (status word, rotated queries, split
 *    partials) lives in a 4 MiB static device array inside the library, which
 *    every GPU that loads the library holds until the process exits;
 *  - this call's device status bits are copied to `status` (device int32,
 *    may be NULL) at the end of the call.
 * The call performs no cudaMalloc, cudaFree or other allocating call.
 * Set-up: the first call on a device resolves the array's address for that
 * device (cudaGetSymbolAddress) and configures the kernels. Every call shares the array and it keeps the
 * last call's contents (the status word is cleared at the start of each
 * call): calls that may overlap on the GPU (different streams, or threads
 * without ordering) race and give wrong results; calls ordered on one stream
 * are safe. The history is split into fewer pieces when needed to fit. A call
 * whose per-query state does not fit even with one history split, i.e. when
 * B * Hq * (560 + 528 * (1 + (sink + recent) / 64)) + B * Hkv * 4096 bytes plus
 * about 1.3 KB of rounding exceed 4 MiB (B * Hq above about 880 with the
 * default windows and Hq / Hkv = 4), returns OSCAR_ERR_TOO_LARGE before any
 * device work. */
int oscar_decode_attention_noalloc(const oscar_layout* layout, void* pool, int layer, int B, const void* q,
                                   const int32_t* seq_lens, const int32_t* hist_pt, int max_hist_pages,
                                   const int32_t* bf16_pt, float sm_scale, void* out, int out_dtype, float* lse,
                                   int* status, void* stream);

/* Record a timeline of the CTAs of every following tensor-core decode launch
 * (each launch overwrites it): for CTA i (linear block index) the eight
 * uint64 values at buf[8 i] are its id, SM id, start time, time its first
 * history page landed, time its last warp finished the main loop, time its
 * partials were written, 0, and the time its wait for the kernel before it
 * returned (history CTAs); times are %globaltimer nanoseconds.
 * buf: device memory for `capacity` records (64 bytes each); NULL stops
 * recording. CTAs beyond `capacity` are not recorded. */
int oscar_trace_ctas(oscar_cache* cache, void* buf, int capacity);

/* Record a timeline of every CTA of the following launches of this cache's
 * kernels (append, prefill, query prologue, decode, merge), accumulating
 * across launches until the buffer is full. buf: device uint64
 * [4 + 4 * capacity]; the caller zeroes buf[0], which counts the records
 * claimed (it may exceed `capacity`; the excess is not written). Record i is
 * buf[4 + 4 i .. 4 + 4 i + 3] = {kind | layer << 8 | SM << 24 | linear CTA
 * index << 32, start, end, mark}, times in %globaltimer nanoseconds, taken by
 * thread 0 on entry and when it leaves the kernel; mark is, for the merge, the
 * time its wait for the decode kernel returned and, for the step prologue,
 * the time its rotation was done, else 0. Kinds: 1 step prologue
 * with an append (oscar_append_kv, or append + query prologue in
 * oscar_decode_step), 2 query prologue alone (oscar_decode_attention),
 * 3 tensor-core decode, 4 merge, 5 CUDA-core history decode, 6 BF16 segment,
 * 7 prefill. Launches issued while a buffer is set keep
 * writing to it, also from CUDA graphs captured meanwhile; NULL stops
 * recording for later launches. */
int oscar_trace_timeline(oscar_cache* cache, void* buf, int capacity);

/* Failure-detection self-check: launches one warp that waits on a device
 * barrier nothing completes. Like every wait in the library it gives up after
 * 2 seconds of %globaltimer time and sets OSCAR_STATUS_TIMEOUT in the status
 * word (read with oscar_get_status). Nothing faults and nothing stays pending;
 * the cache remains usable. */
int oscar_check_wait_timeout(oscar_cache* cache, void* stream);

/* Human-readable name of a status code. */
const char* oscar_error_string(int code);

#ifdef __cplusplus
}
#endif
#endif /* OSCAR_H */
