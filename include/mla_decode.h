/* Paged Multi-head Latent Attention (MLA) decode for one GB300 (sm_103a).
 *
 * C ABI of libmla_decode.so. Plain pointers and sizes only; every pointer
 * named "device" is caller-owned device memory (for example a torch tensor's
 * data_ptr()). The calls below never allocate device memory and never
 * synchronise the stream, except mla_get_error, which is a diagnostic.
 * `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *
 * The operation, as the pages state it:
 *  - Each token of a DeepSeek-V2/V3-style MLA layer is cached as one latent
 *    row: kv_lora_rank 512 (c_kv) plus qk_rope_head_dim 64, with no per-head
 *    K or V (SGLang PR #32972 "Let Kimi-Linear use the paged MLA attention
 *    backends", Validation). With the query absorbed into latent space
 *    (q_nope * W_UK || q_rope, 576-d), every head attends over the same
 *    576-d keys, and the first 512 dims of each row are the shared value.
 *  - The pool is paged; a request's pages are listed in a block table or in
 *    CSR kv_indices (same page, "What this does").
 *  - The pool has a leading layer dimension so layers never alias slots
 *    (MoE-Infinity PR #195 "DeepSeek-V2/V3 paged-attention shim (MLA)",
 *    Root causes 5).
 *  - The new token's latent row is written through slot_mapping on every
 *    decode step (same page, Root causes 2); context_length excludes that
 *    just-generated token (Root causes 4), so the new token sits at position
 *    L = context_lens[b] and is attended.
 *  - The MLA softmax scale is passed explicitly (same page, Changes).
 *  - Optional sliding window over the most recent tokens (FastDeploy PR #8049
 *    "Support MLA_SWA functionality", Motivation): window W > 0 attends
 *    positions [max(0, L + 1 - W), L]; W = 0 attends [0, L].
 *  - Optional fp8_e4m3 cache (SGLang PR #32972, Validation table,
 *    tokenspeed_mla row), dequantised inside the kernel, never materialised
 *    as bf16 (same page, Pre-existing issues 2).
 *
 * Error behaviour: every call returns 0 or a negative MLA_ERR_* code after
 * checking its host-visible arguments. Conditions only the device can see
 * (a page id outside [0, num_pages), a slot outside the layer, a plan that
 * does not match the decode call, a bounded wait that ran out) set bits in a
 * sticky status word inside the workspace and the offending load or store is
 * skipped; no kernel traps. Read the word with mla_get_error.
 */
#ifndef MLA_DECODE_H_
#define MLA_DECODE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_OK 0
#define MLA_ERR_ARG (-1)          /* bad host argument (null, size, range) */
#define MLA_ERR_UNSUPPORTED (-2)  /* shape or dtype this library does not build */
#define MLA_ERR_WORKSPACE (-3)    /* workspace too small or misaligned */
#define MLA_ERR_CUDA (-4)         /* a CUDA runtime call failed */

/* Bits of the device status word (mla_get_error). */
#define MLA_STATUS_BAD_PAGE 0x1     /* page id outside [0, num_pages): load skipped */
#define MLA_STATUS_BAD_SLOT 0x2     /* slot_mapping entry >= num_pages*page_size: write skipped */
#define MLA_STATUS_PLAN_MISMATCH 0x4 /* decode arguments differ from the plan's */
#define MLA_STATUS_TIMEOUT 0x8      /* a bounded wait inside a kernel ran out */
#define MLA_STATUS_BAD_LENGTH 0x10  /* context_lens[b] < 0 or beyond the block table */
#define MLA_STATUS_NO_PAGES 0x20    /* mla_extend_tables: the free pages did not suffice */
#define MLA_STATUS_BAD_POSITION 0x40 /* mla_rope_write: position beyond the angle table: row skipped */

#define MLA_DTYPE_BF16 0
#define MLA_DTYPE_FP8_E4M3 1

#define MLA_KV_LORA_RANK 512
#define MLA_ROPE_DIM 64
#define MLA_LATENT_DIM 576 /* MLA_KV_LORA_RANK + MLA_ROPE_DIM */
#define MLA_V_HEAD_DIM 128 /* output width of mla_uv_project */

/* A paged latent pool: data is [num_layers][num_pages][page_size][576]
 * row-major, element type bf16 or e4m3 (one byte). data must be 16-byte
 * aligned. page_size is 16, 32, 64 or 128. kv_scale (fp8 only, > 0): the
 * stored code is e4m3(x / kv_scale) and the value read is code * kv_scale. */
typedef struct {
  void* data;
  int num_layers;
  int num_pages;
  int page_size;
  int dtype;
  float kv_scale;
} mla_kv_pool;

/* Latent write (the per-step KV persistence of MoE-Infinity PR #195, Root
 * causes 2 and Changes; pad-row rule of SGLang PR #32972, Cuda-graph safety).
 * For i < n: if slot_mapping[i] >= 0, row `new_rows[i]` is stored at
 * pool[layer][slot / page_size][slot % page_size]; negative slots are pad rows
 * and write nothing. fp8 pools store e4m3 with round-to-nearest-even and
 * saturation to +-448 of (float(x) / kv_scale), computed in IEEE fp32.
 *   new_rows:     device, [n][576] bf16, 16-byte aligned rows.
 *   slot_mapping: device, [n] int64, slot within the layer.
 *   workspace:    device decode workspace whose status word records slots
 *                 beyond the layer (write skipped), or NULL to skip silently.
 * Returns MLA_ERR_ARG for a null pool/rows/slots with n > 0 or a layer out of
 * range. */
int mla_kv_write(const mla_kv_pool* pool, int layer, const void* new_rows,
                 const int64_t* slot_mapping, int n, void* workspace,
                 void* stream);

/* Bytes of decode workspace for `batch` requests of `num_heads` heads on the
 * current device (room for the widest schedule, mla_decode_num_clusters()).
 * 0 on bad arguments or when the device cannot run the decode kernel. The
 * workspace must be 256-byte aligned and zeroed once before its first use
 * (its status word starts at 0); later calls keep it consistent. */
size_t mla_decode_workspace_size(int batch, int num_heads);

/* Number of two-CTA clusters of the decode kernel that fit on the current
 * device at once (the default schedule width), or a negative error. */
int mla_decode_num_clusters(void);

/* Split-KV schedule (the plan/run split of FlashInfer's plan(), described in
 * SGLang PR #32972, Correction: the plan writes into a buffer the caller
 * keeps, so a captured decode reads what the last plan wrote).
 * Reads context_lens (device, [batch] int32, tokens cached before this step),
 * splits the attended tokens of all requests into 64-token blocks, and
 * deals the blocks to `num_clusters` clusters. Either the concatenated block
 * sequence is cut into equal contiguous ranges, one per cluster, or (batches
 * of up to 1024 requests, when it is estimated cheaper) only requests
 * heavier than a cluster's share are split into near-equal pieces and the
 * pieces are dealt largest first, at most two per cluster. A request split
 * over several clusters has its partial results merged by mla_decode. The
 * schedule depends only on the lengths and is the same on every call with
 * the same arguments. Must be re-run whenever context_lens,
 * batch, num_heads, page_size or window change, before mla_decode.
 *   num_clusters: 0 = mla_decode_num_clusters(); 1 = no split at all;
 *                 values above mla_decode_num_clusters() are clamped to it.
 *   window:       0 = full attention, else the sliding-window width.
 * Returns MLA_ERR_WORKSPACE if workspace_bytes is below
 * mla_decode_workspace_size(batch, num_heads). */
int mla_decode_plan(const int32_t* context_lens, int batch, int num_heads,
                    int page_size, int window, int num_clusters,
                    void* workspace, size_t workspace_bytes, void* stream);

/* Absorbed paged MLA decode, q_len = 1. For each request b and head h:
 *   s_t = softmax_scale * q[b,h,:] . K_t over t in [start_b, L_b],
 *   out[b,h,:] = sum_t softmax(s)_t * K_t[0:512],
 *   lse[b,h]   = log(sum_t exp(s_t))  (natural log),
 * with K_t the 576-d latent row of position t of request b in `layer`, and
 * start_b = 0 or max(0, L_b + 1 - window). Positions live in block
 * t / page_size of the request's page list: page_indptr != NULL selects the
 * CSR form (page_ids[page_indptr[b] + j]); otherwise page_ids is a block
 * table [batch][max_blocks]. Only the blocks that hold attended positions are
 * read (the bounded-prefix rule of SGLang PR #32972, Correction); a page id
 * outside [0, num_pages) sets MLA_STATUS_BAD_PAGE and its rows read as zero.
 *   q:   device, [batch][num_heads][576] bf16 (absorbed nope 512 || rope 64).
 *   out: device, [batch][num_heads][512] bf16, 32-byte aligned (the kernel
 *        writes whole 32-byte sectors). lse: device [batch][num_heads] fp32
 *        or NULL. q must be 16-byte aligned; MLA_ERR_ARG otherwise.
 *   workspace: the one last given to mla_decode_plan with the same batch,
 *        num_heads, page_size and window.
 * num_heads must be 16, 32, 64 or 128 (MLA_ERR_UNSUPPORTED otherwise). The
 * latent width is fixed at 576/512. Arithmetic: fp32 accumulation; the two
 * CTAs that share a work unit exchange their half-dimension partial scores,
 * scaled to log2 units and rounded to fp16 (relative error at most 2^-11 of
 * a partial; magnitudes beyond 65504 saturate). fp8 pools are dequantised in the kernel, tile by tile: the codes
 * are exact in f16, q is converted to f16 (exact for |q| in [2^-14, 65504],
 * saturating beyond) and kv_scale multiplies the scores and the output.
 * Launches the split kernel and the merge kernel (which returns at once when
 * the plan split no request) on `stream`. */
int mla_decode(const mla_kv_pool* pool, int layer, const void* q,
               const int32_t* page_indptr, const int32_t* page_ids,
               int max_blocks, const int32_t* context_lens, int batch,
               int num_heads, float softmax_scale, int window,
               void* workspace, void* out, float* lse, void* stream);

/* Several query positions per request: multi-token decode (speculative or
 * multi-token-prediction steps, LightLLM PR #1593 "Support dsv4 model",
 * Summary and Validation) and, with longer runs of positions, the absorbed
 * form of chunked prefill over the paged latent (vLLM #12639 "[Attention]
 * MLA with chunked prefill", Future work). Request b holds L_b =
 * context_lens[b] cached tokens before this step; its q_len new tokens sit
 * at positions L_b .. L_b + q_len - 1 (their latent rows written beforehand
 * with mla_kv_write, q_len slots per request), and query position i attends
 * positions [start_i, L_b + i] with start_i = 0, or max(0, L_b + i + 1 -
 * window): causal within the step. q_len = 1 is mla_decode exactly.
 *   q:   device [batch][q_len][num_heads][576] bf16, 16-byte aligned.
 *   out: device [batch][q_len][num_heads][512] bf16, 32-byte aligned;
 *   lse: device [batch][q_len][num_heads] fp32 or NULL.
 * The q_len x num_heads rows of a request run in groups of 128 (one
 * tensor-core tile of rows); each group reads the request's pages once.
 * batch x q_len x num_heads must stay below 2^31 (MLA_ERR_ARG).
 * Workspace and plan: mla_decode_workspace_size_q and mla_decode_plan_q with
 * the same batch, q_len and num_heads (a plan made for another q_len sets
 * MLA_STATUS_PLAN_MISMATCH). Everything else as for mla_decode. */
size_t mla_decode_workspace_size_q(int batch, int q_len, int num_heads);
int mla_decode_plan_q(const int32_t* context_lens, int batch, int q_len,
                      int num_heads, int page_size, int window,
                      int num_clusters, void* workspace,
                      size_t workspace_bytes, void* stream);
int mla_decode_q(const mla_kv_pool* pool, int layer, const void* q,
                 const int32_t* page_indptr, const int32_t* page_ids,
                 int max_blocks, const int32_t* context_lens, int batch,
                 int q_len, int num_heads, float softmax_scale, int window,
                 void* workspace, void* out, float* lse, void* stream);

/* W_UV projection after attention: y[b,h,:] = attn_out[b,h,:] @ w_uv[h],
 * v_head_dim 128 (MoE-Infinity PR #195, Root causes 3).
 *   attn_out: device [batch][num_heads][512] bf16; w_uv: device
 *   [num_heads][512][128] bf16; y: device [batch][num_heads][128] bf16; all
 *   16-byte aligned (MLA_ERR_ARG otherwise).
 *   workspace: a decode workspace (256-byte aligned) whose status word
 *   records MLA_STATUS_TIMEOUT if a bounded wait inside the kernel runs out,
 *   or NULL. Either way the rows such a wait leaves unfinished are written
 *   as NaN, never left stale.
 * fp32 accumulation. */
int mla_uv_project(const void* attn_out, const void* w_uv, void* y, int batch,
                   int num_heads, void* workspace, void* stream);

/* ---------------------------------------------------------------- prefill step
 * Three calls make a step that takes a chunk of new tokens per request (prompt
 * chunks, mixed with single tokens): mla_extend_tables finds the tokens'
 * places, mla_rope_write rotates and stores their latent rows and rotates
 * their queries, mla_prefill attends. context_lens has its meaning of above
 * throughout: the tokens cached before the step, so that the new ones sit at
 * positions context_lens[b] .. and are attended once written. */

/* Page tables of a step from request lengths, on the device. Request b holds
 * context_lens[b] = L tokens, whose pages are the first ceil(L / page_size)
 * entries of its block table row, and gets new_lens[b] = n >= 0 more. The pages
 * that these need are taken off the top of the stack of free pages, in the
 * order of requests and blocks: the first one is free_pages[count - 1].
 *   context_lens, new_lens: device, [batch] int32.
 *   free_pages:   device, [free_capacity] int32, the stack; the first
 *                 *free_count entries are free pages. Not written.
 *   free_count:   device int32. Not written unless state points at it.
 *   block_table:  device, [batch][max_blocks] int32; the entries of new blocks
 *                 are written, all others left as they were.
 *   slot_mapping: device, [max_tokens] int64: the slot of each new token, request
 *                 after request, as mla_kv_write and mla_rope_write take it.
 *   positions:    device, [max_tokens] int32: its position; or NULL.
 *                 Entries behind the last token are -1 in both (pad rows).
 *   q_indptr:     device, [batch + 1] int32: where each request's tokens start.
 *   page_indptr, page_ids: device, [batch + 1] and [max_page_ids] int32: the
 *                 tables as CSR lists, of ceil((L + n) / page_size) pages each;
 *                 or both NULL. Entries behind the last page are left as they were.
 *   state:        device, [2] int32: the free pages left, and the first request
 *                 that was refused for want of pages (batch if none). state may
 *                 be free_count's own address: the count is then updated in place.
 * All outputs are complete when the call is, in the order of the stream; state
 * is written before the others and says nothing of them.
 * A request whose pages do not all remain (MLA_STATUS_NO_PAGES) takes none: its
 * new tokens have slot and position -1, its CSR list only the pages it held.
 * Requests after it that need pages are refused too, those that need none are
 * served. A request with a negative length or more tokens than max_blocks
 * blocks hold (MLA_STATUS_BAD_LENGTH) is refused alike; a negative n counts as
 * no tokens. A free page outside [0, num_pages) (MLA_STATUS_BAD_PAGE) is stored
 * as -1 in the table and its list. Such an id among the pages held already stays
 * as it is in both, and sets the status only where a new token lies in its page
 * (entries before a window, which nothing reads, may hold anything). Either gives
 * the tokens slot and position -1. Tokens beyond max_tokens and ids
 * beyond max_page_ids are not written (MLA_STATUS_BAD_LENGTH).
 *   workspace:    whose status word records this (a decode or prefill
 *                 workspace, 256-byte aligned), or NULL.
 * Outputs share no memory with each other or with inputs (but for state).
 * page_size is 16, 32, 64 or 128; max_blocks * page_size and batch * max_blocks
 * are below 2^31. */
int mla_extend_tables(const int32_t* context_lens, const int32_t* new_lens, int batch, int page_size, int num_pages,
                      const int32_t* free_pages, const int32_t* free_count, int free_capacity, int32_t* block_table,
                      int max_blocks, int64_t* slot_mapping, int32_t* positions, int max_tokens, int32_t* q_indptr,
                      int32_t* page_indptr, int32_t* page_ids, int max_page_ids, int32_t* state, void* workspace,
                      void* stream);

/* Rotary positions of n new tokens, the latent rows' norm and their write.
 * Pair j (of 32) of a row's last 64 dims is dims (2j, 2j + 1) if interleaved
 * is nonzero, else (j, j + 32). It turns by the angle that cos_sin holds for
 * position p = positions[pair_axis[j]][token]:
 *   (x, y) -> (x cos - y sin, x sin + y cos),
 *   cos = cos_sin[p][j], sin = cos_sin[p][32 + j].
 * Rows (rows != NULL): c_kv (the first 512 dims) becomes
 * c_kv / sqrt(mean(c_kv^2) + norm_eps) * norm_weight if norm_weight is given,
 * the rope part turns, and the row is stored at its slot as mla_kv_write does,
 * rounded once from fp32. Queries (q_rope != NULL): the 64 rope dims of every
 * head turn and are rounded to bf16.
 *   rows:         device, [n][576] bf16, 16-byte aligned.
 *   slot_mapping: device, [n] int64, no slot twice; required with rows. A row with a negative
 *                 slot is a pad row: neither its latent nor its queries are
 *                 touched. A slot beyond the layer sets MLA_STATUS_BAD_SLOT and
 *                 its latent row is skipped.
 *   positions:    device, [num_axes][n] int32, 1 to 4 axes (text has one; time,
 *                 height and width are three). A negative one marks a pad row;
 *                 one >= max_position sets MLA_STATUS_BAD_POSITION and the row
 *                 and its queries are skipped.
 *   pair_axis:    host, [32]: each pair's axis; NULL is axis 0 for all.
 *   cos_sin:      device, [max_position][64] fp32, 16-byte aligned.
 *   norm_weight:  device, [512] bf16, 16-byte aligned, or NULL.
 *   q_rope, q_out: device; the rope dims of head h of token t start
 *                 (t * num_heads + h) * pitch elements further. Pitches are
 *                 multiples of 8 and at least 64, pointers 16-byte aligned.
 *                 q_out may be q_rope (in place) or rows that share no element
 *                 with it; other overlaps are refused with MLA_ERR_ARG.
 *   pool, layer:  used with rows only; rows are not the pool's. workspace: for the status word
 *                 (256-byte aligned), or NULL. */
int mla_rope_write(const mla_kv_pool* pool, int layer, const void* rows, const int64_t* slot_mapping, int n,
                   const int32_t* positions, int num_axes, const uint8_t* pair_axis, const float* cos_sin,
                   int max_position, int interleaved, const void* norm_weight, float norm_eps, const void* q_rope,
                   int64_t q_pitch, void* q_out, int64_t q_out_pitch, int num_heads, void* workspace, void* stream);

/* Attention of a ragged chunk of new tokens over the paged cache, in the
 * 192/128 multi-head form (the unabsorbed form of mla_decode_q followed by
 * mla_uv_project, with a number of new tokens of its own for each request).
 * Request b has n_b = q_indptr[b + 1] - q_indptr[b] new tokens (0 is fine) at
 * positions L_b .. L_b + n_b - 1, written beforehand; for its token i, head h:
 *   k_t = (c_kv[t] w_uk[h]^T, k_rope[t]), v_t = c_kv[t] w_uv[h],
 *   s_t = softmax_scale * q[q_indptr[b] + i, h, :] . k_t
 *         over t in [0 or max(0, L_b + i + 1 - window), L_b + i],
 *   out = sum_t softmax(s)_t v_t,  lse = log(sum_t exp(s_t)).
 * Keys and values of all heads are made once (513 bytes per head and attended
 * position, in the workspace) and then attended at 640 flops a pair; making
 * them costs as much as 410 queries' attention. So requests of up to 32 new
 * tokens (56 over 3,000 positions and more) are attended in the latent space, by
 * the kernel of mla_decode, at 2 x 2,176 flops a pair: in calls of 16, 32, 64 or
 * 128 heads with max_kv_tokens * num_heads >= 200,000 (where q_rows <= 8 * batch
 * also from 100,000 or from batch * num_heads >= 400 on). A step of single
 * tokens alone is mla_decode's.
 *   q:        device, [q_rows][num_heads][192] bf16 (nope 128 || rope 64).
 *   q_indptr: device, [batch + 1] int32, non-decreasing, within [0, q_rows].
 *             Rows of out outside [q_indptr[0], q_indptr[batch]) stay as they were.
 *   page_indptr / page_ids / max_blocks: the pages, as for mla_decode. With
 *             page_indptr, NULL page_ids are lists without a page.
 *   max_kv_tokens: at least the sum over requests of attended positions,
 *             L_b + n_b - (0 or max(0, L_b + 1 - window)) where n_b > 0.
 *   w_uk:     device, [num_heads][128][512] bf16; w_uv: [num_heads][512][128].
 *   out:      device, [q_rows][num_heads][128] bf16, 32-byte aligned;
 *   lse:      device, [q_rows][num_heads] fp32 or NULL. q, w_uk, w_uv 16-byte.
 *   workspace: mla_prefill_workspace_size(batch, q_rows, max_kv_tokens,
 *             num_heads, heads_per_pass) bytes, 256-byte aligned, its first 256
 *             zeroed once before the first use. Of its own: not a decode
 *             workspace, and not shared by calls that overlap on the GPU.
 * num_heads is 1 to 1024. Arithmetic: fp32 accumulation and softmax sums; for
 * the tensor core keys are rounded to bf16, values and softmax weights to f16,
 * the values of a row and head with a power of two of their own (beyond 2^76 in
 * size they saturate, below 2^-74 they lose bits), the weights times that power
 * (what lies 2^-21 below a row's largest loses bits, below 2^-32 it is zero).
 * Rows whose largest value of a head lies outside [2^-8, 2^12), and attended
 * rows whose c_kv is zero, cost the call up to 2.3 times its time. In the
 * latent space a pair of bf16 queries stands for the exact one, scores and
 * softmax weights are mla_decode's, but half scores beyond 65504 log2 units are
 * infinite. The result is off by 1.7e-3 to 2.1e-3 (2-norm, of independent
 * normal values; 1.7e-3 is its own rounding to bf16). fp8 pools: the codes are
 * widened exactly and kv_scale multiplies the scores and the output. A call
 * repeated gives the same bits; with other requests, capacities or heads a pass
 * beside it a request's sums may be taken in another order.
 * out and lse share no memory with each other or with inputs.
 * On the device: a bad page id sets MLA_STATUS_BAD_PAGE and its rows read as
 * zero; a request with a bad length (negative, beyond its page list, or beyond
 * max_kv_tokens in the sum) sets MLA_STATUS_BAD_LENGTH and its rows of out and
 * lse are NaN; row pointers outside q set it and nothing is written. A cached
 * row with an infinity or NaN in c_kv gives NaN to the rows that attend it
 * and to no others (finite c_kv whose product with w_uv overflows fp32 may
 * reach others of its request). After MLA_STATUS_TIMEOUT out and lse are
 * unspecified. */
int mla_prefill(const mla_kv_pool* pool, int layer, const void* q, const int32_t* q_indptr, const int32_t* page_indptr,
                const int32_t* page_ids, int max_blocks, const int32_t* context_lens, int batch, int q_rows,
                int64_t max_kv_tokens, int num_heads, const void* w_uk, const void* w_uv, float softmax_scale,
                int window, void* workspace, size_t workspace_bytes, void* out, float* lse, void* stream);

/* Bytes of workspace for mla_prefill with room for the keys and values of
 * heads_per_pass heads (0: of all heads, or of as many as 8 GiB hold). It does
 * for every call of as many heads with no more requests, rows and positions, in
 * no more passes. A workspace of another size is used for as many heads a pass
 * as fit, without the latent space where that does not fit; below one head's
 * mla_prefill returns MLA_ERR_WORKSPACE. 0 on bad arguments. */
size_t mla_prefill_workspace_size(int batch, int q_rows, int64_t max_kv_tokens, int num_heads, int heads_per_pass);

/* ---------------------------------------------------------------- shared prefixes
 * Decode of a batch whose requests share their first positions in groups (one
 * system prompt or document for many requests): a group's prefix is read and
 * attended once for all its requests. The operation is mla_decode_q's with
 * window = 0: request b has context_lens[b] = L_b tokens cached and q_len new
 * ones, written beforehand, and its query i attends [0, L_b + i]. Prefix g
 * belongs to requests prefix_indptr[g] to prefix_indptr[g + 1]: their first
 * P = min(prefix_lens[g], every L_b of theirs) positions are read through the
 * block table row (or page list) of the first of them, the positions from P on
 * through each request's own. So a request's entries of pages that end before P
 * are used of the first request alone, and P need not end a page. A request that
 * has its group to itself is read through its own pages throughout.
 * Requests before prefix_indptr[0] or from prefix_indptr[num_prefixes] on are
 * pad requests: their rows of out and lse stay as they were.
 * Rows of a request do not see another's: a cached row of one request's own
 * positions with an infinity or NaN leaves the results of all others as they are.
 *
 * The plan goes by the lengths alone and serves any number of mla_decode_shared
 * calls (every layer of a step) with the same batch, q_len, num_heads,
 * num_prefixes and page_size; other values set MLA_STATUS_PLAN_MISMATCH and
 * nothing is written.
 *   context_lens, prefix_lens: device, [batch] and [num_prefixes] int32. Lengths
 *             below 0 or from 2^29 on set MLA_STATUS_BAD_LENGTH (of a group without
 *             requests none is looked at). Such a prefix length counts as 0; such
 *             an L_b is left out of P, and its request has the group's P positions
 *             (none by itself) and its new ones: the others' results stay.
 *   prefix_indptr: device, [num_prefixes + 1] int32, non-decreasing, within
 *             [0, batch]; otherwise MLA_STATUS_BAD_LENGTH is set and the plan is
 *             empty (decode calls with it write nothing).
 *   num_clusters: as for mla_decode_plan, of the clusters of this kernel.
 *   page_size is 16, 32, 64 or 128, num_heads 1 to 1024, batch and num_prefixes
 *   at most 2^22; batch * q_len * num_heads stays below 2^31 (q_len * num_heads
 *   below 2^30). */
size_t mla_decode_workspace_size_shared(int batch, int q_len, int num_heads, int num_prefixes);
int mla_decode_plan_shared(const int32_t* context_lens, const int32_t* prefix_indptr, const int32_t* prefix_lens, int batch,
                           int num_prefixes, int q_len, int num_heads, int page_size, int num_clusters, void* workspace,
                           size_t workspace_bytes, void* stream);
/*   q:   device [batch][q_len][num_heads][576] bf16, 16-byte aligned.
 *   page_indptr / page_ids / max_blocks: the pages, as for mla_decode. With
 *        page_indptr, NULL page_ids are lists without a page. A page id outside
 *        [0, num_pages), or a position beyond the request's list, sets
 *        MLA_STATUS_BAD_PAGE and its rows read as zero.
 *   out: device [batch][q_len][num_heads][512] bf16, 32-byte aligned;
 *   lse: device [batch][q_len][num_heads] fp32 or NULL.
 *   workspace: mla_decode_workspace_size_shared bytes (of the same batch, q_len,
 *        num_heads, num_prefixes), 256-byte aligned, its first 256 zeroed once
 *        before the first use: the one last given to mla_decode_plan_shared. Not
 *        shared by calls that overlap on the GPU.
 * Arithmetic: fp32 accumulation and softmax sums; softmax weights are rounded to
 * the cache's type for the tensor core (bf16; f16 for fp8 pools, whose queries
 * are f16 as mla_decode's are and whose kv_scale multiplies the scores and the
 * output). Scores are below 2^24 in size, in log2 units. Calls with the same plan
 * give the same bits. Of a request's new tokens those that a query does not see
 * do not touch its result, whatever they hold. A position that it sees and whose
 * row holds an infinity makes its score infinite: NaN throughout for +inf; for
 * -inf NaN in the infinite dims, or nothing where it is a new token behind the
 * first. After MLA_STATUS_TIMEOUT out and lse are unspecified. */
int mla_decode_shared(const mla_kv_pool* pool, int layer, const void* q, const int32_t* page_indptr, const int32_t* page_ids,
                      int max_blocks, int batch, int q_len, int num_heads, int num_prefixes, float softmax_scale,
                      void* workspace, void* out, float* lse, void* stream);

/* ---------------------------------------------------------------- compact store
 * A paged store of latent rows in fewer bits, with scales of the values' own:
 * for prefixes that wait to be used again. data is [num_layers][num_pages]
 * [page_size][row bytes], 16-byte aligned. A row holds, one after the other,
 *   MLA_QUANT_E4M3: 512 e4m3 codes, 4 fp32 scales (128 dims each),
 *   MLA_QUANT_E2M1: 256 bytes of two e2m1 codes (dims 2i low, 2i + 1 high), 16
 *                   bf16 scales (32 dims each),
 * and the 64 rope dims in bf16. With a the largest |c_kv| of a group, in IEEE
 * fp32: scale = a / 448, or a / 6 rounded to bf16; code = the nearest to x /
 * scale (ties to even, saturating), zero where the scale is zero. A group with an
 * infinity or NaN has a NaN scale and reads as NaN. */
#define MLA_QUANT_E4M3 0
#define MLA_QUANT_E2M1 1
#define MLA_QUANT_E4M3_ROW 656 /* bytes */
#define MLA_QUANT_E2M1_ROW 416

typedef struct {
  void* data;
  int num_layers;
  int num_pages;
  int page_size; /* 16, 32, 64 or 128 */
  int format;    /* MLA_QUANT_E4M3 or MLA_QUANT_E2M1 */
} mla_quant_pool;

/* Writes rows[i] at slot slot_mapping[i] (page * page_size + offset) of `layer`,
 * quantised; i < n. Negative slots are pad rows; a slot beyond the layer sets
 * MLA_STATUS_BAD_SLOT and is skipped. No slot twice.
 *   rows: device [n][576] bf16, 16-byte aligned. slot_mapping: device [n] int64.
 *   workspace: for the status word (256-byte aligned), or NULL. */
int mla_quant_write(const mla_quant_pool* pool, int layer, const void* rows, const int64_t* slot_mapping, int n,
                    void* workspace, void* stream);

/* Reads slot slots[i] of `layer` back, i < n, into row i of `rows` or (into !=
 * NULL) into slot into_slots[i] of layer into_layer of a decode pool. Values are
 * code * scale in fp32, rounded once to bf16; an e4m3 pool stores them as
 * mla_kv_write does (divided by its kv_scale in fp32). If either slot of i is
 * negative nothing is written for it; one beyond its layer sets
 * MLA_STATUS_BAD_SLOT likewise. A slot may be read twice but not written twice.
 *   rows: device [n][576] bf16, 16-byte aligned, or NULL with `into`.
 *   slots, into_slots: device [n] int64; into_slots NULL without `into`.
 * Outputs share no memory with the store. */
int mla_quant_read(const mla_quant_pool* pool, int layer, const int64_t* slots, int n, const mla_kv_pool* into, int into_layer,
                   const int64_t* into_slots, void* rows, void* workspace, void* stream);

/* Reads the status word of `workspace` into *code (MLA_STATUS_* bits) and, if
 * `clear` is nonzero, resets it. Synchronises `stream`: diagnostics only. */
int mla_get_error(void* workspace, int* code, int clear, void* stream);

/* Self-test of the bounded wait that every kernel of this library uses on
 * its mbarriers (the published method has no counterpart of this call): one
 * thread waits for the first phase of a fresh mbarrier, limited to limit_us
 * microseconds of global time. With arrive == 0 nothing ever completes the
 * phase, the wait runs out and MLA_STATUS_TIMEOUT is OR-ed into *status (a
 * device int32); with arrive != 0 the thread arrives first and *status is
 * left unchanged. Either way the kernel returns and the context stays
 * usable. Returns MLA_ERR_ARG for a null status or limit_us outside
 * [1, 1000000]. Asynchronous on `stream`. */
int mla_selftest_bounded_wait(int arrive, unsigned int limit_us, int32_t* status, void* stream);

/* Allocation-free decode, for callers that cannot allocate device memory at
 * all: code running inside a memory pool or arena that it does not own,
 * plugins whose host forbids cudaMalloc while a graph or a tight memory
 * budget is active, or embedded runtimes that only hand out fixed buffers.
 * The published method has no counterpart of this call; it is the same operation as
 * mla_decode_plan followed by mla_decode (same arguments, same results),
 * with the schedule and the split partials kept in a scratch array that the
 * library declares at file scope (MLA_NOALLOC_SCRATCH_BYTES of device
 * memory, held by every GPU that loads the library until the process ends).
 *   - It calls no cudaMalloc, cudaFree or allocating library routine.
 *   - A call needs mla_decode_workspace_size(batch, num_heads) bytes of that
 *     scratch: on a 152-SM GPU about 38 MiB of split partials at 128 heads
 *     plus 64 bytes per request, so up to about 150,000 requests fit; a
 *     larger call returns MLA_ERR_WORKSPACE without launching anything.
 *   - The first call on a device looks up the scratch array's device
 *     address; make that first call before any stream capture.
 *   - Every call shares the one scratch array: calls whose work overlaps on
 *     the GPU (different streams, no ordering between them) race. Order them
 *     on one stream.
 *   - The scratch keeps the last call's contents; each call resets its
 *     status word first. status (device int32 or NULL) receives the
 *     MLA_STATUS_* bits of this call when the decode has finished.
 *   - num_clusters as in mla_decode_plan (0 = full width). */
#define MLA_NOALLOC_SCRATCH_BYTES (48u << 20)
int mla_decode_noalloc(const mla_kv_pool* pool, int layer, const void* q,
                       const int32_t* page_indptr, const int32_t* page_ids,
                       int max_blocks, const int32_t* context_lens, int batch,
                       int num_heads, float softmax_scale, int window,
                       int num_clusters, void* out, float* lse,
                       int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_DECODE_H_ */
