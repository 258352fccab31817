/*
 * mla_serving.h -- C ABI of the operators around the decode of
 * mla_paged_kv.h: what fills a paged latent cache, what shares, frees and
 * moves its pages, attention over the prompts that fill it, the decode
 * that reads a prefix many requests share once for all of them, and what takes
 * chunks of new tokens through it: rotary tables, the rotation of heads, rows
 * read back, and attention of ragged chunks over their requests' pages.
 *
 * The conventions are those of mla_paged_kv.h (types, status codes, the
 * stream, caller-owned memory, asynchronous calls, errors before any launch
 * for what the host can see, *d_status (int32, zeroed by the caller; the first
 * error wins) for what only the device can see).  Every d_* pointer is
 * 16-byte aligned unless a comment says otherwise; int32 arrays need 4.
 * A workspace or plan belongs to one call at a time: calls that may overlap
 * on the GPU (two streams, two captured graphs) each need their own.
 * The current device must be the one the memory belongs to.
 */
#ifndef MLA_SERVING_H_
#define MLA_SERVING_H_

#include "mla_paged_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ append */

/* Write new tokens' latent rows into a paged cache, optionally normalising
 * the latent part and rotating the RoPE part on the way.
 *
 * Token t of the packed inputs belongs to request b with
 * cu[b] <= t < cu[b+1] (d_cu_seqlens; NULL: total_tokens / batch tokens for
 * each request, which must divide) and goes to position
 *   pos = cache_seqlens[b] - (cu[b+1] - t)
 * (cache_seqlens counts the new tokens, as the decode calls want it), that is
 * row pos % 64 of page block_table[b][pos / 64].  Tokens outside
 * [cu[0], cu[batch]) are ignored, and no other byte of the cache is written.
 *   c' = c * rsqrt(mean(c^2) + norm_eps) * norm_weight  (d_norm_weight, else c)
 *   r' = r rotated by the angle of pos (d_cos_sin, else r): pairs are
 *        (r[i], r[i+32]), or (r[2i], r[2i+1]) with rope_interleaved, i < 32;
 *        (x, y) -> (x cos - y sin, y cos + x sin), left where they were.
 * All arithmetic is fp32; each stored value is rounded once.
 * A 16-bit cache takes [c', r'] (576 values of its type).  A cache of FP8
 * records (MLA_DTYPE_FP8_RECORD) takes, for each 128-element group of c',
 * scale = max|c'| / 448 (1 for a group of zeros) and codes = E4M3(c' / scale)
 * (the fp32 quotient, nearest even, saturating), and r' in bf16.
 *
 *   d_c            [total_tokens] rows of 512, `in_dtype`, c_stride elements
 *                  apart (a multiple of 8)
 *   d_r            [total_tokens] rows of 64, same type, r_stride apart (a
 *                  multiple of 8)
 *   in_dtype       MLA_DTYPE_BF16 or MLA_DTYPE_FP16
 *   d_cache        [num_pages, 64, 576] of in_dtype (cache_dtype = in_dtype),
 *                  or uint8 [num_pages, 64, 656] (MLA_DTYPE_FP8_RECORD)
 *   d_block_table  int32 [batch, max_pages]
 *   d_norm_weight  [512] of in_dtype, or NULL
 *   d_cos_sin      fp32 [max_pos, 64]: 32 cosines, then 32 sines; or NULL
 *   d_refcount     int32 [num_pages] or NULL.  When given, a token whose page
 *                  has a count other than 1 (free, or shared by a fork) is
 *                  not written and MLA_ERR_BAD_INDEX is reported.
 * A token whose position is negative, past max_pages * 64 or past max_pos,
 * or whose page is outside the pool, is not written; MLA_ERR_BAD_INDEX.
 * Two tokens must not share a slot (requests that share a page they write). */
int mla_cache_append(const void* d_c, long long c_stride, const void* d_r, long long r_stride, int in_dtype,
                     int total_tokens, const int32_t* d_cu_seqlens, const int32_t* d_cache_seqlens, int batch,
                     const int32_t* d_block_table, int max_pages, void* d_cache, int cache_dtype, int num_pages,
                     const void* d_norm_weight, float norm_eps, const float* d_cos_sin, int max_pos,
                     int rope_interleaved, const int32_t* d_refcount, int32_t* d_status, mla_stream_t stream);

/* ------------------------------------------------------------------- pages */

/* The bookkeeping of a page pool, on the device:
 *   d_refcount    int32 [num_pages]: how many block-table entries name the
 *                 page; 0 = free.
 *   d_block_table int32 [rows, max_pages]; row r's first ceil(seqlens[r]/64)
 *                 entries are its pages, the others are not read.
 *   d_seqlens     int32 [rows].
 * One block table serves every layer; mla_cache_copy_pages moves the data of
 * all layers.  rows <= 65536, at most 4096 list entries a call (else
 * MLA_ERR_UNSUPPORTED).  New pages are always the lowest free ones, in list
 * order, so results do not depend on timing.  A list entry that cannot be
 * served leaves its row as it was and is reported: MLA_ERR_BAD_INDEX for a row
 * outside the table, a length out of range or a repeated row, and
 * MLA_ERR_NO_PAGES when the free pages ran out. */

/* Lengthen rows: seqlens[d_rows[i]] += d_new_tokens[i] (>= 0), with pages for
 * the new positions.  A row listed twice is refused in both places, as is one
 * that would pass max_pages pages.  Pages are handed out in list order; an
 * entry whose pages would pass the last free one gets none (nor do later
 * entries that need any). */
int mla_cache_grow(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                   int32_t* d_seqlens, const int32_t* d_rows, const int32_t* d_new_tokens, int n, int32_t* d_status,
                   mla_stream_t stream);

/* Fork: row d_children[i] (which must be empty, seqlens = 0) becomes a copy of
 * row d_parents[i].  Full pages are shared (their counts go up); a partly
 * filled last page is replaced by a fresh page, and d_pairs[i] = (parent's
 * page, fresh page) for mla_cache_copy_pages, else (-1, -1).  A parent may
 * appear any number of times; an entry whose child is listed twice or is not
 * empty, or whose parent is a child in this call or names a page outside the
 * pool or a free one, is refused.
 *   d_pairs int32 [n, 2] out */
int mla_cache_fork(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                   int32_t* d_seqlens, const int32_t* d_parents, const int32_t* d_children, int n, int32_t* d_pairs,
                   int32_t* d_status, mla_stream_t stream);

/* Free rows: the counts of a row's pages go down (a page whose count is
 * already 0 is left there and reported, MLA_ERR_BAD_INDEX, as an entry that
 * names none is), its entries become -1 and its length 0.  A row listed twice
 * is freed once. */
int mla_cache_free(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                   int32_t* d_seqlens, const int32_t* d_rows, int n, int32_t* d_status, mla_stream_t stream);

/* Bytes of d_workspace for mla_cache_compact. */
size_t mla_cache_compact_workspace_bytes(int num_pages);

/* Compact: with n pages in use, pages n and up move to the free pages below
 * n, the lowest first on both sides.  Counts and tables are rewritten;
 * d_pairs[k] = (old page, new page) for k < *d_count, (-1, -1) after that.  No
 * page is both a source and a target.  A table entry inside a row's length
 * that names a free page or none at all is left and reported; so is a length out
 * of range, whose row is taken as far as the table goes (negative: not at all).
 *   d_pairs int32 [num_pages / 2, 2] out, d_count int32 [1] out */
int mla_cache_compact(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                      const int32_t* d_seqlens, int32_t* d_pairs, int32_t* d_count, void* d_workspace,
                      size_t workspace_bytes, int32_t* d_status, mla_stream_t stream);

/* Copy whole pages inside a pool, for every layer: page d_pairs[i].x to page
 * d_pairs[i].y, i < n (or i < min(n, *d_count) with d_count).
 *   d_pool        layers x [num_pages, page_bytes], layer_stride bytes apart
 *                 (>= num_pages * page_bytes; both multiples of 16); pages of
 *                 at most 16 MB, at most 4096 layers and 2^24 pairs
 * (-1, -1) is skipped, and so is a pair of equal pages.  A pair with a page
 * outside the pool, with a target that an earlier pair also has, or with a
 * target that another pair reads is skipped and reported
 * (MLA_ERR_BAD_INDEX), so the outcome never depends on the order of copies. */
int mla_cache_copy_pages(void* d_pool, int layers, long long layer_stride, int num_pages, long long page_bytes,
                         const int32_t* d_pairs, const int32_t* d_count, int n, int32_t* d_status,
                         mla_stream_t stream);

/* ------------------------------------------------------------------ prompt */

/* Attention over whole prompts, packed one after another:
 *   out_i = sum_j softmax_j(scale q_i . k_j) v_j,  lse_i = ln sum_j exp(scale q_i . k_j)
 * over the keys j of query i's own sequence; causal: j <= i + Lk - Lq
 * (aligned at the end, so a chunk of queries behind earlier keys is the same
 * call with Lk > Lq).  A query that sees no key gets out = 0, lse = -inf.
 * Rows of the outputs outside every sequence are left as they were.
 *
 * Bytes of the plan of a batch. */
size_t mla_prompt_plan_bytes(int batch, int total_q);

/* The plan: the list of query tiles of all sequences, longest first, and the
 * offsets it was made for; made once for a batch and read by every layer.
 * Tiles have 512 queries where total_q / batch > 256, else 256: a plan is of
 * exactly its batch, total_q, total_k and offsets.
 *   d_cu_seqlens_q, d_cu_seqlens_k int32 [batch + 1], not decreasing (NULL k:
 *   the same as q); sequence b has queries cu_q[b] .. cu_q[b+1] - 1 and keys
 *   cu_k[b] .. cu_k[b+1] - 1.  With an offset that decreases or lies outside
 *   [0, total] the plan is empty and MLA_ERR_BAD_INDEX is reported. */
int mla_prompt_get_plan(const int32_t* d_cu_seqlens_q, const int32_t* d_cu_seqlens_k, int batch, int total_q,
                        int total_k, int causal, void* d_plan, size_t plan_bytes, int32_t* d_status,
                        mla_stream_t stream);

/*   d_q [total_q, h_q, d_qk], d_k [total_k, h_kv, d_qk], d_v [total_k, h_kv, 128],
 *       element type `dtype` (MLA_DTYPE_BF16 or _FP16); *_token_stride and
 *       *_head_stride in elements, multiples of 8; the last dimension is
 *       contiguous
 *   d_qk 192 (128 + 64 RoPE, the expanded form of the latent heads) or 128
 *   h_kv divides h_q; query head h reads key head h / (h_q / h_kv)
 *   d_plan from mla_prompt_get_plan with the same batch, total_q, total_k and causal
 *   d_out [total_q, h_q, 128] of `dtype`, d_lse fp32 [total_q, h_q], contiguous
 * Softmax weights are rounded to `dtype` for the product with v and divided by
 * the sum of the unrounded ones; statistics and sums are fp32.  softmax_scale is
 * the model's: heads expanded from a latent cache are scaled for their 192 dims,
 * and the decode of their absorbed form takes the same scale.  Values of a sequence must be finite where a query of
 * the same 128-key tile could reach them; rows of other sequences, and rows
 * past the last one, may hold anything. */
int mla_prompt_attention_fwd(const void* d_q, long long q_token_stride, long long q_head_stride, const void* d_k,
                             long long k_token_stride, long long k_head_stride, const void* d_v,
                             long long v_token_stride, long long v_head_stride, int dtype, int total_q, int total_k,
                             int batch, int h_q, int h_kv, int d_qk, float softmax_scale, const void* d_plan,
                             size_t plan_bytes, void* d_out, float* d_lse, int32_t* d_status, mla_stream_t stream);

/* The same call for a program that holds the offsets: d_cu_seqlens_q and
 * d_cu_seqlens_k (NULL: the same) are compared with the plan on the device, and
 * MLA_ERR_STALE_PLAN is reported where one is another than the plan was made
 * for.  The results are those of the plan either way. */
int mla_prompt_attention_checked_fwd(const void* d_q, long long q_token_stride, long long q_head_stride,
                                     const void* d_k, long long k_token_stride, long long k_head_stride,
                                     const void* d_v, long long v_token_stride, long long v_head_stride, int dtype,
                                     int total_q, int total_k, int batch, int h_q, int h_kv, int d_qk,
                                     float softmax_scale, const int32_t* d_cu_seqlens_q,
                                     const int32_t* d_cu_seqlens_k, const void* d_plan, size_t plan_bytes,
                                     void* d_out, float* d_lse, int32_t* d_status, mla_stream_t stream);

/* ------------------------------------------------------------ shared prefix */

/* Dense decode (mla_decode_fwd with one latent KV head: a bf16 or fp16 cache, or
 * FP8 records with a bf16 query) for a batch whose requests start with the same
 * pages, as after mla_cache_fork: the shared pages are attended once for all
 * requests' queries, 128 rows at a time, and merged with each request's own
 * pages.
 *
 * The plan finds the shared pages itself: the longest run of block-table
 * entries that the requests have in common, in whole pages that every query of
 * each of them sees; it may be none.  Requests whose first query sees less
 * than a page (empty slots of a padded batch) are attended by themselves and
 * leave the others' prefix as it is; a request that none is left to share with
 * shares nothing.  The plan is made once for a batch and
 * read by every layer, while the block table and lengths stay as they were.
 * The prefix is attended together only where that takes at most 7/8 of the
 * 128-row blocks that attending it request by request does:
 * 8 ceil(batch * s_q * h_q / 128) <= 7 batch * ceil(s_q * h_q / 128).  Elsewhere
 * (s_q * h_q a multiple of 128, say) every request fills its blocks alone, the
 * shared pages are one copy in L2 either way, and the call is mla_decode_fwd.
 * As in mla_decode_fwd, a 16-bit cache's softmax weights are rounded to its type
 * for the product with the values and divided by the sum of the unrounded ones;
 * over FP8 records the sum is that of the rounded ones.
 *   num_parts from mla_shared_prefix_num_parts; at most 1024
 * Other arguments as for mla_decode_fwd.  batch * s_q * h_q and
 * batch * max_pages stay below 2^31; s_q * h_q <= 2^20, batch <= 65535. */
int mla_shared_prefix_num_parts(int batch, int s_q, int h_q); /* >= 1, or a negative mla_status_t */
size_t mla_shared_prefix_plan_bytes(int batch, int s_q, int h_q, int num_parts);
size_t mla_shared_prefix_workspace_bytes(int batch, int s_q, int h_q, int num_parts);
int mla_shared_prefix_get_plan(const int32_t* d_block_table, int max_pages, const int32_t* d_cache_seqlens, int batch,
                               int s_q, int h_q, int causal, int num_parts, void* d_plan, size_t plan_bytes,
                               mla_stream_t stream);

/*   d_plan      from mla_shared_prefix_get_plan for the same block table,
 *               batch, s_q, h_q, causal and num_parts; it holds the lengths: a
 *               plan of others is answered by (see the checked call below)
 *   d_workspace >= mla_shared_prefix_workspace_bytes(batch, s_q, h_q, num_parts)
 * A block-table entry outside the pool masks its 64 keys and is reported, as
 * in mla_decode_fwd.  Slots of a page behind a request's last key must hold
 * finite values (they meet a weight of 0). */
int mla_shared_prefix_decode_fwd(const void* d_q, const void* d_kv, const int32_t* d_block_table, int max_pages,
                                 int num_pages, int batch, int s_q, int h_q, int dtype, int causal,
                                 float softmax_scale, const void* d_plan, size_t plan_bytes, int num_parts,
                                 void* d_workspace, size_t workspace_bytes, void* d_out, int out_type, float* d_lse,
                                 int32_t* d_status, mla_stream_t stream);

/* The same call for a program that holds the lengths: d_cache_seqlens int32
 * [batch] is compared with the plan on the device, and MLA_ERR_STALE_PLAN is
 * reported where a request's length is another than the plan's, or its entry of
 * the last shared page is another page than the others'.  The results are those
 * of the plan either way. */
int mla_shared_prefix_decode_checked_fwd(const void* d_q, const void* d_kv, const int32_t* d_block_table,
                                         int max_pages, int num_pages, int batch, int s_q, int h_q, int dtype,
                                         int causal, float softmax_scale, const int32_t* d_cache_seqlens,
                                         const void* d_plan, size_t plan_bytes, int num_parts, void* d_workspace,
                                         size_t workspace_bytes, void* d_out, int out_type, float* d_lse,
                                         int32_t* d_status, mla_stream_t stream);

/* ------------------------------------------------------------------ rotary */

/* How the frequencies of rotary positions are scaled for contexts longer than
 * the one a model was trained on (`original` positions), by `factor` (s):
 *   f_i = base^(-2i / dim), i < dim / 2;  turns_i = original f_i / 2 pi
 *   NONE        f_i
 *   LINEAR      f_i / s  (position interpolation)
 *   NTK         of base s^(dim / (dim - 2)) base
 *   YARN        w f_i / s + (1 - w) f_i, w = clamp((i - a) / max(b - a, 0.001), 0, 1) with
 *               a = max(floor(c(high)), 0), b = min(ceil(c(low)), dim - 1),
 *               c(t) = dim ln(original / 2 pi t) / (2 ln base); the table's values
 *               are multiplied by 0.1 ln s + 1
 *   WAVELENGTH  (1 - w) f_i / s + w f_i, w = clamp((turns_i - low) / (high - low), 0, 1)
 * low and high are numbers of turns over the original context. */
typedef enum {
  MLA_ROPE_NONE = 0,
  MLA_ROPE_LINEAR = 1,
  MLA_ROPE_NTK = 2,
  MLA_ROPE_YARN = 3,
  MLA_ROPE_WAVELENGTH = 4
} mla_rope_scaling_t;

/* The frequencies h_freq[dim / 2] (radians a position) and the magnitude of a
 * table, both in host memory.  dim a multiple of 8, at most 256; base > 1;
 * factor >= 1 and original > 0 where they are used; 0 < low < high (YARN and
 * WAVELENGTH). */
int mla_rope_frequencies(int dim, double base, int scaling, double factor, double original, double low, double high,
                         double* h_freq, double* h_magnitude);

/* The table of positions first_pos .. first_pos + positions - 1:
 *   d_cos_sin[p] = magnitude (cos p f_0 .. cos p f_(dim/2-1), sin p f_0 ..)
 * fp32 [positions, dim], 16-byte aligned, as mla_cache_append (dim 64) and
 * mla_rope_heads read it.  h_freq in host memory, 0 <= f <= 2^10, read before the
 * call returns.  Angles are off by at most 2^-52 of themselves and 2^-64 turns a
 * position (a frequency's turns are cut there), at any position below 2^31
 * (first_pos + positions is at most that); values are within 2^-21 of the cosine
 * and sine of that angle, and next to their zeros within 2^-52 of the magnitude. */
int mla_rope_table(const double* h_freq, int dim, double magnitude, long long first_pos, int positions,
                   float* d_cos_sin, mla_stream_t stream);

/* Rotate part of each head of new tokens' queries (x) and keys (k, or none), each
 * head optionally RMS-normalised first, in one pass:
 *   y = x rsqrt(mean(x^2) + norm_eps) w   over the head's dims (with weights, else x)
 *   dims rope_offset .. rope_offset + rope_dim - 1 of y turned by the angle of the
 *   token's position, pairs as in mla_cache_append: (y[i], y[i + rope_dim/2]), or
 *   (y[2i], y[2i+1]) with rope_interleaved; (a, b) -> (a cos - b sin, b cos + a sin)
 * All arithmetic is fp32; each stored value is rounded once.  A token's position
 * is d_positions[t], or, with d_positions NULL, that of mla_cache_append:
 * cache_seqlens[b] - (cu[b+1] - t) for cu[b] <= t < cu[b+1] (d_cu_seqlens NULL:
 * total_tokens / batch tokens for each request, which must divide); tokens
 * outside [cu[0], cu[batch]) are ignored.  A token whose position is negative or
 * past max_pos is not written, MLA_ERR_BAD_INDEX.  Without d_cos_sin (rope_dim 0)
 * heads are only normalised, and all of d_positions, d_cu_seqlens and
 * d_cache_seqlens are NULL.
 *   d_x, d_k   [total_tokens, heads, dim] of `dtype` (MLA_DTYPE_BF16 or _FP16);
 *              strides in elements, multiples of 8, the last dimension contiguous
 *              (0: one read for all)
 *   d_out, d_k_out  the same shapes, strides of their own, at least dim (no element
 *              may be written twice); may be d_x and d_k
 *              themselves with the same strides (dims that are not changed are
 *              then not moved), else must share no element with any input
 *   dim        a multiple of 8, at most 1024; rope_dim a multiple of 16, at most
 *              256; rope_offset a multiple of 8
 *   d_x_weight, d_k_weight  [dim] of `dtype`, or NULL: no norm of that side
 *   k_heads    0: no keys (their pointers NULL)
 *   d_cos_sin  fp32 [max_pos, rope_dim]: cosines, then sines */
int mla_rope_heads(const void* d_x, long long x_token_stride, long long x_head_stride, void* d_out,
                   long long out_token_stride, long long out_head_stride, int heads, const void* d_x_weight,
                   const void* d_k, long long k_token_stride, long long k_head_stride, void* d_k_out,
                   long long k_out_token_stride, long long k_out_head_stride, int k_heads, const void* d_k_weight,
                   int dim, int dtype, int total_tokens, int rope_dim, int rope_offset, int rope_interleaved,
                   float norm_eps, const int32_t* d_positions, const int32_t* d_cu_seqlens,
                   const int32_t* d_cache_seqlens, int batch, const float* d_cos_sin, int max_pos, int32_t* d_status,
                   mla_stream_t stream);

/* ------------------------------------------------------------------ gather */

/* Rows of a paged cache as packed rows (to be expanded into the heads of
 * mla_prompt_attention_fwd, say): row t of the output, cu[b] <= t < cu[b+1],
 * is the cache's row of request b at position d_starts[b] + t - cu[b] (d_starts
 * NULL: 0).  Rows outside [cu[0], cu[batch]) are left as they were.
 *   d_cache  [num_pages, 64, 576] bf16 or fp16, copied; or FP8 records
 *            [num_pages, 64, 656], whose codes times scales are rounded to bf16
 *            once (the RoPE part is bf16 already)
 *   d_out    [total_rows] rows of 576 of the cache's type (records: bf16),
 *            out_stride elements apart (a multiple of 8, at least 576); must not
 *            overlap the cache
 *   d_cu_seqlens int32 [batch + 1], not decreasing; d_starts int32 [batch]
 * A row whose position is negative or past max_pages * 64, or whose page is
 * outside the pool, is not written; MLA_ERR_BAD_INDEX. */
int mla_cache_gather(const void* d_cache, int cache_dtype, int num_pages, const int32_t* d_block_table, int max_pages,
                     const int32_t* d_cu_seqlens, const int32_t* d_starts, int batch, int total_rows, void* d_out,
                     long long out_stride, int32_t* d_status, mla_stream_t stream);

/* ------------------------------------------------------------------- chunk */

/* Attention of ragged chunks of new tokens over a paged latent cache, all of a
 * batch in one call: drafts to verify, prompts taken in chunks, single tokens
 * beside them.  Token i of request b's n_b = cu[b+1] - cu[b] tokens sees the
 * request's keys 0 .. cache_seqlens[b] - 1 (the new tokens among them, as after
 * mla_cache_append), with causal those up to cache_seqlens[b] - n_b + i:
 *   out = sum_j softmax_j(scale q . k_j) k_j[:512],  lse = ln sum_j exp(scale q . k_j)
 * A query that sees no key gets out = 0, lse = -inf.  Rows of the outputs outside
 * every chunk are left as they were.  Softmax weights are rounded to the cache's
 * type (fp16 over FP8 records) for the product with the values and divided by the
 * sum of the unrounded ones; statistics and sums are fp32.  In fp16 the row's largest
 * weight is held as 2^7 .. 2^15: weights below 2^-21 of it keep fewer bits, at worst
 * (the largest at 2^7) off by 2^-32 of it, and those below 2^-32 of it are 0 beside a
 * sum that has them.  Over FP8 records scores
 * are those of the products code x scale: each group's codes times the query's, a
 * query as two E4M3 numbers (exact down to 2^-9 of its largest latent element;
 * smaller elements are off by 2^-17 of that one), times the scale in fp32.  Values
 * are the products with 11 significant bits of scale and product, where a group's
 * scale is above 2^-13 of its key's largest (fewer below) and that one is within
 * 2^-61 .. 2^68.  Values there are held without a power of two, 2^E, that largest scales
 * within a factor of 256 have in common, and weights with it: what is said of the
 * largest weight holds for the largest product with 2^E.
 *
 * num_parts: pairs of CTAs that share the work; mla_chunk_num_parts gives as many
 * as the device runs at once (>= 1, or a negative mla_status_t).  At most 1024. */
#define MLA_CHUNK_PAGE_BYTES (64 * 512 * 2)
#define MLA_CHUNK_QUERY_BYTES 1040
int mla_chunk_num_parts(void);
size_t mla_chunk_plan_bytes(int batch, int total_q, int h_q, int num_parts); /* 0: sizes out of range */
size_t mla_chunk_workspace_bytes(int num_parts);

/* The plan: blocks of 128 query rows with the keys they see, cut into num_parts
 * runs of equal cost, and the offsets and lengths it was made for; made once for
 * a batch and read by every layer.  total_q * h_q < 2^31, batch <= 2^20.
 *   d_cu_seqlens_q int32 [batch + 1], not decreasing, within [0, total_q];
 *   d_cache_seqlens int32 [batch], at most 2^24 (negative: no keys).  With an
 *   offset or length out of range the plan is empty: MLA_ERR_BAD_INDEX, and a
 *   call with it writes nothing. */
int mla_chunk_get_plan(const int32_t* d_cu_seqlens_q, const int32_t* d_cache_seqlens, int batch, int total_q, int h_q,
                       int causal, int num_parts, void* d_plan, size_t plan_bytes, int32_t* d_status,
                       mla_stream_t stream);

/*   d_q           [total_q, h_q, 576] bf16 or fp16 (FP8 records: bf16)
 *   d_kv          [num_pages, 64, 576] of q's type (`dtype`), or FP8 records
 *                 [num_pages, 64, 656] (MLA_DTYPE_FP8_RECORD)
 *   d_block_table int32 [batch, max_pages]
 *   d_plan        from mla_chunk_get_plan with the same batch, total_q, h_q and
 *                 num_parts
 *   d_cu_seqlens_q, d_cache_seqlens  compared with the plan's on the device:
 *                 MLA_ERR_STALE_PLAN where one is another than the plan was made
 *                 for; the results are those of the plan.  MLA_ERR_BAD_INDEX
 *                 where they are but were out of range then: the plan is empty
 *                 and nothing is written.  NULL: not compared, and such a plan
 *                 is reported by mla_chunk_get_plan alone
 *   d_workspace   >= mla_chunk_workspace_bytes(num_parts), over FP8 records and
 *                 total_q * h_q times MLA_CHUNK_QUERY_BYTES.  There every further
 *                 MLA_CHUNK_PAGE_BYTES hold the values of a page, converted once
 *                 for requests of three 128-row blocks and more, in order; those that do
 *                 not fit are converted by each block that reads them (slower, the
 *                 same results)
 *   d_out         [total_q, h_q, 512] of out_type (bf16, fp16 or fp32), d_lse fp32
 *                 [total_q, h_q]; no output or workspace may overlap an input
 * A block-table entry outside the pool (or past max_pages) masks its 64 keys and
 * is reported, MLA_ERR_BAD_INDEX.  Slots of a page behind a request's last key may
 * hold anything; keys that any of its queries sees must be finite for all of them. */
int mla_chunk_attention_fwd(const void* d_q, const void* d_kv, const int32_t* d_block_table, int max_pages,
                            int num_pages, int batch, int total_q, int h_q, int dtype, float softmax_scale,
                            const int32_t* d_cu_seqlens_q, const int32_t* d_cache_seqlens, const void* d_plan,
                            size_t plan_bytes, int num_parts, void* d_workspace, size_t workspace_bytes, void* d_out,
                            int out_type, float* d_lse, int32_t* d_status, mla_stream_t stream);

/* -------------------------------------------------------------- test hooks */

/* The timeout and unwind paths of the two attention kernels above, as
 * mla_test_decode_timeout does for the plain decode: the arguments and checks of
 * mla_prompt_attention_fwd (bf16 with 192 dims) and of
 * mla_shared_prefix_decode_fwd (bf16, or FP8 records), else MLA_ERR_UNSUPPORTED.
 * Instances whose waits have a 200 us budget and whose first tile is never
 * loaded (FP8 records: whose first scores are never computed): the wait for it
 * runs out, MLA_ERR_TIMEOUT is reported, every role leaves its loop, copies and
 * products in flight end, tensor memory is given back, and the grid ends.  The
 * context and the stream stay usable; outputs and workspace are unspecified. */
int mla_test_prompt_timeout(const void* d_q, long long q_token_stride, long long q_head_stride, const void* d_k,
                            long long k_token_stride, long long k_head_stride, const void* d_v,
                            long long v_token_stride, long long v_head_stride, int dtype, int total_q, int total_k,
                            int batch, int h_q, int h_kv, int d_qk, float softmax_scale, const void* d_plan,
                            size_t plan_bytes, void* d_out, float* d_lse, int32_t* d_status, mla_stream_t stream);
int mla_test_shared_prefix_timeout(const void* d_q, const void* d_kv, const int32_t* d_block_table, int max_pages,
                                   int num_pages, int batch, int s_q, int h_q, int dtype, int causal,
                                   float softmax_scale, const void* d_plan, size_t plan_bytes, int num_parts,
                                   void* d_workspace, size_t workspace_bytes, void* d_out, int out_type, float* d_lse,
                                   int32_t* d_status, mla_stream_t stream);
/* The same of mla_chunk_attention_fwd (bf16, or FP8 records): its first K stage is
 * never loaded. */
int mla_test_chunk_timeout(const void* d_q, const void* d_kv, const int32_t* d_block_table, int max_pages,
                           int num_pages, int batch, int total_q, int h_q, int dtype, float softmax_scale,
                           const int32_t* d_cu_seqlens_q, const int32_t* d_cache_seqlens, const void* d_plan,
                           size_t plan_bytes, int num_parts, void* d_workspace, size_t workspace_bytes, void* d_out,
                           int out_type, float* d_lse, int32_t* d_status, mla_stream_t stream);

/* ---------------------------------------------------------------- one pointer */

/* The calls above with their arguments, in order, as 8-byte words: pointers,
 * sizes and integers as int64, floats as double.  For bindings whose
 * foreign-call cost grows with the number of arguments (0.16 us each from
 * Python on an Arm host, more than the call itself takes). */
typedef enum {
  MLA_CALL_APPEND = 0,
  MLA_CALL_GROW = 1,
  MLA_CALL_FORK = 2,
  MLA_CALL_FREE = 3,
  MLA_CALL_COMPACT = 4,
  MLA_CALL_COPY_PAGES = 5,
  MLA_CALL_PROMPT = 6,       /* mla_prompt_attention_fwd */
  MLA_CALL_SHARED_PREFIX = 7, /* mla_shared_prefix_decode_fwd */
  MLA_CALL_SHARED_PREFIX_CHECKED = 8,
  MLA_CALL_PROMPT_CHECKED = 9,
  MLA_CALL_ROPE_HEADS = 10,
  MLA_CALL_GATHER = 11,
  MLA_CALL_CHUNK = 12
} mla_call_t;
int mla_serving_call(int op, const void* args, size_t bytes); /* bytes = 8 x the call's arguments */

#ifdef __cplusplus
}
#endif

#endif /* MLA_SERVING_H_ */
