/*
 * kvx_attention.h — the libkvx calls that compute on a paged KV cache: the write of rotated new
 * rows, the attention of new tokens over the cache, the weight that attention gives to every
 * cached token, and the eviction of the tokens with the least of it.
 *
 * They belong to the same library as kvx.h (libkvx.so) and follow its conventions: device
 * pointers unless marked [host], arguments validated on the host before anything is enqueued,
 * nothing allocated, no synchronisation, no state between calls, capturable in a HIP graph;
 * data-dependent errors are skipped over and OR-ed into *err_flag as KVX_DEVERR_* bits. Every
 * data pointer and every byte stride is a multiple of 16; index and float arrays need their
 * natural alignment.
 *
 * Unlike the copies of kvx.h these calls do floating-point work. Elements are 16-bit (bf16 or
 * fp16); products are accumulated and softmax statistics, angles and totals held in 32 bits
 * (angles in 64), and results are rounded to the element type once, to nearest even. One more
 * rounding is in kvx_paged_attention: the matrix units take the weights that multiply V in the
 * element type, so each is off by up to half a step (bf16 2^-8, fp16 2^-11; fp16 weights below 2^-25
 * of their row's largest by up to 2^-36 of that one), while the sum that divides them holds them unrounded. Every
 * result is a fixed function of the inputs and the launch parameters: there are no atomics on
 * results, and a repeated call gives the same bits.
 */
#ifndef KVX_ATTENTION_H
#define KVX_ATTENTION_H

#include "kvx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define KVX_DTYPE_BF16 0
#define KVX_DTYPE_FP16 1

/* Largest head_dim; head_dim is a multiple of 8. */
#define KVX_MAX_HEAD_DIM 256
/* Requests times KV heads of a call (in kvx_evict_compact: times 2 KV heads + mass heads), and the tokens of
 * kvx_rope_and_cache, are below 2^22; requests of kvx_paged_attention and kvx_attention_mass below
 * 2^16. Larger ones return KVX_ERR_INVALID_ARGUMENT. */

/* Most axes of a rotary position. */
#define KVX_MAX_AXES 4

/* One layer's paged cache of K and V rows. [host] Element (block b, token o of the block, head h,
 * K: w = 0 or V: w = 1, dimension d) is at
 *     base + b*block_stride + o*token_stride + w*kv_stride + h*head_stride + d*2
 * (strides in bytes), which covers the three layouts of kvx_reshape_and_cache, and caches that
 * are head-major inside a block. Slot j of a request is token j % block_size of block
 * table[j / block_size], as in kvx_slot_mapping. The caller guarantees that every such address
 * with b < num_blocks lies inside the allocation. */
typedef struct kvx_paged_cache {
  void* base;
  int64_t num_blocks;
  int64_t block_stride_bytes;
  int64_t token_stride_bytes;
  int64_t kv_stride_bytes;
  int64_t head_stride_bytes;
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype;
} kvx_paged_cache;

/* The requests of one call. [host] Request r's new tokens are rows q_offsets[r] ..
 * q_offsets[r+1]-1 of the query (int64 [num_reqs+1], from 0, non-decreasing, at most num_tokens;
 * rows from q_offsets[num_reqs] on belong to nobody), and its cached tokens are its slots
 * 0 .. context_lens[r]-1 (int64 [num_reqs]), the new tokens' own among them: their rows have been
 * written before the call. block_table is int32 [num_reqs][bt_row_stride] as in kvx_slot_mapping.
 * max_query_len and max_context_len say how long the longest request is, for the choice of launch
 * shape only: results do not depend on them beyond rounding, and a request may be longer. */
typedef struct kvx_batch {
  const int32_t* block_table;
  const int64_t* q_offsets;
  const int64_t* context_lens;
  int64_t max_blocks_per_req;
  int64_t bt_row_stride;
  int64_t num_tokens;
  int64_t max_query_len;
  int64_t max_context_len;
  int32_t num_reqs;
} kvx_batch;

/*
 * kvx_rope_and_cache — rotate the new tokens' queries and keys by their positions, and write the
 * rotated K row and the V row of each token into its cache slot (kvx_reshape_and_cache with the
 * rotation in front of it, in one pass over the data).
 *   A position has num_axes coordinates (one for text; time, height, width for images and video):
 *   positions is int64 [num_axes][num_tokens], |position| < 2^31. Pair i of a head's first rot_dim
 *   elements, i < rot_dim/2, turns by the angle a = positions[pair_axis[i]][token] * inv_freq[i]:
 *       x' = x cos a - y sin a,   y' = y cos a + x sin a
 *   where (x, y) are elements i and i + rot_dim/2, or 2i and 2i+1 with interleaved != 0. Elements
 *   from rot_dim on keep their bits, and so does V.
 *   query      [num_tokens][num_heads][head_dim]; query_out gets the rotated rows (other strides
 *              allowed; query_out may be query itself with the same strides).
 *   key, value [num_tokens][num_kv_heads][head_dim]; heads of a row at the head stride.
 *   pair_axis  int32 [rot_dim/2] [host], each in [0, num_axes); read before the call returns.
 *   inv_freq   float32 [rot_dim/2]; its values count exactly as they are, and the angle is formed
 *              in 64 bits.
 *   slot_mapping int64 [num_tokens]: slot < 0 writes no K and V (padding); a slot in a block >=
 *              num_blocks is skipped and raises KVX_DEVERR_SLOT_RANGE. The query is rotated either
 *              way. Two tokens of a call must not have the same slot.
 * num_heads may be 0 (query NULL) to rotate and write keys alone. rot_dim is a multiple of 16,
 * 16 <= rot_dim <= head_dim. Errors: INVALID_ARGUMENT, MISALIGNED.
 */
kvx_status kvx_rope_and_cache(const kvx_paged_cache* cache, const void* query,
                              int64_t query_token_stride_bytes, int64_t query_head_stride_bytes,
                              int32_t num_heads, const void* key, int64_t key_token_stride_bytes,
                              int64_t key_head_stride_bytes, const void* value,
                              int64_t value_token_stride_bytes, int64_t value_head_stride_bytes,
                              int64_t num_tokens, const int64_t* positions, int32_t num_axes,
                              const int32_t* pair_axis, const float* inv_freq, int32_t rot_dim,
                              int32_t interleaved, const int64_t* slot_mapping, void* query_out,
                              int64_t out_token_stride_bytes, int64_t out_head_stride_bytes,
                              int32_t* err_flag, hipStream_t stream);

/*
 * kvx_paged_attention — attention of every request's new tokens over its paged cache: one token
 * (decode), a few drafted ones, a chunk of a prompt or the whole of it, mixed in one call.
 *   Query row (token i of request r, head h) with n = q_offsets[r+1]-q_offsets[r] new tokens and
 *   c = context_lens[r] slots sees slot j if j < c and
 *       causal:      j <= last = c - n + i            otherwise: last = c - 1
 *       window > 0:  j > last - window
 *   and its table entry is a block of the cache. With K and V from KV head h / (num_heads /
 *   num_kv_heads):
 *       out = sum_j exp(x_j - lse) V_j,   x_j = scale * (q . K_j),   lse = log sum_j exp(x_j)
 *   A row that sees nothing (no context, or every score -inf) gives out = 0 and lse = -inf. What a
 *   slot that a row does not see holds, NaN and infinities included, does not reach that row; a
 *   NaN or infinity of V that it does see reaches its elements of the same dimension.
 *   query, out   [num_tokens][num_heads][head_dim]; out must not overlap query or the cache.
 *   lse          float32 [num_tokens][num_heads], or NULL.
 *   workspace    device memory of workspace_bytes, 16-byte aligned, contents irrelevant, or NULL:
 *                lets the call split long contexts over more of the GPU and join the parts. With
 *                kvx_paged_attention_workspace() bytes it splits as far as pays, with fewer less far
 *                or, where that would leave the GPU idle, not at all.
 *                Calls that may run at the same time, replayed graphs among them, need one each.
 *   scale        finite and > 0.
 *   window       counts slots, not positions: after an eviction the last `window` tokens that were kept. With
 *                causal == 0 every row of a request sees the same last `window` slots of its context.
 * Rows that belong to nobody are left as they were. A context longer than the block table's row, a
 * negative one, or a table entry outside the cache raises KVX_DEVERR_TABLE_RANGE or
 * KVX_DEVERR_BLOCK_RANGE and the slots concerned count as not seen; offsets that decrease or leave
 * [0, num_tokens] raise KVX_DEVERR_OFFSETS and are clamped.
 * Errors: INVALID_ARGUMENT (num_tokens*num_heads + 128*num_reqs*num_kv_heads above 2^31 - 65537, and
 * max_blocks_per_req*block_size above that, among them), MISALIGNED.
 */
kvx_status kvx_paged_attention(const kvx_paged_cache* cache, const kvx_batch* batch,
                               const void* query, int64_t query_token_stride_bytes,
                               int64_t query_head_stride_bytes, int32_t num_heads, float scale,
                               int32_t causal, int64_t window, void* out,
                               int64_t out_token_stride_bytes, int64_t out_head_stride_bytes,
                               float* lse, void* workspace, int64_t workspace_bytes,
                               int32_t* err_flag, hipStream_t stream);

/* Workspace bytes with which kvx_paged_attention splits such a batch as far as pays (0: not at
 * all). Uses the sizes in the structs, not the pointers. -1 where kvx_paged_attention would refuse the
 * sizes. [host] */
int64_t kvx_paged_attention_workspace(const kvx_paged_cache* cache, const kvx_batch* batch,
                                      int32_t num_heads);

/*
 * kvx_attention_mass — add to every cached token the attention weight that the batch's queries
 * give to it, summed over the query tokens and over the query heads of each KV head:
 *       mass[r][g][j] += sum over r's rows of heads of KV head g that see j of exp(x_j - lse[row])
 *   with x, "sees" and the arguments as for kvx_paged_attention, whose lse this takes. Rows whose
 *   lse is -inf give nothing. Slots no row sees keep their bits.
 *   mass   float32 [num_reqs][num_kv_heads][mass_width] at the given strides (in floats, the last
 *          dimension dense); a context longer than mass_width raises KVX_DEVERR_TABLE_RANGE and
 *          is cut there. With mass_width or max_blocks_per_req 0 the call does nothing.
 * Errors: INVALID_ARGUMENT (num_tokens*num_heads, or max_blocks_per_req*block_size, above 2^31 - 65537 among
 * them), MISALIGNED. Only K is read. The last tokens of a prompt, or each decoded token in turn, are what callers
 * usually accumulate over.
 */
kvx_status kvx_attention_mass(const kvx_paged_cache* cache, const kvx_batch* batch,
                              const void* query, int64_t query_token_stride_bytes,
                              int64_t query_head_stride_bytes, int32_t num_heads, float scale,
                              int32_t causal, int64_t window, const float* lse, float* mass,
                              int64_t mass_req_stride, int64_t mass_head_stride, int64_t mass_width,
                              int32_t* err_flag, hipStream_t stream);

/*
 * kvx_evict_select — choose which cached tokens stay: per request and mass head, the first `sink`
 * slots, the last `recent` slots of the context, and of the others those with the largest mass, up
 * to `budget` in all; of equal masses (0 and -0 are equal) the lowest slots stay, and NaN counts
 * as larger than +inf. A context of at most `budget` slots stays whole.
 *   mass      float32 [num_reqs][num_heads][mass_width] at the given strides (in floats), where
 *             num_heads is the number of heads that choose for themselves: num_kv_heads, or a
 *             divisor of it whose heads keep the same tokens.
 *   keep      int32 [num_reqs][num_heads][budget]: the kept slots in ascending order, then -1.
 *   new_lens  int64 [num_reqs]: min(context, budget); not the context_lens array itself.
 * 1 <= budget < 2^31, sink >= 0, recent >= 0, sink + recent <= budget. A context that is negative
 * or longer than mass_width raises KVX_DEVERR_TABLE_RANGE and is clamped.
 */
kvx_status kvx_evict_select(const float* mass, int64_t mass_req_stride, int64_t mass_head_stride,
                            int64_t mass_width, int32_t num_reqs, int32_t num_heads,
                            const int64_t* context_lens, int64_t budget, int64_t sink,
                            int64_t recent, int32_t* keep, int64_t* new_lens, int32_t* err_flag,
                            hipStream_t stream);

/*
 * kvx_evict_compact — move the kept tokens together: for every request, KV head and i with
 * keep[..][i] >= 0, the K and V rows of slot keep[..][i] go to slot i of the destination table, and
 * the mass with them. KV head h follows list h / (num_kv_heads / num_heads). Order is kept, so the
 * newest token of a request is again its last one; the requests' contexts are then the new_lens of
 * kvx_evict_select. Keys already carry their positions, so moving them changes no score.
 *   dst_block_table  may be block_table itself (same pointer): the move is then in place, the
 *              blocks after the kept slots are free afterwards, and no block may belong to two
 *              requests. Otherwise the destination blocks must be none of the source blocks, and
 *              the sources keep their bytes (a shared prefix stays whole for its other owners). A copy
 *              of the source table is not "in place": a row that would go to the request's own
 *              source block of that column is skipped and raises KVX_DEVERR_BLOCK_RANGE, unless it is
 *              there already. Source blocks at other columns or of other requests are not looked for.
 *   keep       int32 [num_reqs][num_heads][budget], ascending, -1 after the last (as
 *              kvx_evict_select writes it); negative entries move nothing.
 *   mass, mass_out  float32 [num_reqs][num_heads][width] at the given strides, or both NULL:
 *              mass_out[..][i] = mass[..][keep[i]], and 0 where keep[i] is negative and from budget
 *              up to mass_out_width. mass_out may be mass itself with the same strides (only where
 *              the move is in place); else the two must not overlap.
 * Destination slots past the kept ones keep their bytes. An entry outside the tables' (or the
 * masses') width, or in a block id outside the cache, is skipped and raises KVX_DEVERR_TABLE_RANGE
 * or KVX_DEVERR_BLOCK_RANGE; one below its own index (no ascending list has it) is skipped and
 * raises KVX_DEVERR_OFFSETS. The cache has at least one block, both tables at least one column.
 */
kvx_status kvx_evict_compact(const kvx_paged_cache* cache, const int32_t* block_table,
                             int64_t max_blocks_per_req, int64_t bt_row_stride,
                             const int32_t* dst_block_table, int64_t dst_max_blocks_per_req,
                             int64_t dst_bt_row_stride, int32_t num_reqs, int32_t num_heads,
                             const int32_t* keep, int64_t budget, const float* mass,
                             int64_t mass_req_stride, int64_t mass_head_stride, int64_t mass_width,
                             float* mass_out, int64_t mass_out_req_stride,
                             int64_t mass_out_head_stride, int64_t mass_out_width,
                             int32_t* err_flag, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVX_ATTENTION_H */
