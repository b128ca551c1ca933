/*
 * kvx_fp4.h — the libkvx calls on a paged KV cache that is held in 4 bits: the write of rotated
 * new rows, the attention of new tokens over the cache, and the transfer between 16-bit caches
 * and 4-bit blocks.
 *
 * They belong to the same library as kvx.h (libkvx.so) and follow the conventions of kvx.h and
 * kvx_attention.h: device pointers unless marked [host], arguments validated on the host before
 * anything is enqueued, nothing allocated, no synchronisation, no state between calls, capturable
 * in a HIP graph; data-dependent errors are skipped over and OR-ed into *err_flag as KVX_DEVERR_*
 * bits. Every data pointer and every byte stride is a multiple of 16.
 *
 * The format (microscaling, 4.25 bits an element): an element is a sign and one of 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6 (codes 0 to 7, and 8 more where negative), two to a byte, the even one in the low half.
 * 32 neighbouring elements of a row share a power of two, 2^(s - 127) with s a byte; s = 255 makes
 * all of them NaN.
 *   Writing a group whose largest magnitude is A: s - 127 is the smallest exponent from -127 on with
 *   A < 7 * 2^(s-127), at most 125 from bf16 and 13 from fp16, so that what is read back is finite in
 *   that type; every element goes to the nearest value, of two equally near ones to the even code,
 *   and beyond 6 to 6. Values are spaced 2 at the top (4, 6, and 8 if there were one), so below the
 *   bound of the exponent no element is off by more than half the spacing at its place. A group that
 *   holds a NaN or an infinity gets s = 255 and codes 0.
 *   Reading is exact in bf16 for s from 0 to 252, and in fp16 for s from 104 to 140; beyond, values are
 *   rounded to the type, and infinite from there on.
 */
#ifndef KVX_FP4_H
#define KVX_FP4_H

#include "kvx_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Elements that share a scale; head_dim is a multiple of it, up to KVX_MAX_HEAD_DIM. */
#define KVX_FP4_GROUP 32

/* Paged blocks in 4 bits. [host] The rows of head h, K (w = 0) or V (w = 1), of block b make a plane at
 *     base + b*block_stride + h*head_stride + w*kv_stride        (strides in bytes)
 * of block_size rows of head_dim/2 bytes, and behind them block_size rows of head_dim/32 scale
 * bytes: kvx_fp4_plane_bytes() in all, filled up to a multiple of 16. With the planes of a block
 * side by side a block is one byte range, which kvx_pack, kvx_unpack, kvx_copy_direct and their like
 * move as it is, and with the heads outermost (head_stride = 2*plane, kv_stride = plane) their
 * head shards too (rows_per_block = 1). dtype is the 16-bit type (KVX_DTYPE_*) of the rows that the
 * calls below read and write beside it. The caller guarantees that every plane with b < num_blocks lies
 * inside the allocation. */
typedef struct kvx_fp4_cache {
  void* base;
  int64_t num_blocks;
  int64_t block_stride_bytes;
  int64_t kv_stride_bytes;
  int64_t head_stride_bytes;
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype;
} kvx_fp4_cache;

/* Bytes of one plane; -1 for a block_size below 1 or a head_dim that is no multiple of 32 up to
 * KVX_MAX_HEAD_DIM. [host] */
int64_t kvx_fp4_plane_bytes(int32_t block_size, int32_t head_dim);

/*
 * kvx_rope_and_cache_fp4 — kvx_rope_and_cache for a 4-bit cache: rotate the new tokens' queries
 * and keys by their positions, and write the rotated K row and the V row of each token into its slot,
 * quantised on the way. Arguments, positions, padding and errors as kvx_rope_and_cache. A rotated key is
 * formed in 64 bits and rounded once, to its 4-bit value (beyond the range of 32 bits it counts as infinite); a rotated
 * query as there.
 *   key_out, value_out  [num_tokens][num_kv_heads][head_dim] at the given strides, both or neither NULL: what
 *              the cache holds of each token, in the 16-bit type, for an attention over the new
 *              rows that sees them as later steps will. Written for tokens without a slot as
 *              well. They must not overlap each other, key or value.
 * Rows of neighbouring slots share no byte: tokens of a call may fill a block together.
 */
kvx_status kvx_rope_and_cache_fp4(const kvx_fp4_cache* cache, const void* query,
                                  int64_t query_token_stride_bytes, int64_t query_head_stride_bytes,
                                  int32_t num_heads, const void* key, int64_t key_token_stride_bytes,
                                  int64_t key_head_stride_bytes, const void* value,
                                  int64_t value_token_stride_bytes, int64_t value_head_stride_bytes,
                                  int64_t num_tokens, const int64_t* positions, int32_t num_axes,
                                  const int32_t* pair_axis, const float* inv_freq, int32_t rot_dim,
                                  int32_t interleaved, const int64_t* slot_mapping, void* query_out,
                                  int64_t out_token_stride_bytes, int64_t out_head_stride_bytes,
                                  void* key_out, int64_t key_out_token_stride_bytes,
                                  int64_t key_out_head_stride_bytes, void* value_out,
                                  int64_t value_out_token_stride_bytes,
                                  int64_t value_out_head_stride_bytes, int32_t* err_flag,
                                  hipStream_t stream);

/*
 * kvx_paged_attention_fp4 — kvx_paged_attention over a 4-bit cache. Arguments, what a row sees, rows
 * that see nothing, the workspace's use and errors as there. K's and V's values are taken in the
 * 16-bit type (see above).
 */
kvx_status kvx_paged_attention_fp4(const kvx_fp4_cache* cache, const kvx_batch* batch,
                                   const void* query, int64_t query_token_stride_bytes,
                                   int64_t query_head_stride_bytes, int32_t num_heads, float scale,
                                   int32_t causal, int64_t window, void* out,
                                   int64_t out_token_stride_bytes, int64_t out_head_stride_bytes,
                                   float* lse, void* workspace, int64_t workspace_bytes,
                                   int32_t* err_flag, hipStream_t stream);

/* Workspace bytes with which kvx_paged_attention_fp4 splits such a batch as far as pays (0: not at
 * all); -1 where it would refuse the sizes. [host] */
int64_t kvx_paged_attention_fp4_workspace(const kvx_fp4_cache* cache, const kvx_batch* batch,
                                          int32_t num_heads);

/*
 * kvx_pack_fp4 — kvx_pack that quantises: the listed blocks of all layers' 16-bit caches into
 * 4-bit blocks, 0.27 of the bytes to send. Block xfer.src_block + (p - xfer.buf_block) of layer l
 * becomes block l*total_blocks + p of `buffer`, for every run xfer and its positions p.
 *   cache        sizes, strides and type of each layer's cache; base is not used.
 *   layer_bases  DEVICE array [num_layers] of the layers' caches.
 *   xfers, xfer_count, total_blocks  a list from kvx_build_xfer_list in KVX_MODE_PACK or
 *                KVX_MODE_DIRECT, as for kvx_pack.
 *   buffer       the send buffer as 4-bit blocks, num_layers*total_blocks of them at least; sizes and
 *                type as the cache's.
 * Whole blocks are taken, unfilled slots with them. Runs outside the cache or the buffer are skipped and raise
 * KVX_DEVERR_BLOCK_RANGE. total_blocks == 0 or num_layers == 0 enqueues nothing. The received buffer goes into a
 * 4-bit cache with kvx_unpack, into 16-bit caches with kvx_unpack_fp4.
 */
kvx_status kvx_pack_fp4(const kvx_paged_cache* cache, void* const* layer_bases,
                        int32_t num_layers, const kvx_xfer* xfers, const int64_t* xfer_count,
                        int64_t total_blocks, const kvx_fp4_cache* buffer, int32_t* err_flag,
                        hipStream_t stream);

/*
 * kvx_unpack_fp4 — kvx_unpack from 4-bit blocks into 16-bit caches: block l*total_blocks + p of
 * `buffer` is written, in the cache's type, to block xfer.dst_block + (p - xfer.buf_block) of layer l.
 * Runs in KVX_MODE_UNPACK or KVX_MODE_DIRECT; other arguments as kvx_pack_fp4, ids and blocks
 * not listed as kvx_unpack.
 */
kvx_status kvx_unpack_fp4(const kvx_fp4_cache* buffer, const kvx_paged_cache* cache,
                          void* const* layer_bases, int32_t num_layers, const kvx_xfer* xfers,
                          const int64_t* xfer_count, int64_t total_blocks, int32_t* err_flag,
                          hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVX_FP4_H */
