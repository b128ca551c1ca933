// Entry points of kvx_fp4.h: argument validation on the host, then the launches. As in kvx_api.hip, a bad call
// returns its status before any HIP call is made.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kvx_attention_check.h"
#include "kvx_fp4.h"
#include "kvx_fp4_launch.h"

namespace {

bool fp4_sizes_ok(int32_t block_size, int32_t head_dim) {
  return block_size >= 1 && head_dim >= KVX_FP4_GROUP && head_dim <= KVX_MAX_HEAD_DIM && head_dim % KVX_FP4_GROUP == 0;
}

// The sizes of 4-bit blocks (not their pointer): ranges, then alignment.
kvx_status check_fp4(const kvx_fp4_cache* c) {
  if (!c || c->num_blocks < 0 || c->num_blocks > kInt32Max || !fp4_sizes_ok(c->block_size, c->head_dim) ||
      c->num_kv_heads < 1 || c->num_kv_heads > 65535 || (c->dtype != KVX_DTYPE_BF16 && c->dtype != KVX_DTYPE_FP16) ||
      !extent_ok(c->num_blocks, c->block_stride_bytes) || !extent_ok(1, c->kv_stride_bytes) ||
      !extent_ok(c->num_kv_heads, c->head_stride_bytes))
    return KVX_ERR_INVALID_ARGUMENT;
  if (!mult16(c->block_stride_bytes) || !mult16(c->kv_stride_bytes) || !mult16(c->head_stride_bytes))
    return KVX_ERR_MISALIGNED;
  return KVX_SUCCESS;
}

// A 4-bit cache in the terms of the 16-bit calls: rows of head_dim/2 bytes.
kvx_paged_cache paged(const kvx_fp4_cache& c) {
  return {c.base,     c.num_blocks,   c.block_stride_bytes, c.head_dim / 2, c.kv_stride_bytes, c.head_stride_bytes,
          c.block_size, c.num_kv_heads, c.head_dim,           c.dtype};
}

// check_attention of kvx_attention_check.h for a 4-bit cache.
kvx_status check_attention_fp4(const kvx_fp4_cache* c, const kvx_batch* b, int32_t num_heads) {
  const kvx_status st = check_fp4(c);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  const kvx_paged_cache as = paged(*c);
  const kvx_status s = check_attention(&as, b, num_heads);
  return s == KVX_SUCCESS ? st : s;
}

// The sizes of a transfer between 16-bit caches and 4-bit blocks.
kvx_status check_transfer(const kvx_paged_cache* c, const kvx_fp4_cache* b, int32_t num_layers, int64_t total_blocks) {
  kvx_status st = check_cache(c);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  const kvx_status s = check_fp4(b);
  if (s == KVX_ERR_INVALID_ARGUMENT) return s;
  if (s != KVX_SUCCESS) st = s;
  if (num_layers < 0 || total_blocks < 0 || total_blocks > kInt32Max || c->block_size != b->block_size ||
      c->head_dim != b->head_dim || c->num_kv_heads != b->num_kv_heads || c->dtype != b->dtype ||
      (int64_t)num_layers * total_blocks > b->num_blocks ||
      // a block's groups of 32 elements are numbered in 32 bits
      (int64_t)c->block_size * (c->head_dim / KVX_FP4_GROUP) > kInt32Max / (2 * c->num_kv_heads))
    return KVX_ERR_INVALID_ARGUMENT;
  // so are the pieces of 128 of them of a layer, of which a workgroup of 256 threads takes 8: a launch has fewer than 2^32 threads
  const int64_t pieces = ((int64_t)c->block_size * (c->head_dim / KVX_FP4_GROUP) * 2 * c->num_kv_heads + 127) / 128;
  if (total_blocks > ((1 << 27) - 8) / pieces) return KVX_ERR_INVALID_ARGUMENT;
  return st;
}

kvx_status transfer(bool pack, const kvx_paged_cache* c, void* const* layer_bases, int32_t num_layers, const kvx_xfer* xfers,
                    const int64_t* xfer_count, int64_t total_blocks, const kvx_fp4_cache* b, int32_t* err_flag,
                    hipStream_t stream) {
  const kvx_status st = check_transfer(c, b, num_layers, total_blocks);
  if (st != KVX_SUCCESS) return st;
  if (num_layers == 0 || total_blocks == 0) return KVX_SUCCESS;
  if (!layer_bases || !xfers || !xfer_count || !b->base) return KVX_ERR_INVALID_ARGUMENT;
  if (!aligned(b->base, 16) || !aligned(xfers, 16)) return KVX_ERR_MISALIGNED;
  const kvx::Fp4CopyArgs a = {*c, *b, layer_bases, num_layers, xfers, xfer_count, total_blocks, err_flag};
  return from_hip(pack ? kvx::launch_pack_fp4(a, stream) : kvx::launch_unpack_fp4(a, stream));
}

}  // namespace

extern "C" {

int64_t kvx_fp4_plane_bytes(int32_t block_size, int32_t head_dim) {
  if (!fp4_sizes_ok(block_size, head_dim)) return -1;
  return ((int64_t)block_size * (head_dim / 2 + head_dim / KVX_FP4_GROUP) + 15) & ~(int64_t)15;
}

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
                                  hipStream_t stream) {
  kvx_status st = check_fp4(cache);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  if (num_tokens < 0 || num_tokens > kMaxGroups || num_heads < 0 || num_heads > 65535 || num_axes < 1 ||
      num_axes > KVX_MAX_AXES || rot_dim < 16 || rot_dim > cache->head_dim || rot_dim % 16 != 0 ||
      (key_out == nullptr) != (value_out == nullptr))
    return KVX_ERR_INVALID_ARGUMENT;
  const int32_t kv = cache->num_kv_heads;
  const kvx_status rows[] = {check_rows(num_tokens, num_heads, query_token_stride_bytes, query_head_stride_bytes),
                             check_rows(num_tokens, kv, key_token_stride_bytes, key_head_stride_bytes),
                             check_rows(num_tokens, kv, value_token_stride_bytes, value_head_stride_bytes),
                             check_rows(num_tokens, num_heads, out_token_stride_bytes, out_head_stride_bytes),
                             check_rows(num_tokens, kv, key_out_token_stride_bytes, key_out_head_stride_bytes),
                             check_rows(num_tokens, kv, value_out_token_stride_bytes, value_out_head_stride_bytes)};
  for (kvx_status s : rows) {
    if (s == KVX_ERR_INVALID_ARGUMENT) return s;
    if (s != KVX_SUCCESS) st = s;
  }
  if (!pair_axis) return KVX_ERR_INVALID_ARGUMENT;
  kvx::Fp4RopeArgs a = {};
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    if (pair_axis[i] < 0 || pair_axis[i] >= num_axes) return KVX_ERR_INVALID_ARGUMENT;
    a.pair_axis[i] = (uint8_t)pair_axis[i];
  }
  if (st != KVX_SUCCESS) return st;
  if (num_tokens == 0) return KVX_SUCCESS;
  if (!key || !value || !positions || !inv_freq || !slot_mapping || (num_heads > 0 && (!query || !query_out)) ||
      (cache->num_blocks > 0 && !cache->base) || (key_out && (key_out == key || value_out == value || key_out == value_out)))
    return KVX_ERR_INVALID_ARGUMENT;
  for (const void* p : {query, key, value, (const void*)query_out, (const void*)key_out, (const void*)value_out,
                        (const void*)cache->base})
    if (!aligned(p, 16)) return KVX_ERR_MISALIGNED;
  a.cache = *cache;
  a.query = {(const char*)query, query_token_stride_bytes, query_head_stride_bytes};
  a.key = {(const char*)key, key_token_stride_bytes, key_head_stride_bytes};
  a.value = {(const char*)value, value_token_stride_bytes, value_head_stride_bytes};
  a.out = {(const char*)query_out, out_token_stride_bytes, out_head_stride_bytes};
  a.key_out = {(const char*)key_out, key_out_token_stride_bytes, key_out_head_stride_bytes};
  a.value_out = {(const char*)value_out, value_out_token_stride_bytes, value_out_head_stride_bytes};
  a.num_heads = num_heads;
  a.rot_dim = rot_dim;
  a.num_axes = num_axes;
  a.num_tokens = num_tokens;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.slots = slot_mapping;
  a.err = err_flag;
  return from_hip(kvx::launch_rope_fp4(a, interleaved != 0, stream));
}

int64_t kvx_paged_attention_fp4_workspace(const kvx_fp4_cache* cache, const kvx_batch* batch,
                                          int32_t num_heads) {
  if (check_attention_fp4(cache, batch, num_heads) != KVX_SUCCESS) return -1;
  if (batch->num_reqs == 0 || batch->num_tokens == 0) return 0;
  return kvx::attention_fp4_workspace(paged(*cache), *batch, num_heads);
}

kvx_status kvx_paged_attention_fp4(const kvx_fp4_cache* cache, const kvx_batch* batch,
                                   const void* query, int64_t query_token_stride_bytes,
                                   int64_t query_head_stride_bytes, int32_t num_heads, float scale,
                                   int32_t causal, int64_t window, void* out,
                                   int64_t out_token_stride_bytes, int64_t out_head_stride_bytes,
                                   float* lse, void* workspace, int64_t workspace_bytes,
                                   int32_t* err_flag, hipStream_t stream) {
  kvx_status st = check_attention_fp4(cache, batch, num_heads);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  if (!std::isfinite(scale) || !(scale > 0) || window < 0 || workspace_bytes < 0) return KVX_ERR_INVALID_ARGUMENT;
  for (kvx_status s : {check_rows(batch->num_tokens, num_heads, query_token_stride_bytes, query_head_stride_bytes),
                       check_rows(batch->num_tokens, num_heads, out_token_stride_bytes, out_head_stride_bytes)}) {
    if (s == KVX_ERR_INVALID_ARGUMENT) return s;
    if (s != KVX_SUCCESS) st = s;
  }
  if (st != KVX_SUCCESS) return st;
  if (batch->num_reqs == 0 || batch->num_tokens == 0) return KVX_SUCCESS;
  const kvx_paged_cache as = paged(*cache);
  if (!query || !out || !batch_pointers(&as, batch)) return KVX_ERR_INVALID_ARGUMENT;
  if (!aligned(query, 16) || !aligned(out, 16) || !aligned(cache->base, 16) || !aligned(workspace, 16))
    return KVX_ERR_MISALIGNED;
  kvx::AttendArgs a = {};
  a.cache = as;
  a.batch = *batch;
  a.query = {(const char*)query, query_token_stride_bytes, query_head_stride_bytes};
  a.out = {(const char*)out, out_token_stride_bytes, out_head_stride_bytes};
  a.num_heads = num_heads;
  a.causal = causal != 0;
  a.scale = scale;
  a.window = window > 0 && window < kInt32Max ? window : kInt32Max;
  a.lse = lse;
  a.workspace = workspace;
  a.workspace_bytes = workspace ? workspace_bytes : 0;
  a.err = err_flag;
  return from_hip(kvx::launch_attention_fp4(a, stream));
}

kvx_status kvx_pack_fp4(const kvx_paged_cache* cache, void* const* layer_bases,
                        int32_t num_layers, const kvx_xfer* xfers, const int64_t* xfer_count,
                        int64_t total_blocks, const kvx_fp4_cache* buffer, int32_t* err_flag,
                        hipStream_t stream) {
  return transfer(true, cache, layer_bases, num_layers, xfers, xfer_count, total_blocks, buffer, err_flag, stream);
}

kvx_status kvx_unpack_fp4(const kvx_fp4_cache* buffer, const kvx_paged_cache* cache,
                          void* const* layer_bases, int32_t num_layers, const kvx_xfer* xfers,
                          const int64_t* xfer_count, int64_t total_blocks, int32_t* err_flag,
                          hipStream_t stream) {
  return transfer(false, cache, layer_bases, num_layers, xfers, xfer_count, total_blocks, buffer, err_flag, stream);
}

}  // extern "C"
