// Entry points of kvx_attention.h: argument validation on the host, then the launches. As in
// kvx_api.hip, a bad call returns its status before any HIP call is made.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kvx_attention.h"
#include "kvx_attention_check.h"
#include "kvx_attention_launch.h"

extern "C" {

kvx_status kvx_rope_and_cache(const kvx_paged_cache* cache, const void* query,
                              int64_t query_token_stride_bytes, int64_t query_head_stride_bytes,
                              int32_t num_heads, const void* key, int64_t key_token_stride_bytes,
                              int64_t key_head_stride_bytes, const void* value,
                              int64_t value_token_stride_bytes, int64_t value_head_stride_bytes,
                              int64_t num_tokens, const int64_t* positions, int32_t num_axes,
                              const int32_t* pair_axis, const float* inv_freq, int32_t rot_dim,
                              int32_t interleaved, const int64_t* slot_mapping, void* query_out,
                              int64_t out_token_stride_bytes, int64_t out_head_stride_bytes,
                              int32_t* err_flag, hipStream_t stream) {
  kvx_status st = check_cache(cache);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  if (num_tokens < 0 || num_tokens > kMaxGroups || num_heads < 0 || num_heads > 65535 || num_axes < 1 ||
      num_axes > KVX_MAX_AXES || rot_dim < 16 || rot_dim > cache->head_dim || rot_dim % 16 != 0)
    return KVX_ERR_INVALID_ARGUMENT;
  const kvx_status rows[] = {
      check_rows(num_tokens, num_heads, query_token_stride_bytes, query_head_stride_bytes),
      check_rows(num_tokens, cache->num_kv_heads, key_token_stride_bytes, key_head_stride_bytes),
      check_rows(num_tokens, cache->num_kv_heads, value_token_stride_bytes, value_head_stride_bytes),
      check_rows(num_tokens, num_heads, out_token_stride_bytes, out_head_stride_bytes)};
  for (kvx_status s : rows) {
    if (s == KVX_ERR_INVALID_ARGUMENT) return s;
    if (s != KVX_SUCCESS) st = s;
  }
  if (!pair_axis) return KVX_ERR_INVALID_ARGUMENT;
  kvx::RopeArgs a = {};
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    if (pair_axis[i] < 0 || pair_axis[i] >= num_axes) return KVX_ERR_INVALID_ARGUMENT;
    a.pair_axis[i] = (uint8_t)pair_axis[i];
  }
  if (st != KVX_SUCCESS) return st;
  if (num_tokens == 0) return KVX_SUCCESS;
  if (!key || !value || !positions || !inv_freq || !slot_mapping || (num_heads > 0 && (!query || !query_out)) ||
      (cache->num_blocks > 0 && !cache->base))
    return KVX_ERR_INVALID_ARGUMENT;
  if (!aligned(query, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(query_out, 16) ||
      !aligned(cache->base, 16))
    return KVX_ERR_MISALIGNED;
  a.cache = *cache;
  a.query = {(const char*)query, query_token_stride_bytes, query_head_stride_bytes};
  a.key = {(const char*)key, key_token_stride_bytes, key_head_stride_bytes};
  a.value = {(const char*)value, value_token_stride_bytes, value_head_stride_bytes};
  a.out = {(const char*)query_out, out_token_stride_bytes, out_head_stride_bytes};
  a.num_heads = num_heads;
  a.rot_dim = rot_dim;
  a.num_axes = num_axes;
  a.num_tokens = num_tokens;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.slots = slot_mapping;
  a.err = err_flag;
  return from_hip(kvx::launch_rope(a, interleaved != 0, stream));
}

int64_t kvx_paged_attention_workspace(const kvx_paged_cache* cache, const kvx_batch* batch,
                                      int32_t num_heads) {
  if (check_attention(cache, batch, num_heads) != KVX_SUCCESS) return -1;
  if (batch->num_reqs == 0 || batch->num_tokens == 0) return 0;
  return kvx::attention_workspace(*cache, *batch, num_heads);
}

kvx_status kvx_paged_attention(const kvx_paged_cache* cache, const kvx_batch* batch,
                               const void* query, int64_t query_token_stride_bytes,
                               int64_t query_head_stride_bytes, int32_t num_heads, float scale,
                               int32_t causal, int64_t window, void* out,
                               int64_t out_token_stride_bytes, int64_t out_head_stride_bytes,
                               float* lse, void* workspace, int64_t workspace_bytes,
                               int32_t* err_flag, hipStream_t stream) {
  kvx_status st = check_attention(cache, batch, num_heads);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  if (!std::isfinite(scale) || !(scale > 0) || window < 0 || workspace_bytes < 0) return KVX_ERR_INVALID_ARGUMENT;
  for (kvx_status s : {check_rows(batch->num_tokens, num_heads, query_token_stride_bytes, query_head_stride_bytes),
                       check_rows(batch->num_tokens, num_heads, out_token_stride_bytes, out_head_stride_bytes)}) {
    if (s == KVX_ERR_INVALID_ARGUMENT) return s;
    if (s != KVX_SUCCESS) st = s;
  }
  if (st != KVX_SUCCESS) return st;
  if (batch->num_reqs == 0 || batch->num_tokens == 0) return KVX_SUCCESS;
  if (!query || !out || !batch_pointers(cache, batch)) return KVX_ERR_INVALID_ARGUMENT;
  if (!aligned(query, 16) || !aligned(out, 16) || !aligned(cache->base, 16) || !aligned(workspace, 16))
    return KVX_ERR_MISALIGNED;
  kvx::AttendArgs a = {};
  a.cache = *cache;
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
  return from_hip(kvx::launch_attention(a, stream));
}

kvx_status kvx_attention_mass(const kvx_paged_cache* cache, const kvx_batch* batch,
                              const void* query, int64_t query_token_stride_bytes,
                              int64_t query_head_stride_bytes, int32_t num_heads, float scale,
                              int32_t causal, int64_t window, const float* lse, float* mass,
                              int64_t mass_req_stride, int64_t mass_head_stride, int64_t mass_width,
                              int32_t* err_flag, hipStream_t stream) {
  kvx_status st = check_batch(cache, batch, num_heads);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  if (!std::isfinite(scale) || !(scale > 0) || window < 0 || mass_width < 0 ||
      !extent_ok(batch->num_reqs, mass_req_stride) || !extent_ok(cache->num_kv_heads, mass_head_stride) ||
      !extent_ok(1, mass_width))
    return KVX_ERR_INVALID_ARGUMENT;
  const kvx_status s = check_rows(batch->num_tokens, num_heads, query_token_stride_bytes, query_head_stride_bytes);
  if (s != KVX_SUCCESS) return s;
  if (st != KVX_SUCCESS) return st;
  if (batch->num_reqs == 0 || batch->num_tokens == 0 || mass_width == 0 || batch->max_blocks_per_req == 0)
    return KVX_SUCCESS;
  if (!query || !lse || !mass || !batch_pointers(cache, batch)) return KVX_ERR_INVALID_ARGUMENT;
  if (!aligned(query, 16) || !aligned(cache->base, 16)) return KVX_ERR_MISALIGNED;
  kvx::MassArgs m = {};
  m.at.cache = *cache;
  m.at.batch = *batch;
  m.at.query = {(const char*)query, query_token_stride_bytes, query_head_stride_bytes};
  m.at.num_heads = num_heads;
  m.at.causal = causal != 0;
  m.at.scale = scale;
  m.at.window = window > 0 && window < kInt32Max ? window : kInt32Max;
  m.at.lse = const_cast<float*>(lse);
  m.at.err = err_flag;
  m.mass = mass;
  m.mass_req_stride = mass_req_stride;
  m.mass_head_stride = mass_head_stride;
  m.mass_width = mass_width;
  return from_hip(kvx::launch_mass(m, stream));
}

kvx_status kvx_evict_select(const float* mass, int64_t mass_req_stride, int64_t mass_head_stride,
                            int64_t mass_width, int32_t num_reqs, int32_t num_heads,
                            const int64_t* context_lens, int64_t budget, int64_t sink,
                            int64_t recent, int32_t* keep, int64_t* new_lens, int32_t* err_flag,
                            hipStream_t stream) {
  if (num_reqs < 0 || num_heads < 1 || mass_width < 0 || mass_width > kInt32Max || budget < 1 || budget > kInt32Max ||
      sink < 0 || recent < 0 || sink > budget || recent > budget - sink || !extent_ok(num_reqs, mass_req_stride) ||
      !extent_ok(num_heads, mass_head_stride) || (int64_t)num_reqs * num_heads > kMaxGroups)
    return KVX_ERR_INVALID_ARGUMENT;
  if (num_reqs == 0) return KVX_SUCCESS;
  if ((!mass && mass_width > 0) || !context_lens || !keep || !new_lens || new_lens == context_lens)
    return KVX_ERR_INVALID_ARGUMENT;
  const kvx::SelectArgs a = {mass,        mass_req_stride, mass_head_stride, mass_width,
                             num_reqs,    num_heads,       context_lens,     (int32_t)budget,
                             (int32_t)sink, (int32_t)recent, keep,           new_lens, err_flag};
  return from_hip(kvx::launch_evict_select(a, stream));
}

kvx_status kvx_evict_compact(const kvx_paged_cache* cache, const int32_t* block_table,
                             int64_t max_blocks_per_req, int64_t bt_row_stride,
                             const int32_t* dst_block_table, int64_t dst_max_blocks_per_req,
                             int64_t dst_bt_row_stride, int32_t num_reqs, int32_t num_heads,
                             const int32_t* keep, int64_t budget, const float* mass,
                             int64_t mass_req_stride, int64_t mass_head_stride, int64_t mass_width,
                             float* mass_out, int64_t mass_out_req_stride,
                             int64_t mass_out_head_stride, int64_t mass_out_width,
                             int32_t* err_flag, hipStream_t stream) {
  const kvx_status st = check_cache(cache);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  if (num_reqs < 0 || num_heads < 1 || cache->num_kv_heads % num_heads != 0 || budget < 1 || budget > kInt32Max ||
      cache->num_blocks == 0 || max_blocks_per_req < 1 || dst_max_blocks_per_req < 1 ||
      !table_ok(num_reqs, max_blocks_per_req, bt_row_stride, cache->block_size) ||
      !table_ok(num_reqs, dst_max_blocks_per_req, dst_bt_row_stride, cache->block_size) ||
      (int64_t)num_reqs * (2 * cache->num_kv_heads + num_heads) > kMaxGroups || (mass == nullptr) != (mass_out == nullptr))
    return KVX_ERR_INVALID_ARGUMENT;
  if (mass && (mass_width < 0 || mass_width > kInt32Max || mass_out_width < 0 || mass_out_width > kInt32Max ||
               !extent_ok(num_reqs, mass_req_stride) || !extent_ok(num_heads, mass_head_stride) ||
               !extent_ok(num_reqs, mass_out_req_stride) || !extent_ok(num_heads, mass_out_head_stride)))
    return KVX_ERR_INVALID_ARGUMENT;
  // masses moved onto themselves need the ordered move, which the tables choose
  if (mass && mass == mass_out &&
      (block_table != dst_block_table || mass_req_stride != mass_out_req_stride ||
       mass_head_stride != mass_out_head_stride))
    return KVX_ERR_INVALID_ARGUMENT;
  if (st != KVX_SUCCESS) return st;
  if (num_reqs == 0) return KVX_SUCCESS;
  if (!block_table || !dst_block_table || !keep || !cache->base)
    return KVX_ERR_INVALID_ARGUMENT;
  // one table in place: its rows are read the same way on both sides
  if (block_table == dst_block_table &&
      (max_blocks_per_req != dst_max_blocks_per_req || bt_row_stride != dst_bt_row_stride))
    return KVX_ERR_INVALID_ARGUMENT;
  if (!aligned(cache->base, 16)) return KVX_ERR_MISALIGNED;
  kvx::CompactArgs a = {};
  a.cache = *cache;
  a.src_table = block_table;
  a.dst_table = dst_block_table;
  a.src_cols = max_blocks_per_req;
  a.src_row = bt_row_stride;
  a.dst_cols = dst_max_blocks_per_req;
  a.dst_row = dst_bt_row_stride;
  a.num_reqs = num_reqs;
  a.num_heads = num_heads;
  a.budget = (int32_t)budget;
  a.keep = keep;
  a.mass = mass;
  a.mass_out = mass_out;
  a.mass_req_stride = mass_req_stride;
  a.mass_head_stride = mass_head_stride;
  a.mass_width = mass_width;
  a.out_req_stride = mass_out_req_stride;
  a.out_head_stride = mass_out_head_stride;
  a.out_width = mass_out_width;
  a.err = err_flag;
  return from_hip(kvx::launch_evict_compact(a, stream));
}

}  // extern "C"
