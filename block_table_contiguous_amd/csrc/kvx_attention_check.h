// What the entry points of kvx_attention.h and kvx_fp4.h look over on the host before anything is enqueued.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention.h"
#include "kvx_attention_plan.h"

namespace {

constexpr int64_t kInt32Max = 0x7fffffff;
constexpr int64_t kMaxRows = kInt32Max - 65536;  // query rows times heads: the rows of a few tiles past the last are counted too
constexpr int64_t kMaxGroups = (1 << 22) - 1;  // workgroups along a grid dimension, up to 1024 threads each

inline kvx_status from_hip(hipError_t e) { return e == hipSuccess ? KVX_SUCCESS : KVX_ERR_HIP; }
inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
inline bool mult16(int64_t v) { return (v & 15) == 0; }

// count x bytes stays within KVX_MAX_EXTENT_BYTES, so that no offset a kernel forms overflows.
inline bool extent_ok(int64_t count, int64_t bytes) {
  return count >= 0 && bytes >= 0 && (count == 0 || bytes <= KVX_MAX_EXTENT_BYTES / count);
}

// The sizes of a cache (not its pointer): ranges, then alignment.
kvx_status check_cache(const kvx_paged_cache* c) {
  if (!c || c->num_blocks < 0 || c->num_blocks > kInt32Max || c->block_size < 1 || c->num_kv_heads < 1 ||
      c->num_kv_heads > 65535 || c->head_dim < 8 || c->head_dim > KVX_MAX_HEAD_DIM ||
      (c->dtype != KVX_DTYPE_BF16 && c->dtype != KVX_DTYPE_FP16) ||
      !extent_ok(c->num_blocks, c->block_stride_bytes) || !extent_ok(c->block_size, c->token_stride_bytes) ||
      !extent_ok(1, c->kv_stride_bytes) || !extent_ok(c->num_kv_heads, c->head_stride_bytes))
    return KVX_ERR_INVALID_ARGUMENT;
  if (c->head_dim % 8 != 0 || !mult16(c->block_stride_bytes) || !mult16(c->token_stride_bytes) ||
      !mult16(c->kv_stride_bytes) || !mult16(c->head_stride_bytes))
    return KVX_ERR_MISALIGNED;
  return KVX_SUCCESS;
}

// A block table's shape; slots of a request, and those of a few tiles behind them, stay below 2^31.
bool table_ok(int64_t reqs, int64_t cols, int64_t row, int32_t block_size) {
  return cols >= 0 && row >= cols && extent_ok(reqs, row) && cols <= (kInt32Max - 65536) / block_size;
}

kvx_status check_rows(int64_t tokens, int64_t heads, int64_t token_stride, int64_t head_stride) {
  if (!extent_ok(tokens, token_stride) || !extent_ok(heads, head_stride)) return KVX_ERR_INVALID_ARGUMENT;
  if (!mult16(token_stride) || !mult16(head_stride)) return KVX_ERR_MISALIGNED;
  return KVX_SUCCESS;
}

// The sizes of a batch and the heads that attend.
kvx_status check_batch(const kvx_paged_cache* c, const kvx_batch* b, int32_t num_heads) {
  const kvx_status st = check_cache(c);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  if (!b || b->num_reqs < 0 || b->num_reqs > 65535 || b->num_tokens < 0 || b->max_query_len < 0 ||
      b->max_context_len < 0 || num_heads < 1 || num_heads % c->num_kv_heads != 0 ||
      !table_ok(b->num_reqs, b->max_blocks_per_req, b->bt_row_stride, c->block_size) ||
      b->num_tokens > kMaxRows / num_heads || (int64_t)b->num_reqs * c->num_kv_heads > kMaxGroups)
    return KVX_ERR_INVALID_ARGUMENT;
  return st;
}

// check_batch for attention, which launches a workgroup a tile of rows.
kvx_status check_attention(const kvx_paged_cache* c, const kvx_batch* b, int32_t num_heads) {
  const kvx_status st = check_batch(c, b, num_heads);
  if (st == KVX_ERR_INVALID_ARGUMENT) return st;
  const int64_t rows = b->num_tokens * num_heads, least = kvx::kRows * (int64_t)b->num_reqs * c->num_kv_heads;
  return rows <= kMaxRows - least ? st : KVX_ERR_INVALID_ARGUMENT;
}

bool batch_pointers(const kvx_paged_cache* c, const kvx_batch* b) {
  return b->q_offsets && b->context_lens && (b->max_blocks_per_req == 0 || b->block_table) &&
         (b->max_blocks_per_req == 0 || c->num_blocks == 0 || c->base);
}

}  // namespace
