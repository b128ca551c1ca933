// The launch shape of kvx_paged_attention, from the sizes of a call. Host code without any HIP call.
#pragma once

#include <stdint.h>

#include "kvx_attention.h"

namespace kvx {

// The launch shape of a batch: by slots (KEYS) where a request's rows of one KV head fit one tile of
// 32. Where the tiles alone do not fill the GPU with two workgroups a CU (kFill), or leave a decode
// batch's uneven contexts to a few rounds of workgroups, they are shared out evenly to kFill
// workgroups, of kMinSteps steps at least, if there is a workspace for the parts.
// The rule takes every request to be as long as the longest, and sharing ends where tiles fill the GPU once. What that costs: a
// chunk of 2304 tokens of 32 heads on 8 over 32768 slots makes 576 tiles, the last 64 of which run alone (1676 us; 2048 tokens
// 1071, 4096 2034); a decode over 131072 slots beside a chunk of 2048 tokens is one workgroup a KV head, in tiles of 128 rows (3351 us;
// without it 1200); 200 decodes of up to 4096 slots on one KV head are shared out and take 73 us, unshared 55.
constexpr int kFill = 512, kMinSteps = 4;
constexpr int64_t kRowsKeys = 32, kRows = 128;     // of a tile, by slots and otherwise
constexpr int64_t kMaxWorkgroups = (1 << 24) - 1;  // of 256 threads: a launch has fewer than 2^32
constexpr int64_t kMaxContext = 0x7fffffff;

struct Plan {
  bool keys;
  int32_t tiles, shares;
  int64_t busy;  // tiles that have rows, by the hints
};
inline Plan plan_attention(const kvx_paged_cache& c, const kvx_batch& b, int32_t num_heads) {
  const int64_t group = num_heads / c.num_kv_heads;
  const int64_t longest = b.max_query_len < b.num_tokens ? b.max_query_len : b.num_tokens;
  Plan p;
  // tiles of 32 rows also have to be few enough for a launch, as those of requests that keep to the hint are
  p.keys = longest * group <= kRowsKeys && (b.num_tokens * group / kRowsKeys + b.num_reqs) * c.num_kv_heads <= kMaxWorkgroups;
  const int64_t rows = p.keys ? kRowsKeys : kRows, slots = p.keys ? 128 : 64;
  p.tiles = (int32_t)(b.num_tokens * group / rows + b.num_reqs);
  int64_t busy = b.num_reqs * ((longest * group + rows - 1) / rows);
  if (busy > p.tiles) busy = p.tiles;
  if (busy < 1) busy = 1;
  const int64_t context = b.max_context_len < kMaxContext ? b.max_context_len : kMaxContext;
  const int fill = c.head_dim > 128 ? kFill / 2 : kFill;  // the widest heads' tiles leave room for one workgroup a CU
  int64_t shares = fill / c.num_kv_heads, most = busy * (context / slots) / kMinSteps;
  if (shares > most) shares = most;
  const bool uneven = busy * c.num_kv_heads < (p.keys ? 4 * fill : fill);
  p.busy = busy;
  p.shares = uneven && shares > (p.keys ? busy / 4 : busy) ? (int32_t)shares : 0;
  return p;
}

// Bytes of a slot: a part of one tile of every KV head.
inline int64_t slot_bytes(const kvx_paged_cache& c, bool keys) {
  return (int64_t)c.num_kv_heads * (keys ? kRowsKeys : kRows) * 4 * ((int64_t)c.head_dim + 1);
}

// The plan's shares in a workspace of so many bytes. One too small for the plan takes fewer, as long as they are more workgroups
// than the tiles would be without sharing: with as many, shares and tiles take about the same time, below that the GPU
// is left idle (16 requests of up to 8192 slots, 32 heads on 8: 100 us unshared, 534 with 2 shares, 157 with 8, 94 with
// 16, 76 with the plan's 64; 8 chunks of 517 tokens on one KV head: 249 unshared, 374 with 132, 211 with 264, 142 with 512).
inline int32_t shares_within(const Plan& p, const kvx_paged_cache& c, int64_t workspace_bytes) {
  const int64_t fit = workspace_bytes / slot_bytes(c, p.keys) - p.tiles;
  return p.shares <= fit ? p.shares : fit > p.busy ? (int32_t)fit : 0;
}

}  // namespace kvx
