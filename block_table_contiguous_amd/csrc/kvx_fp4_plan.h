// The launch shape of kvx_paged_attention_fp4, from the sizes of a call. Host code without any HIP call.
#pragma once

#include <stdint.h>

#include "kvx_attention.h"

namespace kvx {

// A request's rows of one KV head are taken 16 or 32 at a time, by four wavefronts that take 32 slots each of every 128, or, where there
// are more, 128 at a time, 64 slots a step. Where the tiles do not fill the GPU, or a decode batch's contexts are uneven, the
// batch's steps are shared out evenly (see Shares) to as many workgroups as the GPU holds, of 256 slots at least (with 512, one request of 8000 slots takes 18.1 us
// and not 16.1).
constexpr int kFp4Extra = 2;  // steps of 128 slots that the start of a tile of few rows counts for
constexpr int64_t kFp4MaxWorkgroups = (1 << 24) - 1;  // of 256 threads: a launch has fewer than 2^32

struct Fp4Plan {
  int32_t rows, slots;  // of a tile and a step
  int32_t tiles, shares;
  int64_t busy;  // tiles that have rows, by the hints
};
inline Fp4Plan plan_attention_fp4(const kvx_paged_cache& c, const kvx_batch& b, int32_t num_heads) {
  const int64_t group = num_heads / c.num_kv_heads;
  const int64_t longest = b.max_query_len < b.num_tokens ? b.max_query_len : b.num_tokens;
  Fp4Plan p;
  p.rows = longest * group <= 16 ? 16 : longest * group <= 32 ? 32 : 128;
  // tiles of few rows also have to be few enough for a launch, as those of requests that keep to the hint are
  if ((b.num_tokens * group / p.rows + b.num_reqs) * c.num_kv_heads > kFp4MaxWorkgroups) p.rows = 128;
  const bool few = p.rows < 128;
  p.slots = few ? 128 : 64;
  p.tiles = (int32_t)(b.num_tokens * group / p.rows + b.num_reqs);
  int64_t busy = b.num_reqs * ((longest * group + p.rows - 1) / p.rows);
  if (busy > p.tiles) busy = p.tiles;
  if (busy < 1) busy = 1;
  const int64_t context = b.max_context_len < 0x7fffffff ? b.max_context_len : 0x7fffffff;
  // The workgroups that the registers leave room for, 1 to 4 a CU. 32 requests of up to 8192 slots, 32 heads on 8: one token of
  // dimension 256 takes 82 us, with 768 158; 8 tokens of 128 66 us, with 768 84; one of 128 38 us, with 512 46 and with 1024 49; one of
  // 64 34 us, with 768 36.
  const int dim = c.head_dim;
  const int fill = p.rows == 16 ? (dim > 128 ? 512 : dim > 64 ? 768 : 1024) : dim > 128 ? 256 : few && dim <= 64 ? 768 : 512;
  int64_t shares = fill / c.num_kv_heads, most = busy * (context / 256);
  if (shares > most) shares = most;
  const bool uneven = busy * c.num_kv_heads < (few ? 4 * fill : fill);
  p.busy = busy;
  p.shares = uneven && shares > (few ? busy / 4 : busy) ? (int32_t)shares : 0;
  return p;
}

// Bytes of a slot: a part of one tile of every KV head.
inline int64_t fp4_slot_bytes(const Fp4Plan& p, const kvx_paged_cache& c) {
  return (int64_t)c.num_kv_heads * p.rows * 4 * ((int64_t)c.head_dim + 1);
}

// The plan's shares in a workspace of so many bytes: fewer where it is too small for them, as long as they are more
// workgroups than the tiles would be without sharing.
inline int32_t fp4_shares_within(const Fp4Plan& p, const kvx_paged_cache& c, int64_t workspace_bytes) {
  const int64_t fit = workspace_bytes / fp4_slot_bytes(p, c) - p.tiles;
  return p.shares <= fit ? p.shares : fit > p.busy ? (int32_t)fit : 0;
}

}  // namespace kvx
