// The launch shape of kvx_paged_attention_fp4, from the sizes of a call. Host code without any HIP call.
#pragma once

#include <stdint.h>

#include "kvx_attention.h"

namespace kvx {

// Times in this file are of whole calls, the join's launch among them, queued back to back on one stream.
//
// A request's rows of one KV head are taken 16 or 32 at a time, by four wavefronts that take 32 slots each of every 128, or, where there
// are more, 128 at a time, 64 slots a step, which reads a context once for up to 128 rows but widens it slower than 16-row tiles stream
// it. 32 requests of up to 8192 slots, 32 heads on 8, dimension 128: 1 token (4 rows) takes 44 us in tiles of 16 and 57 in tiles of 32;
// 8 tokens 67 in tiles of 32 and 108 in tiles of 128; 16 tokens, two tiles of 32, 93 and 115; 24 tokens 121 and 111 (at dimension 64 75
// and 81). At dimension 256, where a CU holds one tile of 128, 24 tokens 310 and 328, 32 tokens 377 and 334.
//
// Where the tiles do not fill the GPU, or are uneven, the batch's steps are shared out evenly (see Shares) to as many workgroups as the
// GPU holds, of 256 slots at least (with 512, one request of 8000 slots takes 19 us and not 17).
constexpr int kFp4Extra = 2;  // steps that the start of a tile of few rows counts for: the decode batch takes 44 us, with 0 46
constexpr int64_t kFp4MaxWorkgroups = (1 << 24) - 1;  // of 256 threads: a launch has fewer than 2^32

struct Fp4Plan {
  int32_t rows, slots;  // of a tile and a step
  int32_t tiles, shares;
  int64_t busy;  // tiles that have rows, by the hints
};
inline Fp4Plan plan_attention_fp4(const kvx_paged_cache& c, const kvx_batch& b, int32_t num_heads, int64_t window = INT64_MAX) {
  const int64_t group = num_heads / c.num_kv_heads;
  const int64_t longest = b.max_query_len < b.num_tokens ? b.max_query_len : b.num_tokens;
  const int dim = c.head_dim;
  Fp4Plan p;
  p.rows = longest * group <= 16 ? 16 : longest * group <= (dim > 128 ? 96 : 64) ? 32 : 128;
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
  // dimension 256 takes 76 us, with 768 95; one of 128 44 us, with 512 50 and with 1024 55; one of 64 30 us, with 768 31 and with 512 34;
  // 8 tokens of 256 149 us, with 512 159; of 128 67 us, with 768 83; of 64 44 us, with 512 51 and with 1024 54.
  const int64_t fill = p.rows == 16 ? (dim > 128 ? 512 : dim > 64 ? 768 : 1024) : dim > 128 ? 256 : few && dim <= 64 ? 768 : 512;
  int64_t shares = fill / c.num_kv_heads, most = busy * (context / 256), least = few ? busy / 4 : busy;
  if (shares > most) shares = most;
  // Tiles of 128 rows that fill the GPU, up to four times: shares take every tile of a request to be as long as its context, so only
  // where they nearly are (no prompts, no window), and the rounds come out uneven: by requests, or by a last round that is
  // part empty. 2304 tokens over 32768 slots, 32 heads on 8, take 1230 us and not 1678; 32 chunks of up to 517 over up to 9216, 8 heads on
  // one, 300 and not 392. Shared out all the same, 4096 tokens, two full rounds, would take 2112 us and not 1974, a prompt of 8192 275 and
  // not 195.
  const int64_t work = busy * c.num_kv_heads;
  bool uneven = work < (few ? 4 * fill : fill);
  if (!few && !uneven && work < 4 * fill && longest <= context / 4 && window >= context &&
      (b.num_reqs > 1 || 8 * work < 7 * ((work + fill - 1) / fill * fill))) {
    uneven = true;
    least = busy / 4;
  }
  // Where rows see few slots a second launch costs more than it spares: 8 requests of 896 slots, 32 heads on 8, take 13 us and shared
  // out 14 to 16, of 1024 14 and 14 to 16, of 1200 17 and 15 to 16; 13 requests of 5003 with a window of 256 take 11 and 16, with one of
  // 800 18.2 and 17.1 to 18.0, with one of 1024 20.4 and 18.2 to 19.0. One limit for both lies between what either would like.
  const bool few_slots = (context < window ? context : window) <= 896;
  p.busy = busy;
  p.shares = uneven && !few_slots && shares > least ? (int32_t)shares : 0;
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
