// Prints the launch shape of kvx_paged_attention_fp4 for each line of sizes on standard input:
//   requests tokens max_query_len max_context_len heads kv_heads head_dim workspace
// workspace: bytes, or -1 for the full one, or -1-n for that of n slots. Output: rows of a tile, tiles, shares of the plan, shares
// within the workspace, workgroups that the launch without shares has work for, bytes of a slot.
#include <cstdio>

#include "kvx_fp4_plan.h"

int main() {
  long long reqs, tokens, query, context, heads, kv_heads, dim, bytes;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &reqs, &tokens, &query, &context, &heads, &kv_heads, &dim, &bytes) == 8) {
    kvx_paged_cache c = {};
    c.num_kv_heads = (int32_t)kv_heads;
    c.head_dim = (int32_t)dim;
    c.block_size = 16;
    kvx_batch b = {};
    b.num_reqs = (int32_t)reqs;
    b.num_tokens = tokens;
    b.max_query_len = query;
    b.max_context_len = context;
    const kvx::Fp4Plan p = kvx::plan_attention_fp4(c, b, (int32_t)heads);
    const int64_t slot = kvx::fp4_slot_bytes(p, c);
    const int64_t ws = bytes >= 0 ? bytes : bytes == -1 ? (p.shares + (int64_t)p.tiles) * slot : (-1 - bytes) * slot;
    const long long group = heads / kv_heads;
    // every request as long as the longest, but no more tiles than so many tokens can fill
    const long long each = reqs * ((query * group + p.rows - 1) / p.rows), most = tokens * group / p.rows + reqs;
    printf("%d %d %d %d %lld %lld\n", p.rows, p.tiles, p.shares, kvx::fp4_shares_within(p, c, ws), each < most ? each : most,
           (long long)slot);
  }
  return 0;
}
