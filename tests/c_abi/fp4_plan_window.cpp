// Prints the launch shape of kvx_paged_attention_fp4 with a window for each line of sizes on standard input:
//   requests tokens max_query_len max_context_len heads kv_heads head_dim window
// Output: rows of a tile, tiles, shares, bytes of a workspace that holds the parts of these, and bytes of the one that is planned
// without a window.
#include <cstdio>

#include "kvx_fp4_plan.h"

int main() {
  long long reqs, tokens, query, context, heads, kv_heads, dim, window;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &reqs, &tokens, &query, &context, &heads, &kv_heads, &dim, &window) == 8) {
    kvx_paged_cache c = {};
    c.num_kv_heads = (int32_t)kv_heads;
    c.head_dim = (int32_t)dim;
    c.block_size = 16;
    kvx_batch b = {};
    b.num_reqs = (int32_t)reqs;
    b.num_tokens = tokens;
    b.max_query_len = query;
    b.max_context_len = context;
    const kvx::Fp4Plan p = kvx::plan_attention_fp4(c, b, (int32_t)heads, window), q = kvx::plan_attention_fp4(c, b, (int32_t)heads);
    auto bytes = [&](const kvx::Fp4Plan& x) -> long long {
      return x.shares > 0 ? (x.shares + (int64_t)x.tiles) * kvx::fp4_slot_bytes(x, c) : 0;
    };
    printf("%d %d %d %lld %lld\n", p.rows, p.tiles, p.shares, bytes(p), bytes(q));
  }
  return 0;
}
