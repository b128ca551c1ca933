/* Host-side argument validation of the calls of kvx_attention.h, driven from plain C and built with
 * AddressSanitizer and UndefinedBehaviorSanitizer (see build_attention.py): the entry points are
 * the library's, the launches behind them are stubs that count. A call that is refused, or has
 * nothing to do, must reach no launch; one that is right must reach exactly one. Pointers are real
 * host memory, which the library must not look into except where the header says [host]. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "kvx_attention.h"

extern int launches; /* attention_stub.cpp */

static unsigned char arena[1 << 16] __attribute__((aligned(256)));
#define P ((void*)(arena + 4096))
#define Q ((void*)(arena + 8192))
#define ODD ((void*)(arena + 4104))
#define NUL ((void*)0)

static int calls = 0, failures = 0;

static void expect(const char* what, kvx_status got, kvx_status want, int want_launches) {
  ++calls;
  if (got != want || launches != want_launches) {
    ++failures;
    printf("MISMATCH %s: got %d (%s), want %d; %d launches, want %d\n", what, (int)got, kvx_status_string(got),
           (int)want, launches, want_launches);
  }
  launches = 0;
}
#define REFUSED(what, call, want) expect(what, call, want, 0)
#define DONE(what, call) expect(what, call, KVX_SUCCESS, 1)
#define EMPTY(what, call) expect(what, call, KVX_SUCCESS, 0)

static kvx_paged_cache cache(void) {
  kvx_paged_cache c = {P, 100, 16384, 1024, 512, 256, 16, 2, 128, KVX_DTYPE_BF16};
  return c;
}
static kvx_batch batch(void) {
  kvx_batch b = {(const int32_t*)P, (const int64_t*)P, (const int64_t*)P, 8, 8, 5, 3, 128, 3};
  return b;
}
static kvx_status attend(kvx_paged_cache c, kvx_batch b, const void* q, int32_t heads, float scale, int64_t window,
                         void* out, int64_t out_stride, void* ws, int64_t ws_bytes) {
  return kvx_paged_attention(&c, &b, q, 2048, 256, heads, scale, 1, window, out, out_stride, 256, (float*)P, ws, ws_bytes,
                             NUL, NUL);
}
static kvx_status mass(kvx_paged_cache c, kvx_batch b, const void* q, void* lse, void* m, int64_t stride, int64_t width) {
  return kvx_attention_mass(&c, &b, q, 2048, 256, 4, 0.5f, 1, 0, (const float*)lse, (float*)m, stride, 500, width, NUL, NUL);
}
static kvx_status rope(kvx_paged_cache c, const void* q, const void* k, int64_t tokens, int32_t axes, const int32_t* axis,
                       int32_t rot, void* out) {
  return kvx_rope_and_cache(&c, q, 2048, 256, 4, k, 512, 256, P, 512, 256, tokens, (const int64_t*)P, axes, axis,
                            (const float*)P, rot, 0, (const int64_t*)P, out, 2048, 256, NUL, NUL);
}
static kvx_status choose(const void* m, int32_t reqs, const void* lens, int64_t budget, int64_t sink, int64_t recent,
                         void* new_lens) {
  return kvx_evict_select((const float*)m, 1000, 500, 500, reqs, 2, (const int64_t*)lens, budget, sink, recent, (int32_t*)P,
                          (int64_t*)new_lens, NUL, NUL);
}
static kvx_status move(kvx_paged_cache c, const void* src, const void* dst, int32_t reqs, int32_t heads, const void* m,
                       void* mo, int64_t mo_stride) {
  return kvx_evict_compact(&c, (const int32_t*)src, 8, 8, (const int32_t*)dst, 8, 8, reqs, heads, (const int32_t*)P, 100,
                           (const float*)m, 1000, 500, 500, (float*)mo, 1000, mo_stride, 500, NUL, NUL);
}

int main(void) {
  const kvx_status bad = KVX_ERR_INVALID_ARGUMENT, odd = KVX_ERR_MISALIGNED;
  kvx_paged_cache c = cache();
  kvx_batch b = batch();
  int32_t axis[128];
  for (int i = 0; i < 128; ++i) axis[i] = i % 3;

  DONE("attend", attend(c, b, P, 4, 0.1f, 0, Q, 2048, NUL, 0));
  DONE("attend, widest window", attend(c, b, P, 4, 0.1f, INT64_MAX, Q, 2048, NUL, 0));
  DONE("mass", mass(c, b, P, P, P, 1000, 500));
  DONE("rope", rope(c, P, P, 5, 3, axis, 128, Q));
  DONE("choose", choose(P, 3, P, 100, 4, 96, Q));
  DONE("move", move(c, P, Q, 3, 2, NUL, NUL, 500));
  DONE("move in place", move(c, P, P, 3, 1, P, P, 500));

  /* every size of a cache, at and past its ends */
  for (int k = 0; k < 14; ++k) {
    c = cache();
    kvx_status want = bad;
    switch (k) {
      case 0: c.num_blocks = -1; break;
      case 1: c.num_blocks = INT64_MAX; break;
      case 2: c.block_size = 0; break;
      case 3: c.block_size = INT32_MIN; break;
      case 4: c.num_kv_heads = 0; break;
      case 5: c.num_kv_heads = INT32_MAX; break;
      case 6: c.head_dim = KVX_MAX_HEAD_DIM + 8; break;
      case 7: c.dtype = 7; break;
      case 8: c.block_stride_bytes = INT64_MAX; break;
      case 9: c.token_stride_bytes = INT64_MIN; break;
      case 10: c.kv_stride_bytes = INT64_MAX; break;
      case 11: c.head_stride_bytes = INT64_MAX; break;
      case 12: c.head_dim = 12; want = odd; break;
      case 13: c.block_stride_bytes = 24; want = odd; break;
    }
    REFUSED("attend cache", attend(c, b, P, 4, 0.1f, 0, Q, 2048, NUL, 0), want);
    REFUSED("mass cache", mass(c, b, P, P, P, 1000, 500), want);
    if (k != 12) REFUSED("rope cache", rope(c, P, P, 5, 3, axis, 128, Q), want);
    REFUSED("move cache", move(c, P, Q, 3, 2, NUL, NUL, 500), want);
  }
  c = cache();
  for (int k = 0; k < 9; ++k) {
    b = batch();
    switch (k) {
      case 0: b.num_reqs = -1; break;
      case 1: b.num_reqs = INT32_MAX; break;
      case 2: b.num_tokens = INT64_MAX; break;
      case 3: b.num_tokens = -1; break;
      case 4: b.max_blocks_per_req = INT64_MAX; break;
      case 5: b.max_blocks_per_req = b.bt_row_stride = INT64_MAX / 2; break;
      case 6: b.max_query_len = -1; break;
      case 7: b.max_context_len = INT64_MIN; break;
      case 8: b.block_table = NUL; break;
    }
    REFUSED("attend batch", attend(c, b, P, 4, 0.1f, 0, Q, 2048, NUL, 0), bad);
    REFUSED("mass batch", mass(c, b, P, P, P, 1000, 500), bad);
  }
  b = batch();
  REFUSED("attend NaN scale", attend(c, b, P, 4, NAN, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend infinite scale", attend(c, b, P, 4, INFINITY, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend zero scale", attend(c, b, P, 4, 0.0f, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend heads", attend(c, b, P, 5, 0.1f, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend most heads", attend(c, b, P, INT32_MAX - 1, 0.1f, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend window", attend(c, b, P, 4, 0.1f, INT64_MIN, Q, 2048, NUL, 0), bad);
  REFUSED("attend no out", attend(c, b, P, 4, 0.1f, 0, NUL, 2048, NUL, 0), bad);
  REFUSED("attend odd out", attend(c, b, P, 4, 0.1f, 0, ODD, 2048, NUL, 0), odd);
  REFUSED("attend out stride", attend(c, b, P, 4, 0.1f, 0, Q, INT64_MAX, NUL, 0), bad);
  REFUSED("attend odd workspace", attend(c, b, P, 4, 0.1f, 0, Q, 2048, ODD, 64), odd);
  REFUSED("attend workspace bytes", attend(c, b, P, 4, 0.1f, 0, Q, 2048, P, -1), bad);
  REFUSED("mass no lse", mass(c, b, P, NUL, P, 1000, 500), bad);
  REFUSED("mass stride", mass(c, b, P, P, P, INT64_MAX, 500), bad);
  REFUSED("mass width", mass(c, b, P, P, P, 1000, INT64_MIN), bad);
  EMPTY("mass no width", mass(c, b, P, P, NUL, 1000, 0));
  b.num_tokens = 0;
  EMPTY("attend no tokens", attend(c, b, NUL, 4, 0.1f, 0, NUL, 2048, NUL, 0));
  b = batch();
  b.num_reqs = 0;
  EMPTY("attend no requests", attend(c, b, NUL, 4, 0.1f, 0, NUL, 2048, NUL, 0));
  REFUSED("attend null structs", kvx_paged_attention(NUL, NUL, P, 0, 0, 4, 1.0f, 0, 0, P, 0, 0, NUL, NUL, 0, NUL, NUL), bad);

  REFUSED("rope axes", rope(c, P, P, 5, 5, axis, 128, Q), bad);
  REFUSED("rope axis past the last", rope(c, P, P, 5, 2, axis, 128, Q), bad);
  REFUSED("rope no axis", rope(c, P, P, 5, 3, NUL, 128, Q), bad);
  REFUSED("rope past the head", rope(c, P, P, 5, 3, axis, 144, Q), bad);
  REFUSED("rope INT32_MIN", rope(c, P, P, 5, 3, axis, INT32_MIN, Q), bad);
  REFUSED("rope tokens", rope(c, P, P, INT64_MAX, 3, axis, 128, Q), bad);
  REFUSED("rope no key", rope(c, P, NUL, 5, 3, axis, 128, Q), bad);
  REFUSED("rope odd query", rope(c, ODD, P, 5, 3, axis, 128, Q), odd);
  EMPTY("rope no tokens", rope(c, NUL, NUL, 0, 3, axis, 128, NUL));

  REFUSED("choose budget", choose(P, 3, P, INT64_MAX, 4, 96, Q), bad);
  REFUSED("choose protected", choose(P, 3, P, 100, INT64_MAX, INT64_MAX, Q), bad);
  REFUSED("choose over itself", choose(P, 3, Q, 100, 4, 96, Q), bad);
  REFUSED("choose requests", choose(P, INT32_MAX, P, 100, 4, 96, Q), bad);
  EMPTY("choose no requests", choose(NUL, 0, NUL, 100, 4, 96, NUL));

  REFUSED("move heads", move(c, P, Q, 3, 3, NUL, NUL, 500), bad);
  REFUSED("move requests", move(c, P, Q, INT32_MAX, 2, NUL, NUL, 500), bad);
  REFUSED("move one mass", move(c, P, Q, 3, 2, P, NUL, 500), bad);
  REFUSED("move mass onto itself", move(c, P, Q, 3, 2, P, P, 500), bad);
  REFUSED("move mass strides", move(c, P, P, 3, 2, P, P, 400), bad);
  EMPTY("move no requests", move(c, NUL, NUL, 0, 2, NUL, NUL, 500));

  b = batch();
  if (kvx_paged_attention_workspace(&c, &b, 4) < 0 || kvx_paged_attention_workspace(&c, &b, 3) != -1 ||
      kvx_paged_attention_workspace(NUL, &b, 4) != -1)
    ++failures;
  printf("validated %d calls, %d mismatches\n", calls, failures);
  return failures != 0;
}
