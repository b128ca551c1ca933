/* Host-side argument validation of the calls of kvx_fp4.h, driven from plain C and built with
 * AddressSanitizer and UndefinedBehaviorSanitizer (see build_fp4.py): the entry points are the
 * library's, the launches behind them are stubs that count. A call that is refused, or has
 * nothing to do, must reach no launch; one that is right must reach exactly one. Pointers are real
 * host memory, which the library must not look into except where the header says [host]. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "kvx_fp4.h"

extern int launches; /* fp4_stub.cpp */

static unsigned char arena[1 << 16] __attribute__((aligned(256)));
#define P ((void*)(arena + 4096))
#define Q ((void*)(arena + 8192))
#define R ((void*)(arena + 12288))
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

static kvx_fp4_cache cache(void) {
  kvx_fp4_cache c = {P, 100, 4352, 1088, 2176, 16, 2, 128, KVX_DTYPE_BF16};
  return c;
}
static kvx_paged_cache wide(void) {
  kvx_paged_cache c = {NUL, 100, 16384, 1024, 512, 256, 16, 2, 128, KVX_DTYPE_BF16};
  return c;
}
static kvx_batch batch(void) {
  kvx_batch b = {(const int32_t*)P, (const int64_t*)P, (const int64_t*)P, 8, 8, 5, 3, 128, 3};
  return b;
}
static kvx_status attend(kvx_fp4_cache c, kvx_batch b, const void* q, int32_t heads, float scale, int64_t window,
                         void* out, int64_t out_stride, void* ws, int64_t ws_bytes) {
  return kvx_paged_attention_fp4(&c, &b, q, 2048, 256, heads, scale, 1, window, out, out_stride, 256, (float*)P, ws, ws_bytes,
                                 NUL, NUL);
}
static kvx_status rope(kvx_fp4_cache c, const void* q, const void* k, int64_t tokens, int32_t axes, const int32_t* axis,
                       int32_t rot, void* out, void* ko, int64_t ko_stride, void* vo) {
  return kvx_rope_and_cache_fp4(&c, q, 2048, 256, 4, k, 512, 256, P, 512, 256, tokens, (const int64_t*)P, axes, axis,
                                (const float*)P, rot, 0, (const int64_t*)P, out, 2048, 256, ko, ko_stride, 256, vo, 512, 256,
                                NUL, NUL);
}
static kvx_status pack(kvx_paged_cache c, kvx_fp4_cache f, void* bases, int32_t layers, const void* runs, int64_t blocks) {
  return kvx_pack_fp4(&c, (void* const*)bases, layers, (const kvx_xfer*)runs, (const int64_t*)P, blocks, &f, NUL, NUL);
}
static kvx_status unpack(kvx_paged_cache c, kvx_fp4_cache f, void* bases, int32_t layers, const void* runs, int64_t blocks) {
  return kvx_unpack_fp4(&f, &c, (void* const*)bases, layers, (const kvx_xfer*)runs, (const int64_t*)P, blocks, NUL, NUL);
}

int main(void) {
  const kvx_status bad = KVX_ERR_INVALID_ARGUMENT, odd = KVX_ERR_MISALIGNED;
  kvx_fp4_cache c = cache();
  kvx_paged_cache w = wide();
  kvx_batch b = batch();
  int32_t axis[128];
  for (int i = 0; i < 128; ++i) axis[i] = i % 3;

  DONE("attend", attend(c, b, P, 4, 0.1f, 0, Q, 2048, NUL, 0));
  DONE("attend, widest window", attend(c, b, P, 4, 0.1f, INT64_MAX, Q, 2048, NUL, 0));
  DONE("rope", rope(c, P, Q, 5, 3, axis, 128, Q, NUL, 0, NUL));
  DONE("rope with what is held", rope(c, P, Q, 5, 3, axis, 128, Q, R, 512, (void*)(arena + 16384)));
  DONE("pack", pack(w, c, P, 2, P, 50));
  DONE("unpack", unpack(w, c, P, 2, P, 50));

  /* every size of 4-bit blocks, at and past its ends */
  for (int k = 0; k < 13; ++k) {
    c = cache();
    kvx_status want = bad;
    switch (k) {
      case 0: c.num_blocks = -1; break;
      case 1: c.num_blocks = INT64_MAX; break;
      case 2: c.block_size = 0; break;
      case 3: c.block_size = INT32_MIN; break;
      case 4: c.num_kv_heads = 0; break;
      case 5: c.num_kv_heads = INT32_MAX; break;
      case 6: c.head_dim = KVX_MAX_HEAD_DIM + 32; break;
      case 7: c.head_dim = 72; break;
      case 8: c.dtype = 7; break;
      case 9: c.block_stride_bytes = INT64_MAX; break;
      case 10: c.kv_stride_bytes = INT64_MIN; break;
      case 11: c.head_stride_bytes = INT64_MAX; break;
      case 12: c.block_stride_bytes = 24; want = odd; break;
    }
    REFUSED("attend cache", attend(c, b, P, 4, 0.1f, 0, Q, 2048, NUL, 0), want);
    REFUSED("rope cache", rope(c, P, Q, 5, 3, axis, 64, Q, NUL, 0, NUL), want);
    REFUSED("pack buffer", pack(w, c, P, 2, P, 50), want);
    REFUSED("unpack buffer", unpack(w, c, P, 2, P, 50), want);
  }
  c = cache();
  c.block_size = INT32_MAX;
  DONE("attend, one endless block", attend(c, (b.max_blocks_per_req = 0, b), P, 4, 0.1f, 0, Q, 2048, NUL, 0));
  b = batch();
  REFUSED("attend, endless blocks", attend(c, b, P, 4, 0.1f, 0, Q, 2048, NUL, 0), bad);
  w.block_size = INT32_MAX;
  REFUSED("pack, endless blocks", pack(w, c, P, 2, P, 50), bad);
  c = cache();
  w = wide();
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
  }
  b = batch();
  REFUSED("attend NaN scale", attend(c, b, P, 4, NAN, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend zero scale", attend(c, b, P, 4, 0.0f, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend heads", attend(c, b, P, 5, 0.1f, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend most heads", attend(c, b, P, INT32_MAX - 1, 0.1f, 0, Q, 2048, NUL, 0), bad);
  REFUSED("attend window", attend(c, b, P, 4, 0.1f, INT64_MIN, Q, 2048, NUL, 0), bad);
  REFUSED("attend no out", attend(c, b, P, 4, 0.1f, 0, NUL, 2048, NUL, 0), bad);
  REFUSED("attend odd out", attend(c, b, P, 4, 0.1f, 0, ODD, 2048, NUL, 0), odd);
  REFUSED("attend out stride", attend(c, b, P, 4, 0.1f, 0, Q, INT64_MAX, NUL, 0), bad);
  REFUSED("attend odd workspace", attend(c, b, P, 4, 0.1f, 0, Q, 2048, ODD, 64), odd);
  REFUSED("attend workspace bytes", attend(c, b, P, 4, 0.1f, 0, Q, 2048, P, -1), bad);
  b.num_tokens = 0;
  EMPTY("attend no tokens", attend(c, b, NUL, 4, 0.1f, 0, NUL, 2048, NUL, 0));
  b = batch();
  b.num_reqs = 0;
  EMPTY("attend no requests", attend(c, b, NUL, 4, 0.1f, 0, NUL, 2048, NUL, 0));
  REFUSED("attend null structs", kvx_paged_attention_fp4(NUL, NUL, P, 0, 0, 4, 1.0f, 0, 0, P, 0, 0, NUL, NUL, 0, NUL, NUL), bad);
  b = batch();
  REFUSED("attend null batch", kvx_paged_attention_fp4(&c, NUL, P, 0, 0, 4, 1.0f, 0, 0, P, 0, 0, NUL, NUL, 0, NUL, NUL), bad);

  REFUSED("rope axes", rope(c, P, Q, 5, 5, axis, 128, Q, NUL, 0, NUL), bad);
  REFUSED("rope axis past the last", rope(c, P, Q, 5, 2, axis, 128, Q, NUL, 0, NUL), bad);
  REFUSED("rope no axis", rope(c, P, Q, 5, 3, NUL, 128, Q, NUL, 0, NUL), bad);
  REFUSED("rope past the head", rope(c, P, Q, 5, 3, axis, 144, Q, NUL, 0, NUL), bad);
  REFUSED("rope INT32_MIN", rope(c, P, Q, 5, 3, axis, INT32_MIN, Q, NUL, 0, NUL), bad);
  REFUSED("rope tokens", rope(c, P, Q, INT64_MAX, 3, axis, 128, Q, NUL, 0, NUL), bad);
  REFUSED("rope no key", rope(c, P, NUL, 5, 3, axis, 128, Q, NUL, 0, NUL), bad);
  REFUSED("rope odd query", rope(c, ODD, Q, 5, 3, axis, 128, Q, NUL, 0, NUL), odd);
  REFUSED("rope half of what is held", rope(c, P, Q, 5, 3, axis, 128, Q, R, 512, NUL), bad);
  REFUSED("rope over the key", rope(c, P, Q, 5, 3, axis, 128, Q, Q, 512, R), bad);
  REFUSED("rope stride of what is held", rope(c, P, Q, 5, 3, axis, 128, Q, R, INT64_MAX, (void*)(arena + 16384)), bad);
  REFUSED("rope odd stride of what is held", rope(c, P, Q, 5, 3, axis, 128, Q, R, 520, (void*)(arena + 16384)), odd);
  EMPTY("rope no tokens", rope(c, NUL, NUL, 0, 3, axis, 128, NUL, NUL, 0, NUL));

  for (int k = 0; k < 2; ++k) {
    kvx_status (*fn)(kvx_paged_cache, kvx_fp4_cache, void*, int32_t, const void*, int64_t) = k ? unpack : pack;
    REFUSED("transfer layers", fn(w, c, P, -1, P, 50), bad);
    REFUSED("transfer most layers", fn(w, c, P, INT32_MAX, P, 50), bad);
    REFUSED("transfer blocks", fn(w, c, P, 2, P, INT64_MAX), bad);
    REFUSED("transfer too many", fn(w, c, P, 2, P, 51), bad);
    REFUSED("transfer no bases", fn(w, c, NUL, 2, P, 50), bad);
    REFUSED("transfer odd list", fn(w, c, P, 2, ODD, 50), odd);
    EMPTY("transfer nothing", fn(w, c, NUL, 0, NUL, 50));
    w.dtype = KVX_DTYPE_FP16;
    REFUSED("transfer types", fn(w, c, P, 2, P, 50), bad);
    w = wide();
    w.num_kv_heads = INT32_MAX;
    REFUSED("transfer heads", fn(w, c, P, 2, P, 50), bad);
    w = wide();
    w.head_stride_bytes = 24;
    REFUSED("transfer odd heads", fn(w, c, P, 2, P, 50), odd);
    w = wide();
  }
  REFUSED("pack null structs", kvx_pack_fp4(NUL, P, 2, P, P, 50, NUL, NUL, NUL), bad);
  REFUSED("unpack null structs", kvx_unpack_fp4(NUL, NUL, P, 2, P, P, 50, NUL, NUL), bad);

  if (kvx_paged_attention_fp4_workspace(&c, &b, 4) < 0 || kvx_paged_attention_fp4_workspace(&c, &b, 3) != -1 ||
      kvx_paged_attention_fp4_workspace(NUL, &b, 4) != -1 || kvx_fp4_plane_bytes(16, 128) != 1088 ||
      kvx_fp4_plane_bytes(INT32_MIN, 128) != -1 || kvx_fp4_plane_bytes(INT32_MAX, 256) < 0)
    ++failures;
  printf("validated %d calls, %d mismatches\n", calls, failures);
  return failures != 0;
}
