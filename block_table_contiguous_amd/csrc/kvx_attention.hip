// gfx950 kernels of kvx_paged_attention and kvx_attention_mass.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_launch.h"
#include "kvx_paged.h"

namespace kvx {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// A token of the batch: its request, and the slots [lo, hi) it sees.
struct Token {
  int32_t r, lo, hi;
  bool used;
};

__device__ __forceinline__ int32_t context_of(const AttendArgs& a, int r, int32_t* errs) {
  const int64_t c = a.batch.context_lens[r], cap = a.batch.max_blocks_per_req * a.cache.block_size;
  const int64_t x = c < 0 ? 0 : c > cap ? cap : c;
  if (x != c) *errs |= KVX_DEVERR_TABLE_RANGE;
  return (int32_t)x;
}

// One workgroup of a launch looks every request's offsets over.
__device__ void check_offsets(const AttendArgs& a, int tid, int threads) {
  for (int r = tid; r < a.batch.num_reqs; r += threads) {
    const int64_t b = a.batch.q_offsets[r], e = a.batch.q_offsets[r + 1];
    if (b < 0 || e < b || e > a.batch.num_tokens) raise(a.err, KVX_DEVERR_OFFSETS);
  }
}

__device__ Token token_of(const AttendArgs& a, int64_t t, int32_t* errs) {
  int lo = 0, hi = a.batch.num_reqs;  // the last request that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.batch.q_offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t b = a.batch.q_offsets[lo], e = a.batch.q_offsets[lo + 1];
  Token k = {lo, 0, 0, t >= b && t < e};
  if (!k.used) return k;
  const int32_t c = context_of(a, lo, errs);
  const int64_t last = a.causal ? (int64_t)c - (e - t) : (int64_t)c - 1;
  k.hi = (int32_t)(last + 1 < 0 ? 0 : last + 1);
  const int64_t first = last - a.window + 1;
  k.lo = (int32_t)(first < 0 ? 0 : first);
  return k;
}

// One wavefront a query row, a slot at a time.
template <class E>
__global__ __launch_bounds__(64) void attend_simple(AttendArgs a, BlockDiv div) {
  const int64_t t = blockIdx.x / a.num_heads;
  const int h = blockIdx.x - t * a.num_heads, lane = threadIdx.x;
  int32_t errs = 0;
  if (blockIdx.x == 0) check_offsets(a, lane, 64);
  const Token k = token_of(a, t, &errs);
  if (!k.used) return;
  const int g = h / (a.num_heads / a.cache.num_kv_heads), vecs = a.cache.head_dim / 8;
  f32x8 q = {}, o = {};
  if (lane < vecs)
    q = widen<E>(gload<u32x4>(a.query.base + t * a.query.token_stride + h * a.query.head_stride + lane * 16));
  float m = -INFINITY, l = 0;
  for (int j = k.lo; j < k.hi; ++j) {
    const int b = block_of(div, j);
    const int64_t id = a.batch.block_table[k.r * a.batch.bt_row_stride + b];
    if (id < 0 || id >= a.cache.num_blocks) {
      errs |= KVX_DEVERR_BLOCK_RANGE;
      continue;
    }
    const char* row = (const char*)a.cache.base + id * a.cache.block_stride_bytes +
                      (int64_t)(j - b * div.size) * a.cache.token_stride_bytes + g * a.cache.head_stride_bytes;
    float s = 0;
    f32x8 v = {};
    if (lane < vecs) {
      const f32x8 kk = widen<E>(gload<u32x4>(row + lane * 16));
      v = widen<E>(gload<u32x4>(row + a.cache.kv_stride_bytes + lane * 16));
      for (int i = 0; i < 8; ++i) s += q[i] * kk[i];
    }
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    s *= a.scale * kLog2e;
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0 : top;
    const float p = exp2f(s - base), keep = exp2f(m - base);
    l = l * keep + p;
    for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + p * v[i];
    m = top;
  }
  const float inv = l == 0 ? 0 : 1 / l;
  if (lane < vecs) {
    for (int i = 0; i < 8; ++i) o[i] = l == 0 ? 0 : o[i] * inv;
    gstore((char*)a.out.base + t * a.out.token_stride + h * a.out.head_stride + lane * 16, narrow<E>(o));
  }
  if (a.lse && lane == 0) a.lse[t * a.num_heads + h] = l == 0 ? -INFINITY : (m + log2f(l)) / kLog2e;
  if (errs) raise(a.err, errs);
}

// One wavefront a slot of one KV head, a query row at a time.
template <class E>
__global__ __launch_bounds__(64) void mass_simple(MassArgs m, BlockDiv div) {
  const AttendArgs& a = m.at;
  const int r = blockIdx.z, g = blockIdx.y, lane = threadIdx.x;
  int32_t errs = 0;
  int64_t c = context_of(a, r, &errs);
  if (c > m.mass_width) {
    c = m.mass_width;
    errs |= KVX_DEVERR_TABLE_RANGE;
  }
  const int64_t b0 = a.batch.q_offsets[r], e0 = a.batch.q_offsets[r + 1];
  const int64_t b = b0 < 0 ? 0 : b0, e = e0 > a.batch.num_tokens ? a.batch.num_tokens : e0;
  if (b != b0 || e != e0 || e < b) errs |= KVX_DEVERR_OFFSETS;
  const int group = a.num_heads / a.cache.num_kv_heads, vecs = a.cache.head_dim / 8;
  for (int64_t j = blockIdx.x; j < c; j += gridDim.x) {
    const int blk = block_of(div, (int32_t)j);
    const int64_t id = a.batch.block_table[r * a.batch.bt_row_stride + blk];
    if (id < 0 || id >= a.cache.num_blocks) {
      errs |= KVX_DEVERR_BLOCK_RANGE;
      continue;
    }
    const char* row = (const char*)a.cache.base + id * a.cache.block_stride_bytes +
                      (int64_t)(j - (int64_t)blk * div.size) * a.cache.token_stride_bytes + g * a.cache.head_stride_bytes;
    f32x8 kk = {};
    if (lane < vecs) kk = widen<E>(gload<u32x4>(row + lane * 16));
    float total = 0;
    bool any = false;
    for (int64_t t = b; t < e; ++t) {
      const int64_t full = context_of(a, r, &errs);
      const int64_t last = a.causal ? full - (e - t) : full - 1;
      if (j > last || j <= last - a.window) continue;
      any = true;
      for (int i = 0; i < group; ++i) {
        const int h = g * group + i;
        const float lse = a.lse[t * a.num_heads + h];
        if (lse == -INFINITY) continue;
        float s = 0;
        if (lane < vecs) {
          const f32x8 q =
              widen<E>(gload<u32x4>(a.query.base + t * a.query.token_stride + h * a.query.head_stride + lane * 16));
          for (int x = 0; x < 8; ++x) s += q[x] * kk[x];
        }
        for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
        total += exp2f((s * a.scale - lse) * kLog2e);
      }
    }
    if (any && lane == 0) m.mass[r * m.mass_req_stride + g * m.mass_head_stride + j] += total;
  }
  if (errs && lane == 0) raise(a.err, errs);
}

}  // namespace

hipError_t launch_attention(const AttendArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.batch.num_tokens * a.num_heads));
  const BlockDiv div = block_div(a.cache.block_size);
  if (a.cache.dtype == KVX_DTYPE_BF16) attend_simple<Bf16><<<grid, 64, 0, stream>>>(a, div);
  else attend_simple<Fp16><<<grid, 64, 0, stream>>>(a, div);
  return hipGetLastError();
}

int64_t attention_workspace(const kvx_paged_cache&, const kvx_batch&, int32_t) { return 0; }

hipError_t launch_mass(const MassArgs& m, hipStream_t stream) {
  const kvx_batch& b = m.at.batch;
  const int64_t cap = b.max_blocks_per_req * m.at.cache.block_size;
  const dim3 grid((unsigned)(cap < m.mass_width ? cap : m.mass_width), m.at.cache.num_kv_heads, b.num_reqs);
  const BlockDiv div = block_div(m.at.cache.block_size);
  if (m.at.cache.dtype == KVX_DTYPE_BF16) mass_simple<Bf16><<<grid, 64, 0, stream>>>(m, div);
  else mass_simple<Fp16><<<grid, 64, 0, stream>>>(m, div);
  return hipGetLastError();
}

}  // namespace kvx
