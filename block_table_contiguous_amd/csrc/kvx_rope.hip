// gfx950 kernel of kvx_rope_and_cache: rotate queries and keys, write K and V through the slots.
//
// One workgroup a token. Its first rot_dim/2 threads form the angles' cosines and sines once for
// all heads: position x inv_freq in 64 bits, reduced to a fraction of a turn there, because a
// 32-bit product is off by up to 1/16 of a radian at an angle of 2^20, by a whole one from 2^24 on and by 64 below 2^31;
// the functions themselves then take the fraction in 32 bits. The rows are moved as 16-byte vectors,
// a thread holding both halves of its pairs; each is read and written once, and that is the bound:
// HBM bytes for many tokens, one launch and two dependent loads for a few. The first rows are on their
// way while the angles are formed, and the next ones while a thread turns its own (9461
// tokens of 32 + 8 heads of 128: 233 MB in 45-47 us with the pairs half a rotation apart, 50 side by side, where a thread
// has one vector in flight and not two; 49-56 where only 64 or 16 of the dimensions turn). Stores go by the caches' default policy: the attention reads
// the rows next.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_launch.h"
#include "kvx_paged.h"

namespace kvx {
namespace {

constexpr int kRopeThreads = 256;

// What one thread moves at a time: a vector of whole pairs (INTERLEAVED), a pair of vectors half a
// rotation apart, or a vector that passes through.
struct Unit {
  u32x4 a, b;
  char* dst;
  int pair;  // first pair of the vector; < 0: passes through
};

template <class E, bool INTERLEAVED>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, BlockDiv div) {
  __shared__ float turn[KVX_MAX_HEAD_DIM];  // cos of pair i, then sin
  const int64_t t = blockIdx.x;
  const int half = a.rot_dim / 2;
  const kvx_paged_cache& cache = a.cache;
  const int64_t slot = a.slots[t];
  bool write = slot >= 0;
  char* row = nullptr;
  if (write) {
    const int64_t block = slot / div.size;
    if (block >= cache.num_blocks) {
      write = false;
      if (threadIdx.x == 0) raise(a.err, KVX_DEVERR_SLOT_RANGE);
    } else {
      row = (char*)cache.base + block * cache.block_stride_bytes +
            (slot - block * div.size) * cache.token_stride_bytes;
    }
  }
  const int vecs = cache.head_dim / 8;
  const int rot_units = INTERLEAVED ? a.rot_dim / 8 : a.rot_dim / 16;
  const int head_units = rot_units + (cache.head_dim - a.rot_dim) / 8;
  const int q_units = a.num_heads * head_units;
  const int k_units = write ? cache.num_kv_heads * head_units : 0;
  const int v_units = write ? cache.num_kv_heads * vecs : 0;
  const int units = q_units + k_units + v_units;
  auto load = [&](int u, Unit* x) {
    if (u >= q_units + k_units) {  // V
      const int y = u - q_units - k_units, h = y / vecs, c = y - h * vecs;
      x->dst = row + cache.kv_stride_bytes + h * cache.head_stride_bytes + c * 16;
      x->a = gload<u32x4>(a.value.base + t * a.value.token_stride + h * a.value.head_stride + c * 16);
      x->pair = -1;
      return;
    }
    const bool is_q = u < q_units;
    const int y = is_q ? u : u - q_units, h = y / head_units, c = y - h * head_units;
    const RowView& in = is_q ? a.query : a.key;
    const char* src = in.base + t * in.token_stride + h * in.head_stride;
    char* dst = is_q ? (char*)a.out.base + t * a.out.token_stride + h * a.out.head_stride
                     : row + h * cache.head_stride_bytes;
    const int off = c < rot_units ? c * 16 : a.rot_dim * 2 + (c - rot_units) * 16;
    x->pair = c < rot_units ? c * (INTERLEAVED ? 4 : 8) : -1;
    x->dst = dst + off;
    x->a = gload<u32x4>(src + off);
    if (!INTERLEAVED && c < rot_units) x->b = gload<u32x4>(src + half * 2 + off);
  };
  Unit x;
  const int first = threadIdx.x;
  if (first < units) load(first, &x);
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const int64_t pos = a.positions[a.pair_axis[i] * a.num_tokens + t];
    const double turns = (double)pos * (double)a.inv_freq[i] * 0.15915494309189533577;
    const float f = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * f, &s, &c);
    turn[i] = c;
    turn[half + i] = s;
  }
  __syncthreads();
  for (int u = first; u < units; u += kRopeThreads) {
    Unit y = x;
    if (u + kRopeThreads < units) load(u + kRopeThreads, &x);
    if (y.pair < 0) {
      gstore(y.dst, y.a);
    } else if constexpr (INTERLEAVED) {
      f32x8 v = widen<E>(y.a);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float cs = turn[y.pair + j], sn = turn[half + y.pair + j];
        const float p = v[2 * j], q = v[2 * j + 1];
        v[2 * j] = p * cs - q * sn;
        v[2 * j + 1] = q * cs + p * sn;
      }
      gstore(y.dst, narrow<E>(v));
    } else {
      f32x8 p = widen<E>(y.a), q = widen<E>(y.b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float cs = turn[y.pair + j], sn = turn[half + y.pair + j];
        const float x0 = p[j], y0 = q[j];
        p[j] = x0 * cs - y0 * sn;
        q[j] = y0 * cs + x0 * sn;
      }
      gstore(y.dst, narrow<E>(p));
      gstore(y.dst + half * 2, narrow<E>(q));
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, bool interleaved, hipStream_t stream) {
  const dim3 grid((unsigned)a.num_tokens), block(kRopeThreads);
  const BlockDiv div = block_div(a.cache.block_size);
  if (a.cache.dtype == KVX_DTYPE_BF16) {
    if (interleaved) rope_kernel<Bf16, true><<<grid, block, 0, stream>>>(a, div);
    else rope_kernel<Bf16, false><<<grid, block, 0, stream>>>(a, div);
  } else {
    if (interleaved) rope_kernel<Fp16, true><<<grid, block, 0, stream>>>(a, div);
    else rope_kernel<Fp16, false><<<grid, block, 0, stream>>>(a, div);
  }
  return hipGetLastError();
}

}  // namespace kvx
