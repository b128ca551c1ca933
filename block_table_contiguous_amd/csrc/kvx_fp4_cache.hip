// gfx950 kernels that bring rows into the 4-bit form and back: kvx_rope_and_cache_fp4, kvx_pack_fp4, kvx_unpack_fp4.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_fp4_format.h"
#include "kvx_fp4_launch.h"

namespace kvx {
namespace {

// --------------------------------------------------------------------------------------
// the write of rotated new rows
// --------------------------------------------------------------------------------------

constexpr int kRopeThreads = 256;

// A 64-bit number to 32 bits so that a later rounding to fewer bits is as if it were the only one: toward zero, with the
// last bit set where anything was cut off (no value that the 4-bit rounding or the scale's bound breaks at has it set).
__device__ __forceinline__ float sticky(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x), low = b & 0x1fffffffull;
  return (float)__builtin_bit_cast(double, (b ^ low) | (low ? 0x20000000ull : 0));
}

// One workgroup a token. Its first rot_dim/2 threads form the angles' cosines and sines once, in 64 bits: a rotated key is rounded
// to 4 bits, and 32 bits on the way there would decide some of the elements next to a border between two codes.
// The rows of q are then moved as 16-byte vectors, turned in 32 bits; of K and V four neighbouring lanes hold a group
// of 32 elements, eight each, with the partners of the eight read beside them.
template <class E, bool INTERLEAVED>
__global__ __launch_bounds__(kRopeThreads) void rope_fp4_kernel(Fp4RopeArgs a, BlockDiv div) {
  __shared__ double turn[KVX_MAX_HEAD_DIM];  // cos of pair i, then sin
  const int64_t t = blockIdx.x;
  const int half = a.rot_dim / 2, dim = a.cache.head_dim, vecs = dim / 8;
  const kvx_fp4_cache& cache = a.cache;
  const int64_t slot = a.slots[t];
  char* block = nullptr;  // of the slot; NULL: none
  int row = 0;
  if (slot >= 0) {
    const int64_t b = slot / div.size;
    if (b >= cache.num_blocks) {
      if (threadIdx.x == 0) raise(a.err, KVX_DEVERR_SLOT_RANGE);
    } else {
      block = (char*)cache.base + b * cache.block_stride_bytes;
      row = (int)(slot - b * div.size);
    }
  }
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const int64_t pos = a.positions[a.pair_axis[i] * a.num_tokens + t];
    const double turns = (double)pos * (double)a.inv_freq[i] * 0.15915494309189533577;
    double s, c;
    sincospi(2.0 * (turns - rint(turns)), &s, &c);
    turn[i] = c;
    turn[half + i] = s;
  }
  __syncthreads();

  // query rows: a vector of whole pairs, a pair of vectors half a rotation apart, or a vector that passes through
  const int rot_units = INTERLEAVED ? a.rot_dim / 8 : a.rot_dim / 16, head_units = rot_units + (dim - a.rot_dim) / 8;
  for (int u = threadIdx.x; u < a.num_heads * head_units; u += kRopeThreads) {
    const int h = u / head_units, c = u - h * head_units;
    const char* src = a.query.base + t * a.query.token_stride + h * a.query.head_stride;
    char* dst = (char*)a.out.base + t * a.out.token_stride + h * a.out.head_stride;
    const int off = c < rot_units ? c * 16 : a.rot_dim * 2 + (c - rot_units) * 16;
    const u32x4 first = gload<u32x4>(src + off);
    if (c >= rot_units) {
      gstore(dst + off, first);
    } else if constexpr (INTERLEAVED) {
      f32x8 v = widen<E>(first);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float cs = (float)turn[c * 4 + j], sn = (float)turn[half + c * 4 + j];
        const float p = v[2 * j], q = v[2 * j + 1];
        v[2 * j] = p * cs - q * sn;
        v[2 * j + 1] = q * cs + p * sn;
      }
      gstore(dst + off, narrow<E>(v));
    } else {
      f32x8 p = widen<E>(first), q = widen<E>(gload<u32x4>(src + half * 2 + off));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float cs = (float)turn[c * 8 + j], sn = (float)turn[half + c * 8 + j];
        const float x = p[j], y = q[j];
        p[j] = x * cs - y * sn;
        q[j] = y * cs + x * sn;
      }
      gstore(dst + off, narrow<E>(p));
      gstore(dst + half * 2 + off, narrow<E>(q));
    }
  }

  // K, then V; a wavefront's lanes beyond the last vector are whole groups of four
  if (!block && !a.key_out.base) return;
  const int per = cache.num_kv_heads * vecs;
  for (int u = threadIdx.x; u < 2 * per; u += kRopeThreads) {
    const bool is_v = u >= per;
    const int y = is_v ? u - per : u, h = y / vecs, c = y - h * vecs;
    const RowView& in = is_v ? a.value : a.key;
    const char* src = in.base + t * in.token_stride + h * in.head_stride;
    f32x8 v = widen<E>(gload<u32x4>(src + c * 16));
    if (!is_v && c * 8 < a.rot_dim) {
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double cs = turn[c * 4 + j], sn = turn[half + c * 4 + j], p = v[2 * j], q = v[2 * j + 1];
          v[2 * j] = sticky(p * cs - q * sn);
          v[2 * j + 1] = sticky(q * cs + p * sn);
        }
      } else {
        const bool second = c * 8 >= half;
        const int pair = second ? c * 8 - half : c * 8;
        const f32x8 o = widen<E>(gload<u32x4>(src + c * 16 + (second ? -half * 2 : half * 2)));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double cs = turn[pair + j], sn = second ? turn[half + pair + j] : -turn[half + pair + j];
          v[j] = sticky((double)v[j] * cs + (double)o[j] * sn);
        }
      }
    }
    const uint32_t s = scale_byte<E>(top_of_quad(top_of(v))), codes = encode(v, s);
    if (block) {
      char* plane = block + h * cache.head_stride_bytes + (is_v ? cache.kv_stride_bytes : 0);
      gstore(plane + row * (dim / 2) + c * 4, codes);
      if (c % 4 == 0) gstore(plane + cache.block_size * (dim / 2) + row * (dim / kGroup) + c / 4, (uint8_t)s);
    }
    if (a.key_out.base) {
      const RowView& o = is_v ? a.value_out : a.key_out;
      gstore((char*)o.base + t * o.token_stride + h * o.head_stride + c * 16, decode<E>(codes, scale_of(s)));
    }
  }
}

// --------------------------------------------------------------------------------------
// transfer
// --------------------------------------------------------------------------------------

constexpr int kCopyThreads = 256;

// Index of the last run whose buf_block <= p, or -1: a 64-way search, one probe a lane and round.
__device__ __forceinline__ int64_t find_run(const kvx_xfer* xfers, int64_t count, int64_t p, int lane) {
  int64_t lo = 0, hi = count;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64, i = lo + lane * step;
    const uint64_t hit = __ballot(i < hi && xfers[i].buf_block <= p);
    if (hit == 0) return lo - 1;
    lo += (63 - __builtin_clzll(hit)) * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return hi - lo == 1 && xfers[lo].buf_block > p ? lo - 1 : lo;
}

// How a block's groups are numbered: plane by plane (head, K or V), in the order of the plane's bytes.
struct Groups {
  Divisor per_plane, per_row;  // groups of a plane and of a row
  uint32_t of_block;           // groups
};
struct Place {
  uint32_t head, w, row, at, in_row;  // at: in the plane
};
__device__ __forceinline__ Place place(const Groups& g, uint32_t i) {
  const uint32_t plane = i / g.per_plane, at = i - plane * g.per_plane.by, row = at / g.per_row;
  return {plane >> 1, plane & 1, row, at, at - row * g.per_row.by};
}

// A wavefront's block: its layer's cache at the block, and the 4-bit block; false if there is none.
struct Pair {
  char* wide;
  char* narrow;
};
template <bool PACK>
__device__ __forceinline__ bool find_pair(const Fp4CopyArgs& a, int64_t item, int lane, Pair* at) {
  const int64_t l = item / a.total_blocks, p = item - l * a.total_blocks;
  int64_t count = *a.xfer_count;
  if (count > a.total_blocks) count = a.total_blocks;
  if (count <= 0) return false;
  const int64_t k = find_run(a.xfers, count, p, lane);
  if (k < 0) return false;
  const kvx_xfer x = a.xfers[k];
  if (p - x.buf_block >= x.num_blocks) return false;
  const int64_t id = (PACK ? x.src_block : x.dst_block) + (p - x.buf_block);
  if (id < 0 || id >= a.cache.num_blocks) {
    if (lane == 0) raise(a.err, KVX_DEVERR_BLOCK_RANGE);
    return false;
  }
  at->wide = (char*)a.layer_bases[l] + id * a.cache.block_stride_bytes;
  at->narrow = (char*)a.buffer.base + item * a.buffer.block_stride_bytes;
  return true;
}

// Four lanes a group, eight elements each.
template <class E, bool PACK>
__global__ __launch_bounds__(kCopyThreads) void copy_fp4_kernel(Fp4CopyArgs a, Groups g) {
  const int lane = threadIdx.x & 63;
  const int dim = a.cache.head_dim, c = lane & 3;
  const int64_t items = a.num_layers * a.total_blocks;
  for (int64_t item = (int64_t)blockIdx.x * (kCopyThreads / 64) + threadIdx.x / 64; item < items;
       item += (int64_t)gridDim.x * (kCopyThreads / 64)) {
  Pair to;
  if (!find_pair<PACK>(a, item, lane, &to)) continue;
  for (uint32_t i = lane >> 2; i < g.of_block; i += 16) {
    const Place x = place(g, i);
    char* wide = to.wide + x.row * a.cache.token_stride_bytes + x.w * a.cache.kv_stride_bytes +
                 x.head * a.cache.head_stride_bytes + x.in_row * (kGroup * 2) + c * 16;
    char* plane = to.narrow + x.head * a.buffer.head_stride_bytes + x.w * a.buffer.kv_stride_bytes;
    char* codes = plane + x.at * (kGroup / 2) + c * 4;
    char* scale = plane + a.cache.block_size * (dim / 2) + x.at;
    if constexpr (PACK) {
      const f32x8 v = widen<E>(gload<u32x4>(wide));
      const uint32_t s = scale_byte<E>(top_of_quad(top_of(v)));
      gstore(codes, encode(v, s));
      if (c == 0) gstore(scale, (uint8_t)s);
    } else {
      gstore(wide, decode<E>(gload<uint32_t>(codes), scale_of(gload<uint8_t>(scale))));
    }
  }
  }
}

template <bool PACK>
hipError_t launch_copy(const Fp4CopyArgs& a, hipStream_t stream) {
  const uint32_t row = a.cache.head_dim / kGroup, plane = row * a.cache.block_size;
  const uint32_t of_block = plane * 2 * a.cache.num_kv_heads;
  const Groups g = {divisor(plane), divisor(row), of_block};
  const int64_t items = a.num_layers * a.total_blocks, per = kCopyThreads / 64;
  const int64_t groups = (items + per - 1) / per, most = (1 << 24) - 1;  // a launch has fewer than 2^32 threads
  const dim3 grid((unsigned)(groups < most ? groups : most));
  if (a.cache.dtype == KVX_DTYPE_BF16) copy_fp4_kernel<Bf16, PACK><<<grid, kCopyThreads, 0, stream>>>(a, g);
  else copy_fp4_kernel<Fp16, PACK><<<grid, kCopyThreads, 0, stream>>>(a, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_fp4(const Fp4RopeArgs& a, bool interleaved, hipStream_t stream) {
  const dim3 grid((unsigned)a.num_tokens), block(kRopeThreads);
  const BlockDiv div = block_div(a.cache.block_size);
  if (a.cache.dtype == KVX_DTYPE_BF16) {
    if (interleaved) rope_fp4_kernel<Bf16, true><<<grid, block, 0, stream>>>(a, div);
    else rope_fp4_kernel<Bf16, false><<<grid, block, 0, stream>>>(a, div);
  } else {
    if (interleaved) rope_fp4_kernel<Fp16, true><<<grid, block, 0, stream>>>(a, div);
    else rope_fp4_kernel<Fp16, false><<<grid, block, 0, stream>>>(a, div);
  }
  return hipGetLastError();
}

hipError_t launch_pack_fp4(const Fp4CopyArgs& a, hipStream_t stream) { return launch_copy<true>(a, stream); }
hipError_t launch_unpack_fp4(const Fp4CopyArgs& a, hipStream_t stream) { return launch_copy<false>(a, stream); }

}  // namespace kvx
