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

// Data that is read, or written, once goes past the caches: with cached loads packing 48 layers takes 414 us and not 400, with cached
// stores both directions 937 us and not 905 (of an earlier step).
template <class T>
__device__ __forceinline__ T gload_once(const void* p) {
  return __builtin_nontemporal_load((const __attribute__((address_space(1))) T*)p);
}
template <class T>
__device__ __forceinline__ void gstore_once(void* p, T v) {
  __builtin_nontemporal_store(v, (__attribute__((address_space(1))) T*)p);
}

constexpr int kRopeThreads = 256;

// A 64-bit number to 32 bits so that a later rounding to 4 bits is as if it were the only one: its upper half, with the last bit set
// where anything was cut off. No value that the 4-bit rounding or the scale's bound breaks at has that bit set. The half has 21
// bits, so the cast is exact down to 2^-129, the smallest border of any scale, although 32 bits end at 2^-149; what lies below ends
// there at most, on a tie that goes to 0, which is what it is itself.
__device__ __forceinline__ float sticky(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t upper = (uint32_t)(b >> 32) | (uint32_t)((uint32_t)b != 0);
  return (float)__builtin_bit_cast(double, (uint64_t)upper << 32);
}

// One workgroup a token. Its first rot_dim/2 threads form the angles' cosines and sines, once for all heads and in 64 bits: a rotated
// key is rounded to 4 bits, and 32 bits on the way there would decide some of the elements next to a border between two codes.
// Rows are moved as 16-byte vectors, the first on their way while the angles are formed and the next while a thread turns its own: of K
// and V four neighbouring lanes hold a group of 32 elements, eight each, with the partners of the eight beside them; of q a thread holds
// whole pairs. Bound by HBM bytes for many tokens (9461 tokens of 32 + 8 heads, 243 MB: 45 us, 5.4 TB/s; with 128, 384 and 512 threads a token 53, 62
// and 61 us), by a launch and the chain positions, angles, stores for a few (32 tokens: 5 us). Angles in 32 bits for K save nothing.
struct RopeUnits {
  Divisor of_head, of_q_head;  // vectors of a K or V head, units of a q head
  int32_t kv, all;             // vectors of K and V, and all units
};
struct Unit {
  u32x4 a, b;
  int32_t head, at;  // at: vector of the head, or unit of a q head
  int32_t kind;      // 1: K, 2: V, 3: q
};
template <class E, bool INTERLEAVED>
__global__ __launch_bounds__(kRopeThreads) void rope_fp4_kernel(Fp4RopeArgs a, BlockDiv div, RopeUnits n) {
  __shared__ double turn[KVX_MAX_HEAD_DIM];  // cos of pair i, then sin
  __shared__ float turn32[KVX_MAX_HEAD_DIM];
  const int64_t t = blockIdx.x;
  const int half = a.rot_dim / 2, dim = a.cache.head_dim;
  const kvx_fp4_cache& cache = a.cache;
  const int rot_units = INTERLEAVED ? a.rot_dim / 8 : a.rot_dim / 16;
  auto q_offset = [&](int c) { return c < rot_units ? c * 16 : a.rot_dim * 2 + (c - rot_units) * 16; };
  auto load = [&](int u, Unit* x) {
    if (u < n.kv) {
      const int h2 = (uint32_t)u / n.of_head, heads = cache.num_kv_heads;
      const bool is_v = h2 >= heads;
      x->kind = is_v ? 2 : 1;
      x->head = is_v ? h2 - heads : h2;
      x->at = u - h2 * n.of_head.by;
      const RowView& in = is_v ? a.value : a.key;
      const char* src = in.base + t * in.token_stride + x->head * in.head_stride + x->at * 16;
      x->a = gload_once<u32x4>(src);
      if (!INTERLEAVED && !is_v && x->at * 8 < a.rot_dim) x->b = gload_once<u32x4>(src + (x->at * 8 < half ? half * 2 : -half * 2));
    } else {
      x->kind = 3;
      x->head = (uint32_t)(u - n.kv) / n.of_q_head;
      x->at = u - n.kv - x->head * n.of_q_head.by;
      const char* src = a.query.base + t * a.query.token_stride + x->head * a.query.head_stride + q_offset(x->at);
      x->a = gload_once<u32x4>(src);
      if (!INTERLEAVED && x->at < rot_units) x->b = gload_once<u32x4>(src + half * 2);
    }
  };
  Unit x;
  if (threadIdx.x < n.all) load(threadIdx.x, &x);
  const int64_t slot = a.slots[t];
  char* block = nullptr;  // of the slot; NULL: none
  int64_t row = 0;
  if (slot >= 0) {
    const int64_t b = slot / div.size;
    if (b >= cache.num_blocks) {
      if (threadIdx.x == 0) raise(a.err, KVX_DEVERR_SLOT_RANGE);
    } else {
      block = (char*)cache.base + b * cache.block_stride_bytes;
      row = slot - b * div.size;
    }
  }
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const int64_t pos = a.positions[a.pair_axis[i] * a.num_tokens + t];
    const double turns = (double)pos * (double)a.inv_freq[i] * 0.15915494309189533577;
    double s, c;
    sincospi(2.0 * (turns - rint(turns)), &s, &c);
    turn[i] = c;
    turn[half + i] = s;
    turn32[i] = (float)c;
    turn32[half + i] = (float)s;
  }
  __syncthreads();

  for (int u = threadIdx.x; u < n.all; u += kRopeThreads) {
    const Unit y = x;
    if (u + kRopeThreads < n.all) load(u + kRopeThreads, &x);
    if (y.kind == 3) {
      char* dst = (char*)a.out.base + t * a.out.token_stride + y.head * a.out.head_stride + q_offset(y.at);
      if (y.at >= rot_units) {
        gstore(dst, y.a);
      } else if constexpr (INTERLEAVED) {
        f32x8 v = widen<E>(y.a);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float cs = turn32[y.at * 4 + j], sn = turn32[half + y.at * 4 + j];
          const float p = v[2 * j], q = v[2 * j + 1];
          v[2 * j] = p * cs - q * sn;
          v[2 * j + 1] = q * cs + p * sn;
        }
        gstore(dst, narrow<E>(v));
      } else {
        f32x8 p = widen<E>(y.a), q = widen<E>(y.b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float cs = turn32[y.at * 8 + j], sn = turn32[half + y.at * 8 + j];
          const float v = p[j], w = q[j];
          p[j] = v * cs - w * sn;
          q[j] = w * cs + v * sn;
        }
        gstore(dst, narrow<E>(p));
        gstore(dst + half * 2, narrow<E>(q));
      }
    } else {
      f32x8 v = widen<E>(y.a);
      const int at = y.at * 8;
      if (y.kind == 1 && at < a.rot_dim) {
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double cs = turn[y.at * 4 + j], sn = turn[half + y.at * 4 + j], p = v[2 * j], q = v[2 * j + 1];
            v[2 * j] = sticky(p * cs - q * sn);
            v[2 * j + 1] = sticky(q * cs + p * sn);
          }
        } else {
          const bool second = at >= half;
          const int pair = second ? at - half : at;
          const f32x8 o = widen<E>(y.b);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const double cs = turn[pair + j], sn = second ? turn[half + pair + j] : -turn[half + pair + j];
            v[j] = sticky((double)v[j] * cs + (double)o[j] * sn);
          }
        }
      }
      const uint32_t s = scale_byte<E>(top_of_quad(top_of(v))), codes = encode(v, s);
      if (block) {
        char* plane = block + y.head * cache.head_stride_bytes + (y.kind == 2 ? cache.kv_stride_bytes : 0);
        gstore(plane + row * (dim / 2) + y.at * 4, codes);
        if (y.at % 4 == 0)
          gstore(plane + (int64_t)cache.block_size * (dim / 2) + row * (dim / kGroup) + y.at / 4, (uint8_t)s);
      }
      if (a.key_out.base) {
        const RowView& o = y.kind == 2 ? a.value_out : a.key_out;
        gstore((char*)o.base + t * o.token_stride + y.head * o.head_stride + y.at * 16, decode<E>(codes, scale_of(s)));
      }
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
  Divisor pieces;              // wavefronts' shares of a block
};
struct Place {
  uint32_t head, w, row, at, in_row;  // at: in the plane
};
__device__ __forceinline__ Place place(const Groups& g, uint32_t i) {
  const uint32_t plane = i / g.per_plane, at = i - plane * g.per_plane.by, row = at / g.per_row;
  return {plane >> 1, plane & 1, row, at, at - row * g.per_row.by};
}

__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)(uint32_t)uniform((int32_t)x) | (int64_t)uniform((int32_t)(x >> 32)) << 32;
}

// The runs of a wavefront's blocks, one after another. Runs, counts and bases come by the scalar unit: vector loads would queue
// behind the data.
template <bool PACK>
struct Runs {
  const Fp4CopyArgs& a;
  int64_t count, k;   // runs, and the present one
  int64_t from, to;   // its blocks of the buffer
  int64_t id;         // cache block of the first
  char* base;         // of the layer
  __device__ __forceinline__ Runs(const Fp4CopyArgs& args, int l, uint32_t p, int lane) : a(args) {
    count = constant(a.xfer_count);
    if (count > a.total_blocks) count = a.total_blocks;
    base = (char*)constant(a.layer_bases + l);
    k = count > 0 ? uniform(find_run(a.xfers, count, p, lane)) : -1;
    if (k < 0) k = 0;
    read();
  }
  __device__ __forceinline__ void read() {
    from = to = INT64_MAX;
    if (k >= count) return;
    from = constant(&a.xfers[k].buf_block);
    to = from + constant(&a.xfers[k].num_blocks);
    id = PACK ? constant(&a.xfers[k].src_block) : constant(&a.xfers[k].dst_block);
  }
  // The cache's block for block p of the buffer, p not falling; NULL if there is none.
  __device__ __forceinline__ char* block(uint32_t p, int lane) {
    while (p >= to) {
      ++k;
      read();
    }
    if (p < from) return nullptr;
    const int64_t at = id + (p - from);
    if (at < 0 || at >= a.cache.num_blocks) {
      if (lane == 0) raise(a.err, KVX_DEVERR_BLOCK_RANGE);
      return nullptr;
    }
    return base + at * a.cache.block_stride_bytes;
  }
};

// Runs that leave the buffer, which no block of it finds: one a thread, of the first layer's workgroups (no more runs than blocks
// count, and a workgroup takes the pieces of 8 blocks at most).
__device__ __forceinline__ void check_runs(const Fp4CopyArgs& a) {
  const int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  if (i >= a.total_blocks || i >= constant(a.xfer_count)) return;
  const int64_t at = a.xfers[i].buf_block;
  if (at < 0 || at > a.total_blocks || a.xfers[i].num_blocks > a.total_blocks - at) raise(a.err, KVX_DEVERR_BLOCK_RANGE);
}

// The 4x4 words of four neighbouring lanes transposed: lane c ends with the c-th word of each.
__device__ __forceinline__ u32x4 transposed(u32x4 v, int c) {
  auto swap = [](uint32_t& low, uint32_t& high, bool upper, auto dpp) {
    const uint32_t got = dpp(upper ? low : high);
    if (upper) low = got;
    else high = got;
  };
  uint32_t a = v[0], b = v[1], d = v[2], e = v[3];
  auto by1 = [](uint32_t x) -> uint32_t { return __builtin_amdgcn_mov_dpp(x, 0xb1, 0xf, 0xf, true); };
  auto by2 = [](uint32_t x) -> uint32_t { return __builtin_amdgcn_mov_dpp(x, 0x4e, 0xf, 0xf, true); };
  swap(a, b, c & 1, by1);
  swap(d, e, c & 1, by1);
  swap(a, d, c & 2, by2);
  swap(b, e, c & 2, by2);
  return {a, b, d, e};
}
template <int I>
__device__ __forceinline__ uint32_t of_lane(uint32_t x) {  // of the four neighbours
  return __builtin_amdgcn_mov_dpp(x, I * 0x55, 0xf, 0xf, true);
}

// A wavefront takes 128 groups at a time, 8 KiB of the 16-bit side, and kPieces such pieces one after another, the next one's loads
// before the present one's stores. On the 16-bit side four lanes hold a group, 16 bytes each; on the 4-bit side a lane holds one, and words
// change lanes between the two, so that both move 1 KiB an instruction. Bound by HBM bytes, read and written once: 48 layers of
// 4608 blocks of 8 KiB (2.29 GB on both sides) are packed in 400 us, 5.7 TB/s, and unpacked to random blocks in 429 us, 5.3 TB/s; with 1, 4
// and 8 pieces a wavefront the two took 915, 887 and 916 us together where 2 took 842, with the groups in the 16-bit side's order 907.
//   EVEN, where rows are 1, 2, 4 or 8 groups and planes whole times 16: 16 groups are rows of one plane, whose place the scalar
//   unit finds; a lane's place among them never changes. Packing so takes 400 us and not 420; unpacking is no faster.
constexpr int kPiece = 128, kLoads = kPiece / 16, kPieces = 2;
template <class E, bool PACK, bool EVEN>
__global__ __launch_bounds__(kCopyThreads) void copy_fp4_kernel(Fp4CopyArgs a, Groups g, uint32_t pieces) {
  const int lane = threadIdx.x & 63, c = lane & 3, quad = lane >> 2;
  const int64_t scales = (int64_t)a.cache.block_size * (a.cache.head_dim / 2);
  const uint32_t my_row = quad / g.per_row;
  const int64_t my_wide = my_row * a.cache.token_stride_bytes + (quad - my_row * g.per_row.by) * (kGroup * 2) + c * 16;
  constexpr int NV = PACK ? kLoads : kLoads / 4;
  struct Piece {
    char* cache;   // the cache's block; NULL: none
    char* buffer;  // and the buffer's
    uint32_t first;
    u32x4 v[NV];
    uint32_t s[NV];
  };
  // the 16-bit side of group first + i * 16 + quad, or NULL behind the block's last
  auto wide = [&](const Piece& x, int i) -> char* {
    const uint32_t at = x.first + i * 16 + (EVEN ? 0 : quad);
    if (at >= g.of_block) return nullptr;
    const Place y = place(g, at);
    char* p = x.cache + y.row * a.cache.token_stride_bytes + y.w * a.cache.kv_stride_bytes + y.head * a.cache.head_stride_bytes;
    return EVEN ? p + my_wide : p + y.in_row * (kGroup * 2) + c * 16;
  };
  // the 4-bit side of group first + (i + c) * 16 + quad, i a multiple of 4
  auto narrow = [&](const Piece& x, int i, char** scale) -> char* {
    const uint32_t at = x.first + (i + c) * 16 + quad;
    if (at >= g.of_block) return nullptr;
    const Place y = place(g, at);
    char* plane = x.buffer + y.head * a.buffer.head_stride_bytes + y.w * a.buffer.kv_stride_bytes;
    *scale = plane + scales + y.at;
    return plane + (int64_t)y.at * (kGroup / 2);
  };
  auto load = [&](Piece& x) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      char* scale;
      const char* p = PACK ? wide(x, i) : narrow(x, i * 4, &scale);
      x.v[i] = u32x4{0, 0, 0, 0};
      x.s[i] = 0;
      if (p) {
        x.v[i] = gload_once<u32x4>(p);
        if (!PACK) x.s[i] = gload_once<uint8_t>(scale);
      }
    }
  };
  auto store = [&](const Piece& x) {
#pragma unroll
    for (int i = 0; i < kLoads; i += 4) {
      if constexpr (PACK) {
        u32x4 codes;
        uint32_t s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x8 y = widen<E>(x.v[i + k]);
          s[k] = scale_byte<E>(top_of_quad(top_of(y)));
          codes[k] = encode(y, s[k]);
        }
        codes = transposed(codes, c);
        char* scale;
        char* p = narrow(x, i, &scale);
        if (!p) continue;
        gstore_once(p, codes);
        gstore(scale, (uint8_t)(c & 2 ? (c & 1 ? s[3] : s[2]) : (c & 1 ? s[1] : s[0])));
      } else {
        const u32x4 codes = transposed(x.v[i / 4], c);
        const uint32_t s = x.s[i / 4], of[4] = {of_lane<0>(s), of_lane<1>(s), of_lane<2>(s), of_lane<3>(s)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          char* p = wide(x, i + k);
          if (p) gstore_once(p, decode<E>(codes[k], scale_of(of[k])));
        }
      }
    }
  };
  if (blockIdx.y == 0) check_runs(a);
  const uint32_t share = blockIdx.x * (kCopyThreads / 64) + uniform((int32_t)(threadIdx.x / 64));
  for (int l = blockIdx.y; l < a.num_layers; l += gridDim.y) {
    if (share >= (pieces + kPieces - 1) / kPieces) break;
    const uint32_t begin = share * kPieces, end = begin + kPieces < pieces ? begin + kPieces : pieces;
    Runs<PACK> runs(a, l, begin / g.pieces, lane);
    auto find = [&](Piece& x, uint32_t i) {
      const uint32_t block = i / g.pieces;
      x.first = (i - block * g.pieces.by) * kPiece;
      x.cache = runs.block(block, lane);
      x.buffer = (char*)a.buffer.base + (l * a.total_blocks + block) * a.buffer.block_stride_bytes;
      if (x.cache) load(x);
    };
    Piece now, next;
    find(now, begin);
    for (uint32_t i = begin; i < end; ++i) {
      next.cache = nullptr;
      if (i + 1 < end) find(next, i + 1);
      if (now.cache) store(now);
      now = next;
    }
  }
}

template <class E, bool PACK>
void launch_copy_type(const Fp4CopyArgs& a, const Groups& g, uint32_t pieces, dim3 grid, hipStream_t stream) {
  if constexpr (PACK) {
    if (16 % g.per_row.by == 0 && g.per_plane.by % 16 == 0) {
      copy_fp4_kernel<E, true, true><<<grid, kCopyThreads, 0, stream>>>(a, g, pieces);
      return;
    }
  }
  copy_fp4_kernel<E, PACK, false><<<grid, kCopyThreads, 0, stream>>>(a, g, pieces);
}

template <bool PACK>
hipError_t launch_copy(const Fp4CopyArgs& a, hipStream_t stream) {
  const uint32_t row = a.cache.head_dim / kGroup, plane = row * a.cache.block_size;
  const uint32_t of_block = plane * 2 * a.cache.num_kv_heads, in_block = (of_block + kPiece - 1) / kPiece;
  const Groups g = {divisor(plane), divisor(row), of_block, divisor(in_block)};
  // a layer's pieces by column, and layers by row; a launch has fewer than 2^32 threads, layers beyond are taken in turn
  const int64_t pieces = a.total_blocks * in_block, per = kPieces * (kCopyThreads / 64);
  const int64_t columns = (pieces + per - 1) / per;
  int64_t rows = ((1 << 24) - 1) / columns;
  if (rows > a.num_layers) rows = a.num_layers;
  if (rows > 65535) rows = 65535;
  const dim3 grid((unsigned)columns, (unsigned)rows);
  if (a.cache.dtype == KVX_DTYPE_BF16) launch_copy_type<Bf16, PACK>(a, g, (uint32_t)pieces, grid, stream);
  else launch_copy_type<Fp16, PACK>(a, g, (uint32_t)pieces, grid, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_fp4(const Fp4RopeArgs& a, bool interleaved, hipStream_t stream) {
  const dim3 grid((unsigned)a.num_tokens), block(kRopeThreads);
  const BlockDiv div = block_div(a.cache.block_size);
  const int32_t vecs = a.cache.head_dim / 8, kv = 2 * a.cache.num_kv_heads * vecs;
  const int32_t q_head = (interleaved ? a.rot_dim / 8 : a.rot_dim / 16) + (a.cache.head_dim - a.rot_dim) / 8;
  const RopeUnits n = {divisor(vecs), divisor(q_head), kv, kv + a.num_heads * q_head};
  if (a.cache.dtype == KVX_DTYPE_BF16) {
    if (interleaved) rope_fp4_kernel<Bf16, true><<<grid, block, 0, stream>>>(a, div, n);
    else rope_fp4_kernel<Bf16, false><<<grid, block, 0, stream>>>(a, div, n);
  } else {
    if (interleaved) rope_fp4_kernel<Fp16, true><<<grid, block, 0, stream>>>(a, div, n);
    else rope_fp4_kernel<Fp16, false><<<grid, block, 0, stream>>>(a, div, n);
  }
  return hipGetLastError();
}

hipError_t launch_pack_fp4(const Fp4CopyArgs& a, hipStream_t stream) { return launch_copy<true>(a, stream); }
hipError_t launch_unpack_fp4(const Fp4CopyArgs& a, hipStream_t stream) { return launch_copy<false>(a, stream); }

}  // namespace kvx
