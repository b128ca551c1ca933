// gfx950 kernels of kvx_paged_attention_fp4.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_rows.h"
#include "kvx_fp4_format.h"
#include "kvx_fp4_launch.h"
#include "kvx_fp4_plan.h"

namespace kvx {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// --------------------------------------------------------------------------------------
// matrix pieces
// --------------------------------------------------------------------------------------

// 16x16x32: lane l = 16 g + n holds row (or column) n and elements 8 g to 8 g + 7 of the summed dimension; result register i of
// lane l is row 4 g + i, column n. Products of 4-bit K with q split into 8-bit floats (the scaled products' types) would spare K's
// conversion, but they cut off what is 2^-11 of the largest of the products they add at once, which a sum of weights shows.
__device__ __forceinline__ f32x4 product(Bf16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Bf16::V8, a), __builtin_bit_cast(Bf16::V8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 product(Fp16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Fp16::V8, a), __builtin_bit_cast(Fp16::V8, b), c, 0, 0, 0);
}

// Largest and sum over the lanes l, l ^ 16, l ^ 32, l ^ 48.
template <class F>
__device__ __forceinline__ float over_rows(float x, F f) {
  uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  x = f(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
  b = __builtin_bit_cast(uint32_t, x);
  const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t s0 = s[0], s1 = s[1];
  return f(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
}
__device__ __forceinline__ float max_over_rows(float x) {
  return over_rows(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float sum_over_rows(float x) {
  return over_rows(x, [](float a, float b) { return a + b; });
}

// Where v may read back infinite or NaN in the type.
template <class E>
constexpr uint32_t kFiniteScales = __is_same(E, Bf16) ? 252 : 140;

// One code in the type, widened.
template <class E>
__device__ __forceinline__ f32x4 decode4(uint32_t codes, float scale) {
  const u32x4 r = decode<E>(codes, scale);
  const u32x2 two = {r[0], r[1]};
  return __builtin_convertvector(__builtin_bit_cast(typename E::V4, two), f32x4);
}

// --------------------------------------------------------------------------------------
// attention
// --------------------------------------------------------------------------------------

// One pass over the slots with a running maximum and sum, scores transposed (S^T = K q^T), so that a lane holds one query
// row and four slots of each 16, and the weights are where O^T += V^T P^T takes them. RT tiles of 16 rows are the same for the
// four wavefronts of a workgroup, which take 32 slots each of every 128 and meet only at the end. A lane loads whole groups of 32
// elements (of heads of up to 64, half groups) with their scales. Of K, widened to 16 bits, they are the matrix unit's operand as they
// stand, because the summed dimension may be numbered in any order; V goes widened to LDS and is read from there with the transposing
// load. DP is head_dim padded to 64, 128 or 256.
// A decode batch of 32 requests of up to 8192 slots, 32 heads on 8, reads its 156 MB in 38 us, 4.1 TB/s, two requests of 131071 and 114412
// slots their 267 MB in 55 us, 4.8 TB/s. Without anything computed the same loads take 33 and 51 us: their count bounds it, rows of 64
// bytes and scales of 4, then the start and the end of the shares. Two steps' loads in flight spill or take a wavefront's
// place (40.6 us where one took 38.8), a fourth workgroup a CU spills (44.5 us).
//   SHARED: the grid's workgroups take equal shares of the whole batch's steps (see Shares).
template <class E, int DP, int RT, bool SHARED>
__global__ __launch_bounds__(256, DP > 128 ? 3 - RT : 4 - RT) void attend_fp4_kernel(AttendArgs args, BlockDiv div, Split sp) {
  const AttendArgs a = argument<AttendArgs>();
  constexpr int ROWS = 16 * RT, KW = 32, BN = 4 * KW, KT = KW / 16;
  constexpr int KS = DP > 128 ? 2 : 1, DT = DP / 16;
  constexpr int W = DP > 64 ? 4 : 2;  // words of a row that a lane loads at a time: a piece
  constexpr int VROW = DP * 2 + 32;  // bytes of a row of V in LDS
  constexpr int TILE = 4 * KW * VROW, JOIN = 4 * 16 * DP * 4;
  __shared__ __align__(16) char smem[TILE > JOIN ? TILE : JOIN];
  __shared__ float sm[2][4][ROWS];

  const int tid = threadIdx.x, lane = tid & 63, w = uniform((int32_t)(tid >> 6));
  const int n = lane & 15, hq = lane >> 4;
  const int group = a.num_heads / a.cache.num_kv_heads, dim = a.cache.head_dim, groups = dim / kGroup, pieces = dim / (W * 8);
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  int g = blockIdx.x % a.cache.num_kv_heads, index = blockIdx.x / a.cache.num_kv_heads;
  if constexpr (SHARED) {  // shares that follow one another to one XCD: workgroup i runs on XCD i % 8
    const int xcd = blockIdx.x % 8, per = gridDim.x / 8, more = gridDim.x % 8;
    const int at = xcd * per + (xcd < more ? xcd : more) + blockIdx.x / 8;
    g = at / sp.shares;
    index = at - g * sp.shares;
  }
  if (blockIdx.x == 0) check_batch(a, cap, tid, 256);

  char* const own = smem + w * KW * VROW;  // this wavefront's rows of V
  // the 16-byte pieces of every second four rows change places in pairs, so that eight rows' writes of one, which go out
  // together, fall on different 16 bytes of 128
  const int odd_row = (n >> 2 & 1) * 16;
  char* const put[2] = {own + n * VROW + hq * (W * 16) + odd_row, own + n * VROW + hq * (W * 16) - odd_row};
  const char* const get = own + (4 * hq + (n >> 2)) * VROW + ((((n >> 1) & 1) ^ (hq & 1)) * 16) + (n & 1) * 8;

  Rows x;
  Shares all;
  int32_t tiles = 0, steps = 1, from = 0, to = 1;  // steps [from, to) of tile x.tile
  uint32_t tile0 = 0;
  int64_t left = 1;
  if constexpr (SHARED) {
    const Requests q = locate<ROWS, BN, kFp4Extra>(a, group, cap, lane, sp.shares, &all, [&](const Shares& s, const Requests& q) {
      const int64_t begin = share_begin(s, index);
      return index < s.count && q.step0 <= begin && begin < q.step0 + (int64_t)q.tiles * q.steps;
    });
    if (q.steps == 0) return;
    const int64_t begin = share_begin(all, index);
    left = share_begin(all, index + 1) - begin;
    tile0 = q.tile0;
    tiles = q.tiles;
    steps = q.steps;
    x = q.x;
    x.tile = (int32_t)quotient(begin - q.step0, steps);
    from = (int32_t)(begin - q.step0 - (int64_t)x.tile * steps);
  } else {
    x = find_rows<ROWS>(a, sp.tiles - 1 - index, group, cap, lane);
    if (x.tile < 0 || (int64_t)x.tile * ROWS >= (int64_t)x.tokens * group) return;
  }
  bool bad_blocks = false;
  for (;;) {
  if constexpr (SHARED) {
    if (tile0 + x.tile >= (uint32_t)sp.tiles) break;  // offsets that are not a CSR: the workspace has no slots for more
    to = from + left < steps ? (int)(from + left) : steps;
  }
  const int row0 = x.tile * ROWS, rows = x.tokens * group;

  // this lane's rows, what they see, and what any row of the workgroup sees
  int2 see[RT];
  int head[RT];
  int64_t q_row[RT];
  bool used[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = row0 + rt * 16 + n;
    used[rt] = row < rows;
    const int token = used[rt] ? row / group : 0;
    head[rt] = g * group + (used[rt] ? row - token * group : 0);
    q_row[rt] = x.q0 + token;
    see[rt] = sees(a, x, token);
    if (!used[rt]) see[rt] = {0, 0};
  }
  const int last_row = row0 + ROWS < rows ? row0 + ROWS - 1 : rows - 1;
  const int2 first = sees_uniform(a, x, row0 / group), last = sees_uniform(a, x, last_row / group);
  const int kend = last.y;
  const int t_first = first.x / BN, t_all = (kend + BN - 1) / BN - t_first;
  int tb = t_first, te = t_first + (t_all > 0 ? t_all : 0);
  if constexpr (SHARED) {
    // the first kFp4Extra steps of a tile stand for its start
    const int own = steps - kFp4Extra, b = from > kFp4Extra ? from - kFp4Extra : 0, e = to > kFp4Extra ? to - kFp4Extra : 0;
    if (t_all == own) {
      tb = t_first + b;
      te = t_first + e;
    } else {  // a tile whose rows see less than all of the request's: its steps in proportion
      const int64_t mine = te - tb;
      te = tb + (int)quotient(mine * e, own);
      tb = tb + (int)quotient(mine * b, own);
    }
  }
  tb = uniform(tb);
  te = uniform(te);

  // q: lane 16 g + n has piece g (and g + 4) of row n, as it will have of K
  u32x4 q[RT][KS][W];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const char* p = a.query.base + q_row[rt] * a.query.token_stride + head[rt] * a.query.head_stride;
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
      for (int k = 0; k < W; ++k) {
        q[rt][c][k] = u32x4{0, 0, 0, 0};
        if (used[rt] && c * 4 + hq < pieces) q[rt][c][k] = gload<u32x4>(p + (c * 4 + hq) * (W * 16) + k * 16);
      }
  }

  const char* const base = (const char*)a.cache.base + g * a.cache.head_stride_bytes;
  const int64_t scales = (int64_t)a.cache.block_size * (dim / 2);
  const int32_t* const table = a.batch.block_table + x.r * a.batch.bt_row_stride;
  const int cols = (int)a.batch.max_blocks_per_req;

  f32x4 acc[RT][DT];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[rt][d] = f32x4{};
  }
  const float c1 = a.scale * kLog2e;

  // Lane 16 g + n of a wavefront stages piece g (and g + 4) of slots n and 16 + n of its 32. A slot that is not there is read
  // from the cache's first rows; its scale of V becomes 0 and its weight is. Lanes past a narrower head's last piece load that
  // one again: q is zero there and K's scale 1, and such columns of V reach no element of the result.
  typedef uint32_t Words __attribute__((ext_vector_type(W)));
  struct {
    Words k[KT][KS], v[KT][KS];
    uint32_t ks[KT][KS], vs[KT][KS];
    uint32_t there;  // one bit a slot
  } in;
  uint32_t at[KS];
#pragma unroll
  for (int c = 0; c < KS; ++c) at[c] = c * 4 + hq < pieces ? c * 4 + hq : pieces - 1;
  int32_t ids[KT];
  auto load_ids = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const int b = block_of(div, t * BN + w * KW + i * 16 + n);
      ids[i] = gload<int32_t>(table + (b < cols ? b : cols - 1));
    }
  };
  auto fetch = [&](int t) __attribute__((always_inline)) {
    in.there = 0;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const int j = t * BN + w * KW + i * 16 + n;
      const bool wanted = j < kend, ok = wanted && (uint32_t)ids[i] < (uint64_t)a.cache.num_blocks;
      bad_blocks |= wanted && !ok;
      in.there |= (uint32_t)(__ballot(ok) & 0xffff) << (16 * i);
      const int64_t o = ok ? j - block_of(div, j) * div.size : 0;
      const char* k = base + (ok ? ids[i] * a.cache.block_stride_bytes : 0);
      const char* e = k + o * (dim / 2);
      const char* s = k + scales + o * groups;
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        in.k[i][c] = gload<Words>(e + at[c] * (W * 4));
        in.ks[i][c] = gload<uint8_t>(s + at[c] * W / 4);
        in.v[i][c] = gload<Words>(e + a.cache.kv_stride_bytes + at[c] * (W * 4));
        in.vs[i][c] = gload<uint8_t>(s + a.cache.kv_stride_bytes + at[c] * W / 4);
      }
    }
  };
  bool far = false;  // some row's scores are (see is_far)
  auto step = [&](int t) __attribute__((always_inline)) {
    const int k0 = t * BN + w * KW;
    const bool inner = t * BN >= last.x && t * BN + BN <= first.y;
    f32x4 s[RT][KT];
#pragma unroll
    for (int i = 0; i < KT; ++i) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][i] = f32x4{};
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        const float scale = c * 4 + hq < pieces ? scale_of(in.ks[i][c]) : 1.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const u32x4 wide = decode<E>(in.k[i][c][k], scale);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) s[rt][i] = product(E(), wide, q[rt][c][k], s[rt][i]);
        }
      }
    }
    // A weight of zero times a NaN or infinity is NaN: pieces of V that may read back as one are left out of the products
    // and added below for the rows that see them.
    uint64_t odd[KT][KS], any_odd = 0;
    if (!inner || in.there != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          if (!(in.there >> (16 * i + n) & 1)) in.vs[i][c] = 0;
          const bool bad = in.vs[i][c] > kFiniteScales<E> && c * 4 + hq < pieces;
          any_odd |= odd[i][c] = __ballot(bad);
          if (in.vs[i][c] > kFiniteScales<E>) in.vs[i][c] = 0, in.v[i][c] = Words(0);
        }
    }
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        const float scale = scale_of(in.vs[i][c]);
#pragma unroll
        for (int k = 0; k < W; ++k) *(u32x4*)(put[k & 1] + i * 16 * VROW + c * 256 + k * 16) = decode<E>(in.v[i][c][k], scale);
      }
    __builtin_amdgcn_wave_barrier();
    const uint32_t there = in.there;
    if (t + 1 < te) {
      fetch(t + 1);
      load_ids(t + 2);
    }

    u32x4 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (!inner || there != 0xffffffffu) {
        const int at = k0 + 4 * hq, lo = see[rt].x - at, hi = see[rt].y - at;
        const uint32_t mine = there >> (4 * hq);
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int o = 16 * i + r;
            if (o < lo || o >= hi || !(mine >> o & 1)) s[rt][i][r] = -INFINITY;
          }
      }
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, s[rt][i][r]);
      top = max_over_rows(top) * c1;
      // the reference moves only when the maximum leaves its range: the sums keep their 32 bits
      if (__any(top > m[rt] + (kLift<E> + kLag<E>))) {
        const float held = m[rt];
        const float to = top - held > kLift<E> + kLag<E> ? (is_far(top) ? top : top - kLift<E>) : held;
        const float shrink = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(held - to);
        m[rt] = to;
        l[rt] *= shrink;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[rt][d] *= shrink;
        far |= __any(is_far(to));
      }
      const float ref = m[rt] == -INFINITY ? 0.0f : m[rt];
      f32x8 pv;
      if (far) {  // rounded before the reference is taken from it, as the maximum was
#pragma unroll
        for (int i = 0; i < KT * 4; ++i) pv[i] = rounded_difference(rounded_product(s[rt][i / 4][i % 4], c1), ref);
      } else {
#pragma unroll
        for (int i = 0; i < KT * 4; ++i) pv[i] = __builtin_fmaf(s[rt][i / 4][i % 4], c1, -ref);
      }
#pragma unroll
      for (int i = 0; i < KT * 4; ++i) {
        pv[i] = __builtin_amdgcn_exp2f(pv[i]);
        l[rt] += pv[i];
        s[rt][i / 4][i % 4] = pv[i];
      }
      p[rt] = narrow<E>(pv);  // one rounding of each weight to the element type, which the matrix unit takes
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const char* at = get + d * 32;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KVX_LDS s16x4*)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KVX_LDS s16x4*)(at + 16 * VROW));
      const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) acc[rt][d] = product(E(), __builtin_bit_cast(u32x4, v), p[rt], acc[rt][d]);
    }
    if (any_odd) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int c = 0; c < KS; ++c)
          for (uint64_t todo = odd[i][c]; todo; todo &= todo - 1) {
            const int from = __builtin_ctzll(todo), o = from & 15, at = c * 4 + (from >> 4), j = k0 + i * 16 + o;
            const int b = block_of(div, j);
            const char* plane = base + table[b] * a.cache.block_stride_bytes + a.cache.kv_stride_bytes;
            const int64_t row = j - b * div.size;
            const float scale = scale_of(gload<uint8_t>(plane + scales + row * groups + at * W / 4));
            const uint32_t parts = W == 4 ? 3u << (2 * at) : 1u << at;  // a bit each, so that no index into the sums is made of it
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const float mine = o % 4 == 0 ? s[rt][i][0] : o % 4 == 1 ? s[rt][i][1] : o % 4 == 2 ? s[rt][i][2] : s[rt][i][3];
              const float pj = __shfl(mine, n + 16 * (o >> 2));
              if (j < see[rt].x || j >= see[rt].y) continue;
#pragma unroll
              for (int d = 0; d < DT; ++d) {
                if (!(parts >> d & 1)) continue;
                const uint32_t codes = gload<uint16_t>(plane + row * (dim / 2) + d * 8 + 2 * hq);
                acc[rt][d] += pj * decode4<E>(codes, scale);
              }
            }
          }
    }
    __builtin_amdgcn_wave_barrier();
  };

  // a step's loads go out while the one before forms its weights, the block ids a step ahead of them
  if (tb < te) {
    load_ids(tb);
    fetch(tb);
    load_ids(tb + 1);
  }
  for (int t = tb; t < te; ++t) step(t);

  // join the wavefronts: weights of each one's sum, then the sums themselves through LDS
  const AttendArgs end = argument<AttendArgs>();
  const bool whole = !SHARED || (from == 0 && to == steps);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = sum_over_rows(l[rt]);
    if (hq == 0) {
      sm[0][w][rt * 16 + n] = m[rt];
      sm[1][w][rt * 16 + n] = l[rt];
    }
  }
  __syncthreads();
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float top = -INFINITY, total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, sm[0][i][rt * 16 + n]);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < 4; ++i) total += sm[1][i][rt * 16 + n] * __builtin_amdgcn_exp2f(sm[0][i][rt * 16 + n] - ref);
    const float mine = __builtin_amdgcn_exp2f(m[rt] - ref);
    // [wavefront][row][16-byte pieces, swizzled by row]
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *(f32x4*)(smem + ((w * 16 + n) * (DP / 4) + ((d * 4 + hq) ^ n)) * 16) = acc[rt][d] * mine;
    __syncthreads();
    const float inv = total == 0 ? 0.0f : 1.0f / total;
    // where a part's row goes: share index of tile tile0 + x.tile
    const int64_t part = ((int64_t)(index + (int32_t)(tile0 + x.tile)) * end.cache.num_kv_heads + g) * ROWS + rt * 16 + n;
#pragma unroll
    for (int i = 0; i < DT / 4; ++i) {
      const int d = i * 4 + w, e = d * 16 + 4 * hq;
      f32x4 v = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) v += *(const f32x4*)(smem + ((k * 16 + n) * (DP / 4) + ((d * 4 + hq) ^ n)) * 16);
      v = total == 0 ? f32x4{} : v * inv;
      if (!used[rt] || e >= end.cache.head_dim) continue;
      if (SHARED && !whole) {
        gstore(sp.acc + part * end.cache.head_dim + e, v);
      } else {
        gstore((char*)end.out.base + q_row[rt] * end.out.token_stride + head[rt] * end.out.head_stride + e * 2,
               __builtin_convertvector(v, typename E::V4));
      }
    }
    if (used[rt] && hq == 0 && w == 0) {
      const float lse2 = total == 0 ? -INFINITY : top + __builtin_amdgcn_logf(total);
      if (SHARED && !whole) sp.lse[part] = lse2;
      else if (end.lse) end.lse[q_row[rt] * end.num_heads + head[rt]] = lse2 * kLn2;
    }
    __syncthreads();
  }

  if constexpr (!SHARED) break;
  left -= to - from;
  if (left <= 0) break;
  // the next tile, of this request or of the next one that has any
  from = 0;
  if (++x.tile == tiles) {
    tile0 += tiles;
    do {
      x = request_uniform(a, x.r + 1, cap);
      extent<ROWS, BN, kFp4Extra>(a, x, group, &tiles, &steps);
      tiles = uniform(tiles);
      steps = uniform(steps);
    } while (tiles == 0);
  }
  }
  if (bad_blocks) raise(a.err, KVX_DEVERR_BLOCK_RANGE);
}

// In the 32x32x16 products lane l holds column (or row) l % 32 and, with hf = l / 32, elements 8 hf to 8 hf + 7 of the summed
// dimension; result register i of lane l is row 8 (i / 4) + 4 hf + i % 4, column l % 32.
__device__ __forceinline__ f32x16 product(Bf16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Bf16::V8, a), __builtin_bit_cast(Bf16::V8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 product(Fp16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(Fp16::V8, a), __builtin_bit_cast(Fp16::V8, b), c, 0, 0, 0);
}

// Many rows: 128 of them a workgroup, 32 a wavefront, and 64 slots a step, which the four wavefronts widen to 16 bits on their
// way to LDS, 16 slots each. Scores transposed as above, with the 32x32x16 products. 2048 tokens over 32768 slots, 32 heads on 8, take 1020 us,
// 1040 TFLOP/s: the matrix units are busy 46% of the time and the vector units 52%, which share a SIMD's issue and run side by
// side only as far as its two wavefronts are at different work.
//   SHARED: the grid's workgroups take equal shares of the whole batch's steps (see Shares).
template <class E, int DP, bool SHARED>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attend_fp4_rows_kernel(AttendArgs args, BlockDiv div, Split sp) {
  const AttendArgs a = argument<AttendArgs>();
  constexpr int ROWS = 128, BN = 64, KW = 16, KT = 2, KSTEPS = DP / 16, DT = DP / 32;
  constexpr int KS = DP > 128 ? 2 : 1;                   // groups of K, and of V, that a lane stages
  constexpr int KROW = DP * 2 + 16, VROW = DP * 2 + 64;  // bytes of a row in LDS
  __shared__ __align__(16) char smem[BN * (KROW + VROW) + BN];
  char* const sk = smem;
  char* const sv = smem + BN * KROW;
  uint8_t* const flags = (uint8_t*)(smem + BN * (KROW + VROW));

  const int tid = threadIdx.x, lane = tid & 63, w = uniform((int32_t)(tid >> 6));
  const int n = lane & 31, hf = lane >> 5;
  const int group = a.num_heads / a.cache.num_kv_heads, dim = a.cache.head_dim, groups = dim / kGroup;
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  int g = blockIdx.x % a.cache.num_kv_heads, index = blockIdx.x / a.cache.num_kv_heads;
  if constexpr (SHARED) {  // shares that follow one another to one XCD: workgroup i runs on XCD i % 8
    const int xcd = blockIdx.x % 8, per = gridDim.x / 8, more = gridDim.x % 8;
    const int at = xcd * per + (xcd < more ? xcd : more) + blockIdx.x / 8;
    g = at / sp.shares;
    index = at - g * sp.shares;
  }
  if (blockIdx.x == 0) check_batch(a, cap, tid, 256);

  // lane 16 q + s stages group q (and q + 4) of slot s of its wavefront's 16
  const int slot = lane & 15, quarter = lane >> 4;
  char* const sk_put = sk + (w * KW + slot) * KROW + quarter * 64;
  // The 16-byte pieces of a row's groups in V change places by row: piece i of row r is at i ^ (r / 2 % 4). Eight lanes write at a
  // time, eight rows' pieces, which then fall on different 16 bytes of 128; unchanged, they take four times as long.
  const uint32_t sv_put = BN * KROW + (w * KW + slot) * VROW + quarter * 64 + (slot >> 1 & 3) * 16;
  const char* const sk_get = sk + n * KROW + hf * 16;
  const int of_row = 4 * hf + ((lane & 15) >> 2), piece = ((lane >> 4) & 1) * 2 + ((lane >> 1) & 1);
  const char* const sv_get = sv + of_row * VROW + (piece ^ (of_row >> 1 & 3)) * 16 + (lane & 1) * 8;

  Rows x;
  Shares all;
  int32_t tiles = 0, steps = 1, from = 0, to = 1;  // steps [from, to) of tile x.tile
  uint32_t tile0 = 0;
  int64_t left = 1;
  if constexpr (SHARED) {
    const Requests q = locate<ROWS, BN>(a, group, cap, lane, sp.shares, &all, [&](const Shares& s, const Requests& q) {
      const int64_t begin = share_begin(s, index);
      return index < s.count && q.step0 <= begin && begin < q.step0 + (int64_t)q.tiles * q.steps;
    });
    if (q.steps == 0) return;
    const int64_t begin = share_begin(all, index);
    left = share_begin(all, index + 1) - begin;
    tile0 = q.tile0;
    tiles = q.tiles;
    steps = q.steps;
    x = q.x;
    x.tile = (int32_t)quotient(begin - q.step0, steps);
    from = (int32_t)(begin - q.step0 - (int64_t)x.tile * steps);
  } else {
    // The longest tiles first; every other round of 256 workgroups (one a CU) the other way round, so that a CU's second
    // tile makes up for its first.
    const int per = 256 / a.cache.num_kv_heads > 0 ? 256 / a.cache.num_kv_heads : 1, round = index / per;
    const int back = (round + 1) * per < sp.tiles ? (round + 1) * per : sp.tiles;
    x = find_rows<ROWS>(a, sp.tiles - 1 - (round & 1 ? back - 1 - (index - round * per) : index), group, cap, lane);
    if (x.tile < 0 || (int64_t)x.tile * ROWS >= (int64_t)x.tokens * group) return;
  }
  bool bad_blocks = false;
  for (;;) {
  const AttendArgs a = argument<AttendArgs>();
  if constexpr (SHARED) {
    if (tile0 + x.tile >= (uint32_t)sp.tiles) break;  // offsets that are not a CSR: the workspace has no slots for more
    to = from + left < steps ? (int)(from + left) : steps;
  }
  const int row0 = x.tile * ROWS, rows = x.tokens * group;

  // this lane's row, what it sees, and what any row of the workgroup sees
  const int row = row0 + w * 32 + n;
  const bool used = row < rows;
  const int token = used ? row / group : 0, head = g * group + (used ? row - token * group : 0);
  const int64_t q_row = x.q0 + token;
  int2 see = sees(a, x, token);
  if (!used) see = {0, 0};
  const int last_row = row0 + ROWS < rows ? row0 + ROWS - 1 : rows - 1;
  const int2 first = sees_uniform(a, x, row0 / group), last = sees_uniform(a, x, last_row / group);
  const int kend = last.y;
  const int t_first = first.x / BN, t_all = (kend + BN - 1) / BN - t_first;
  int tb = t_first, te = t_first + (t_all > 0 ? t_all : 0);
  if constexpr (SHARED) {
    if (t_all == steps) {
      tb = t_first + from;
      te = t_first + to;
    } else {  // a tile whose rows see less than all of the request's: its steps in proportion
      const int64_t mine = te - tb;
      te = tb + (int)quotient(mine * to, steps);
      tb = tb + (int)quotient(mine * from, steps);
    }
  }
  tb = uniform(tb);
  te = uniform(te);

  // q: lane n's row, eight elements a step
  u32x4 q[KSTEPS];
  {
    const char* p = a.query.base + q_row * a.query.token_stride + head * a.query.head_stride;
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      q[s] = u32x4{0, 0, 0, 0};
      if (used && 2 * s + hf < dim / 8) q[s] = gload<u32x4>(p + (2 * s + hf) * 16);
    }
  }

  const char* const base = (const char*)a.cache.base + g * a.cache.head_stride_bytes;
  const int64_t scales = (int64_t)a.cache.block_size * (dim / 2);
  const int32_t* const table = a.batch.block_table + x.r * a.batch.bt_row_stride;
  const int cols = (int)a.batch.max_blocks_per_req;

  f32x16 acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = f32x16{};
  float m = -INFINITY, l = 0;
  const float c1 = a.scale * kLog2e;

  auto load_id = [&](int t) -> int32_t {
    const int b = block_of(div, t * BN + w * KW + slot);
    return gload<int32_t>(table + (b < cols ? b : cols - 1));
  };
  u32x4 rk[KS], rv[KS];
  uint32_t ks[KS], vs[KS];
  uint32_t ok_mask = 0;
  auto fetch = [&](int t, int32_t id) {
    // a slot that is not there is read from the cache's first rows; its scale of V becomes 0, and its weight is
    const int j = t * BN + w * KW + slot;
    const bool wanted = j < kend, ok = wanted && (uint32_t)id < (uint64_t)a.cache.num_blocks;
    bad_blocks |= wanted && !ok;
    ok_mask = (uint32_t)(__ballot(ok) & 0xffff);
    const int64_t o = ok ? j - block_of(div, j) * div.size : 0;
    const char* k = base + (ok ? id * a.cache.block_stride_bytes : 0);
    const char* e = k + o * (dim / 2);
    const char* s = k + scales + o * groups;
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      const int at = c * 4 + quarter;
      rk[c] = rv[c] = u32x4{0, 0, 0, 0};
      ks[c] = vs[c] = 0;
      if (at < groups) {
        rk[c] = gload<u32x4>(e + at * 16);
        ks[c] = gload<uint8_t>(s + at);
        rv[c] = gload<u32x4>(e + at * 16 + a.cache.kv_stride_bytes);
        vs[c] = gload<uint8_t>(s + at + a.cache.kv_stride_bytes);
      }
    }
  };

  int32_t id = 0;
  if (tb < te) {
    fetch(tb, load_id(tb));
    id = load_id(tb + 1);
  }
  // q is here before the loop: a wait for it inside would be one for the loads in flight as well
#pragma unroll
  for (int st = 0; st < KSTEPS; ++st) asm volatile("" : "+v"(q[st]));
  for (int t = tb; t < te; ++t) {
    const int k0 = t * BN;
    // every row sees every slot of an inner tile
    const bool inner = k0 >= last.x && k0 + BN <= first.y;
    if (lane < KW) flags[w * KW + lane] = (ok_mask >> lane) & 1;
    if (ok_mask != 0xffff) {
#pragma unroll
      for (int c = 0; c < KS; ++c)
        if (!(ok_mask >> here(slot) & 1)) ks[c] = vs[c] = 0;
    }
    if (!inner) {
      // A weight of zero times a NaN or infinity is NaN: slots of V that may read back as one are left out of the products and
      // added below for the rows that see them.
      uint64_t bad = 0;
#pragma unroll
      for (int c = 0; c < KS; ++c) bad |= __ballot(vs[c] > kFiniteScales<E>);
      bad |= bad >> 32;
      bad |= bad >> 16;
      if ((bad >> here(slot)) & 1) {
#pragma unroll
        for (int c = 0; c < KS; ++c) vs[c] = 0, rv[c] = u32x4{0, 0, 0, 0};
        if (quarter == 0) flags[w * KW + slot] = 3;
      }
    }
    if (DP >= 128 || quarter * 32 < DP) {
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        const float k_scale = scale_of(ks[c]), v_scale = scale_of(vs[c]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          *(u32x4*)(sk_put + c * 256 + k * 16) = decode<E>(rk[c][k], k_scale);
          *(u32x4*)(smem + ((sv_put + c * 256) ^ (k * 16))) = decode<E>(rv[c][k], v_scale);
        }
      }
    }
    lds_barrier();
    if (t + 1 < te) {
      fetch(t + 1, id);
      id = load_id(t + 2);
    }

    const uint8_t flag = flags[lane];
    // one bit a slot
    const uint64_t there = __ballot(flag & 1), skipped = __ballot(flag & 2);
    // The wavefront that has begun on a tile goes first until it is done: the SIMD's other one does its own part better
    // while these products run.
    __builtin_amdgcn_s_setprio(1);
    f32x16 s[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) s[kt] = f32x16{};
#pragma unroll
    for (int st = 0; st < KSTEPS; ++st)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)  // no product waits for the one before it
        s[kt] = product(E(), *(const u32x4*)(sk_get + kt * 32 * KROW + st * 32), q[st], s[kt]);
    // K is read eight pieces ahead of the products: read as they are needed, each would wait for LDS
    if constexpr (KT * KSTEPS > 8) {
      __builtin_amdgcn_sched_group_barrier(kDsRead, 8, 0);
#pragma unroll
      for (int i = 0; i < KT * KSTEPS - 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(kMfma, 8, 0);
    }
    if (!inner || ~there) {
      const int at = here(k0 + 4 * hf), lo = see.x - at, hi = see.y - at;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const uint32_t mine = (uint32_t)(there >> (kt * 32)) >> here(4 * hf);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int o = 8 * (i / 4) + i % 4;
          if (kt * 32 + o < lo || kt * 32 + o >= hi || !(mine & (1u << o))) s[kt][i] = -INFINITY;
        }
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kt][i]);
    top = fmaxf(top, other_half(top)) * c1;
    // the reference moves only when the maximum leaves its range: the sums keep their 32 bits
    if (__any(top > m + (kLift<E> + kLag<E>))) {
      const float held = m, now = here(top);
      const float to = now - held > kLift<E> + kLag<E> ? (is_far(now) ? now : now - kLift<E>) : held;
      const float shrink = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(held - to);
      m = to;
      l *= shrink;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] *= shrink;
    }
    if (__any(is_far(m))) {
      // the scores become what they stand above the reference, rounded before it is taken from them, as the maximum was
      const float from = m == -INFINITY ? 0.0f : m, factor = here(c1), back = 1.0f / factor;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float up = rounded_difference(rounded_product(s[kt][i], factor), from);
          if (is_far(from)) s[kt][i] = up * back;
        }
    }
    const float ref = m == -INFINITY || is_far(m) ? 0.0f : m;
    // Weights and products by 16 slots: V is read one group ahead, and the weights of a group are formed in the shadow of
    // the products of the one before.
#pragma unroll
    for (int gr = 0; gr < 2 * KT; ++gr) {
      f32x8 pv;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = 8 * (gr % 2) + i;
        pv[i] = s[gr / 2][at] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[gr / 2][at], c1, -ref));
        l += pv[i];
      }
      // one rounding of each weight to the element type, which the matrix unit takes
      const u32x4 p = narrow<E>(pv);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const char* at = sv_get + 16 * gr * VROW + d * 64;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KVX_LDS s16x4*)at);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KVX_LDS s16x4*)(at + 8 * VROW));
        const s16x8 va = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        acc[d] = product(E(), __builtin_bit_cast(u32x4, va), p, acc[d]);
      }
    }
    __builtin_amdgcn_sched_group_barrier(kDsRead, 2 * DT, 1);
    __builtin_amdgcn_sched_group_barrier(kVector, 28, 1);
#pragma unroll
    for (int gr = 0; gr < 2 * KT; ++gr) {
      if (gr + 1 < 2 * KT) __builtin_amdgcn_sched_group_barrier(kDsRead, 2 * DT, 1);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 1);
        if (gr + 1 < 2 * KT) __builtin_amdgcn_sched_group_barrier(kVector, 28 / DT, 1);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (skipped) {
      for (uint64_t todo = skipped; todo; todo &= todo - 1) {
        const int o = __builtin_ctzll(todo), j = k0 + o;
        float pj = 0;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (kt * 32 + 8 * (i / 4) + i % 4 == o - here(4 * hf)) pj = s[kt][i];
        pj += other_half(pj);
        if (j < see.x || j >= see.y) continue;
        const int b = block_of(div, j), in = j - b * div.size;
        const char* plane = base + table[b] * a.cache.block_stride_bytes + a.cache.kv_stride_bytes;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if (d >= groups) break;
          const float scale = scale_of(gload<uint8_t>(plane + scales + (int64_t)in * groups + d));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 v = decode4<E>(gload<uint16_t>(plane + (int64_t)in * (dim / 2) + d * 16 + i * 4 + hf * 2), scale);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[d][4 * i + e] += pj * v[e];
          }
          __builtin_amdgcn_sched_barrier(0);  // a few at a time: this branch must not set the registers of the loop
        }
      }
    }
    lds_barrier();
  }
  l += other_half(l);

  const AttendArgs end = argument<AttendArgs>();
  const bool whole = !SHARED || (from == 0 && to == steps);
  const float inv = l == 0 ? 0.0f : 1.0f / l;
  // where a part's row goes: share index of tile tile0 + x.tile
  const int64_t part = ((int64_t)(index + (int32_t)(tile0 + x.tile)) * end.cache.num_kv_heads + g) * ROWS + (row - row0);
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = d * 32 + 8 * i + 4 * hf;
      if (!used || e >= end.cache.head_dim) continue;
      f32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = l == 0 ? 0.0f : acc[d][4 * i + k] * inv;
      if (SHARED && !whole) {
        gstore(sp.acc + part * end.cache.head_dim + e, v);
      } else {
        gstore((char*)end.out.base + q_row * end.out.token_stride + head * end.out.head_stride + e * 2,
               __builtin_convertvector(v, typename E::V4));
      }
    }
  if (used && hf == 0) {
    const float lse2 = l == 0 ? -INFINITY : m + __builtin_amdgcn_logf(l);
    if (SHARED && !whole) sp.lse[part] = lse2;
    else if (end.lse) end.lse[q_row * end.num_heads + head] = lse2 * kLn2;
  }

  if constexpr (!SHARED) break;
  left -= to - from;
  if (left <= 0) break;
  // the next tile, of this request or of the next one that has any
  from = 0;
  if (++x.tile == tiles) {
    tile0 += tiles;
    do {
      x = request_uniform(a, x.r + 1, cap);
      extent<ROWS, BN>(a, x, group, &tiles, &steps);
      tiles = uniform(tiles);
      steps = uniform(steps);
    } while (tiles == 0);
  }
  }
  if (bad_blocks) raise(a.err, KVX_DEVERR_BLOCK_RANGE);
}

template <class E, int DP>
void launch_attend(const AttendArgs& a, BlockDiv div, const Split& sp, int rows, hipStream_t stream) {
  const int heads = a.cache.num_kv_heads;
  if (sp.shares == 0) {
    const dim3 grid((unsigned)(sp.tiles * heads));
    if (rows == 16) attend_fp4_kernel<E, DP, 1, false><<<grid, 256, 0, stream>>>(a, div, sp);
    else if (rows == 32) attend_fp4_kernel<E, DP, 2, false><<<grid, 256, 0, stream>>>(a, div, sp);
    else attend_fp4_rows_kernel<E, DP, false><<<grid, 256, 0, stream>>>(a, div, sp);
    return;
  }
  const dim3 grid((unsigned)(sp.shares * heads));
  // a tile's rows are joined by one workgroup, or by several while that is up to 2048 in all and they have 32 threads' work each
  // (177 tiles of 128 rows: 13.4 us by 11 workgroups each, 14.3 by 4, 19.8 by 2, 14.7 by 16)
  const int64_t blocks = (int64_t)sp.tiles * heads;
  const int64_t longest = a.batch.max_query_len < a.batch.num_tokens ? a.batch.max_query_len : a.batch.num_tokens;
  const int64_t most = longest * (a.num_heads / heads) * a.cache.head_dim / 128;
  int64_t several = 2048 / blocks;
  several = several < most ? several : most;
  several = several < 1 ? 1 : several < 16 ? several : 16;
  const dim3 join((unsigned)blocks, (unsigned)several);
  if (rows == 16) {
    attend_fp4_kernel<E, DP, 1, true><<<grid, 256, 0, stream>>>(a, div, sp);
    join_kernel<E, 16, 128, kFp4Extra><<<join, 256, 0, stream>>>(a, sp);
  } else if (rows == 32) {
    attend_fp4_kernel<E, DP, 2, true><<<grid, 256, 0, stream>>>(a, div, sp);
    join_kernel<E, 32, 128, kFp4Extra><<<join, 256, 0, stream>>>(a, sp);
  } else {
    attend_fp4_rows_kernel<E, DP, true><<<grid, 256, 0, stream>>>(a, div, sp);
    join_kernel<E, 128, 64><<<join, 256, 0, stream>>>(a, sp);
  }
}

template <class E>
void launch_dims(const AttendArgs& a, BlockDiv div, const Split& sp, int rows, hipStream_t stream) {
  if (a.cache.head_dim <= 64) launch_attend<E, 64>(a, div, sp, rows, stream);
  else if (a.cache.head_dim <= 128) launch_attend<E, 128>(a, div, sp, rows, stream);
  else launch_attend<E, 256>(a, div, sp, rows, stream);
}

}  // namespace

hipError_t launch_attention_fp4(const AttendArgs& a, hipStream_t stream) {
  const Fp4Plan p = plan_attention_fp4(a.cache, a.batch, a.num_heads, a.window);
  Split sp = {fp4_shares_within(p, a.cache, a.workspace_bytes), p.tiles, nullptr, nullptr};
  if (sp.shares > 0) {
    sp.acc = (float*)a.workspace;  // first: rows of 16-byte vectors
    sp.lse = sp.acc + (int64_t)(sp.shares + p.tiles) * a.cache.num_kv_heads * p.rows * a.cache.head_dim;
  }
  const BlockDiv div = block_div(a.cache.block_size);
  if (a.cache.dtype == KVX_DTYPE_BF16) launch_dims<Bf16>(a, div, sp, p.rows, stream);
  else launch_dims<Fp16>(a, div, sp, p.rows, stream);
  return hipGetLastError();
}

int64_t attention_fp4_workspace(const kvx_paged_cache& c, const kvx_batch& b, int32_t num_heads) {
  const Fp4Plan p = plan_attention_fp4(c, b, num_heads);
  return p.shares > 0 ? (p.shares + (int64_t)p.tiles) * fp4_slot_bytes(p, c) : 0;
}

}  // namespace kvx
