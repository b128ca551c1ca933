// gfx950 kernels of kvx_paged_attention and kvx_attention_mass.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_launch.h"
#include "kvx_attention_plan.h"
#include "kvx_attention_rows.h"
#include "kvx_paged.h"

namespace kvx {
namespace {

// --------------------------------------------------------------------------------------
// matrix pieces
// --------------------------------------------------------------------------------------

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mfma(Bf16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Bf16::V8, a), __builtin_bit_cast(Bf16::V8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(Fp16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(Fp16::V8, a), __builtin_bit_cast(Fp16::V8, b), c, 0, 0, 0);
}

// In the 32x32x16 products lane l holds column (or row) l % 32 and, with hf = l / 32, elements
// 8 hf .. 8 hf + 7 of the summed dimension; result register i of lane l is row 8 (i / 4) + 4 hf + i % 4,
// column l % 32.

template <class E>
__device__ __forceinline__ bool non_finite(u32x4 v) {
  constexpr uint32_t exp = sizeof(E) && __is_same(E, Bf16) ? 0x7f80u : 0x7c00u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (v[i] & exp) == exp || ((v[i] >> 16) & exp) == exp;
  return bad;
}

// A buffer that starts at p (the same in all lanes) for loads whose offsets the caller keeps inside
// the memory: a scalar base, a scalar step and a lane's constant offset make an address for nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const char* p) {
  const uint64_t at = (uint64_t)uniform((int64_t)p);
  return __builtin_amdgcn_make_buffer_rsrc((void*)at, 0, 0x7fffffff, 0x00027000);
}

// --------------------------------------------------------------------------------------
// attention
// --------------------------------------------------------------------------------------

// One pass over the slots with a running maximum and sum. Scores are computed transposed, S^T = K Q^T, so that a lane
// holds one query row and 16 slots of each 32: the row's maximum and sum need one exchange between two
// lanes, and the weights are already where O^T += V^T P^T takes them, because the summed dimension may be
// numbered in any order: V is read from LDS with the transposing load, four slots a lane, in the order in
// which the score registers hold them. DP is head_dim padded to 64, 128 or 256.
//   KEYS = false: the four wavefronts hold 32 rows each and share every 64 slots staged in LDS.
//   KEYS = true (up to 32 rows): they hold the same rows and 32 slots each of every 128, meet
//     only at the end, and need no barrier before it: bound by the bytes of K and V.
//   SHARED: the grid's workgroups take equal shares of the whole batch's steps (see Shares).
// K and V go from memory to registers one tile ahead and then to LDS, in rows padded so that the reads of
// 16 rows (K: 16 bytes a row), or of 4 slots x 64 bytes (V: 64 bytes a row), fall on different banks;
// padding, unlike a swizzle, leaves every address one register and a constant.
// The shared variants do not fit their registers whole: at 128 dimensions 10 to 17 values a lane are in scratch (44-72 bytes), at 256
// 70 to 84 (284-340 bytes), all of them what a tile's start and end use, none in the loop over the slots.
template <class E, int DP, bool KEYS, bool BY_BLOCK, bool SHARED>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attend_kernel(AttendArgs args, BlockDiv div, Split sp) {
  const AttendArgs a = argument<AttendArgs>();
  constexpr int ROWS = KEYS ? kRowsKeys : kRows, BN = KEYS ? 128 : 64, KW = BN / 4;
  constexpr int VPR = DP / 8, RPI = 64 / VPR, NI = KW / RPI;
  constexpr int KT = KEYS ? 1 : 2, KSTEPS = DP / 16, DT = DP / 32;
  constexpr int KROW = DP * 2 + 16, VROW = DP * 2 + 64;  // bytes of a row in LDS
  // Q in registers, but for the widest heads' few rows in LDS: their tiles and sums take the registers
  constexpr bool Q_LDS = KEYS && DP > 128;
  __shared__ __align__(16) char smem[BN * (KROW + VROW) + BN + (Q_LDS ? 32 * KROW : 0)];
  char* const sk = smem;
  char* const sv = smem + BN * KROW;
  uint8_t* const flags = (uint8_t*)(smem + BN * (KROW + VROW));

  const int tid = threadIdx.x, lane = tid & 63, w = uniform((int32_t)(tid >> 6));
  const int n = lane & 31, hf = lane >> 5;
  const int group = a.num_heads / a.cache.num_kv_heads, vecs = a.cache.head_dim / 8;
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  // Workgroup i runs on XCD i % 8, each with an L2 of its own: a head's tiles, or shares that follow one another and read
  // the same K and V, to one XCD (8 requests' chunks on one KV head 129 -> 124 us).
  int g = blockIdx.x % a.cache.num_kv_heads, index = blockIdx.x / a.cache.num_kv_heads;
  if constexpr (SHARED) {
    const int xcd = blockIdx.x % 8, per = gridDim.x / 8, more = gridDim.x % 8;
    const int at = xcd * per + (xcd < more ? xcd : more) + blockIdx.x / 8;
    g = at / sp.shares;
    index = at - g * sp.shares;
  }
  if (blockIdx.x == 0) check_batch(a, cap, tid, 256);

  // the padding of every row is zero, once
  const int c = lane % VPR, sub = lane / VPR;  // the 16-byte piece and row this lane stages
  char* const sk_put = sk + (w * KW + sub) * KROW + c * 16;
  char* const sv_put = sv + (w * KW + sub) * VROW + c * 16;
  const int kw = KEYS ? w * KW : 0;  // first slot of a tile that this wavefront computes
  const char* const sk_get = sk + (kw + n) * KROW + hf * 16;
  const char* const sv_get = sv + (kw + 4 * hf + ((lane & 15) >> 2)) * VROW + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
  // This lane's place for the reference of its row: in the padding of the V rows that it stages.
  auto reference = [&]() -> float* {
    const int piece = lane_here() % VPR;
    return (float*)(sv_put - 16 * piece + DP * 2 + 4 * piece + (piece >= 16 ? RPI * VROW - 64 : 0));
  };
  auto clear_padding = [&]() {
    if (vecs < VPR && c >= vecs) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        *(u32x4*)(sk_put + i * RPI * KROW) = u32x4{0, 0, 0, 0};
        *(u32x4*)(sv_put + i * RPI * VROW) = u32x4{0, 0, 0, 0};
      }
    }
  };
  clear_padding();

  // the tiles of rows, and the steps of each, that this workgroup computes
  Rows x;
  Shares all;
  int32_t tiles = 0, steps = 1, from = 0, to = 1;  // steps [from, to) of tile x.tile
  uint32_t tile0 = 0;
  int64_t left = 1;                                           // steps of this share, with those
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
    // The longest tiles first; every other round of 256 workgroups (one a CU) the other way round, so
    // that a CU's second tile makes up for its first.
    const int per = 256 / a.cache.num_kv_heads > 0 ? 256 / a.cache.num_kv_heads : 1, round = index / per;
    const int back = (round + 1) * per < sp.tiles ? (round + 1) * per : sp.tiles;
    x = find_rows<ROWS>(a, sp.tiles - 1 - (round & 1 ? back - 1 - (index - round * per) : index), group, cap, lane);
    // a spare tile, or offsets that are not a CSR
    if (x.tile < 0 || (int64_t)x.tile * ROWS >= (int64_t)x.tokens * group) return;
  }
  int errs = 0;
  bool bad_blocks = false;
  for (;;) {
  const AttendArgs a = argument<AttendArgs>();
  if constexpr (SHARED) {
    if (tile0 + x.tile >= (uint32_t)sp.tiles) break;  // offsets that are not a CSR: the workspace has no slots for more
    to = from + left < steps ? (int)(from + left) : steps;
  }
  const int row0 = x.tile * ROWS, rows = x.tokens * group;

  // this lane's row, what it sees, and what any row of the workgroup sees
  const int row = row0 + (KEYS ? 0 : w * 32) + n;
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

  // Q: lane n's row, eight elements a step
  u32x4 q[Q_LDS ? 1 : KSTEPS];
  char* const sq = smem + BN * (KROW + VROW) + BN + n * KROW + hf * 16;
  {
    const char* p = a.query.base + q_row * a.query.token_stride + head * a.query.head_stride;
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      u32x4 v = {0, 0, 0, 0};
      if (used && 2 * s + hf < vecs) v = gload<u32x4>(p + (2 * s + hf) * 16);
      if constexpr (!Q_LDS) q[s] = v;
      else if (s % 4 == w) *(u32x4*)(sq + s * 32) = v;  // a quarter of the steps each
    }
    if constexpr (Q_LDS) __syncthreads();
  }

  const char* const kbase = (const char*)a.cache.base + g * a.cache.head_stride_bytes + (c < vecs ? c : 0) * 16;
  const int32_t* const table = a.batch.block_table + x.r * a.batch.bt_row_stride;
  const int cols = (int)a.batch.max_blocks_per_req;

  f32x16 acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = f32x16{};
  float m = -INFINITY, l = 0;
  *reference() = m;
  const float c1 = a.scale * kLog2e;

  // Staging. BY_BLOCK, where 16 slots always lie in one block: their rows are token_stride apart, and the block
  // is looked up and the rows' addresses formed once a wavefront, in scalar registers. Otherwise lane
  // l looks up slot l % KW of the wavefront's share and passes the row's offset on.
  constexpr int BLKS = KW / 16;
  const uint32_t v_off = (uint32_t)(sub * (int32_t)a.cache.token_stride_bytes) + (c < vecs ? c : 0) * 16;
  auto load_id = [&](int t) -> int32_t {
    const int b = block_of(div, t * BN + w * KW + lane % KW);
    return gload<int32_t>(table + (b < cols ? b : cols - 1));
  };
  u32x4 rk[NI], rv[NI];
  uint64_t ok_mask = 0;
  auto fetch = [&](int t, int32_t id) {
    // a slot that is not there is read from the cache's first rows and then set to zero
    if constexpr (BY_BLOCK) {
      ok_mask = 0;
#pragma unroll
      for (int k = 0; k < BLKS; ++k) {
        const int32_t block = lane_of(id, k * 16);
        const int j = t * BN + w * KW + k * 16;
        int there = kend - j < 16 ? kend - j : 16;
        if (there < 0) there = 0;
        int64_t off = 0;
        if ((uint32_t)block < (uint64_t)a.cache.num_blocks) {
          off = block * a.cache.block_stride_bytes +
                (int64_t)(j - block_of(div, j) * div.size) * a.cache.token_stride_bytes;
          ok_mask |= (uint64_t)((1u << there) - 1) << (k * 16);
        } else if (there > 0) {
          bad_blocks = true;
        }
        const char* p = (const char*)a.cache.base + g * a.cache.head_stride_bytes + off;
        const auto kr = rows_at(p), vr = rows_at(p + a.cache.kv_stride_bytes);
#pragma unroll
        for (int i = 0; i < NI / BLKS; ++i) {
          const int down = i * RPI * (int32_t)a.cache.token_stride_bytes;
          rk[k * (NI / BLKS) + i] = __builtin_amdgcn_raw_buffer_load_b128(kr, v_off, down, 0);
          rv[k * (NI / BLKS) + i] = __builtin_amdgcn_raw_buffer_load_b128(vr, v_off, down, 0);
        }
      }
      ok_mask |= ok_mask << 32;  // lanes l and l + 32 stand for the same slot
      if (KW == 16) ok_mask |= ok_mask << 16;
      return;
    } else {
    const int j = t * BN + w * KW + lane % KW;
    const bool in = j < kend, ok = in && (uint32_t)id < (uint64_t)a.cache.num_blocks;
    if (in && !ok) errs |= KVX_DEVERR_BLOCK_RANGE;
    const int64_t off = ok ? id * a.cache.block_stride_bytes +
                                 (int64_t)(j - block_of(div, j) * div.size) * a.cache.token_stride_bytes
                           : 0;
    ok_mask = __ballot(ok);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const char* p = kbase + __shfl(off, i * RPI + sub);
      rk[i] = gload<u32x4>(p);
      rv[i] = gload<u32x4>(p + a.cache.kv_stride_bytes);
    }
    }
  };

  int32_t id = 0;
  tb = uniform(tb);
  te = uniform(te);
  if (tb < te) {
    fetch(tb, load_id(tb));
    id = load_id(tb + 1);
  }
  // Q is here before the loop: a wait for it inside would be one for the loads in flight as well
#pragma unroll
  for (int st = 0; st < (Q_LDS ? 0 : KSTEPS); ++st) asm volatile("" : "+v"(q[st]));
  for (int t = tb; t < te; ++t) {
    const int k0 = t * BN;
    // every row sees every slot of an inner tile
    const bool inner = k0 >= last.x && k0 + BN <= first.y;
    if (lane < KW) flags[w * KW + lane] = (ok_mask >> lane) & 1;
    if (~ok_mask) {
      const uint32_t mine = (uint32_t)(ok_mask >> here(sub));
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (!(mine & (1u << (i * RPI)))) rk[i] = rv[i] = u32x4{0, 0, 0, 0};
    }
    if (!inner) {
      // A weight of zero times a NaN or infinity is NaN: rows of V that hold one are left out of the
      // products and added below for the query rows that see them.
      const int from = here(sub);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint64_t bad = __ballot(c < vecs && non_finite<E>(rv[i]));
        if (bad == 0) continue;
        if ((bad >> (from * VPR)) & ((1ull << VPR) - 1)) {
          rv[i] = u32x4{0, 0, 0, 0};
          if (c == 0) flags[w * KW + i * RPI + from] = 3;
        }
      }
    }
    if (c < vecs) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        *(u32x4*)(sk_put + i * RPI * KROW) = rk[i];
        *(u32x4*)(sv_put + i * RPI * VROW) = rv[i];
      }
    }
    if constexpr (KEYS) __builtin_amdgcn_wave_barrier();
    else lds_barrier();
    if (t + 1 < te) {
      fetch(t + 1, id);
      id = load_id(t + 2);
    }

    const uint8_t flag = flags[kw + (lane & (KT * 32 - 1))];
    // one bit a slot of this wavefront; with KEYS its 32 slots are read twice
    const uint64_t there = __ballot(flag & 1), skipped = __ballot((flag & 2) && lane < KT * 32);
    // The wavefront that has begun on a tile goes first until it is done: the SIMD's other one does its own part better
    // while these products run (1192 -> 1122 us at 2048 queries of 32 heads over 32768 slots from the weights on, 1112 from here).
    __builtin_amdgcn_s_setprio(1);
    f32x16 s[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) s[kt] = f32x16{};
#pragma unroll
    for (int st = 0; st < KSTEPS; ++st)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)  // no product waits for the one before it
        s[kt] = mfma(E(), *(const u32x4*)(sk_get + kt * 32 * KROW + st * 32),
                     Q_LDS ? *(const u32x4*)(sq + st * 32) : q[Q_LDS ? 0 : st], s[kt]);
    // K is read eight pieces ahead of the products: read as they are needed, each would wait for LDS. The compiler keeps to
    // this order in the unshared variants at 128 dimensions (rows: by block) and in part at 64 and 256, but not in the shared ones,
    // whose registers are full.
    if constexpr (!Q_LDS) {
    __builtin_amdgcn_sched_group_barrier(kDsRead, 8, 0);
#pragma unroll
    for (int i = 0; i < KT * KSTEPS - 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, 8, 0);
    }
    if (!inner || ~there) {
      const int at = here(k0 + kw + 4 * hf), lo = see.x - at, hi = see.y - at;
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
    // The reference moves only when the maximum leaves its range: the sums keep their 32 bits. What only this needs is kept
    // in LDS or formed here: with a register more in the loop the compiler no longer reads K ahead of the products above
    // (1042 -> 1150 us at 2048 queries of 32 heads over 32768 slots).
    if (__any(top > m + (kLift<E> + kLag<E>))) {
      float* const mine = reference();
      const float held = *mine, now = here(top);
      const float to = now - held > kLift<E> + kLag<E> ? (is_far(now) ? now : now - kLift<E>) : held;
      const float shrink = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(held - to);
      *mine = m = to;
      l *= shrink;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] *= shrink;
      if (__any(is_far(to))) {
        // the scores become what they stand above the reference, and m is such that the next tile comes here again
        const float from = to == -INFINITY ? 0.0f : to, factor = here(c1), back = 1.0f / factor;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[kt][i] = rounded_difference(rounded_product(s[kt][i], factor), from) * back;
        m = -INFINITY;
      }
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    // Weights and products by 16 slots: V is read one group ahead, and the weights of a group are
    // formed in the shadow of the products of the one before.
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
        acc[d] = mfma(E(), __builtin_bit_cast(u32x4, va), p, acc[d]);
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
        const int o = __builtin_ctzll(todo), j = k0 + kw + o;
        float pj = 0;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (kt * 32 + 8 * (i / 4) + i % 4 == o - here(4 * hf)) pj = s[kt][i];
        pj += other_half(pj);
        if (j < see.x || j >= see.y) continue;
        const int b = block_of(div, j);
        const char* p = (const char*)a.cache.base + table[b] * a.cache.block_stride_bytes +
                        (int64_t)(j - b * div.size) * a.cache.token_stride_bytes + a.cache.kv_stride_bytes +
                        g * a.cache.head_stride_bytes + hf * 8;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (d * 32 + 8 * i >= a.cache.head_dim) break;
            const f32x4 v = __builtin_convertvector(gload<typename E::V4>(p + d * 64 + i * 16), f32x4);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[d][4 * i + e] += pj * v[e];
          }
          __builtin_amdgcn_sched_barrier(0);  // a few at a time: this branch must not set the registers of the loop
        }
      }
    }
    if constexpr (KEYS) __builtin_amdgcn_wave_barrier();
    else lds_barrier();
  }
  l += other_half(l);
  m = *reference();

  if constexpr (KEYS) {
    // join the wavefronts: weights of each one's sum, then the sums themselves through LDS
    float* const sm = (float*)smem;
    __syncthreads();
    if (lane < 32) {
      sm[w * 32 + n] = m;
      sm[128 + w * 32 + n] = l;
    }
    __syncthreads();
    float top = -INFINITY, total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, sm[i * 32 + n]);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < 4; ++i) total += sm[128 + i * 32 + n] * __builtin_amdgcn_exp2f(sm[i * 32 + n] - ref);
    const float mine = __builtin_amdgcn_exp2f(m - ref);
    __syncthreads();
    // [wavefront][row][16-byte pieces, swizzled by row]
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[d][4 * i + e] * mine;
        const int piece = d * 8 + 2 * i + hf;
        *(f32x4*)(smem + ((w * 32 + n) * (DP / 4) + (piece ^ (n & 15))) * 16) = v;
      }
    m = top;
    l = total;
    __syncthreads();
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      // wavefront w takes register quad w of each 32 dimensions
      f32x4 v = {};
      const int piece = d * 8 + 2 * w + hf;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v += *(const f32x4*)(smem + ((i * 32 + n) * (DP / 4) + (piece ^ (n & 15))) * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[d][e] = v[e];
    }
  }

  const AttendArgs end = argument<AttendArgs>();
  const bool whole = !SHARED || (from == 0 && to == steps);
  const float inv = l == 0 ? 0.0f : 1.0f / l;
  // where a part's row goes: share index of tile tile0 + x.tile
  const int64_t part = ((int64_t)(index + (int32_t)(tile0 + x.tile)) * end.cache.num_kv_heads + g) * ROWS + (row - row0);
  constexpr int QUADS = KEYS ? 1 : 4;  // register quads of each 32 dimensions that this lane stores
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < QUADS; ++i) {
      const int e = d * 32 + 8 * (KEYS ? w : i) + 4 * hf;
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
  if (used && hf == 0 && (!KEYS || w == 0)) {
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
  if constexpr (KEYS) {
    __syncthreads();  // the join above has used the tiles' LDS
    clear_padding();
  }
  }
  if (bad_blocks) errs |= KVX_DEVERR_BLOCK_RANGE;
  if (errs) raise(a.err, errs);
}

template <class E, int DP>
void launch_attend(const AttendArgs& a, BlockDiv div, const Split& sp, bool keys, hipStream_t stream) {
  const int heads = a.cache.num_kv_heads;
  // Blocks of a multiple of 16 tokens, as they usually are: addresses by block, which spares the vector unit (a
  // long chunk 1125 -> 1081 us). The decode kernel waits for memory instead, and is faster without (138 against 148 us).
  const bool by_block = a.cache.block_size % 16 == 0 && a.cache.token_stride_bytes <= (1 << 24);
  if (sp.shares == 0) {
    const dim3 grid((unsigned)(sp.tiles * heads));
    if (keys) attend_kernel<E, DP, true, false, false><<<grid, 256, 0, stream>>>(a, div, sp);
    else if (by_block) attend_kernel<E, DP, false, true, false><<<grid, 256, 0, stream>>>(a, div, sp);
    else attend_kernel<E, DP, false, false, false><<<grid, 256, 0, stream>>>(a, div, sp);
    return;
  }
  const dim3 grid((unsigned)(sp.shares * heads));
  // A tile's rows are joined by one workgroup, or by several while that is up to 2048 in all (one round of them on
  // the CUs) and they have 32 threads' work each: each first finds its tile again, so more cost more than they read.
  const int64_t blocks = (int64_t)sp.tiles * heads;
  const int64_t longest = a.batch.max_query_len < a.batch.num_tokens ? a.batch.max_query_len : a.batch.num_tokens;
  const int64_t most = longest * (a.num_heads / heads) * a.cache.head_dim / 128;
  int64_t several = 2048 / blocks;
  several = several < most ? several : most;
  several = several < 1 ? 1 : several < 16 ? several : 16;
  const dim3 join((unsigned)blocks, (unsigned)several);
  if (keys) {
    attend_kernel<E, DP, true, false, true><<<grid, 256, 0, stream>>>(a, div, sp);
    join_kernel<E, kRowsKeys, 128><<<join, 256, 0, stream>>>(a, sp);
  } else {
    if (by_block) attend_kernel<E, DP, false, true, true><<<grid, 256, 0, stream>>>(a, div, sp);
    else attend_kernel<E, DP, false, false, true><<<grid, 256, 0, stream>>>(a, div, sp);
    join_kernel<E, kRows, 64><<<join, 256, 0, stream>>>(a, sp);
  }
}

template <class E>
void launch_attend_dims(const AttendArgs& a, BlockDiv div, const Split& sp, bool keys, hipStream_t stream) {
  if (a.cache.head_dim <= 64) launch_attend<E, 64>(a, div, sp, keys, stream);
  else if (a.cache.head_dim <= 128) launch_attend<E, 128>(a, div, sp, keys, stream);
  else launch_attend<E, 256>(a, div, sp, keys, stream);
}

// --------------------------------------------------------------------------------------
// attention mass
// --------------------------------------------------------------------------------------

// The rows of a request that a mass kernel works on, and what it may touch of the masses.
struct MassRows {
  Rows x;
  int rows, from, end;  // query rows; slots [from, end) that some row sees and the masses hold
};
__device__ __forceinline__ bool mass_rows(const MassArgs& ma, int r, int group, int64_t cap, MassRows* m) {
  const AttendArgs& a = ma.at;
  m->x = request(a, r, cap);
  const Rows& x = m->x;
  if (x.context > ma.mass_width && blockIdx.y == 0) raise(a.err, KVX_DEVERR_TABLE_RANGE);
  if (x.tokens == 0) return false;
  m->rows = x.tokens * group;
  m->from = sees(a, x, 0).x;
  const int last = sees(a, x, x.tokens - 1).y;
  m->end = last < ma.mass_width ? last : (int)ma.mass_width;
  return true;
}

// Loads a tile of rows as the memory holds them, 16 consecutive bytes a lane and whole rows by
// neighbouring lanes, and passes it through LDS to the lanes that the products want it in: read
// by those lanes directly, each would touch a line of its own, and the address unit, not
// memory, would set the pace (a decode batch's masses: 108 us against 92).
template <int DP, int TILE>
struct RowTile {
  static constexpr int VPR = DP / 8, RPI = 64 / VPR, NI = TILE / RPI, ROW = DP * 2 + 16;
  u32x4 v[NI];
  // where(i): address of row i * RPI + lane / VPR, whose piece lane % VPR this lane loads
  template <class F>
  __device__ __forceinline__ void load(F where, int lane, int vecs) {
    const int c = lane % VPR, from = c < vecs ? c * 16 : 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = gload<u32x4>(where(i) + from);
  }
  __device__ __forceinline__ void put(char* lds, int lane, int vecs) const {
    const int c = lane % VPR;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      *(u32x4*)(lds + (i * RPI + lane / VPR) * ROW + c * 16) = v[i];
    if (c >= vecs) {
#pragma unroll
      for (int i = 0; i < NI; ++i) *(u32x4*)(lds + (i * RPI + lane / VPR) * ROW + c * 16) = u32x4{0, 0, 0, 0};
    }
  }
};

// A lane's way through the rows (token, head of the group) of one KV head: found by a division once, and by a
// comparison from then on, as the rows pass by in equal steps. Divided anew, the rows of a tile took
// half as many instructions as its weights (61 tokens of 32 heads over 32749 slots and 56 over 9295 48 -> 45 us; a prompt's
// 8192 tokens of 8 heads 558 -> 345 us).
struct RowWalk {
  int32_t token, head;
  int64_t off;  // in bytes, from the request's first row
  __device__ __forceinline__ void start(int row, int group, int64_t token_stride, int64_t head_stride) {
    token = row / group;
    head = row - token * group;
    off = token * token_stride + head * head_stride;
  }
  __device__ __forceinline__ void advance(int rows, int group, int64_t token_stride, int64_t head_stride) {
    const int tokens = rows / group, heads = rows - tokens * group;  // the same in every lane
    const int64_t by = tokens * token_stride + heads * head_stride;
    head += heads;
    const bool over = head >= group;
    head -= over ? group : 0;
    token += over ? tokens + 1 : tokens;
    off += over ? by + token_stride - group * head_stride : by;
  }
};
// The rows of the mass kernels' loops.
template <class Q>
struct RowLoads {
  const char *query, *lse;  // the request's first row's
  int64_t lse_stride;       // of a token
  int32_t first_end, window;  // the first token sees slots up to first_end
  RowWalk qs, ls;
  __device__ __forceinline__ void setup(const AttendArgs& a, const Rows& x, int g, int group) {
    query = a.query.base + x.q0 * a.query.token_stride + (int64_t)g * group * a.query.head_stride;
    lse = (const char*)(a.lse + x.q0 * a.num_heads + g * group);
    lse_stride = (int64_t)a.num_heads * 4;
    first_end = x.context - x.tokens + 1;
    window = a.window < 0x7fffffff ? (int32_t)a.window : 0x7fffffff;
  }
  // row: of the tile's rows, the first that this lane loads a piece of; mine: the one whose weights it forms
  __device__ __forceinline__ void start(const AttendArgs& a, int group, int row, int mine) {
    qs.start(row, group, a.query.token_stride, a.query.head_stride);
    ls.start(mine, group, lse_stride, 4);
  }
  // Loads tile rows from row on; left: of the rows from that one on, those that there are; a row past
  // the last reads the first token's and sees nothing. Then on by step rows.
  __device__ __forceinline__ void load(const AttendArgs& a, const Rows& x, int group, int lane, int vecs, int left, int n,
                                       int first, int step, Q& q, int2* see, float* l) {
    RowWalk w = qs;
    q.load([&](int i) {
      const int64_t off = first + i * Q::RPI + lane / Q::VPR < left ? w.off : 0;
      w.advance(Q::RPI, group, a.query.token_stride, a.query.head_stride);
      return query + off;
    }, lane, vecs);
    qs.advance(step, group, a.query.token_stride, a.query.head_stride);
    const bool used = n < left;
    *l = gload<float>((const float*)(lse + (used ? ls.off : 0)));
    int hi = a.causal ? first_end + ls.token : x.context;
    hi = hi < 0 || !used ? 0 : hi;
    *see = {hi > window ? hi - window : 0, hi};
    ls.advance(step, group, lse_stride, 4);
  }
};

// Adds the weights exp(x - lse) of 64 slots from k0 to a lane's sums: its row sees slots [now.x, now.y).
struct Nothing {
  __device__ __forceinline__ void operator()() const {}
};
template <class F = Nothing>  // order: of the weights and what stands before them
__device__ __forceinline__ void add_weights(f32x16 (&s)[2], f32x16 (&sum)[2], int2 now, int k0, int hf, float c1, float ref,
                                            F order = F()) {
  const bool whole = __all(now.x <= k0 && now.y >= k0 + 64);
#pragma unroll
  for (int kt = 0; kt < 2; ++kt)
#pragma unroll
    for (int i = 0; i < 16; ++i) s[kt][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][i], c1, -ref));
#pragma unroll
  for (int kt = 0; kt < 2; ++kt)
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+v"(s[kt][i]));  // all formed here, not behind the branch
  order();
#pragma unroll
  for (int kt = 0; kt < 2; ++kt) {
    if (!whole) {
      const int to = here(k0 + kt * 32 + 4 * hf), lo = now.x - to, hi = now.y - to;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int o = 8 * (i / 4) + i % 4;
        if (o < lo || o >= hi) s[kt][i] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[kt][i] += s[kt][i];
  }
}
// The lanes' sums of 64 slots joined through LDS of the wavefront's own: lane l gets slot l's.
template <int LROW>
__device__ __forceinline__ float row_sums(char* own, const f32x16 (&sum)[2], int lane) {
  float* const mine = (float*)own;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int kt = 0; kt < 2; ++kt)
#pragma unroll
    for (int i = 0; i < 16; ++i) mine[(kt * 32 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4) * LROW + (lane & 31)] = sum[kt][i];
  __builtin_amdgcn_wave_barrier();
  f32x4 t = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) t += *(const f32x4*)(mine + lane * LROW + i * 4);
  return (t[0] + t[1]) + (t[2] + t[3]);
}

// A wavefront owns 64 slots of one KV head: their K stays in registers, the query rows pass by 32 at a
// time (through LDS, for all four wavefronts), and the weights exp(x - lse) of S^T = K Q^T add up in the
// score registers' own layout, a partial sum a lane; the lanes' sums meet once at the end, through
// LDS. Every slot belongs to one wavefront, so nothing is joined between workgroups and the order of
// the sum is fixed. The exponentials bound it, then the products.
constexpr int kMassSlots = 256;  // of a workgroup
// Workgroups that fill the GPU with few rows. A decode step's time hardly changes with their size between a launch too large (128
// slots each) and too uneven (8192): 32 requests of up to 8192 slots, 8 KV heads, 101 us with 128 slots, 90 with the rule's 512,
// 101 with 2048, 116 with 8192; 256 on one KV head 101, 83 (rule), 87, 102; one of 131072 58, 48 with the rule's 256, 46, 103. The
// most, 4096 slots, keeps a batch too large for the rule from that end.
constexpr int kMassFill = 4096;

template <class E, int DP>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void mass_kernel(MassArgs ma, BlockDiv div) {
  typedef RowTile<DP, 32> KTile;
  typedef RowTile<DP, 8> QTile;  // a wavefront's share of 32 rows
  constexpr int KSTEPS = DP / 16, LROW = 36, ROW = KTile::ROW;  // LROW: floats of a slot's partial sums in LDS
  constexpr int OWN = 32 * ROW > 64 * LROW * 4 ? 32 * ROW : 64 * LROW * 4;
  __shared__ __align__(16) char smem[4 * OWN + 2 * 32 * ROW];
  const AttendArgs& a = ma.at;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, hf = lane >> 5, g = blockIdx.x, r = blockIdx.z;
  const int group = a.num_heads / a.cache.num_kv_heads, vecs = a.cache.head_dim / 8;
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  if (blockIdx.y == 0 && g == 0 && r == 0) check_batch(a, cap, tid, 256);
  MassRows m;
  if (!mass_rows(ma, r, group, cap, &m)) return;
  const Rows& x = m.x;
  const float c1 = a.scale * kLog2e;
  const int32_t* const table = a.batch.block_table + r * a.batch.bt_row_stride;
  RowLoads<QTile> rows;
  rows.setup(a, x, g, group);
  char* const own = smem + w * OWN;       // K on its way to registers, then partial sums
  char* const qs = smem + 4 * OWN;        // two tiles of query rows
  int errs = 0;

  for (int64_t at = (int64_t)blockIdx.y * kMassSlots; at < m.end; at += (int64_t)gridDim.y * kMassSlots) {
    if (at + kMassSlots <= m.from) continue;
    const int k0 = (int)at + w * 64;
    // lanes look up one slot each
    const int j = k0 + lane;
    const bool in = j >= m.from && j < m.end;
    const int32_t id = in ? table[block_of(div, j)] : -1;
    const bool ok = in && (uint32_t)id < (uint64_t)a.cache.num_blocks;
    if (in && !ok) errs |= KVX_DEVERR_BLOCK_RANGE;
    const int64_t off = ok ? id * a.cache.block_stride_bytes +
                                 (int64_t)(j - block_of(div, j) * div.size) * a.cache.token_stride_bytes
                           : 0;
    float* const mass = ma.mass + r * ma.mass_req_stride + g * ma.mass_head_stride + j;
    float before = 0;
    if (ok) before = gload<float>(mass);
    u32x4 k[2][KSTEPS];
    {
      KTile t[2];
      const char* const base = (const char*)a.cache.base + g * a.cache.head_stride_bytes;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
        t[kt].load([&](int i) { return base + __shfl(off, kt * 32 + i * KTile::RPI + lane / KTile::VPR); }, lane, vecs);
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        t[kt].put(own, lane, vecs);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int st = 0; st < KSTEPS; ++st) k[kt][st] = *(const u32x4*)(own + n * ROW + st * 32 + hf * 16);
        __builtin_amdgcn_wave_barrier();
      }
    }
    // the rows that see some of the workgroup's slots
    int row_from = 0, row_to = m.rows;
    if (a.causal) {
      const int64_t t0 = at - x.context + x.tokens, t1 = t0 + kMassSlots + a.window;
      if (t0 > 0) row_from = t0 < x.tokens ? (int)t0 * group : m.rows;
      if (t1 < x.tokens) row_to = t1 > 0 ? (int)t1 * group : 0;
    }
    f32x16 sum[2] = {f32x16{}, f32x16{}};
    QTile q;
    int2 see;
    float lse;
    rows.start(a, group, row_from + w * 8 + lane / QTile::VPR, row_from + n);
    auto load_rows = [&](int row0) {
      rows.load(a, x, group, lane, vecs, row_to - row0, n, w * 8, 32, q, &see, &lse);
    };
    // The products of one tile of rows run while the weights of the one before are formed.
    f32x16 s[2][2];
    int2 now[2];
    float ref[2];
    int row0 = row_from, turn = 0;
    auto scores = [&](int to) {
      char* const tile = qs + turn * 32 * ROW;
      q.put(tile + w * 8 * ROW, lane, vecs);
      ref[to] = lse * kLog2e;
      now[to] = lse == -INFINITY ? int2{0, 0} : see;
      // The other tile is written next, which every wavefront has read before this barrier.
      lds_barrier();
      row0 += 32;
      turn ^= 1;
      if (row0 < row_to) load_rows(row0);
      s[to][0] = s[to][1] = f32x16{};
#pragma unroll
      for (int st = 0; st < KSTEPS; ++st) {
        const u32x4 qf = *(const u32x4*)(tile + n * ROW + st * 32 + hf * 16);
        s[to][0] = mfma(E(), k[0][st], qf, s[to][0]);
        s[to][1] = mfma(E(), k[1][st], qf, s[to][1]);
      }
    };
    auto interleave = [&]() {
      __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 2);
#pragma unroll
      for (int st = 0; st < KSTEPS; ++st) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 2);
        __builtin_amdgcn_sched_group_barrier(kVector, 64 / (2 * KSTEPS), 2);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 2);
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 2);
        __builtin_amdgcn_sched_group_barrier(kVector, 64 / (2 * KSTEPS), 2);
      }
    };
    if (row0 < row_to) {
      load_rows(row0);
      scores(0);
      for (;;) {
        if (row0 >= row_to) {
          add_weights(s[0], sum, now[0], k0, hf, c1, ref[0]);
          break;
        }
        scores(1);
        add_weights(s[0], sum, now[0], k0, hf, c1, ref[0], interleave);
        if (row0 >= row_to) {
          add_weights(s[1], sum, now[1], k0, hf, c1, ref[1]);
          break;
        }
        scores(0);
        add_weights(s[1], sum, now[1], k0, hf, c1, ref[1], interleave);
      }
    }
    const float total = row_sums<LROW>(own, sum, lane);
    if (ok) gstore(mass, before + total);
    lds_barrier();  // the query tiles and the partial sums are free again
  }
  if (errs) raise(a.err, errs);
}

// The same where there are too few slots to fill the GPU that way, as with a whole prompt's rows: a workgroup's
// wavefronts share 64 slots and take the tiles of rows in turn, each through LDS of its own; their sums
// meet at the end, in order (a prompt of 8192 tokens of 8 heads on one KV head: 2084 us by mass_kernel, 345 so).
// The widest heads have four, which leaves each the registers for its rows (1682 -> 839 us at 256).
template <int DP>
constexpr int kMassWaves = DP <= 128 ? 8 : 4;

template <class E, int DP>
__global__ __launch_bounds__(64 * kMassWaves<DP>, DP <= 128 ? 2 : 1) void mass_rows_kernel(MassArgs ma, BlockDiv div) {
  typedef RowTile<DP, 64 / kMassWaves<DP>> KTile;  // a wavefront's share of 64 slots
  typedef RowTile<DP, 32> QTile;
  constexpr int KSTEPS = DP / 16, LROW = 36, ROW = QTile::ROW;
  constexpr int OWN = 32 * ROW > 64 * LROW * 4 ? 32 * ROW : 64 * LROW * 4;
  __shared__ __align__(16) char smem[kMassWaves<DP> * OWN];
  __shared__ float sums[kMassWaves<DP>][64];
  const AttendArgs& a = ma.at;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform((int32_t)(tid >> 6));
  const int n = lane & 31, hf = lane >> 5, g = blockIdx.x, r = blockIdx.z;
  const int group = a.num_heads / a.cache.num_kv_heads, vecs = a.cache.head_dim / 8;
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  if (blockIdx.y == 0 && g == 0 && r == 0) check_batch(a, cap, tid, 64 * kMassWaves<DP>);
  MassRows m;
  if (!mass_rows(ma, r, group, cap, &m)) return;
  const Rows& x = m.x;
  const float c1 = a.scale * kLog2e;
  const int32_t* const table = a.batch.block_table + r * a.batch.bt_row_stride;
  RowLoads<QTile> rows;
  rows.setup(a, x, g, group);
  char* const own = smem + w * OWN;
  int errs = 0;

  for (int64_t at = (int64_t)blockIdx.y * 64; at < m.end; at += (int64_t)gridDim.y * 64) {
    if (at + 64 <= m.from) continue;
    const int k0 = (int)at, j = k0 + lane;
    const bool in = j >= m.from && j < m.end;
    const int32_t id = in ? table[block_of(div, j)] : -1;
    const bool ok = in && (uint32_t)id < (uint64_t)a.cache.num_blocks;
    if (in && !ok) errs |= KVX_DEVERR_BLOCK_RANGE;
    const int64_t off = ok ? id * a.cache.block_stride_bytes +
                                 (int64_t)(j - block_of(div, j) * div.size) * a.cache.token_stride_bytes
                           : 0;
    u32x4 k[2][KSTEPS];
    {
      KTile t;
      const char* const base = (const char*)a.cache.base + g * a.cache.head_stride_bytes;
      constexpr int SHARE = 64 / kMassWaves<DP>;
      t.load([&](int i) { return base + __shfl(off, w * SHARE + i * KTile::RPI + lane / KTile::VPR); }, lane, vecs);
      t.put(smem + w * SHARE * ROW, lane, vecs);
      lds_barrier();
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int st = 0; st < KSTEPS; ++st)
          k[kt][st] = *(const u32x4*)(smem + (kt * 32 + n) * ROW + st * 32 + hf * 16);
      lds_barrier();
    }
    int row_from = 0, row_to = m.rows;
    if (a.causal) {
      const int64_t t0 = at - x.context + x.tokens, t1 = t0 + 64 + a.window;
      if (t0 > 0) row_from = t0 < x.tokens ? (int)t0 * group : m.rows;
      if (t1 < x.tokens) row_to = t1 > 0 ? (int)t1 * group : 0;
    }
    f32x16 sum[2] = {f32x16{}, f32x16{}};
    QTile q;
    int2 see;
    float lse;
    rows.start(a, group, row_from + w * 32 + lane / QTile::VPR, row_from + w * 32 + n);
    auto load_rows = [&](int row0) {
      rows.load(a, x, group, lane, vecs, row_to - row0, n, 0, 32 * kMassWaves<DP>, q, &see, &lse);
    };
    constexpr int STEP = 32 * kMassWaves<DP>;
    int row0 = row_from + w * 32;
    if (row0 < row_to) load_rows(row0);
    for (; row0 < row_to; row0 += STEP) {
      q.put(own, lane, vecs);
      const float ref = lse * kLog2e;
      const int2 now = lse == -INFINITY ? int2{0, 0} : see;
      __builtin_amdgcn_wave_barrier();
      if (row0 < row_to - STEP) load_rows(row0 + STEP);
      f32x16 s[2] = {f32x16{}, f32x16{}};
#pragma unroll
      for (int st = 0; st < KSTEPS; ++st) {
        const u32x4 qf = *(const u32x4*)(own + n * ROW + st * 32 + hf * 16);
        s[0] = mfma(E(), k[0][st], qf, s[0]);
        s[1] = mfma(E(), k[1][st], qf, s[1]);
      }
      __builtin_amdgcn_wave_barrier();
      add_weights(s, sum, now, k0, hf, c1, ref);
    }
    const float total = row_sums<LROW>(own, sum, lane);
    sums[w][lane] = total;
    lds_barrier();
    if (w == 0 && ok) {
      float* const mass = ma.mass + r * ma.mass_req_stride + g * ma.mass_head_stride + j;
      float t = 0;
#pragma unroll
      for (int i = 0; i < kMassWaves<DP>; ++i) t += sums[i][lane];
      gstore(mass, gload<float>(mass) + t);
    }
    lds_barrier();
  }
  if (errs && w == 0) raise(a.err, errs);
}

// The same for up to 32 query rows of a KV head, a decode step's: the rows stay in registers and the
// slots pass by, 32 a wavefront and step with the next step's K on its way: the bytes of K bound it.
template <class E, int DP>
__global__ __launch_bounds__(256, DP <= 128 ? 3 : 2) void mass_few_kernel(MassArgs ma, BlockDiv div, int span) {
  typedef RowTile<DP, 32> Tile;
  constexpr int KSTEPS = DP / 16, LROW = 36, ROW = Tile::ROW;
  constexpr int OWN = 32 * ROW > 32 * LROW * 4 ? 32 * ROW : 32 * LROW * 4;
  __shared__ __align__(16) char smem[4 * OWN];
  const AttendArgs& a = ma.at;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, hf = lane >> 5, g = blockIdx.x, r = blockIdx.z;
  const int group = a.num_heads / a.cache.num_kv_heads, vecs = a.cache.head_dim / 8;
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  if (blockIdx.y == 0 && g == 0 && r == 0) check_batch(a, cap, tid, 256);
  MassRows m;
  if (!mass_rows(ma, r, group, cap, &m)) return;
  const Rows& x = m.x;
  const int32_t* const table = a.batch.block_table + r * a.batch.bt_row_stride;
  const char* const base = (const char*)a.cache.base + g * a.cache.head_stride_bytes;
  float* const masses = ma.mass + r * ma.mass_req_stride + g * ma.mass_head_stride;
  const float c1 = a.scale * kLog2e;
  char* const own = smem + w * OWN;  // K, then the weights
  int errs = 0;

  u32x4 q[KSTEPS];
  int2 see;
  float ref;
  auto load_rows = [&](int row0) {
    const int row = row0 + n;
    const bool used = row < m.rows;
    const int token = used ? row / group : 0, head = g * group + (used ? row - token * group : 0);
    const char* p = a.query.base + (x.q0 + token) * a.query.token_stride + head * a.query.head_stride;
    const float lse = gload<float>(a.lse + (x.q0 + token) * a.num_heads + head);
#pragma unroll
    for (int st = 0; st < KSTEPS; ++st) {
      const int c = 2 * st + hf;
      q[st] = gload<u32x4>(p + (c < vecs ? c : 0) * 16);
      if (DP / 8 != vecs && c >= vecs) q[st] = u32x4{0, 0, 0, 0};
    }
    see = used && lse != -INFINITY ? sees(a, x, token) : int2{0, 0};
    ref = lse * kLog2e;
  };

  for (int64_t at = (int64_t)blockIdx.y * span; at < m.end; at += (int64_t)gridDim.y * span) {
    // this wavefront's steps: slots from, from + 128, ... below to
    const int to = at + span < m.end ? (int)at + span : m.end;
    const int skip = m.from > at ? (int)((m.from - at) / 128 * 128) : 0;
    const int from = (int)at + skip + w * 32;
    if (from >= to) continue;
    bool ok;
    Tile k;
    float before;
    auto look_up = [&](int k0) -> int32_t {  // lanes l and l + 32: slot k0 + l
      const int j = k0 + n;
      return j >= m.from && j < to ? table[block_of(div, j)] : -1;
    };
    auto load_k = [&](int k0, int32_t id) {
      const int j = k0 + n;
      const bool in = j >= m.from && j < to;
      ok = in && (uint32_t)id < (uint64_t)a.cache.num_blocks;
      if (in && !ok) errs |= KVX_DEVERR_BLOCK_RANGE;
      const int64_t off = ok ? id * a.cache.block_stride_bytes +
                                   (int64_t)(j - block_of(div, j) * div.size) * a.cache.token_stride_bytes
                             : 0;
      k.load([&](int i) { return base + __shfl(off, i * Tile::RPI + lane / Tile::VPR); }, lane, vecs);
      before = ok ? gload<float>(masses + j) : 0.0f;
    };
    // one pass over the slots; more only where a request has more rows than the hint said
    for (int row0 = 0; row0 < m.rows; row0 += 32) {
      load_k(from, look_up(from));
      int32_t id = from + 128 < to ? look_up(from + 128) : -1;
      load_rows(row0);
      // here before the loop: a wait for them inside would be one for the loads in flight as well
#pragma unroll
      for (int st = 0; st < KSTEPS; ++st) asm volatile("" : "+v"(q[st]));
      asm volatile("" : "+v"(ref));
      for (int k0 = from; k0 < to; k0 += 128) {
        const bool store = ok;
        const float old = before;
        k.put(own, lane, vecs);
        __builtin_amdgcn_wave_barrier();
        if (k0 + 128 < to) {
          load_k(k0 + 128, id);
          id = k0 + 256 < to ? look_up(k0 + 256) : -1;
        }
        f32x16 s = {};
#pragma unroll
        for (int st = 0; st < KSTEPS; ++st)
          s = mfma(E(), *(const u32x4*)(own + n * ROW + st * 32 + hf * 16), q[st], s);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c1, -ref));
        if (!__all(see.x <= k0 && see.y >= k0 + 32)) {
          const int origin = here(k0 + 4 * hf), lo = see.x - origin, hi = see.y - origin;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int o = 8 * (i / 4) + i % 4;
            if (o < lo || o >= hi) s[i] = 0;
          }
        }
        float* const mine = (float*)own;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 16; ++i) mine[(8 * (i / 4) + 4 * hf + i % 4) * LROW + n] = s[i];
        __builtin_amdgcn_wave_barrier();
        // lane l sums half of slot l % 32's weights
        float total = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 t = *(const f32x4*)(mine + n * LROW + hf * 16 + i * 4);
          total += (t[0] + t[1]) + (t[2] + t[3]);
        }
        total += other_half(total);
        __builtin_amdgcn_wave_barrier();
        if (store && hf == 0) gstore(masses + k0 + n, old + total);
      }
    }
  }
  if (errs) raise(a.err, errs);
}

enum { kMassBySlots, kMassByRows, kMassFew };

template <class E, int DP>
void launch_mass_dim(const MassArgs& m, BlockDiv div, dim3 grid, int how, int span, hipStream_t stream) {
  if (how == kMassFew) mass_few_kernel<E, DP><<<grid, 256, 0, stream>>>(m, div, span);
  else if (how == kMassByRows) mass_rows_kernel<E, DP><<<grid, 64 * kMassWaves<DP>, 0, stream>>>(m, div);
  else mass_kernel<E, DP><<<grid, 256, 0, stream>>>(m, div);
}

template <class E>
void launch_mass_dims(const MassArgs& m, BlockDiv div, dim3 grid, int how, int span, hipStream_t stream) {
  const int dim = m.at.cache.head_dim;
  if (dim <= 64) launch_mass_dim<E, 64>(m, div, grid, how, span, stream);
  else if (dim <= 128) launch_mass_dim<E, 128>(m, div, grid, how, span, stream);
  else launch_mass_dim<E, 256>(m, div, grid, how, span, stream);
}

}  // namespace

hipError_t launch_attention(const AttendArgs& a, hipStream_t stream) {
  const Plan p = plan_attention(a.cache, a.batch, a.num_heads);
  Split sp = {shares_within(p, a.cache, a.workspace_bytes), p.tiles, nullptr, nullptr};
  if (sp.shares > 0) {
    sp.acc = (float*)a.workspace;  // first: rows of 16-byte vectors
    sp.lse = sp.acc + (int64_t)(sp.shares + p.tiles) * a.cache.num_kv_heads * (p.keys ? kRowsKeys : kRows) * a.cache.head_dim;
  }
  const BlockDiv div = block_div(a.cache.block_size);
  if (a.cache.dtype == KVX_DTYPE_BF16) launch_attend_dims<Bf16>(a, div, sp, p.keys, stream);
  else launch_attend_dims<Fp16>(a, div, sp, p.keys, stream);
  return hipGetLastError();
}

int64_t attention_workspace(const kvx_paged_cache& c, const kvx_batch& b, int32_t num_heads) {
  const Plan p = plan_attention(c, b, num_heads);
  return p.shares > 0 ? (p.shares + (int64_t)p.tiles) * slot_bytes(c, p.keys) : 0;
}

hipError_t launch_mass(const MassArgs& m, hipStream_t stream) {
  const kvx_batch& b = m.at.batch;
  int64_t slots = b.max_blocks_per_req * m.at.cache.block_size;
  if (slots > m.mass_width) slots = m.mass_width;
  // as many workgroups as the hint asks for; they go on over the slots of a longer request
  if (slots > b.max_context_len) slots = b.max_context_len > 0 ? b.max_context_len : 1;
  const int64_t longest = b.max_query_len < b.num_tokens ? b.max_query_len : b.num_tokens;
  const int64_t lists = (int64_t)b.num_reqs * m.at.cache.num_kv_heads;
  // slots of a workgroup
  int64_t per = kMassSlots;
  int how = kMassBySlots;
  if (longest * (m.at.num_heads / m.at.cache.num_kv_heads) <= 32) {
    // a whole number of steps of its four wavefronts, few enough to fill the GPU
    how = kMassFew;
    per = (slots * lists / kMassFill + 127) / 128 * 128;
    if (per < 128) per = 128;
    if (per > 4096) per = 4096;
  } else if ((slots + kMassSlots - 1) / kMassSlots * lists < (m.at.cache.head_dim <= 128 ? kFill : kFill / 3)) {
    // Two workgroups a CU of mass_kernel, or one where the widest heads take the registers of two. Many rows, 512 tokens of 8 heads
    // on one over 4096 slots: 64, 256 and 512 workgroups by slots 124, 130 and 174 us, by rows 32, 111 and 217; at 256
    // dimensions 64, 128 and 256 of them 207, 206 and 209 against 70, 128 and 243. A prompt of 8192 tokens (32): 1522
    // against 340, at 256 dimensions 2806 against 840. With few rows the two meet earlier (61 tokens of 4 heads a KV head: 128
    // workgroups 14 against 12 us, 256 15 against 22, 384 17 against 32), at a loss of microseconds.
    how = kMassByRows;
    per = 64;
  }
  const int span = (int)per;
  const int64_t pieces = (slots + per - 1) / per;
  const dim3 grid(m.at.cache.num_kv_heads, (unsigned)(pieces < 65535 ? pieces : 65535), b.num_reqs);
  const BlockDiv div = block_div(m.at.cache.block_size);
  if (m.at.cache.dtype == KVX_DTYPE_BF16) launch_mass_dims<Bf16>(m, div, grid, how, span, stream);
  else launch_mass_dims<Fp16>(m, div, grid, how, span, stream);
  return hipGetLastError();
}

}  // namespace kvx
