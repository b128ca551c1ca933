// What the attention kernels share: which rows and slots a workgroup computes, the sharing of a batch's work and the join of
// its parts, and helpers of the running softmax.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_launch.h"
#include "kvx_paged.h"

namespace kvx {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// --------------------------------------------------------------------------------------
// which rows a workgroup computes
// --------------------------------------------------------------------------------------

// A query row of request r is one (token, head of the KV head's group) pair, token by token, so a
// tile of rows shares its K and V whatever the number of heads in a group. The tiles of all
// requests are numbered without any sum over the requests: request r's begin at
// floor(first row / ROWS) + r, which leaves it at least the tiles it needs and at most one spare.
struct Rows {
  int32_t r;         // the request
  int32_t context;   // its slots
  int32_t tokens;    // its new tokens
  int32_t tile;      // index of the tile in the request
  int64_t q0;        // its first query row
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) {
  return x < lo ? lo : x > hi ? hi : x;
}

// Values that are the same in every lane, kept in scalar registers.
__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)(uint32_t)uniform((int32_t)x) | (int64_t)uniform((int32_t)(x >> 32)) << 32;
}
// One lane's value in all.
__device__ __forceinline__ int32_t lane_of(int32_t x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ int64_t lane_of(int64_t x, int lane) {
  return (int64_t)(uint32_t)lane_of((int32_t)x, lane) | (int64_t)lane_of((int32_t)(x >> 32), lane) << 32;
}

// Request r: its rows and slots, clamped to the tensors.
__device__ __forceinline__ Rows request(const AttendArgs& a, int r, int64_t cap) {
  Rows x;
  x.r = r;
  x.tile = 0;
  x.q0 = clamp64(a.batch.q_offsets[r], 0, a.batch.num_tokens);
  x.tokens = (int32_t)(clamp64(a.batch.q_offsets[r + 1], x.q0, a.batch.num_tokens) - x.q0);
  x.context = a.cache.num_blocks > 0 ? (int32_t)clamp64(a.batch.context_lens[r], 0, cap) : 0;
  return x;
}
// The same of a request that all lanes ask for.
__device__ __forceinline__ Rows request_uniform(const AttendArgs& a, int r, int64_t cap) {
  Rows x = request(a, uniform(r), cap);
  x.q0 = uniform(x.q0);
  x.tokens = uniform(x.tokens);
  x.context = uniform(x.context);
  return x;
}

// One workgroup of a launch looks every request's offsets and contexts over.
__device__ void check_batch(const AttendArgs& a, int64_t cap, int tid, int threads) {
  int errs = 0;
  for (int r = tid; r < a.batch.num_reqs; r += threads) {
    const int64_t b = a.batch.q_offsets[r], e = a.batch.q_offsets[r + 1], c = a.batch.context_lens[r];
    if (b < 0 || e < b || e > a.batch.num_tokens) errs |= KVX_DEVERR_OFFSETS;
    if (c < 0 || c > cap) errs |= KVX_DEVERR_TABLE_RANGE;
  }
  if (errs) raise(a.err, errs);
}

// The slots [lo, hi) that new token i of a request sees.
__device__ __forceinline__ int2 sees(const AttendArgs& a, const Rows& x, int token) {
  const int64_t hi = a.causal ? (int64_t)x.context - x.tokens + token + 1 : (int64_t)x.context;
  const int64_t lo = hi - a.window;
  return {(int)(lo < 0 ? 0 : lo), (int)(hi < 0 ? 0 : hi)};
}

// The request of a tile: a 64-way search over the offsets, one probe a lane and round (one round
// up to 64 requests). All lanes get the same answer; whatever the offsets hold, r is a request.
template <int ROWS>
__device__ __forceinline__ Rows find_rows(const AttendArgs& a, int32_t tile, int group, int64_t cap, int lane) {
  int lo = 0, len = a.batch.num_reqs;
  int64_t begin;
  for (;;) {
    const int step = (len + 63) / 64;
    const int i = lane * step < len ? lo + lane * step : lo;
    begin = clamp64(a.batch.q_offsets[i], 0, a.batch.num_tokens);
    const bool at = lane * step < len && begin * group / ROWS + i <= tile;
    const uint64_t hit = __ballot(at);
    const int pick = hit ? 63 - __builtin_clzll(hit) : 0;
    lo += pick * step;
    if (step == 1) break;
    len = len - pick * step < step ? len - pick * step : step;
  }
  Rows x = request_uniform(a, lo, cap);
  x.tile = tile - (int32_t)(x.q0 * group / ROWS + x.r);
  return x;
}

// Shared work: the tiles of all requests in a row, each of its request's nominal number of steps (tiles
// of slots that any of the request's rows sees, at least one), cut into equal shares for the
// workgroups of one KV head. A share begins and ends anywhere, so a batch of any lengths is even; a tile
// that several shares meet in is joined from its parts, which lie in consecutive slots of the
// workspace: the part of share i in tile q is in slot i + q, since either number grows by
// one from each part to the next.
struct Shares {
  int64_t steps;  // of all requests
  int32_t count;  // shares that are not empty: the first `longer` have each + 1 steps, the others each
  int32_t longer;
  int64_t each;
};
// a / b of non-negative numbers; the 64-bit division costs an order of magnitude more than the 32-bit one
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}
// EXTRA: steps that stand for a tile's start, before its own, where a share that meets several tiles should get less of them.
template <int ROWS, int BN, int EXTRA = 0>
__device__ __forceinline__ void extent(const AttendArgs& a, const Rows& x, int group, int32_t* tiles, int32_t* steps) {
  *tiles = (int32_t)(((int64_t)x.tokens * group + ROWS - 1) / ROWS);
  const int lo = sees(a, x, 0).x, hi = sees(a, x, x.tokens - 1).y;
  *steps = (hi > lo ? (hi + BN - 1) / BN - lo / BN : 1) + EXTRA;
}
// 64 requests of the batch, one a lane: their tiles and steps, and those of all requests before them. Offsets that
// give the same rows to many requests can make more tiles than 32 bits hold: tile0 then wraps around, and who takes a
// tile's number for a place checks that there is one.
struct Requests {
  Rows x;
  int32_t tiles, steps;
  uint32_t tile0;
  int64_t step0;
};
template <int ROWS, int BN, int EXTRA>
__device__ __forceinline__ Requests sixty_four(const AttendArgs& a, int group, int64_t cap, int lane, int r0, uint32_t tile0,
                                               int64_t step0) {
  Requests q = {};
  if (r0 + lane < a.batch.num_reqs) {
    q.x = request(a, r0 + lane, cap);
    extent<ROWS, BN, EXTRA>(a, q.x, group, &q.tiles, &q.steps);
  }
  int64_t sum = (int64_t)q.tiles * q.steps;
  uint32_t num = q.tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t s = __shfl_up(sum, d);
    const uint32_t t = __shfl_up(num, d);
    if (lane >= d) sum += s, num += t;
  }
  q.tile0 = tile0 + num - q.tiles;
  q.step0 = step0 + sum - (int64_t)q.tiles * q.steps;
  return q;
}
// Counts the steps of the batch, and finds the request for which holds(shares, a lane's request) is
// true: its lane's values in every lane, steps == 0 where there is none.
template <int ROWS, int BN, int EXTRA = 0, class F>
__device__ __forceinline__ Requests locate(const AttendArgs& a, int group, int64_t cap, int lane, int shares, Shares* all,
                                           F holds) {
  Requests q = {};
  const int reqs = a.batch.num_reqs;
  for (int r0 = 0; r0 < reqs; r0 += 64)
    q = sixty_four<ROWS, BN, EXTRA>(a, group, cap, lane, r0, lane_of((int32_t)(q.tile0 + q.tiles), 63),
                             lane_of(q.step0 + (int64_t)q.tiles * q.steps, 63));
  all->steps = lane_of(q.step0 + (int64_t)q.tiles * q.steps, 63);
  all->count = all->steps < shares ? (int32_t)all->steps : shares;
  if (all->count == 0) return {};
  all->each = quotient(all->steps, all->count);
  all->longer = (int32_t)(all->steps - all->each * all->count);
  Requests f = q;
  for (int r0 = 0;; r0 += 64) {
    if (reqs > 64)  // up to 64 requests the first pass holds them all
      f = sixty_four<ROWS, BN, EXTRA>(a, group, cap, lane, r0, r0 ? lane_of((int32_t)(f.tile0 + f.tiles), 63) : 0,
                               r0 ? lane_of(f.step0 + (int64_t)f.tiles * f.steps, 63) : 0);
    const uint64_t there = __ballot(f.tiles > 0 && holds(*all, f));
    if (there) {
      const int l = __builtin_ctzll(there);
      return {{r0 + l, lane_of(f.x.context, l), lane_of(f.x.tokens, l), 0, lane_of(f.x.q0, l)},
              lane_of(f.tiles, l), lane_of(f.steps, l), (uint32_t)lane_of((int32_t)f.tile0, l), lane_of(f.step0, l)};
    }
    if (r0 + 64 >= reqs) return {};
  }
}
__device__ __forceinline__ int64_t share_begin(const Shares& s, int i) {
  return s.each * i + (i < s.longer ? i : s.longer);
}
__device__ __forceinline__ int share_of(const Shares& s, int64_t step) {  // the share that step falls into
  const int64_t split = (s.each + 1) * s.longer;
  return step < split ? (int)quotient(step, s.each + 1) : s.longer + (int)quotient(step - split, s.each);
}

__device__ __forceinline__ int2 sees_uniform(const AttendArgs& a, const Rows& x, int token) {
  const int2 s = sees(a, x, uniform(token));
  return {uniform(s.x), uniform(s.y)};
}

// --------------------------------------------------------------------------------------
// pieces
// --------------------------------------------------------------------------------------

#define KVX_LDS __attribute__((address_space(3)))

// max or sum over the two lanes l and l ^ 32
__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? r[0] : r[1]);
}

// The reference that weights are formed against, 2^(x - m): kLift below the row's maximum when it is set, and left
// there until the maximum stands kLift + kLag above it, so that weights end at 2^(kLift + kLag). fp16 ends at 2^16 and
// rounds to steps of 2^-24 at the lower end: lifted, weights keep all their bits down to 2^-25 of the largest, and round
// off by 2^-36 of it below (unlifted, a tail of slots that weigh less than 2^-25 each, as behind an attention sink, would be
// lost whole). bf16 has the exponents of 32 bits and needs no lift.
template <class E>
constexpr float kLift = __is_same(E, Fp16) ? 11.0f : 0.0f;
template <class E>
constexpr float kLag = __is_same(E, Fp16) ? 4.0f : 8.0f;
// Scores of 2^20 and more, in base 2, are far: 32 bits hold them in steps of 2^-3, and from 2^24 on the rounding of x alone decides
// over the weight's exponent. x is then rounded before the reference is taken from it, as the maximum was, so that the largest
// weight is what the reference says; in one step, unrounded, it could end anywhere up to half a step of x.
__device__ __forceinline__ bool is_far(float x) { return __builtin_amdgcn_frexp_expf(x) > 20; }  // not of an infinity
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}
__device__ __forceinline__ float rounded_difference(float a, float b) {
#pragma clang fp contract(off)
  return a - b;
}

// A kernel's first argument, read from the argument segment where it stands: the loops' registers
// need not hold what only their ends use.
template <class T>
__device__ __forceinline__ const T& argument() {
  const __attribute__((address_space(4))) char* p =
      (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const T*)p;
}

// The same value, computed where it stands: keeps what the rare branches of a loop need out of the
// registers of the loop.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ float here(float x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ int lane_here() { return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, here(0))); }

// Kinds of instructions for __builtin_amdgcn_sched_group_barrier.
constexpr int kMfma = 0x8, kDsRead = 0x100, kVector = 0x402;

// Barrier for data passed through LDS: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// --------------------------------------------------------------------------------------
// shared work's parts
// --------------------------------------------------------------------------------------

struct Split {
  int32_t shares;  // workgroups of a KV head that share the work evenly; 0: one a tile of rows
  int32_t tiles;   // tiles of rows, at most
  float* acc;      // [slot][KV head][row of the tile][head_dim], and the base-2 lse of each row
  float* lse;
};

// Joins the parts of a tile: out = sum_s 2^(lse_s - top) o_s / sum_s 2^(lse_s - top). A thread takes four
// dimensions of one row, and with many parts only every second or eighth of them, the threads of a row and
// dimension side by side. What bounds it is one chain of loads: the batch, then the parts.
template <class E, int ROWS, int BN, int EXTRA = 0>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a, Split sp) {
  __shared__ f32x4 sums[256];
  __shared__ float tops[256], totals[256];
  const int group = a.num_heads / a.cache.num_kv_heads, quads = a.cache.head_dim / 4;
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  const int tid = threadIdx.x, lane = tid & 63;
  const int g = blockIdx.x % a.cache.num_kv_heads, tile = blockIdx.x / a.cache.num_kv_heads;
  Shares all;
  const Requests q = locate<ROWS, BN, EXTRA>(a, group, cap, lane, sp.shares, &all, [&](const Shares&, const Requests& q) {
    return tile - q.tile0 < (uint32_t)q.tiles;
  });
  if (q.steps == 0) return;  // no such tile
  const int64_t begin = q.step0 + (int64_t)(int32_t)(tile - q.tile0) * q.steps;
  const int s_from = share_of(all, begin), s_to = share_of(all, begin + q.steps - 1) + 1;
  if (s_to - s_from == 1) return;  // one share computed it whole
  Rows x = q.x;
  x.tile = (int32_t)(tile - q.tile0);
  const int rows = x.tokens * group - x.tile * ROWS, items = (rows < ROWS ? rows : ROWS) * quads;
  const int ways_log = s_to - s_from <= 8 ? 0 : s_to - s_from <= 16 ? 1 : 3;
  const int ways = 1 << ways_log, per = 256 >> ways_log, way = tid >> (8 - ways_log);
  for (int at = blockIdx.y * per; at < items; at += gridDim.y * per) {
    const int item = at + (tid & (per - 1)), row = item / quads, e = (item - row * quads) * 4;
    const bool used = item < items;
    auto part = [&](int s) { return ((int64_t)(s + tile) * a.cache.num_kv_heads + g) * ROWS + row; };
    float top = -INFINITY, total = 0;
    f32x4 o = {};
    if (used) {
      for (int s0 = s_from + way; s0 < s_to; s0 += 4 * ways) {
        float lse[4];
        f32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // four parts side by side, the last one again where there are fewer
          const int s = s0 + k * ways < s_to ? s0 + k * ways : s0;
          lse[k] = gload<float>(sp.lse + part(s));
          v[k] = gload<f32x4>(sp.acc + part(s) * a.cache.head_dim + e);
          if (s0 + k * ways >= s_to) lse[k] = -INFINITY;
        }
        const float m = fmaxf(fmaxf(fmaxf(lse[0], lse[1]), fmaxf(lse[2], lse[3])), top);
        const float ref = m == -INFINITY ? 0.0f : m, keep = __builtin_amdgcn_exp2f(top - ref);
        total *= keep;
        o *= keep;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float wgt = __builtin_amdgcn_exp2f(lse[k] - ref);
          total += wgt;
          if (lse[k] != -INFINITY) o += wgt * v[k];
        }
        top = m;
      }
    }
    if (ways > 1) {
      __syncthreads();
      sums[tid] = o;
      tops[tid] = top;
      totals[tid] = total;
      __syncthreads();
      if (way) continue;
      for (int k = 1; k < ways; ++k) top = fmaxf(top, tops[k * per + tid]);
      const float ref = top == -INFINITY ? 0.0f : top;
      total = 0;
      o = f32x4{};
      for (int k = 0; k < ways; ++k) {
        const float m = tops[k * per + tid];
        if (m == -INFINITY) continue;
        const float wgt = __builtin_amdgcn_exp2f(m - ref);
        total += wgt * totals[k * per + tid];
        o += wgt * sums[k * per + tid];
      }
    }
    if (!used) continue;
    const int flat = x.tile * ROWS + row, token = flat / group, head = g * group + flat - token * group;
    const int64_t t = x.q0 + token;
    const float inv = total == 0 ? 0.0f : 1.0f / total;
    gstore((char*)a.out.base + t * a.out.token_stride + head * a.out.head_stride + e * 2,
           __builtin_convertvector(o * inv, typename E::V4));
    if (e == 0 && a.lse)
      a.lse[t * a.num_heads + head] = total == 0 ? -INFINITY : (top + __builtin_amdgcn_logf(total)) * kLn2;
  }
}

}  // namespace
}  // namespace kvx
