// gfx950 kernels of kvx_paged_attention and kvx_attention_mass.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_launch.h"
#include "kvx_attention_plan.h"
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
template <int ROWS, int BN>
__device__ __forceinline__ void extent(const AttendArgs& a, const Rows& x, int group, int32_t* tiles, int32_t* steps) {
  *tiles = (int32_t)(((int64_t)x.tokens * group + ROWS - 1) / ROWS);
  const int lo = sees(a, x, 0).x, hi = sees(a, x, x.tokens - 1).y;
  *steps = hi > lo ? (hi + BN - 1) / BN - lo / BN : 1;
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
template <int ROWS, int BN>
__device__ __forceinline__ Requests sixty_four(const AttendArgs& a, int group, int64_t cap, int lane, int r0, uint32_t tile0,
                                               int64_t step0) {
  Requests q = {};
  if (r0 + lane < a.batch.num_reqs) {
    q.x = request(a, r0 + lane, cap);
    extent<ROWS, BN>(a, q.x, group, &q.tiles, &q.steps);
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
template <int ROWS, int BN, class F>
__device__ __forceinline__ Requests locate(const AttendArgs& a, int group, int64_t cap, int lane, int shares, Shares* all,
                                           F holds) {
  Requests q = {};
  const int reqs = a.batch.num_reqs;
  for (int r0 = 0; r0 < reqs; r0 += 64)
    q = sixty_four<ROWS, BN>(a, group, cap, lane, r0, lane_of((int32_t)(q.tile0 + q.tiles), 63),
                             lane_of(q.step0 + (int64_t)q.tiles * q.steps, 63));
  all->steps = lane_of(q.step0 + (int64_t)q.tiles * q.steps, 63);
  all->count = all->steps < shares ? (int32_t)all->steps : shares;
  if (all->count == 0) return {};
  all->each = quotient(all->steps, all->count);
  all->longer = (int32_t)(all->steps - all->each * all->count);
  Requests f = q;
  for (int r0 = 0;; r0 += 64) {
    if (reqs > 64)  // up to 64 requests the first pass holds them all
      f = sixty_four<ROWS, BN>(a, group, cap, lane, r0, r0 ? lane_of((int32_t)(f.tile0 + f.tiles), 63) : 0,
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
// matrix pieces
// --------------------------------------------------------------------------------------

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
#define KVX_LDS __attribute__((address_space(3)))

__device__ __forceinline__ f32x16 mfma(Bf16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Bf16::V8, a), __builtin_bit_cast(Bf16::V8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(Fp16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(Fp16::V8, a), __builtin_bit_cast(Fp16::V8, b), c, 0, 0, 0);
}

// In the 32x32x16 products lane l holds column (or row) l % 32 and, with hf = l / 32, elements
// 8 hf .. 8 hf + 7 of the summed dimension; result register i of lane l is row 8 (i / 4) + 4 hf + i % 4,
// column l % 32.

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

template <class E>
__device__ __forceinline__ bool non_finite(u32x4 v) {
  constexpr uint32_t exp = sizeof(E) && __is_same(E, Bf16) ? 0x7f80u : 0x7c00u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (v[i] & exp) == exp || ((v[i] >> 16) & exp) == exp;
  return bad;
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

// A buffer that starts at p (the same in all lanes) for loads whose offsets the caller keeps inside
// the memory: a scalar base, a scalar step and a lane's constant offset make an address for nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const char* p) {
  const uint64_t at = (uint64_t)uniform((int64_t)p);
  return __builtin_amdgcn_make_buffer_rsrc((void*)at, 0, 0x7fffffff, 0x00027000);
}

// Kinds of instructions for __builtin_amdgcn_sched_group_barrier.
constexpr int kMfma = 0x8, kDsRead = 0x100, kVector = 0x402;

// Barrier for data passed through LDS: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// --------------------------------------------------------------------------------------
// attention
// --------------------------------------------------------------------------------------

struct Split {
  int32_t shares;  // workgroups of a KV head that share the work evenly; 0: one a tile of rows
  int32_t tiles;   // tiles of rows, at most
  float* acc;      // [slot][KV head][row of the tile][head_dim], and the base-2 lse of each row
  float* lse;
};

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

// Joins the parts of a tile: out = sum_s 2^(lse_s - top) o_s / sum_s 2^(lse_s - top). A thread takes four
// dimensions of one row, and with many parts only every second or eighth of them, the threads of a row and
// dimension side by side. What bounds it is one chain of loads: the batch, then the parts.
template <class E, int ROWS, int BN>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a, Split sp) {
  __shared__ f32x4 sums[256];
  __shared__ float tops[256], totals[256];
  const int group = a.num_heads / a.cache.num_kv_heads, quads = a.cache.head_dim / 4;
  const int64_t cap = a.batch.max_blocks_per_req * a.cache.block_size;
  const int tid = threadIdx.x, lane = tid & 63;
  const int g = blockIdx.x % a.cache.num_kv_heads, tile = blockIdx.x / a.cache.num_kv_heads;
  Shares all;
  const Requests q = locate<ROWS, BN>(a, group, cap, lane, sp.shares, &all, [&](const Shares&, const Requests& q) {
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
