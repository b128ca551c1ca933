// gfx950 kernels of kvx_evict_select and kvx_evict_compact.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_launch.h"
#include "kvx_paged.h"

namespace kvx {
namespace {

// --------------------------------------------------------------------------------------
// selection
// --------------------------------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

// Masses as integers of the same order: protected slots above NaN above +inf, -0 as 0.
__device__ __forceinline__ uint32_t rank_of(float m) {
  if (m != m) return 0xfffffffeu;
  const uint32_t b = __builtin_bit_cast(uint32_t, m + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One workgroup a list. The masses are read once, into registers (lists beyond kSelSlots in pieces, again for every
// digit). The rank of the last kept slot is found digit by digit from the top, 11, 11 and 10 bits: a histogram a round
// over the slots that agree with the digits found. A digit of 11 bits spreads masses of like size, which share sign and
// exponent, over some bins: the additions of a wavefront to one bin come one after the other.
// Then the slots above the rank and the lowest ones that equal it are written in order, their places from counts by wavefront
// and 64 slots. What bounds it is the chain of rounds, each a pass through LDS (8 x 8 lists of 9216: 13.2 us, 17.6 with
// four digits of 8 bits; 8 lists of 32768: 27 us, 62 with half as many registers and four digits).
constexpr int kSelRegs = 32;
constexpr int kSelSlots = kSelRegs * kSelThreads;
constexpr int kSelBins = 2048;
constexpr int kSelCopies = 2;  // histograms, by wavefront: equal digits of different wavefronts collide less

__global__ __launch_bounds__(kSelThreads) void select_kernel(SelectArgs a) {
  __shared__ __align__(16) uint32_t hist[kSelCopies][kSelBins];
  __shared__ uint32_t tops[kSelWaves];
  __shared__ uint32_t counts[2][kSelRegs * kSelWaves];  // above the rank, equal to it: of 64 slots each, in order
  __shared__ uint32_t found[4];  // digit, slots still wanted among those that have it; totals of a piece
  const int r = blockIdx.x / a.num_heads, h = blockIdx.x - r * a.num_heads;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t c = a.context_lens[r];
  const int64_t clamped = c < 0 ? 0 : c > a.width ? a.width : c;
  if (c != clamped && tid == 0) raise(a.err, KVX_DEVERR_TABLE_RANGE);
  const uint32_t n = (uint32_t)clamped, budget = (uint32_t)a.budget, want_all = n < budget ? n : budget;
  if (h == 0 && tid == 0) a.new_lens[r] = want_all;
  int32_t* keep = a.keep + (int64_t)blockIdx.x * a.budget;
  if (n <= budget) {
    for (uint32_t i = tid; i < budget; i += kSelThreads) keep[i] = i < n ? (int32_t)i : -1;
    return;
  }
  const float* mass = a.mass + r * a.req_stride + h * a.head_stride;
  const uint32_t last = n - (uint32_t)a.recent, sink = (uint32_t)a.sink;
  uint32_t k[kSelRegs];
  auto load = [&](uint32_t j0) {
    float m[kSelRegs];
#pragma unroll
    for (int i = 0; i < kSelRegs; ++i) {
      const uint32_t j = j0 + i * kSelThreads + tid;
      if (j - tid < n) m[i] = gload<float>(mass + (j < n ? j : 0));
    }
#pragma unroll
    for (int i = 0; i < kSelRegs; ++i) {
      const uint32_t j = j0 + i * kSelThreads + tid;
      if (j - tid < n) k[i] = j < sink || j >= last ? 0xffffffffu : rank_of(m[i]);
    }
  };
  load(0);
  uint32_t prefix = 0, mask = 0, want = want_all;
  for (int shift = 21;; shift = shift > 11 ? shift - 11 : 0) {
    *(u32x4*)(&hist[0][0] + 4 * tid) = u32x4{0, 0, 0, 0};
    __syncthreads();
    for (uint32_t j0 = 0; j0 < n; j0 += kSelSlots) {
      if (n > kSelSlots) load(j0);
#pragma unroll
      for (int i = 0; i < kSelRegs; ++i) {
        const uint32_t j = j0 + i * kSelThreads + tid;
        if (j - tid >= n) break;
        if (j < n && (k[i] & mask) == prefix) atomicAdd(&hist[wave % kSelCopies][(k[i] >> shift) & (kSelBins - 1)], 1u);
      }
    }
    __syncthreads();
    // this thread: two bins, from the largest down
    const uint32_t bin = kSelBins - 2 - 2 * tid;
    uint32_t high = 0, low = 0;
#pragma unroll
    for (int v = 0; v < kSelCopies; ++v) {
      const u32x2 b = *(const u32x2*)&hist[v][bin];
      low += b[0];
      high += b[1];
    }
    uint32_t upto = high + low;
    for (uint32_t d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 63) tops[wave] = upto;
    __syncthreads();
    uint32_t before = upto - high - low;
    for (uint32_t v = 0; v < wave; ++v) before += tops[v];
    if (before < want && want <= before + high + low) {
      const bool first = want <= before + high;
      found[0] = bin + first;
      found[1] = want - before - (first ? 0 : high);
    }
    __syncthreads();
    prefix |= found[0] << shift;  // the last digit's top bit is the one before's lowest
    mask |= (uint32_t)(kSelBins - 1) << shift;
    want = found[1];
    if (shift == 0) break;
  }
  uint32_t base = 0, ties = want;  // slots written so far; equal slots still to write
  for (uint32_t j0 = 0; j0 < n; j0 += kSelSlots) {
    if (n > kSelSlots) load(j0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelRegs; ++i) {
      const uint32_t j = j0 + i * kSelThreads + tid;
      if (j - tid >= n) break;  // this row of 1024 slots and the ones after it are behind the list
      const uint32_t above = __popcll(__ballot(j < n && k[i] > prefix));
      const uint32_t equal = __popcll(__ballot(j < n && k[i] == prefix));
      if (lane < 2) counts[lane][i * kSelWaves + wave] = lane ? equal : above;
    }
    __syncthreads();
    if (wave < 2) {  // each count becomes the sum of those before it: lane l's are kEach l .. kEach l + kEach - 1
      constexpr int kEach = kSelRegs * kSelWaves / 64;
      uint32_t* const at = counts[wave] + kEach * lane;
      const uint32_t written = (n - j0 + kSelThreads - 1) / kSelThreads * kSelWaves;
      uint32_t v[kEach], sum = 0;
      for (int i = 0; i < kEach; ++i) {
        v[i] = sum;
        sum += kEach * lane + i < written ? at[i] : 0;
      }
      uint32_t upto = sum;
      for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
      }
      for (int i = 0; i < kEach; ++i) at[i] = v[i] + upto - sum;
      if (lane == 63) found[2 + wave] = upto;
    }
    __syncthreads();
    const uint64_t under = (1ull << lane) - 1;
#pragma unroll
    for (int i = 0; i < kSelRegs; ++i) {
      const uint32_t j = j0 + i * kSelThreads + tid;
      if (j - tid >= n) break;
      const bool gt = j < n && k[i] > prefix, eq = j < n && k[i] == prefix;
      const uint32_t g = counts[0][i * kSelWaves + wave] + __popcll(__ballot(gt) & under);
      const uint32_t e = counts[1][i * kSelWaves + wave] + __popcll(__ballot(eq) & under);
      if (gt || (eq && e < ties)) keep[base + g + (e < ties ? e : ties)] = (int32_t)j;
    }
    const uint32_t e_kept = found[3] < ties ? found[3] : ties;
    base += found[2] + e_kept;
    ties -= e_kept;
  }
}
static_assert(kSelRegs * kSelWaves % 64 == 0 && kSelBins == 2 * kSelThreads && kSelCopies * kSelBins == 4 * kSelThreads,
              "two bins and four entries a thread, whole counts a lane");

// --------------------------------------------------------------------------------------
// moving
// --------------------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
// Rows in flight a thread, moved past the caches like the copies of whole blocks: 4 against 8 (a batch's eviction 75 against
// 78 us), and 73 with non-temporal loads and stores.
constexpr int kMoveUnroll = 4;

// Every load of the workgroup has its value before any wavefront goes on to store.
__device__ __forceinline__ void loads_landed() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// A workgroup moves one column: the K or V rows of one KV head of one request, or one row of
// masses, a tile of slots at a time: all its loads, then all its stores. An ascending list has
// keep[i] >= i, so a slot is read in its own tile or an earlier one; with the tiles of a column in
// one workgroup (grid.y = 1), in order and with a barrier between a tile's loads and its stores,
// the move is right in place. Where source and destination differ, grid.y spreads the tiles; a row whose destination
// block is the source's own of that place (a copy of the table, or part of one) would then race with the reads of it, and
// is left alone. In place, a column's tiles follow one another and each waits for its chain of three loads, 2.4 us for 64 rows of
// 128 dimensions, so a move in place is bound by the longest list and hardly by the bytes (lists of 32768 to 16384: one 621 us, 8
// of them 651; into other blocks 10 and 34).
__global__ __launch_bounds__(kMoveThreads) void compact_kernel(CompactArgs a, BlockDiv div) {
  const kvx_paged_cache& cache = a.cache;
  const int columns = 2 * cache.num_kv_heads + (a.mass ? a.num_heads : 0);
  // Workgroup i runs on XCD i % 8: a request's columns, whose rows lie side by side, to one XCD where they can be (72 -> 70 us)
  const int xcd = blockIdx.x % 8, per = gridDim.x / 8, more = gridDim.x % 8;
  const int at_column = xcd * per + (xcd < more ? xcd : more) + blockIdx.x / 8;
  const int r = at_column / columns, col = at_column - r * columns;
  const int tid = threadIdx.x;
  const bool in_place = a.src_table == a.dst_table;
  int errs = 0;
  if (col >= 2 * cache.num_kv_heads) {
    const int h = col - 2 * cache.num_kv_heads;
    const int32_t* keep = a.keep + ((int64_t)r * a.num_heads + h) * a.budget;
    const float* in = a.mass + r * a.mass_req_stride + h * a.mass_head_stride;
    float* out = a.mass_out + r * a.out_req_stride + h * a.out_head_stride;
    const int64_t tile = kMoveThreads * kMoveUnroll;
    for (int64_t t0 = blockIdx.y * tile; t0 < a.out_width; t0 += gridDim.y * tile) {
      float v[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int64_t i = t0 + u * kMoveThreads + tid;
        const int32_t k = i < a.budget && i < a.out_width ? keep[i] : -1;
        v[u] = 0;
        if (k >= 0 && k < i) errs |= KVX_DEVERR_OFFSETS;
        else if (k >= a.mass_width) errs |= KVX_DEVERR_TABLE_RANGE;
        else if (k >= 0) v[u] = in[k];
      }
      loads_landed();
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int64_t i = t0 + u * kMoveThreads + tid;
        if (i < a.out_width) out[i] = v[u];
      }
    }
  } else {
    const int h = col >> 1;
    const int64_t at = (col & 1) * cache.kv_stride_bytes + h * cache.head_stride_bytes;
    const int list = h / (cache.num_kv_heads / a.num_heads);
    const int32_t* keep = a.keep + ((int64_t)r * a.num_heads + list) * a.budget;
    const int32_t* from = a.src_table + r * a.src_row;
    const int32_t* to = a.dst_table + r * a.dst_row;
    const uint32_t vecs = cache.head_dim / 8;
    const int tile_rows = kMoveThreads * kMoveUnroll / vecs;
    // this thread's rows and pieces of a tile, the same in every tile
    int row[kMoveUnroll], piece[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const uint32_t x = u * kMoveThreads + tid;
      row[u] = x / vecs;
      piece[u] = (x - row[u] * vecs) * 16;
    }
    for (int64_t t0 = (int64_t)blockIdx.y * tile_rows; t0 < a.budget; t0 += (int64_t)gridDim.y * tile_rows) {
      // Three rounds of loads, each issued whole: list entries, table entries, rows. What is not to be
      // moved reads the first entry or row instead, and is not stored.
      int32_t k[kMoveUnroll], sb[kMoveUnroll], db[kMoveUnroll], own[kMoveUnroll];  // own: the source's block at d
      bool move[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        move[u] = row[u] < tile_rows && t0 + row[u] < a.budget;
        k[u] = gload<int32_t>(keep + (move[u] ? t0 + row[u] : 0));
      }
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int32_t i = (int32_t)(t0 + row[u]);
        move[u] = move[u] && k[u] >= 0;
        if (move[u] && k[u] < i) errs |= KVX_DEVERR_OFFSETS, move[u] = false;
        const int32_t s = block_of(div, k[u]), d = block_of(div, i);
        if (move[u] && (s >= a.src_cols || d >= a.dst_cols)) errs |= KVX_DEVERR_TABLE_RANGE, move[u] = false;
        k[u] = move[u] ? k[u] - s * div.size : 0;  // places in the blocks from here on
        piece[u] = (piece[u] & 0xffff) | (move[u] && s == d && k[u] == i - d * div.size ? 1 << 16 : 0);
        sb[u] = gload<int32_t>(from + (move[u] ? s : 0));
        db[u] = gload<int32_t>(to + (move[u] ? d : 0));
        own[u] = in_place ? 0 : gload<int32_t>(from + (move[u] ? d : 0));  // d <= s
      }
      u32x4 v[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        if (move[u] && ((uint32_t)sb[u] >= (uint64_t)cache.num_blocks || (uint32_t)db[u] >= (uint64_t)cache.num_blocks))
          errs |= KVX_DEVERR_BLOCK_RANGE, move[u] = false;
        if (in_place || own[u] == db[u]) {  // one block on both sides: its row may be there already
          if (move[u] && !in_place && !(piece[u] >> 16)) errs |= KVX_DEVERR_BLOCK_RANGE, move[u] = false;
          move[u] = move[u] && !(piece[u] >> 16);
        }
        const char* src = (const char*)cache.base + at + (piece[u] & 0xffff);
        if (move[u]) src += sb[u] * cache.block_stride_bytes + (int64_t)k[u] * cache.token_stride_bytes;
        v[u] = __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x4*)src);
      }
      loads_landed();
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int32_t i = (int32_t)(t0 + row[u]);
        if (move[u])
          __builtin_nontemporal_store(
              v[u], (__attribute__((address_space(1))) u32x4*)(
                        (char*)cache.base + db[u] * cache.block_stride_bytes +
                        (int64_t)(i - block_of(div, i) * div.size) * cache.token_stride_bytes + at + (piece[u] & 0xffff)));
      }
    }
  }
  if (errs) raise(a.err, errs);
}

}  // namespace

hipError_t launch_evict_select(const SelectArgs& a, hipStream_t stream) {
  select_kernel<<<dim3((unsigned)(a.num_reqs * a.num_heads)), dim3(kSelThreads), 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_evict_compact(const CompactArgs& a, hipStream_t stream) {
  const int columns = 2 * a.cache.num_kv_heads + (a.mass ? a.num_heads : 0);
  const int tile_rows = kMoveThreads * kMoveUnroll / (a.cache.head_dim / 8);
  int64_t tiles = 1;
  if (a.src_table != a.dst_table) {
    tiles = ((int64_t)a.budget + tile_rows - 1) / tile_rows;
    if (tiles > 65535) tiles = 65535;
  }
  compact_kernel<<<dim3((unsigned)(a.num_reqs * columns), (unsigned)tiles), dim3(kMoveThreads), 0, stream>>>(
      a, block_div(a.cache.block_size));
  return hipGetLastError();
}

}  // namespace kvx
