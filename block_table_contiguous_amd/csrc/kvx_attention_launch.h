// Internal interface between the entry points of kvx_attention.h (kvx_attention_api.hip) and
// their gfx950 kernels. Arguments are already validated when these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention.h"

namespace kvx {

// Byte strides of a [tokens][heads][head_dim] tensor.
struct RowView {
  const char* base;
  int64_t token_stride;
  int64_t head_stride;
};

struct RopeArgs {
  kvx_paged_cache cache;
  RowView query, key, value, out;
  int32_t num_heads, rot_dim, num_axes;
  int64_t num_tokens;
  const int64_t* positions;
  const float* inv_freq;
  const int64_t* slots;
  int32_t* err;
  uint8_t pair_axis[KVX_MAX_HEAD_DIM / 2];
};
hipError_t launch_rope(const RopeArgs& a, bool interleaved, hipStream_t stream);

struct AttendArgs {
  kvx_paged_cache cache;
  kvx_batch batch;
  RowView query, out;
  int32_t num_heads, causal;
  float scale;
  int64_t window;  // INT32_MAX where there is none
  float* lse;
  void* workspace;
  int64_t workspace_bytes;
  int32_t* err;
};
hipError_t launch_attention(const AttendArgs& a, hipStream_t stream);
int64_t attention_workspace(const kvx_paged_cache& c, const kvx_batch& b, int32_t num_heads);

struct MassArgs {
  AttendArgs at;  // out, workspace unused; lse is read
  float* mass;
  int64_t mass_req_stride, mass_head_stride, mass_width;
};
hipError_t launch_mass(const MassArgs& a, hipStream_t stream);

struct SelectArgs {
  const float* mass;
  int64_t req_stride, head_stride, width;
  int32_t num_reqs, num_heads;
  const int64_t* context_lens;
  int32_t budget, sink, recent;
  int32_t* keep;
  int64_t* new_lens;
  int32_t* err;
};
hipError_t launch_evict_select(const SelectArgs& a, hipStream_t stream);

struct CompactArgs {
  kvx_paged_cache cache;
  const int32_t* src_table;
  const int32_t* dst_table;
  int64_t src_cols, src_row, dst_cols, dst_row;
  int32_t num_reqs, num_heads, budget;
  const int32_t* keep;
  const float* mass;
  float* mass_out;
  int64_t mass_req_stride, mass_head_stride, mass_width;
  int64_t out_req_stride, out_head_stride, out_width;
  int32_t* err;
};
hipError_t launch_evict_compact(const CompactArgs& a, hipStream_t stream);

}  // namespace kvx
