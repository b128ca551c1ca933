// Internal interface between the entry points of kvx_fp4.h (kvx_fp4_api.hip) and their gfx950 kernels.
// Arguments are already validated when these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvx_attention_launch.h"
#include "kvx_fp4.h"

namespace kvx {

struct Fp4RopeArgs {
  kvx_fp4_cache cache;
  RowView query, key, value, out, key_out, value_out;  // key_out.base NULL: not wanted
  int32_t num_heads, rot_dim, num_axes;
  int64_t num_tokens;
  const int64_t* positions;
  const float* inv_freq;
  const int64_t* slots;
  int32_t* err;
  uint8_t pair_axis[KVX_MAX_HEAD_DIM / 2];
};
hipError_t launch_rope_fp4(const Fp4RopeArgs& a, bool interleaved, hipStream_t stream);

// The attention's arguments are those of the 16-bit cache, with the 4-bit one described in its terms: a row is
// head_dim/2 bytes at token_stride_bytes of the same, its scales head_dim/32 bytes from block_size rows on, and
// dtype that of query and out.
hipError_t launch_attention_fp4(const AttendArgs& a, hipStream_t stream);
int64_t attention_fp4_workspace(const kvx_paged_cache& c, const kvx_batch& b, int32_t num_heads);

struct Fp4CopyArgs {
  kvx_paged_cache cache;  // of each layer, base unused
  kvx_fp4_cache buffer;
  void* const* layer_bases;
  int32_t num_layers;
  const kvx_xfer* xfers;
  const int64_t* xfer_count;
  int64_t total_blocks;
  int32_t* err;
};
hipError_t launch_pack_fp4(const Fp4CopyArgs& a, hipStream_t stream);
hipError_t launch_unpack_fp4(const Fp4CopyArgs& a, hipStream_t stream);

}  // namespace kvx
