// What stands behind the entry points of kvx_fp4.h in the sanitizer build: launches that count, and
// kvx_status_string for the driver's messages.
#include "kvx_fp4_launch.h"

extern "C" int launches = 0;
extern "C" const char* kvx_status_string(kvx_status) { return "status"; }

namespace kvx {
static hipError_t count() {
  ++launches;
  return hipSuccess;
}
hipError_t launch_rope_fp4(const Fp4RopeArgs&, bool, hipStream_t) { return count(); }
hipError_t launch_attention_fp4(const AttendArgs&, hipStream_t) { return count(); }
hipError_t launch_pack_fp4(const Fp4CopyArgs&, hipStream_t) { return count(); }
hipError_t launch_unpack_fp4(const Fp4CopyArgs&, hipStream_t) { return count(); }
int64_t attention_fp4_workspace(const kvx_paged_cache&, const kvx_batch&, int32_t) { return 0; }
}  // namespace kvx
