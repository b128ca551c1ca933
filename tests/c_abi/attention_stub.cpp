// What stands behind the entry points of kvx_attention.h in the sanitizer build: launches that
// count, and kvx_status_string for the driver's messages.
#include "kvx_attention_launch.h"

extern "C" int launches = 0;
extern "C" const char* kvx_status_string(kvx_status) { return "status"; }

namespace kvx {
static hipError_t count() {
  ++launches;
  return hipSuccess;
}
hipError_t launch_rope(const RopeArgs&, bool, hipStream_t) { return count(); }
hipError_t launch_attention(const AttendArgs&, hipStream_t) { return count(); }
hipError_t launch_mass(const MassArgs&, hipStream_t) { return count(); }
hipError_t launch_evict_select(const SelectArgs&, hipStream_t) { return count(); }
hipError_t launch_evict_compact(const CompactArgs&, hipStream_t) { return count(); }
int64_t attention_workspace(const kvx_paged_cache&, const kvx_batch&, int32_t) { return 0; }
}  // namespace kvx
