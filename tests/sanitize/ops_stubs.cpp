// Stand-ins for the cache's, attention's and expert layer's launches, so that their host-side code
// (kv_api.cpp, moe_api.cpp) links into the sanitizer build without any device code.
#include <hip/hip_runtime.h>

#include "kv.h"
#include "moe.h"

namespace bsg {
hipError_t kv_append_launch(const KvArgs&, int, int, bool, hipStream_t) { return hipErrorUnknown; }
hipError_t kv_read_launch(const KvArgs&, int, int, hipStream_t) { return hipErrorUnknown; }
hipError_t kv_attend_launch(const KvArgs&, int, int, int, hipStream_t) { return hipErrorUnknown; }
void kv_workspace(const bsg_kv_problem&, int, size_t* part, size_t* counters, size_t* groups) { *part = *counters = *groups = 0; }
size_t moe_workspace(const bsg_moe_problem&, uint8_t*, MoeArgs*, size_t* at, size_t* bytes) { return *at = *bytes = 0; }
hipError_t moe_launch(const MoeArgs&, int, int, hipStream_t) { return hipErrorUnknown; }
}  // namespace bsg
