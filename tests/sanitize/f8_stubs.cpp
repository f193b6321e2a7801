// Stand-ins for the launches of the products in 8-bit floating point, so that their host-side code (f8_api.cpp) links into
// the sanitizer build without any device code.
#include <hip/hip_runtime.h>

#include "f8.h"

namespace bsg {
hipError_t f8_quantize_launch(Src, int64_t, int64_t, const void*, int64_t, void*, int64_t, float*, int64_t, hipStream_t) {
  return hipErrorUnknown;
}
hipError_t f8_few_launch(const F8Args&, Src, bool, int, hipStream_t) { return hipErrorUnknown; }
hipError_t f8_tiled_launch(const F8Args&, bool, int, int, hipStream_t) { return hipErrorUnknown; }
void f8_workspace(int64_t, int, uint64_t* part_bytes, uint64_t* counter_bytes) { *part_bytes = *counter_bytes = 0; }
}  // namespace bsg
