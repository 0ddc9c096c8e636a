// Dense causal attention over int8 pages.
#include "attend_launch.cuh"

namespace i8kv {
cudaError_t launch_attend_int8(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s) {
  return ap::launch_of<ap::kI8>(p, two_tiles, ctas, s);
}
}  // namespace i8kv
