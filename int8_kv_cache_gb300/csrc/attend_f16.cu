// Dense causal attention over fp16 rows and pages.
#include "attend_launch.cuh"

namespace i8kv {
cudaError_t launch_attend_f16(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s) {
  return ap::launch_of<ap::kF16>(p, two_tiles, ctas, s);
}
}  // namespace i8kv
