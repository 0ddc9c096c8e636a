// Dense causal attention over MX4 records.
#include "attend_launch.cuh"

namespace i8kv {
cudaError_t launch_attend_mx4(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s) {
  return ap::launch_of<ap::kMx4>(p, two_tiles, ctas, s);
}
}  // namespace i8kv
