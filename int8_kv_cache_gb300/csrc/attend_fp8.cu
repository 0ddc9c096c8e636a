// Dense causal attention over float8 e4m3fn pages.
#include "attend_launch.cuh"

namespace i8kv {
cudaError_t launch_attend_fp8(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s) {
  return ap::launch_of<ap::kE4>(p, two_tiles, ctas, s);
}
}  // namespace i8kv
