// Instantiations of the MX4 decode: 8-warp CTAs over balanced pieces of few long rows, whose
// partials the combine kernel joins.
#include "mx4_kernel.cuh"

namespace i8kv {
cudaError_t launch_paged_mx4_wide(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                  KernelInfo* info) {
  return dispatch_mx4<kMx4WideWarps, Mx4Way::kPieces>(key, p, s, info);
}
}  // namespace i8kv
