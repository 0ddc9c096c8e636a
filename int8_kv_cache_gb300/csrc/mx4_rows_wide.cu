// Instantiations of the MX4 decode: one 8-warp CTA per row and KV head.
#include "mx4_kernel.cuh"

namespace i8kv {
cudaError_t launch_paged_mx4_rows_wide(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                       KernelInfo* info) {
  return dispatch_mx4<kMx4WideWarps, Mx4Way::kRows>(key, p, s, info);
}
}  // namespace i8kv
