// Instantiations of the MX4 decode: one 4-warp CTA per row and KV head.
#include "mx4_kernel.cuh"

namespace i8kv {
cudaError_t launch_paged_mx4_rows(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                  KernelInfo* info) {
  return dispatch_mx4<kMx4Warps, Mx4Way::kRows>(key, p, s, info);
}
}  // namespace i8kv
