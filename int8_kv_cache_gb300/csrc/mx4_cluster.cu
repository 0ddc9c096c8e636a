// Instantiations of the MX4 decode: clusters of 8-warp CTAs, one per row and KV head,
// which join through distributed shared memory.
#include "mx4_kernel.cuh"

namespace i8kv {
cudaError_t launch_paged_mx4_cluster(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                     KernelInfo* info) {
  return dispatch_mx4<kMx4WideWarps, Mx4Way::kCluster>(key, p, s, info);
}
}  // namespace i8kv
