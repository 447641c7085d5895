// 4-bit-cache split kernel instantiated for 32 query rows per CTA.
#include "split_kv4.cuh"

namespace mlav {
cudaError_t launch_split_kv4_32(const SplitArgs& a, dim3 grid, cudaStream_t stream) {
  return launch_split_kv4_nq<32>(a, grid, stream);
}
int split_kv4_smem_32() { return kv4_smem_bytes<32>(); }
}  // namespace mlav
