// The block norms' kernels for fp32 x.
#include "block_norm.cuh"

namespace dt {

cudaError_t block_rows_fp32(const BlockSmall& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  return block_rows<float, float>(p, bwd, s, stream);
}
cudaError_t block_rows_fp32(const BlockLarge& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  return block_rows<float, float>(p, bwd, s, stream);
}

}  // namespace dt
