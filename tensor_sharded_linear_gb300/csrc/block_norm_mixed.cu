// The block norms' kernels for bf16 x in a fp32 residual stream.
#include "block_norm.cuh"

namespace dt {

cudaError_t block_rows_mixed(const BlockSmall& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  return block_rows<__nv_bfloat16, float>(p, bwd, s, stream);
}
cudaError_t block_rows_mixed(const BlockLarge& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  return block_rows<__nv_bfloat16, float>(p, bwd, s, stream);
}

}  // namespace dt
