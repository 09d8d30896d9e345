// The block norms' kernels for bf16 x in a bf16 residual stream.
#include "block_norm.cuh"

namespace dt {

cudaError_t block_rows_bf16(const BlockSmall& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  return block_rows<__nv_bfloat16, __nv_bfloat16>(p, bwd, s, stream);
}
cudaError_t block_rows_bf16(const BlockLarge& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  return block_rows<__nv_bfloat16, __nv_bfloat16>(p, bwd, s, stream);
}

}  // namespace dt
