// The attention kernels over the 4-bit cache for heads of 64 channels.
#include <exception>

#include "kv4_attention.cuh"

namespace dt {
namespace kv4 {

template cudaError_t variant<64>(int, bool, int64_t, Variant*);
template cudaError_t launch<64>(const AttnParams&, int, bool, int64_t, int, cudaStream_t);

}  // namespace kv4
}  // namespace dt
