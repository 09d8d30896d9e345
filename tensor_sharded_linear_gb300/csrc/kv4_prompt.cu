// The tensor-core attention kernel for prompts: instantiations and launch.
#include <atomic>
#include <exception>

#include "kv4_prompt.cuh"

namespace dt {
namespace kv4 {

namespace {

template <int D, int G>
cudaError_t prepare() {
  static std::atomic<bool> done[64];  // by device; calls come from any thread
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv4_prompt_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PromptShape<D, G>::SMEM);
    if (e != cudaSuccess) return e;
    done[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

template <int D, int G>
cudaError_t launch_one(const AttnParams& p, int grid, cudaStream_t s) {
  cudaError_t e =
      launch_early(kv4_prompt_kernel<D, G>, dim3(grid), 32 * PROMPT_WARPS, PromptShape<D, G>::SMEM, s, p);
  if (e != cudaSuccess) return e;
  return launch_early(kv4_join_kernel<__nv_bfloat16, D>, join_grid(grid, p.rb, D), 32 * JOIN_WARPS, 0, s, p);
}

}  // namespace

cudaError_t prompt_variant(int D, int G, Variant* out) {
  cudaError_t e = D == 64    ? (G == 32 ? prepare<64, 32>() : prepare<64, 64>())
                  : D == 128 ? (G == 32 ? prepare<128, 32>() : prepare<128, 64>())
                             : (G == 32 ? prepare<256, 32>() : prepare<256, 64>());
  if (e != cudaSuccess) return e;
  out->grid = device_sm_count();
  out->rows = D == 64 ? PromptShape<64, 64>::ROWS : D == 128 ? PromptShape<128, 64>::ROWS : PromptShape<256, 64>::ROWS;
  const size_t splits = ((size_t)out->grid * sizeof(Split) + 255) / 256 * 256;
  out->bytes = splits + (size_t)2 * out->grid * out->rows * (D + 4) * sizeof(float);
  return cudaSuccess;
}

cudaError_t prompt_launch(const AttnParams& p, int D, int G, int grid, cudaStream_t s) {
  if (D == 64) return G == 32 ? launch_one<64, 32>(p, grid, s) : launch_one<64, 64>(p, grid, s);
  if (D == 128) return G == 32 ? launch_one<128, 32>(p, grid, s) : launch_one<128, 64>(p, grid, s);
  return G == 32 ? launch_one<256, 32>(p, grid, s) : launch_one<256, 64>(p, grid, s);
}

}  // namespace kv4
}  // namespace dt
