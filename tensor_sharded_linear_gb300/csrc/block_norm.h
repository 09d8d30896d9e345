// Arguments and launch shapes of the block norms.
#pragma once

#include <cuda_runtime.h>

#include "row_operands.h"

namespace dt {

struct BlockArgs {
  RowTable x, r, h, y;    // forward: h and y are written; backward: they are dh and dy
  RowTable dx, dr;        // backward
  const void *post, *gate, *pre;
  void *dpost, *dgate, *dpre;
  int32_t post_dtype, gate_dtype, pre_dtype, dpost_dtype, dgate_dtype, dpre_dtype;
  const int32_t* rng;     // NULL: no dropout
  uint32_t drop_below;    // words below this are dropped
  float drop_scale;       // 1 / (1 - p)
  float eps, scale;
  int64_t tokens;
  int32_t n;
  int64_t gate_rows, gate_per;  // rows of the gate, consecutive tokens of each
  // backward: sums per run of tokens (a CTA's, or a cluster's), [run][pitch] for
  // pre and post, [run + gate row][pitch] for the gate
  float *part_pre, *part_post, *part_gate;
  int32_t runs, pitch;
  // tokens of a run: run_tokens, and one more in the first run_more runs
  int32_t run_tokens, run_more;
};

#ifdef __CUDACC__
__device__ __forceinline__ int64_t run_begin(const BlockArgs& p, int run) {
  return (int64_t)run * p.run_tokens + min(run, p.run_more);
}
__device__ __forceinline__ int64_t run_of(const BlockArgs& p, int64_t t) {
  const int64_t longer = (int64_t)p.run_more * (p.run_tokens + 1);
  return t < longer ? t / (p.run_tokens + 1) : p.run_more + (t - longer) / max(p.run_tokens, 1);
}
#endif

// The launch's tables of row blocks; most launches need few.
template <int CAP>
struct BlockParams : BlockArgs {
  static constexpr int kCap = CAP;
  RowBlock blocks[CAP];
};
using BlockSmall = BlockParams<64>;
using BlockLarge = BlockParams<6 * DT_MAX_SLOTS>;

// How a launch covers its rows.
struct BlockShape {
  int threads = 0, vpt = 0, grid = 0;  // vpt: vectors of 8 channels a thread; 0: the kernels for any size
  int cluster = 1;     // backward: CTAs that share a row's channels
  int stages = 0;      // backward: rows of the ring
  bool ahead = false;  // forward: the next row's loads go out early
  bool even = true;    // rows of a multiple of 8 channels on 16-byte boundaries
  size_t smem = 0;
};
constexpr int BN_SMEM = 224 * 1024;  // of an SM, for rings
constexpr int BN_STATIC = 2560;      // a CTA's other shared memory, at most
// Threads of forward CTAs that an SM's registers are shared among, measured
// together with the vectors a thread at 8192 x 4096 with dropout: four vectors
// and 640 threads 51.6 us, two and 768 57.7, eight and 512 64.7.
constexpr int block_forward_resident(int vpt, bool ahead, int esize) {
  return vpt == 1 ? 1024 : vpt == 2 ? (ahead ? 768 : 1024) : ahead ? (esize == 4 ? 512 : 640) : 768;
}

// Launches of the kernels on vectors of 8 channels, by the types of x and of
// the residual stream (one translation unit each).
#define DT_BLOCK_LAUNCHES(name)                                                                        \
  cudaError_t name(const BlockSmall& p, bool bwd, const BlockShape& s, cudaStream_t stream);           \
  cudaError_t name(const BlockLarge& p, bool bwd, const BlockShape& s, cudaStream_t stream);
DT_BLOCK_LAUNCHES(block_rows_bf16)
DT_BLOCK_LAUNCHES(block_rows_mixed)
DT_BLOCK_LAUNCHES(block_rows_fp32)

}  // namespace dt
