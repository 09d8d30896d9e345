// Host and device description of one attention call over the 4-bit cache.
#pragma once

#include <cuda_runtime.h>

#include "heads_sm103.cuh"
#include "kv4.h"

namespace dt {
namespace kv4 {

constexpr int WARPS = 4;             // each takes every fourth tile of keys
constexpr int THREADS = 32 * WARPS;
// Least multiplier of S, the least positive fp32 number: |S| stays below
// 2^123, so what is smaller makes logits of 0 as this does; but 0 itself would
// make NaN of the -inf that hidden keys have.
constexpr float LEAST_SCALE = 1.401298464324817e-45f;

// What a CTA left unfinished: the unit whose keys begin in its range and end
// in CTA `last`'s (unit < 0: none).  The join kernel adds those pieces.
struct Split {
  int32_t unit;  // >= 0: the row block below is split
  int32_t q_row; // first (query, head) row of the block
  int32_t rows;  // rows of the block
  int32_t q0;    // first token of the sequence
  int32_t head;  // kv head
  int32_t last;  // CTA that holds the last piece
};

struct AttnParams {
  HeadMap q, out, lse;
  CacheMap cache;
  SeqTable seq;
  const int32_t* page_table;
  int32_t table_width;
  int32_t g;  // query heads per kv head
  uint32_t page_mul, page_shift;  // division by the page size (Kv4Batch)
  int32_t causal, window;
  int32_t want_lse;
  int32_t rb;        // rows of a unit (for the join)
  float scale_log2;  // softmax scale * log2(e)
  float* part;       // [2 CTAs][rows][D + 4]: sums, then maximum (log2 units), denominator, padding
  Split* split;      // [CTA]
  int32_t* status;
  unsigned long long wait_limit_ns;
  uint32_t starve;  // test hook: from this step (tile) on copies stay short of what their barrier awaits
};

#ifdef __CUDACC__
// First key that a query at position pos sees through the window (0: none).
// Positions are negative where a sequence has more queries than keys, and
// windows may be any size: pos - window itself can leave 32 bits.
__device__ __forceinline__ int window_begin(int pos, int window) {
  return window && pos >= window ? pos - window + 1 : 0;
}
#endif

// Grid of the device-filling launch, rows of a unit and workspace of one
// variant; and its launch (defined per head_dim).
struct Variant {
  int grid = 0;
  int rows = 0;
  size_t bytes = 0;
};
template <int D>
cudaError_t variant(int G, bool fp32, int64_t rows_per_seq, Variant* out);
template <int D>
cudaError_t launch(const AttnParams& p, int G, bool fp32, int64_t rows_per_seq, int grid, cudaStream_t s);

// The tensor-core kernel for prompts (bf16).
cudaError_t prompt_variant(int D, int G, Variant* out);
cudaError_t prompt_launch(const AttnParams& p, int D, int G, int grid, cudaStream_t s);

}  // namespace kv4
}  // namespace dt
