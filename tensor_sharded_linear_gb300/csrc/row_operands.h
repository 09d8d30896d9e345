// Operands of rows: [..., N] activations whose tokens lie on one slot, in row
// blocks on several (Shard(0)), or as partial sums (Partial) on the shards of
// tp, as the column- and row-parallel linears take and leave them.
#pragma once

#include <cstdint>

#include "head_operands.h"

namespace dt {

// Rows [begin, begin of the next block) of a tensor, or of one part of a sum.
struct RowBlock {
  char* ptr;      // row `begin`
  int64_t ld;     // elements between rows
  int64_t begin;  // first token
};

// A tensor's blocks in a launch's table: `count` blocks, ascending, for each
// of `parts` parts of a sum (1: no sum), part after part.
struct RowTable {
  int16_t first = 0, count = 0, parts = 0, dtype = 0;
};

#ifdef __CUDACC__
// The block of token t in a table of ascending blocks; `at` remembers it, and
// later tokens only move on.
__device__ __forceinline__ int row_block(const RowBlock* blocks, const RowTable& r, int64_t t, int& at) {
  while (at + 1 < r.count && blocks[r.first + at + 1].begin <= t) ++at;
  return r.first + at;
}
__device__ __forceinline__ char* row_at(const RowBlock& b, int64_t t, int esize) {
  return b.ptr + (t - b.begin) * b.ld * esize;
}
#endif

struct RowOperand {
  RowBlock block[DT_MAX_SLOTS];  // parts after parts
  int count = 0, parts = 1;
  int64_t tokens = 0, n = 0;
  int dtype = 0;
  bool vec16 = true;  // every row starts on a 16-byte boundary
};

// Check `in` as a [..., N] operand of rows and fill `out`: Replicate or
// Shard(0) on every mesh dim, or (sum) Partial(sum) on tp; leading dims
// collapse to one token dim; unit inner stride.  Outputs must not have
// materialised replicas, nor rows that overlap.
dt_status row_operand(const dt_dtensor* in, const char* what, int tp, bool output, bool sum, RowOperand* out,
                      Layout* layout);

}  // namespace dt
