// Operands that are sharded by attention heads: [..., H * D] activations as
// the column-parallel q/k/v projections leave them (Shard(-1) on tp, every
// shard holding whole heads), and the small int32 / fp32 tensors that go
// with them (positions, page tables, lengths, rotation tables, weights).
#pragma once

#include <cstdint>

#include "dt_internal.h"

namespace dt {

// Where head h of token t lives: slot h / per_slot, at
// ptr + (t * stride + (h % per_slot) * D) * element size.
struct HeadMap {
  struct Slot {
    char* ptr;
    int64_t stride;  // elements between consecutive tokens
  } slot[DT_MAX_SLOTS];
  int32_t per_slot;  // heads of a full slot
  uint32_t mul;      // ceil(2^31 / per_slot): h / per_slot = umulhi(2 h + 1, mul) for h < 2^15
  int32_t heads;     // heads in all
};
constexpr int MAX_HEADS = 1 << 15;
// Tokens, and (query, head) rows of a kv head, stay below this: kernels count
// them in 32 bits and add a grid's stride of them (a few thousand).
constexpr int64_t MAX_ROWS = (1ll << 31) - (1ll << 16);

#ifdef __CUDACC__
// Address of head h of token t.
template <class T>
__device__ __forceinline__ T* head_ptr(const HeadMap& m, int64_t t, int h, int d) {
  const int s = __umulhi(2u * (uint32_t)h + 1u, m.mul);
  const HeadMap::Slot& v = m.slot[s];
  return reinterpret_cast<T*>(v.ptr) + (t * v.stride + (h - s * m.per_slot) * d);
}
#endif

// What the host learns about a head-sharded operand besides its HeadMap.
struct HeadOperand {
  HeadMap map;
  int64_t tokens = 0;
  int heads = 0;
  int dtype = 0;
  bool vec16 = true;  // every head of every token starts on a 16-byte boundary
};

// Check `in` as a [..., H * D] operand and fill `out`.  Its last dim is
// Shard(-1) or Replicate on tp (tp < 0: Replicate everywhere) and Replicate
// on the other mesh dims; shards hold whole heads; leading dims collapse to
// one token dim.  Outputs must not have materialised replicas.
dt_status head_operand(const dt_dtensor* in, const char* what, int tp, int head_dim, bool output, HeadOperand* out,
                       Layout* layout);

// A Replicate, contiguous tensor: slot 0's pointer and its shape.
struct PlainOperand {
  const char* ptr = nullptr;
  int ndim = 0;
  int64_t shape[DT_MAX_TENSOR_DIMS] = {1, 1, 1, 1};
  int64_t numel = 0;
  int dtype = 0;
};
dt_status plain_operand(const dt_dtensor* in, const char* what, const Layout& mesh_of, bool output, PlainOperand* out);

// Both layouts on the same mesh?
dt_status same_mesh(const Layout& a, const Layout& b, const char* what);

// Run `body` (a callable returning dt_status) with no C++ exception leaving it.
template <class F>
dt_status no_throw(F&& body) {
  try {
    return body();
  } catch (const std::exception& e) {
    return fail(DT_ERR_CAPACITY, "host memory: %s", e.what());
  } catch (...) {
    return fail(DT_ERR_CAPACITY, "host error");
  }
}

}  // namespace dt
