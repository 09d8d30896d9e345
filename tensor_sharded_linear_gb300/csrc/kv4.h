// The paged 4-bit cache of keys and values.
//
// int32 [pages, kv heads, page size, words]: one record per token and kv
// head, all of a token's key and value for a head in one contiguous run, so
// an append writes one run and an attention tile is one bulk copy per page:
//   D/8 words   key codes, nibble i of word w = channel 8 w + i
//   D/8 words   value codes
//   D/G words   key parameters, one word per group of G channels:
//               bf16 step in the low half, bf16 minimum in the high half
//   D/G words   value parameters
//   padding to a multiple of 4 words (records start on 16 bytes)
// A code c stands for minimum + c * step, held exactly in fp32 but for the
// one rounding of that sum.
#pragma once

#include "head_operands.h"

namespace dt {

__host__ __device__ constexpr int kv4_words(int D, int G) { return (2 * (D / 8) + 2 * (D / G) + 3) / 4 * 4; }

inline bool kv4_format_ok(int D, int G) { return (D == 64 || D == 128 || D == 256) && (G == 32 || G == 64); }

// Heads of the cache: slot h / per_slot at ptr[slot] + page * page_stride +
// (h % per_slot) * head_stride (in words), records contiguous after that.
struct CacheMap {
  int32_t* ptr[DT_MAX_SLOTS];
  int64_t page_stride[DT_MAX_SLOTS];
  int64_t head_stride[DT_MAX_SLOTS];
  int32_t per_slot, heads, pages, page_size;
};

#ifdef __CUDACC__
__device__ __forceinline__ int32_t* cache_page(const CacheMap& m, int64_t page, int h) {
  const int s = static_cast<unsigned>(h) / static_cast<unsigned>(m.per_slot);
  return m.ptr[s] + page * m.page_stride[s] + static_cast<int64_t>(h - s * m.per_slot) * m.head_stride[s];
}
#endif

// The cache and the batch it serves, checked: cache [pages, heads, page
// size, words] Shard(1) or Replicate on tp; page_table int32 [batch, n],
// kv_lens int32 [batch], q_starts int32 [batch + 1] or NULL, all Replicate.
// query: kv_lens and q_starts are not looked at (nor set).
struct Kv4Batch {
  CacheMap cache;
  const int32_t* page_table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int32_t batch, table_width, q_len;
  int32_t capacity;  // keys a row of the page table can address
  uint32_t page_mul, page_shift;  // j / page_size = umulhi(2 j, page_mul) >> page_shift for j < 2^31
};
dt_status kv4_batch(const dt_dtensor* cache, const dt_dtensor* page_table, const dt_dtensor* kv_lens,
                    const dt_dtensor* q_starts, int tp, int D, int G, int64_t tokens, const Layout& mesh_of,
                    bool query, Kv4Batch* out);

}  // namespace dt
