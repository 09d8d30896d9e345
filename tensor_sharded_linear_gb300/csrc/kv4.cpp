// Host checks of the paged 4-bit cache.
#include <algorithm>
#include <exception>

#include "kv4.h"

namespace dt {

dt_status kv4_batch(const dt_dtensor* cache, const dt_dtensor* page_table, const dt_dtensor* kv_lens,
                    const dt_dtensor* q_starts, int tp, int D, int G, int64_t tokens, const Layout& mesh_of,
                    bool query, Kv4Batch* out) {
  DTensor C;
  dt_status st = parse_dtensor(cache, &C, "cache");
  if (st != DT_OK) return st;
  const Layout& L = C.layout;
  if ((st = same_mesh(L, mesh_of, "cache")) != DT_OK) return st;
  if (L.dtype != DT_INT32) return fail(DT_ERR_INVALID_ARG, "cache must be int32");
  const int W = kv4_words(D, G);
  if (L.ndim != 4 || L.gshape[3] != W)
    return fail(DT_ERR_SHAPE, "cache must be [pages, heads, page_size, %d] for head_dim %d in groups of %d", W, D, G);
  if (L.gshape[0] >= (1ll << 31) || L.gshape[1] > MAX_HEADS || L.gshape[2] > (1 << 20))
    return fail(DT_ERR_CAPACITY, "cache dims");
  if (L.gshape[2] < 1) return fail(DT_ERR_SHAPE, "cache: page_size must be at least 1");
  const bool sharded = tp >= 0 && L.is_shard(tp, 1);
  for (int m = 0; m < L.mesh_ndim; ++m) {
    if (m == tp && sharded) continue;
    if (!L.is_replicate(m))
      return fail(DT_ERR_PLACEMENT, "cache must be Shard(1) or Replicate on tp and Replicate on other mesh dims");
  }
  if (L.materialize && L.nslots > (sharded ? L.mesh[tp] : 1))
    return fail(DT_ERR_UNSUPPORTED, "cache with materialised replicas");
  CacheMap& M = out->cache;
  const int parts = sharded ? L.mesh[tp] : 1;
  M.heads = (int32_t)L.gshape[1];
  M.per_slot = (int32_t)std::max<int64_t>(1, (L.gshape[1] + parts - 1) / parts);
  M.pages = (int32_t)L.gshape[0];
  M.page_size = (int32_t)L.gshape[2];
  for (int j = 0; j < parts; ++j) {
    int c[DT_MAX_MESH_DIMS] = {0, 0, 0, 0};
    if (sharded) c[tp] = j;
    const SlotView& v = C.slots[L.slot_of_coords(c)];
    M.ptr[j] = reinterpret_cast<int32_t*>(v.ptr);
    M.page_stride[j] = v.stride[0];
    M.head_stride[j] = v.stride[1];
    if (v.numel == 0) continue;
    if (v.stride[3] != 1 || (v.shape[2] > 1 && v.stride[2] != W))
      return fail(DT_ERR_UNSUPPORTED, "cache: the records of a page and head must be contiguous");
    if (reinterpret_cast<uintptr_t>(v.ptr) % 16 || (v.shape[0] > 1 && v.stride[0] % 4) ||
        (v.shape[1] > 1 && v.stride[1] % 4))
      return fail(DT_ERR_ALIGNMENT, "cache: records must start on 16-byte boundaries");
  }
  // m = ceil(2^(31 + s) / d) with 2^s >= d: j m / 2^(31 + s) has the floor of j / d for every j < 2^31
  out->page_shift = 0;
  while ((1 << out->page_shift) < M.page_size) ++out->page_shift;
  out->page_mul = (uint32_t)(((1ull << (31 + out->page_shift)) + M.page_size - 1) / M.page_size);
  PlainOperand pt, kl, qs;
  if ((st = plain_operand(page_table, "page_table", mesh_of, false, &pt)) != DT_OK) return st;
  if (pt.dtype != DT_INT32) return fail(DT_ERR_INVALID_ARG, "page_table must be int32");
  if (pt.ndim != 2) return fail(DT_ERR_SHAPE, "page_table must be [batch, pages]");
  if (pt.shape[0] > (1 << 20) || pt.shape[1] >= (1ll << 31)) return fail(DT_ERR_CAPACITY, "page_table dims");
  out->batch = (int32_t)pt.shape[0];
  out->table_width = (int32_t)pt.shape[1];
  out->capacity = (int32_t)std::min<int64_t>(pt.shape[1] * (int64_t)M.page_size, (1ll << 31) - (1ll << 22));
  if (M.pages == 0) out->capacity = 0;
  out->page_table = reinterpret_cast<const int32_t*>(pt.ptr);
  out->kv_lens = nullptr;
  out->q_starts = nullptr;
  out->q_len = 0;
  if (query) return DT_OK;
  if ((st = plain_operand(kv_lens, "kv_lens", mesh_of, false, &kl)) != DT_OK) return st;
  if (kl.dtype != DT_INT32) return fail(DT_ERR_INVALID_ARG, "kv_lens must be int32");
  if (kl.ndim != 1 || kl.shape[0] != pt.shape[0]) return fail(DT_ERR_SHAPE, "kv_lens must be [batch]");
  out->kv_lens = reinterpret_cast<const int32_t*>(kl.ptr);
  if (q_starts) {
    if ((st = plain_operand(q_starts, "q_starts", mesh_of, false, &qs)) != DT_OK) return st;
    if (qs.dtype != DT_INT32) return fail(DT_ERR_INVALID_ARG, "q_starts must be int32");
    if (qs.ndim != 1 || qs.shape[0] != pt.shape[0] + 1) return fail(DT_ERR_SHAPE, "q_starts must be [batch + 1]");
    out->q_starts = reinterpret_cast<const int32_t*>(qs.ptr);
  } else {
    if (out->batch == 0 ? tokens != 0 : tokens % out->batch != 0)
      return fail(DT_ERR_SHAPE, "%lld tokens are not the same number for each of %d sequences: q_starts is needed",
                  (long long)tokens, out->batch);
    out->q_len = out->batch ? (int32_t)(tokens / out->batch) : 0;
  }
  return DT_OK;
}

}  // namespace dt

using namespace dt;

extern "C" dt_status dt_kv4_record_words(int32_t head_dim, int32_t group, int32_t* words) {
  clear_error();
  if (!words) return fail(DT_ERR_INVALID_ARG, "words is NULL");
  if (!kv4_format_ok(head_dim, group))
    return fail(DT_ERR_UNSUPPORTED, "head_dim %d in groups of %d (64, 128, 256 in groups of 32 or 64)", head_dim, group);
  *words = kv4_words(head_dim, group);
  return DT_OK;
}
