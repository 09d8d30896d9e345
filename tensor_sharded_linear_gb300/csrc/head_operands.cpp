// Checks of head-sharded operands and of the Replicate tensors beside them.
//
// Model parallelism (wineandchord), "Tensor-parallel linear layers": q/k/v
// are column-parallel, so a rank holds the columns of whole heads; nanotron
// tutorial, 5.1: attention runs on each rank's heads between the column- and
// the row-parallel linear.
#include <exception>

#include "head_operands.h"

namespace dt {

dt_status same_mesh(const Layout& a, const Layout& b, const char* what) {
  bool ok = a.mesh_ndim == b.mesh_ndim;
  for (int m = 0; ok && m < a.mesh_ndim; ++m) ok = a.mesh[m] == b.mesh[m];
  return ok ? DT_OK : fail(DT_ERR_SHAPE, "%s: meshes differ", what);
}

dt_status head_operand(const dt_dtensor* in, const char* what, int tp, int head_dim, bool output, HeadOperand* out,
                       Layout* layout) {
  DTensor X;
  dt_status st = parse_dtensor(in, &X, what);
  if (st != DT_OK) return st;
  const Layout& L = X.layout;
  *layout = L;
  if (L.ndim < 2) return fail(DT_ERR_SHAPE, "%s must be [..., heads * head_dim]", what);
  if (tp >= L.mesh_ndim) return fail(DT_ERR_INVALID_ARG, "tp_mesh_dim %d", tp);
  if (L.dtype != DT_BF16 && L.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "%s must be bf16 or fp32", what);
  const int last = L.ndim - 1;
  const int64_t width = L.gshape[last];
  if (width % head_dim != 0)
    return fail(DT_ERR_SHAPE, "%s: last dim %lld is not a multiple of head_dim %d", what, (long long)width, head_dim);
  if (width / head_dim > MAX_HEADS) return fail(DT_ERR_CAPACITY, "%s: more than %d heads", what, MAX_HEADS);
  const bool sharded = tp >= 0 && L.is_shard(tp, last);
  for (int m = 0; m < L.mesh_ndim; ++m) {
    if (m == tp && sharded) continue;
    if (!L.is_replicate(m))
      return fail(DT_ERR_PLACEMENT, "%s must be Shard(-1) or Replicate on tp and Replicate on other mesh dims", what);
  }
  if (output && L.materialize && L.nslots > (sharded ? L.mesh[tp] : 1))
    return fail(DT_ERR_UNSUPPORTED, "%s: an output with materialised replicas", what);
  const int parts = sharded ? L.mesh[tp] : 1;
  const int64_t chunk = width > 0 ? (width + parts - 1) / parts : 0;
  if (chunk % head_dim != 0)
    return fail(DT_ERR_SHAPE, "%s: shards of %lld columns do not hold whole heads of %d", what, (long long)chunk,
                head_dim);
  out->heads = (int)(width / head_dim);
  out->dtype = L.dtype;
  out->tokens = 1;
  for (int d = 0; d < last; ++d) out->tokens *= L.gshape[d];
  if (out->tokens >= MAX_ROWS) return fail(DT_ERR_CAPACITY, "%s: 2^31 - 2^16 tokens or more", what);
  HeadMap& M = out->map;
  M.heads = out->heads;
  M.per_slot = chunk > 0 ? (int32_t)(chunk / head_dim) : 1;
  M.mul = (uint32_t)(((1ull << 31) + M.per_slot - 1) / M.per_slot);
  out->vec16 = true;
  for (int j = 0; j < parts; ++j) {
    int c[DT_MAX_MESH_DIMS] = {0, 0, 0, 0};
    if (sharded) c[tp] = j;
    const SlotView& v = X.slots[L.slot_of_coords(c)];
    M.slot[j].ptr = v.ptr;
    M.slot[j].stride = 0;
    if (v.numel == 0) continue;  // an empty slot's strides are arbitrary
    if (v.shape[last] > 1 && v.stride[last] != 1)
      return fail(DT_ERR_UNSUPPORTED, "%s must have unit inner stride", what);
    int64_t rs = 0;
    bool have = false;
    int64_t span = 0;  // elements between rows of the next outer dim
    for (int d = last - 1; d >= 0; --d) {
      if (v.shape[d] == 1) continue;
      if (!have) {
        rs = v.stride[d];
        span = rs * v.shape[d];
        have = true;
      } else {
        if (v.stride[d] != span) return fail(DT_ERR_UNSUPPORTED, "%s: leading dims must be collapsible", what);
        span *= v.shape[d];
      }
    }
    if (output && out->tokens > 1 && rs < v.shape[last])
      return fail(DT_ERR_UNSUPPORTED, "%s: rows of an output overlap", what);
    M.slot[j].stride = rs;
    out->vec16 = out->vec16 && reinterpret_cast<uintptr_t>(v.ptr) % 16 == 0 && (rs * L.esize) % 16 == 0;
  }
  out->vec16 = out->vec16 && (head_dim * L.esize) % 16 == 0;
  return DT_OK;
}

dt_status plain_operand(const dt_dtensor* in, const char* what, const Layout& mesh_of, bool output,
                        PlainOperand* out) {
  DTensor X;
  dt_status st = parse_dtensor(in, &X, what);
  if (st != DT_OK) return st;
  const Layout& L = X.layout;
  if ((st = same_mesh(L, mesh_of, what)) != DT_OK) return st;
  for (int m = 0; m < L.mesh_ndim; ++m)
    if (!L.is_replicate(m)) return fail(DT_ERR_PLACEMENT, "%s must be Replicate", what);
  if (output && L.nslots > 1) return fail(DT_ERR_UNSUPPORTED, "%s: an output with materialised replicas", what);
  const SlotView& v = X.slots[0];
  out->ptr = v.ptr;
  out->ndim = L.ndim;
  out->numel = v.numel;
  out->dtype = L.dtype;
  int64_t expect = 1;
  for (int d = L.ndim - 1; d >= 0; --d) {
    out->shape[d] = v.shape[d];
    if (v.numel > 0 && v.shape[d] > 1 && v.stride[d] != expect)
      return fail(DT_ERR_UNSUPPORTED, "%s must be contiguous", what);
    expect *= v.shape[d];
  }
  return DT_OK;
}

}  // namespace dt
