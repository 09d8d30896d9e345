// Checks of operands of rows.
//
// Model parallelism (wineandchord), "Sequence parallel": norms, dropout and
// residual work on token shards between the tensor-parallel layers; DTorch
// user guide, "Module parallel": RowParallelLinear leaves Partial.
#include <algorithm>

#include "row_operands.h"

namespace dt {

dt_status row_operand(const dt_dtensor* in, const char* what, int tp, bool output, bool sum, RowOperand* out,
                      Layout* layout) {
  DTensor X;
  dt_status st = parse_dtensor(in, &X, what);
  if (st != DT_OK) return st;
  const Layout& L = X.layout;
  *layout = L;
  if (L.ndim < 2) return fail(DT_ERR_SHAPE, "%s must be [..., channels]", what);
  if (tp >= L.mesh_ndim) return fail(DT_ERR_INVALID_ARG, "tp_mesh_dim %d", tp);
  if (L.dtype != DT_BF16 && L.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "%s must be bf16 or fp32", what);
  const int last = L.ndim - 1;
  int slots = 1;
  for (int m = 0; m < L.mesh_ndim; ++m) {
    if (L.is_replicate(m)) continue;
    slots *= L.mesh[m];
    if (L.is_shard(m, 0)) continue;
    if (sum && m == tp && L.is_partial(m)) {
      if (L.op[m] != DT_SUM) return fail(DT_ERR_UNSUPPORTED, "%s: parts are summed, Partial(sum) only", what);
      continue;
    }
    return fail(DT_ERR_PLACEMENT, "%s must be Replicate or Shard(0)%s", what, sum ? ", or Partial on tp" : "");
  }
  if (output && L.nslots > slots)
    return fail(DT_ERR_UNSUPPORTED, "%s: an output with materialised replicas", what);
  out->n = L.gshape[last];
  out->dtype = L.dtype;
  out->tokens = 1;
  int64_t inner = 1;
  for (int d = 0; d < last; ++d) out->tokens *= L.gshape[d];
  for (int d = 1; d < last; ++d) inner *= L.gshape[d];
  if (out->tokens >= MAX_ROWS) return fail(DT_ERR_CAPACITY, "%s: 2^31 - 2^16 tokens or more", what);
  if (out->n > (1 << 30)) return fail(DT_ERR_CAPACITY, "%s: more than 2^30 channels", what);
  out->parts = tp >= 0 && L.is_partial(tp) ? L.mesh[tp] : 1;
  out->vec16 = true;
  // the row blocks, by the first rank that holds each
  struct At {
    int64_t begin;
    int coords[DT_MAX_MESH_DIMS];
  } at[DT_MAX_SLOTS];
  int n = 0;
  for (int r = 0; r < L.mesh_size; ++r) {
    At a;
    L.rank_coords(r, a.coords);
    bool first = true;
    for (int m = 0; m < L.mesh_ndim; ++m) first = first && (L.kind[m] == DT_SHARD || a.coords[m] == 0);
    const Box b = L.box_of_coords(a.coords);
    if (!first || b.size[0] * inner * out->n == 0) continue;
    a.begin = b.off[0] * inner;
    at[n++] = a;  // (at most one per slot)
  }
  std::sort(at, at + n, [](const At& a, const At& b) { return a.begin < b.begin; });
  out->count = n;
  for (int part = 0; part < out->parts; ++part)
    for (int i = 0; i < n; ++i) {
      if (L.nslots > 0 && out->parts > 1) at[i].coords[tp] = part;
      const SlotView& v = X.slots[L.slot_of_coords(at[i].coords)];
      if (v.shape[last] > 1 && v.stride[last] != 1) return fail(DT_ERR_UNSUPPORTED, "%s must have unit inner stride", what);
      int64_t ld = 0, span = 0, rows = 1;
      bool have = false;
      for (int d = last - 1; d >= 0; --d) {
        rows *= v.shape[d];
        if (v.shape[d] == 1) continue;
        if (!have) {
          ld = v.stride[d];
          span = ld * v.shape[d];
          have = true;
        } else {
          if (v.stride[d] != span) return fail(DT_ERR_UNSUPPORTED, "%s: leading dims must be collapsible", what);
          span *= v.shape[d];
        }
      }
      if (output && rows > 1 && ld < out->n) return fail(DT_ERR_UNSUPPORTED, "%s: rows of an output overlap", what);
      out->block[part * n + i] = RowBlock{v.ptr, ld, at[i].begin};
      out->vec16 = out->vec16 && reinterpret_cast<uintptr_t>(v.ptr) % 16 == 0 && ld * L.esize % 16 == 0;
    }
  return DT_OK;
}

}  // namespace dt
