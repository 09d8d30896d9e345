// Entry points of attention over the paged 4-bit cache: checks, choice of
// the kernel variant, workspace.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <exception>

#include "kv4_attention.h"
#include "ptx_sm103.cuh"

namespace dt {

namespace kv4 {
extern template cudaError_t variant<64>(int, bool, int64_t, Variant*);
extern template cudaError_t variant<128>(int, bool, int64_t, Variant*);
extern template cudaError_t variant<256>(int, bool, int64_t, Variant*);
extern template cudaError_t launch<64>(const AttnParams&, int, bool, int64_t, int, cudaStream_t);
extern template cudaError_t launch<128>(const AttnParams&, int, bool, int64_t, int, cudaStream_t);
extern template cudaError_t launch<256>(const AttnParams&, int, bool, int64_t, int, cudaStream_t);
}  // namespace kv4

namespace {

using namespace kv4;

// The kernel for prompts from this many (query, head) rows per sequence and
// kv head.  It works on blocks of 256 rows (128 at head_dim 256) whatever
// their number, the other in passes of 16.  16 sequences of 4096 keys, the
// other kernel's time first: 32/8 heads of 128, 64 rows 111 and 76 us, 256
// rows 405 and 98, and 48 rows 87 where 64 take 76 here; 16/16 heads of 64, 64
// rows 125 and 100; 16/2 heads of 256, 48 rows 60 where 64 take 45 here.  With
// two sequences of 2048 keys, too little for the whole device, the two meet
// at about 96 to 128 rows (64 rows: 17.6 and 21.9 us).  The number is the
// call's average, since the host does not know the lengths: where they differ
// much, some rows run on the kernel that suits them less.  All measured with
// equal lengths.
constexpr int64_t PROMPT_FROM = 64;
bool prompt_kernel(bool fp32, int64_t rows) { return !fp32 && rows >= PROMPT_FROM; }

cudaError_t variant_any(int D, int G, bool fp32, int64_t rows, Variant* v) {
  if (prompt_kernel(fp32, rows)) return prompt_variant(D, G, v);
  return D == 64 ? variant<64>(G, fp32, rows, v) : D == 128 ? variant<128>(G, fp32, rows, v)
                                                            : variant<256>(G, fp32, rows, v);
}

// Test hooks, read once from the environment: DT_KV4_WAIT_LIMIT_MS bounds the
// kernels' waits (default 2000 ms); DT_KV4_STARVE=n makes the barriers of the
// n-th step of each CTA (tile of each warp) and of those after it await more
// bytes than are copied, so the waits run out and the kernel reports
// DT_DEV_ERR_TIMEOUT.
struct Hooks {
  unsigned long long wait_limit_ns = WAIT_LIMIT_NS;
  uint32_t starve = ~0u;  // a step's number; no share has that many
};
const Hooks& hooks() {
  static const Hooks h = [] {
    Hooks x;
    const char* e = getenv("DT_KV4_WAIT_LIMIT_MS");
    const long ms = e ? atol(e) : 0;
    if (ms > 0 && ms <= 10000) x.wait_limit_ns = (unsigned long long)ms * 1000000ull;
    e = getenv("DT_KV4_STARVE");
    const long n = e ? atol(e) : 0;
    if (n > 0 && n <= 1000000) x.starve = (uint32_t)n - 1;
    return x;
  }();
  return h;
}

// The operands that decide the variant, checked.
struct Checked {
  HeadOperand Q;
  Layout lq;
  Kv4Batch B;
  int64_t rows_per_seq = 0;  // on average: (query, head) rows per kv head
  bool nothing = false;      // no output elements
};

dt_status check(const dt_dtensor* q, const dt_dtensor* cache, const dt_dtensor* page_table, const dt_dtensor* kv_lens,
                const dt_dtensor* q_starts, int D, int G, int tp, bool query,
                Checked* c) {
  if (!kv4_format_ok(D, G))
    return fail(DT_ERR_UNSUPPORTED, "head_dim %d in groups of %d (64, 128, 256 in groups of 32 or 64)", D, G);
  dt_status st = head_operand(q, "q", tp, D, false, &c->Q, &c->lq);
  if (st != DT_OK) return st;
  if ((st = kv4_batch(cache, page_table, kv_lens, q_starts, tp, D, G, c->Q.tokens, c->lq, query, &c->B)) != DT_OK) return st;
  c->nothing = c->Q.tokens == 0 || c->Q.heads == 0;
  if (c->B.cache.heads == 0 ? c->Q.heads != 0 : c->Q.heads % c->B.cache.heads != 0)
    return fail(DT_ERR_SHAPE, "q has %d heads, the cache %d: not a multiple", c->Q.heads, c->B.cache.heads);
  if (!c->Q.vec16) return fail(DT_ERR_ALIGNMENT, "q must have 16-byte aligned rows");
  if (!c->nothing && c->B.batch > 0) {
    const int64_t g = c->Q.heads / c->B.cache.heads;
    c->rows_per_seq = (c->Q.tokens + c->B.batch - 1) / c->B.batch * g;
    if (c->Q.tokens * g >= MAX_ROWS) return fail(DT_ERR_CAPACITY, "q: 2^31 - 2^16 rows per kv head or more");
  }
  return DT_OK;
}

dt_status attention_call(const dt_dtensor* q, const dt_dtensor* cache, const dt_dtensor* page_table,
                         const dt_dtensor* kv_lens, const dt_dtensor* q_starts, const dt_dtensor* out,
                         const dt_dtensor* lse, int D, int G, float scale, int causal, int window, int tp,
                         void* workspace, size_t workspace_bytes, int32_t* d_status, cudaStream_t stream) {
  clear_error();
  Checked c;
  dt_status st = check(q, cache, page_table, kv_lens, q_starts, D, G, tp, false, &c);
  if (st != DT_OK) return st;
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(DT_ERR_INVALID_ARG, "scale must be positive and finite");
  if (window < 0) return fail(DT_ERR_INVALID_ARG, "window %d", window);
  if (window > 0 && !causal) return fail(DT_ERR_INVALID_ARG, "a window needs the causal mask");
  AttnParams p;
  HeadOperand o, ls;
  Layout lo;
  if ((st = head_operand(out, "out", tp, D, true, &o, &lo)) != DT_OK) return st;
  if ((st = same_mesh(lo, c.lq, "out")) != DT_OK) return st;
  if (o.tokens != c.Q.tokens || o.heads != c.Q.heads) return fail(DT_ERR_SHAPE, "out must have the shape of q");
  if (o.dtype != c.Q.dtype) return fail(DT_ERR_INVALID_ARG, "out must have the dtype of q");
  if (!o.vec16) return fail(DT_ERR_ALIGNMENT, "out must have 16-byte aligned rows");
  p.want_lse = lse != nullptr;
  p.lse = o.map;
  if (lse) {
    if ((st = head_operand(lse, "lse", tp, 1, true, &ls, &lo)) != DT_OK) return st;
    if ((st = same_mesh(lo, c.lq, "lse")) != DT_OK) return st;
    if (ls.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "lse must be fp32");
    if (ls.tokens != c.Q.tokens || ls.heads != c.Q.heads) return fail(DT_ERR_SHAPE, "lse must be [tokens, heads]");
    p.lse = ls.map;
  }
  if (c.nothing || c.B.batch == 0) return DT_OK;
  p.q = c.Q.map;
  p.out = o.map;
  p.cache = c.B.cache;
  p.seq = SeqTable{c.B.q_starts, c.B.kv_lens, c.B.batch, c.B.q_len, (int32_t)c.Q.tokens, c.B.capacity};
  p.page_table = c.B.page_table;
  p.table_width = c.B.table_width;
  p.g = c.Q.heads / c.B.cache.heads;
  p.page_mul = c.B.page_mul;
  p.page_shift = c.B.page_shift;
  p.causal = causal != 0;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = hooks().wait_limit_ns;
  p.starve = hooks().starve;
  if ((st = bind_device_of(c.B.kv_lens)) != DT_OK) return st;
  const bool fp32 = c.Q.dtype == DT_FP32;
  Variant v;
  cudaError_t e = variant_any(D, G, fp32, c.rows_per_seq, &v);
  if (e != cudaSuccess) return fail(DT_ERR_CUDA, "kv4_attention: %s", cudaGetErrorString(e));
  if (!workspace || workspace_bytes < v.bytes)
    return fail(DT_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0,
                v.bytes);
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(DT_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  p.split = static_cast<Split*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                    ((size_t)v.grid * sizeof(Split) + 255) / 256 * 256);
  p.status = device_status_word(d_status);
  if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
  p.rb = v.rows;
  e = prompt_kernel(fp32, c.rows_per_seq) ? prompt_launch(p, D, G, v.grid, stream)
      : D == 64 ? launch<64>(p, G, fp32, c.rows_per_seq, v.grid, stream)
              : D == 128 ? launch<128>(p, G, fp32, c.rows_per_seq, v.grid, stream)
                         : launch<256>(p, G, fp32, c.rows_per_seq, v.grid, stream);
  if (e != cudaSuccess) return fail(DT_ERR_CUDA, "kv4_attention launch: %s", cudaGetErrorString(e));
  count_launch();
  count_launch();
  return DT_OK;
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" dt_status dt_tp_kv4_attention(const dt_dtensor* q, const dt_dtensor* cache, const dt_dtensor* page_table,
                                         const dt_dtensor* kv_lens, const dt_dtensor* q_starts, const dt_dtensor* out,
                                         const dt_dtensor* lse, int32_t head_dim, int32_t group, float scale,
                                         int32_t causal, int32_t window, int32_t tp_mesh_dim, void* workspace,
                                         size_t workspace_bytes, int32_t* d_status, dt_stream_t stream) {
  return no_throw([&] {
    return attention_call(q, cache, page_table, kv_lens, q_starts, out, lse, head_dim, group, scale, causal, window,
                          tp_mesh_dim, workspace, workspace_bytes, d_status, reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" dt_status dt_tp_kv4_attention_workspace_size(const dt_dtensor* q, const dt_dtensor* cache,
                                                        const dt_dtensor* page_table, int32_t head_dim, int32_t group,
                                                        int32_t tp_mesh_dim, size_t* bytes) {
  return no_throw([&]() -> dt_status {
    clear_error();
    if (!bytes) return fail(DT_ERR_INVALID_ARG, "bytes is NULL");
    Checked c;
    dt_status st = check(q, cache, page_table, nullptr, nullptr, head_dim, group, tp_mesh_dim, true, &c);
    if (st != DT_OK) return st;
    *bytes = 0;
    if (c.nothing || c.B.batch == 0) return DT_OK;
    Variant v;
    cudaError_t e = variant_any(head_dim, group, c.Q.dtype == DT_FP32, c.rows_per_seq, &v);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(DT_ERR_CUDA, "kv4_attention: %s", cudaGetErrorString(e));
    }
    *bytes = v.bytes;
    return DT_OK;
  });
}
