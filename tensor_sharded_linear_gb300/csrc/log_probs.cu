// Log probabilities of given tokens over a vocabulary that is sharded on tp,
// with the entropy and the most likely alternatives, and their gradient.
//
// Per token, z = scale * logits (V of them, all arithmetic fp32):
//   M = max z      S = sum exp(z - M)      lse = M + ln S
//   logp(id) = (z_id - M) - ln S           H = ln S - (sum (z - M) exp(z - M)) / S
//   top: the k largest logits, ties to the lowest id, with their logp
// and for gradients g_c of logp(id_c) and e of H, with p = exp(z - lse):
//   dlogit_j = scale (sum over c with id_c = j of g_c  -  p_j (sum_c g_c)  -  e p_j (z_j - lse + H))
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "heads_sm103.cuh"
#include "row_operands.h"

namespace dt {
namespace {

constexpr int LP_MAX_TOP = 32;
constexpr int LP_MAX_GIVEN = 64;

// Columns [begin, begin of the next shard) of every token.
struct VocabShard {
  char* ptr;
  int64_t ld;  // elements between tokens
  int64_t begin;
};

struct LogProbArgs {
  VocabShard z[DT_MAX_SLOTS], dz[DT_MAX_SLOTS];
  int32_t shards, dz_shards;
  int64_t tokens, vocab;
  const int32_t* ids;  // [tokens, given]; NULL: none
  int32_t given, ignore, top;
  float scale;
  float *logp, *lse, *entropy, *top_logp;  // backward: lse and entropy are read
  int32_t* top_ids;
  const float *dlogp, *dentropy;
  int32_t* status;
};

// Bits whose order as unsigned numbers is that of the values; -0 equals +0, NaN is above all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FFFFFFFu);
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr int LP_THREADS = 256;

template <class F>
__device__ __forceinline__ void cta_reduce(uint64_t* buf, uint64_t& v, F&& join) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int o = 16; o; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < LP_THREADS / 32; ++w) v = join(v, buf[w]);
}

template <class T>
__device__ __forceinline__ float logit(const LogProbArgs& p, int64_t t, int64_t j) {
  int s = 0;
  while (s + 1 < p.shards && p.z[s + 1].begin <= j) ++s;
  return to_f32(reinterpret_cast<const T*>(p.z[s].ptr)[t * p.z[s].ld + (j - p.z[s].begin)]);
}

// The id at place i: its column, or -1 (and the status bit unless it is the one to be ignored).
__device__ __forceinline__ int64_t given_id(const LogProbArgs& p, int64_t i, bool report) {
  const int32_t id = load_plain(p.ids + i);
  if (id >= 0 && id < p.vocab) return id;
  if (report && id != p.ignore) atomicOr(p.status, DT_DEV_ERR_INDEX);
  return -1;
}

template <class T>
__global__ void __launch_bounds__(LP_THREADS) log_probs_kernel(const __grid_constant__ LogProbArgs p) {
  __shared__ uint64_t buf[LP_THREADS / 32];
  wait_for_previous_kernel();
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    float m = -INFINITY, s = 0.f, e = 0.f;
    auto each = [&](auto&& body) {
      for (int k = 0; k < p.shards; ++k) {
        const T* z = reinterpret_cast<const T*>(p.z[k].ptr) + t * p.z[k].ld;
        const int64_t n = (k + 1 < p.shards ? p.z[k + 1].begin : p.vocab) - p.z[k].begin;
        for (int64_t j = threadIdx.x; j < n; j += LP_THREADS) body(to_f32(z[j]), p.z[k].begin + j);
      }
    };
    each([&](float z, int64_t) { m = max_nan(m, z); });
    uint64_t v = __float_as_uint(m);
    cta_reduce(buf, v, [](uint64_t a, uint64_t b) {
      return (uint64_t)__float_as_uint(max_nan(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)b)));
    });
    m = __uint_as_float((uint32_t)v);
    const bool none = m == -INFINITY;  // no token is possible
    each([&](float z, int64_t) {
      const float d = none ? -INFINITY : (z - m) * p.scale, x = __expf(d);
      s += x;
      e += x * fmaxf(d, -1e30f);
    });
    auto add = [](uint64_t a, uint64_t b) {
      return (uint64_t)__float_as_uint(__uint_as_float((uint32_t)a) + __uint_as_float((uint32_t)b));
    };
    v = __float_as_uint(s);
    cta_reduce(buf, v, add);
    s = __uint_as_float((uint32_t)v);
    v = __float_as_uint(e);
    cta_reduce(buf, v, add);
    e = __uint_as_float((uint32_t)v);
    const float ln = logf(s);
    auto logp = [&](float z) { return none ? -INFINITY : (z - m) * p.scale - ln; };
    if (threadIdx.x == 0) {
      if (p.lse) p.lse[t] = none ? -INFINITY : m * p.scale + ln;
      if (p.entropy) p.entropy[t] = none ? 0.f : ln - e / s;
    }
    for (int c = threadIdx.x; c < p.given; c += LP_THREADS) {
      const int64_t id = given_id(p, t * p.given + c, true);
      p.logp[t * p.given + c] = id >= 0 ? logp(logit<T>(p, t, id)) : 0.f;
    }
    uint64_t last = ~0ull;
    for (int k = 0; k < p.top; ++k) {
      uint64_t best = 0;
      each([&](float z, int64_t j) {
        const uint64_t x = (uint64_t)order_key(z) << 32 | (0xFFFFFFFFu - (uint32_t)j);
        if (x < last && x > best) best = x;
      });
      cta_reduce(buf, best, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
      last = best;
      if (threadIdx.x == 0) {
        p.top_logp[t * p.top + k] = logp(key_value((uint32_t)(best >> 32)));
        p.top_ids[t * p.top + k] = (int32_t)(0xFFFFFFFFu - (uint32_t)best);
      }
    }
  }
}

template <class T>
__global__ void __launch_bounds__(LP_THREADS) log_probs_backward_kernel(const __grid_constant__ LogProbArgs p) {
  wait_for_previous_kernel();
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    float g = 0.f;
    for (int c = 0; c < p.given; ++c) {
      const int64_t id = given_id(p, t * p.given + c, threadIdx.x == 0);
      if (id >= 0) g += load_plain(p.dlogp + t * p.given + c);
    }
    const float lse = load_plain(p.lse + t), ge = p.dentropy ? load_plain(p.dentropy + t) : 0.f;
    const float h = p.dentropy ? load_plain(p.entropy + t) : 0.f;
    const bool none = lse == -INFINITY;
    for (int k = 0; k < p.shards; ++k) {
      const T* z = reinterpret_cast<const T*>(p.z[k].ptr) + t * p.z[k].ld;
      T* dz = reinterpret_cast<T*>(p.dz[k].ptr) + t * p.dz[k].ld;
      const int64_t n = (k + 1 < p.shards ? p.z[k + 1].begin : p.vocab) - p.z[k].begin;
      for (int64_t j = threadIdx.x; j < n; j += LP_THREADS) {
        const float l = to_f32(z[j]) * p.scale - lse, q = __expf(l);
        float d = -q * g - ge * q * (fmaxf(l, -1e30f) + h);
        for (int c = 0; c < p.given; ++c)
          if (load_plain(p.ids + t * p.given + c) == p.z[k].begin + j) d += load_plain(p.dlogp + t * p.given + c);
        from_f32(dz + j, none || (g == 0.f && ge == 0.f && p.given <= 1) ? 0.f : d * p.scale);
      }
    }
  }
}

// ---------------------------------------------------------------- host

// Check `in` as [..., V] logits, Shard(-1) or Replicate on tp and Replicate
// on the other mesh dims, and fill the shards in order (empty ones left out).
dt_status vocab_operand(const dt_dtensor* in, const char* what, int tp, bool output, VocabShard* out, int32_t* shards,
                        Layout* layout) {
  DTensor X;
  dt_status st = parse_dtensor(in, &X, what);
  if (st != DT_OK) return st;
  const Layout& L = X.layout;
  *layout = L;
  if (L.ndim < 2) return fail(DT_ERR_SHAPE, "%s must be [..., vocabulary]", what);
  if (tp >= L.mesh_ndim) return fail(DT_ERR_INVALID_ARG, "tp_mesh_dim %d", tp);
  if (L.dtype != DT_BF16 && L.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "%s must be bf16 or fp32", what);
  const int last = L.ndim - 1;
  const bool sharded = tp >= 0 && L.is_shard(tp, last);
  for (int m = 0; m < L.mesh_ndim; ++m)
    if (!(m == tp && sharded) && !L.is_replicate(m))
      return fail(DT_ERR_PLACEMENT, "%s must be Shard(-1) or Replicate on tp and Replicate on other mesh dims", what);
  const int parts = sharded ? L.mesh[tp] : 1;
  if (output && L.nslots > parts) return fail(DT_ERR_UNSUPPORTED, "%s: an output with materialised replicas", what);
  int64_t tokens = 1;
  for (int d = 0; d < last; ++d) tokens *= L.gshape[d];
  if (tokens >= MAX_ROWS) return fail(DT_ERR_CAPACITY, "%s: 2^31 - 2^16 tokens or more", what);
  if (L.gshape[last] >= MAX_ROWS) return fail(DT_ERR_CAPACITY, "%s: a vocabulary of 2^31 - 2^16 or more", what);
  *shards = 0;
  for (int j = 0; j < parts; ++j) {
    int c[DT_MAX_MESH_DIMS] = {0, 0, 0, 0};
    if (sharded) c[tp] = j;
    const SlotView& v = X.slots[L.slot_of_coords(c)];
    if (v.numel == 0) continue;
    if (v.shape[last] > 1 && v.stride[last] != 1) return fail(DT_ERR_UNSUPPORTED, "%s must have unit inner stride", what);
    int64_t ld = 0, span = 0;
    bool have = false;
    for (int d = last - 1; d >= 0; --d) {
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
    if (output && tokens > 1 && ld < v.shape[last]) return fail(DT_ERR_UNSUPPORTED, "%s: rows of an output overlap", what);
    out[(*shards)++] = VocabShard{v.ptr, ld, v.goff[last]};
  }
  return DT_OK;
}

// A Replicate, contiguous tensor beside the logits: [...] or [..., inner].
dt_status beside(const dt_dtensor* in, const char* what, const Layout& of, int dtype, bool output, bool has_inner,
                 int64_t* inner, const void** ptr) {
  PlainOperand o;
  dt_status st = plain_operand(in, what, of, output, &o);
  if (st != DT_OK) return st;
  if (o.dtype != dtype) return fail(DT_ERR_INVALID_ARG, "%s must be %s", what, dtype == DT_INT32 ? "int32" : "fp32");
  const int lead = of.ndim - 1;
  bool shape = o.ndim == lead || (has_inner && o.ndim == lead + 1);
  for (int d = 0; shape && d < lead; ++d) shape = o.shape[d] == of.gshape[d];
  const int64_t n = shape && o.ndim == lead + 1 ? o.shape[lead] : 1;
  if (shape && *inner >= 0) shape = n == *inner;
  if (!shape) return fail(DT_ERR_SHAPE, "%s must have the leading dims of logits%s", what, has_inner ? " (and ids)" : "");
  *inner = n;
  *ptr = o.ptr;
  return DT_OK;
}

dt_status common_checks(const LogProbArgs& p, const Layout& l) {
  if (!(p.scale > 0.f) || !std::isfinite(p.scale)) return fail(DT_ERR_INVALID_ARG, "scale must be positive and finite");
  if (p.given > LP_MAX_GIVEN) return fail(DT_ERR_CAPACITY, "%d ids per token (at most %d)", p.given, LP_MAX_GIVEN);
  if (p.tokens > 0 && p.vocab == 0) return fail(DT_ERR_SHAPE, "logits of an empty vocabulary");
  (void)l;
  return DT_OK;
}

template <class K, class P>
cudaError_t launch_rows(K kernel, const P& p, cudaStream_t s) {
  const int grid = (int)std::min<int64_t>(p.tokens, (int64_t)device_sm_count() * 8);
  return launch_early(kernel, dim3(grid), LP_THREADS, 0, s, p);
}

void sizes(const Layout& l, LogProbArgs* p) {
  p->tokens = 1;
  for (int d = 0; d + 1 < l.ndim; ++d) p->tokens *= l.gshape[d];
  p->vocab = l.gshape[l.ndim - 1];
}

template <class T>
T* writable(const void* p) {
  return static_cast<T*>(const_cast<void*>(p));
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" dt_status dt_tp_log_probs(const dt_dtensor* logits, const dt_dtensor* ids, const dt_dtensor* logprobs,
                                     const dt_dtensor* lse, const dt_dtensor* entropy, const dt_dtensor* top_logprobs,
                                     const dt_dtensor* top_ids, float scale, int32_t ignore_index, int32_t tp_mesh_dim,
                                     int32_t* d_status, dt_stream_t stream) {
  return no_throw([&]() -> dt_status {
    clear_error();
    LogProbArgs p{};
    Layout lz;
    dt_status st;
    if (!logits) return fail(DT_ERR_INVALID_ARG, "logits is NULL");
    if ((st = vocab_operand(logits, "logits", tp_mesh_dim, false, p.z, &p.shards, &lz)) != DT_OK) return st;
    sizes(lz, &p);
    p.scale = scale;
    p.ignore = ignore_index;
    if ((ids != nullptr) != (logprobs != nullptr)) return fail(DT_ERR_INVALID_ARG, "ids and logprobs go together");
    if ((top_logprobs != nullptr) != (top_ids != nullptr))
      return fail(DT_ERR_INVALID_ARG, "top_logprobs and top_ids go together");
    if (!logprobs && !lse && !entropy && !top_ids) return fail(DT_ERR_INVALID_ARG, "no output");
    const void* ptr = nullptr;
    const void* anchor = nullptr;
    if (ids) {
      int64_t given = -1;
      if ((st = beside(ids, "ids", lz, DT_INT32, false, true, &given, &ptr)) != DT_OK) return st;
      p.ids = static_cast<const int32_t*>(ptr);
      if ((st = beside(logprobs, "logprobs", lz, DT_FP32, true, true, &given, &ptr)) != DT_OK) return st;
      p.logp = writable<float>(ptr);
      p.given = (int32_t)std::min<int64_t>(given, LP_MAX_GIVEN + 1);
      if (given > 0) anchor = ptr;
    }
    int64_t one = 1;
    if (lse) {
      if ((st = beside(lse, "lse", lz, DT_FP32, true, false, &one, &ptr)) != DT_OK) return st;
      anchor = p.lse = writable<float>(ptr);
    }
    if (entropy) {
      if ((st = beside(entropy, "entropy", lz, DT_FP32, true, false, &one, &ptr)) != DT_OK) return st;
      anchor = p.entropy = writable<float>(ptr);
    }
    if (top_ids) {
      int64_t k = -1;
      if ((st = beside(top_ids, "top_ids", lz, DT_INT32, true, true, &k, &ptr)) != DT_OK) return st;
      p.top_ids = writable<int32_t>(ptr);
      if ((st = beside(top_logprobs, "top_logprobs", lz, DT_FP32, true, true, &k, &ptr)) != DT_OK) return st;
      p.top_logp = writable<float>(ptr);
      if (k > LP_MAX_TOP) return fail(DT_ERR_CAPACITY, "%lld alternatives (at most %d)", (long long)k, LP_MAX_TOP);
      if (p.tokens > 0 && k > p.vocab) return fail(DT_ERR_SHAPE, "more alternatives than tokens in the vocabulary");
      p.top = (int32_t)k;
      if (k > 0) anchor = ptr;
    }
    if ((st = common_checks(p, lz)) != DT_OK) return st;
    if (p.tokens == 0 || !anchor) return DT_OK;
    if ((st = bind_device_of(anchor)) != DT_OK) return st;
    p.status = device_status_word(d_status);
    if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = lz.dtype == DT_BF16 ? launch_rows(log_probs_kernel<__nv_bfloat16>, p, s)
                                              : launch_rows(log_probs_kernel<float>, p, s);
    if (e != cudaSuccess) return fail(DT_ERR_CUDA, "log_probs launch: %s", cudaGetErrorString(e));
    count_launch();
    return DT_OK;
  });
}

extern "C" dt_status dt_tp_log_probs_backward(const dt_dtensor* dlogprobs, const dt_dtensor* dentropy,
                                              const dt_dtensor* logits, const dt_dtensor* ids, const dt_dtensor* lse,
                                              const dt_dtensor* entropy, const dt_dtensor* dlogits, float scale,
                                              int32_t ignore_index, int32_t tp_mesh_dim, int32_t* d_status,
                                              dt_stream_t stream) {
  return no_throw([&]() -> dt_status {
    clear_error();
    LogProbArgs p{};
    Layout lz, ld;
    dt_status st;
    if (!logits || !dlogits) return fail(DT_ERR_INVALID_ARG, "logits or dlogits is NULL");
    if (!lse) return fail(DT_ERR_INVALID_ARG, "lse is NULL");
    if ((ids != nullptr) != (dlogprobs != nullptr)) return fail(DT_ERR_INVALID_ARG, "ids and dlogprobs go together");
    if (!dlogprobs && !dentropy) return fail(DT_ERR_INVALID_ARG, "neither dlogprobs nor dentropy");
    if (dentropy && !entropy) return fail(DT_ERR_INVALID_ARG, "dentropy needs entropy");
    if ((st = vocab_operand(logits, "logits", tp_mesh_dim, false, p.z, &p.shards, &lz)) != DT_OK) return st;
    if ((st = vocab_operand(dlogits, "dlogits", tp_mesh_dim, true, p.dz, &p.dz_shards, &ld)) != DT_OK) return st;
    if ((st = same_mesh(ld, lz, "dlogits")) != DT_OK) return st;
    bool same = ld.ndim == lz.ndim;
    for (int d = 0; same && d < lz.ndim; ++d) same = ld.gshape[d] == lz.gshape[d];
    if (!same) return fail(DT_ERR_SHAPE, "dlogits must have the shape of logits");
    if (ld.dtype != lz.dtype) return fail(DT_ERR_INVALID_ARG, "dlogits must have the dtype of logits");
    if (p.shards != p.dz_shards) return fail(DT_ERR_PLACEMENT, "dlogits must be placed as logits");
    sizes(lz, &p);
    p.scale = scale;
    p.ignore = ignore_index;
    const void* ptr = nullptr;
    if (ids) {
      int64_t given = -1;
      if ((st = beside(ids, "ids", lz, DT_INT32, false, true, &given, &ptr)) != DT_OK) return st;
      p.ids = static_cast<const int32_t*>(ptr);
      if ((st = beside(dlogprobs, "dlogprobs", lz, DT_FP32, false, true, &given, &ptr)) != DT_OK) return st;
      p.dlogp = static_cast<const float*>(ptr);
      p.given = (int32_t)std::min<int64_t>(given, LP_MAX_GIVEN + 1);
    }
    int64_t one = 1;
    if ((st = beside(lse, "lse", lz, DT_FP32, false, false, &one, &ptr)) != DT_OK) return st;
    p.lse = writable<float>(ptr);
    if (dentropy) {
      if ((st = beside(entropy, "entropy", lz, DT_FP32, false, false, &one, &ptr)) != DT_OK) return st;
      p.entropy = writable<float>(ptr);
      if ((st = beside(dentropy, "dentropy", lz, DT_FP32, false, false, &one, &ptr)) != DT_OK) return st;
      p.dentropy = static_cast<const float*>(ptr);
    }
    if ((st = common_checks(p, lz)) != DT_OK) return st;
    if (p.tokens == 0) return DT_OK;
    if ((st = bind_device_of(p.dz[0].ptr)) != DT_OK) return st;
    p.status = device_status_word(d_status);
    if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = lz.dtype == DT_BF16 ? launch_rows(log_probs_backward_kernel<__nv_bfloat16>, p, s)
                                              : launch_rows(log_probs_backward_kernel<float>, p, s);
    if (e != cudaSuccess) return fail(DT_ERR_CUDA, "log_probs_backward launch: %s", cudaGetErrorString(e));
    count_launch();
    return DT_OK;
  });
}
