// Appending keys and values to the paged 4-bit cache, the position rotation
// applied on the way to the keys and to the queries that go with them.
//
// Token i of sequence b's new ones is its key number kv_lens[b] - n_b + i
// (kv_lens counts them already), its position in the rotation table too, and
// goes to page page_table[b, position / page_size].  Per group of G channels
// of a key (after the rotation, in fp32, unrounded) or value:
//   m = bf16(min)    s = bf16((max - min) * (1/15))    inv = 1 / s
//   code = clamp(rint((x - m) * inv), 0, 15)
// Steps below the least normal fp32 number would make inv overflow: such a
// group is held as its minimum (inv = 0).  A group with a value that is not
// finite, or whose range is not, is held as NaN (s = m = NaN, codes 0).
// Each operation rounds on its own (no fused multiply-adds), so the codes
// are a function of these formulas alone.
//
// Bound by memory: q, k and v are read once, q and one record per token and
// kv head written once.
//
// Layout.  D/16 lanes hold a head row, two chunks of 8 channels each: chunk
// l and chunk l + D/16, the partners of a full rotation.  The codes of a
// chunk are one word of the record, and a group's minimum and maximum are a
// few shuffles (a group of 64 is 8 neighbouring lanes' chunk).  A warp takes
// rows of one token: sequence, position and page are looked up once per warp.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <exception>

#include "heads_sm103.cuh"
#include "kv4.h"

namespace dt {
namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_WARPS = AP_THREADS / 32;

struct AppendParams {
  HeadMap k, v, q, q_out, k_st, v_st;  // q*: heads 0 without queries; *_st: per_slot 0 when not wanted
  CacheMap cache;
  SeqTable seq;
  const int32_t* page_table;
  int32_t table_width;
  const float* cos_sin;  // NULL: no rotation
  int64_t table_rows;
  int32_t rotary, interleaved;
  int32_t has_stored;
  int32_t* status;
};

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Turns the lane's two chunks (channels 8 l.. and 8 (l + D/16)..) of row x.
template <class T, int D>
__device__ __forceinline__ void rotate_row(const AppendParams& p, const T* x, const float* cs, int l, float (&a)[8],
                                           float (&b)[8]) {
  constexpr int L = D / 16;
  const int R = p.rotary;
  float c8[8], s8[8];
  if (!p.interleaved && R == D) {  // the partners are this lane's own chunks
    load8_keep(cs + 8 * l, c8);
    load8_keep(cs + R / 2 + 8 * l, s8);
#pragma unroll
    for (int e = 0; e < 8; ++e) rotate_pair(a[e], b[e], c8[e], s8[e]);
    return;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float(&y)[8] = half ? b : a;
    const int c = half ? l + L : l;  // chunk
    if (8 * c >= R) continue;
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 4 * c + e;
        rotate_pair(y[2 * e], y[2 * e + 1], __ldg(cs + i), __ldg(cs + R / 2 + i));
      }
    } else {  // R a multiple of 16: the partner is another chunk of the row
      const int hc = R / 16;
      const bool low = c < hc;
      const int i = 8 * (low ? c : c - hc);
      float z[8];
      load8(x + 8 * (low ? c + hc : c - hc), z);
      load8_keep(cs + i, c8);
      load8_keep(cs + R / 2 + i, s8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (low) rotate_pair(y[e], z[e], c8[e], s8[e]);
        else rotate_pair(z[e], y[e], c8[e], s8[e]);
      }
    }
  }
}

// Codes and parameters of one chunk whose group spans `lanes` neighbouring
// lanes and `both` chunks; y becomes the values as the cache holds them.
__device__ __forceinline__ void quantise(float lo, float hi, float (&y)[8], uint32_t* word, uint32_t* param) {
  float m = __bfloat162float(__float2bfloat16_rn(lo));
  float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 0.06666667014360428f)));
  float inv = s >= 1.1754943508222875e-38f ? __fdiv_rn(1.f, s) : 0.f;
  if (!isfinite(m) || !isfinite(s)) m = s = __int_as_float(0x7fc00000), inv = 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(y[e], m), inv)), 0.f), 15.f);  // NaN -> 0
    w |= static_cast<uint32_t>(c) << (4 * e);
    y[e] = __fadd_rn(__fmul_rn(c, s), m);
  }
  *word = w;
  *param = (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xffff0000u);
}

template <class T, int D, int G>
__global__ void __launch_bounds__(AP_THREADS) kv4_append_kernel(const __grid_constant__ AppendParams p, int units) {
  constexpr int L = D / 16, SG = 32 / L, W = kv4_words(D, G), NG = D / G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / L, l = lane % L;
  const int rows = p.q.heads + 2 * p.cache.heads;  // q heads, key heads, value heads
  const int64_t total = (int64_t)p.seq.tokens * units;
  for (int64_t w = (int64_t)blockIdx.x * AP_WARPS + warp; w < total; w += (int64_t)gridDim.x * AP_WARPS) {
    const int t = (int)(w / units);
    const int row = (int)(w - (int64_t)t * units) * SG + sub;
    const int hk = p.cache.heads, hq = p.q.heads;
    const int kind = row < hq ? 0 : row < hq + hk ? 1 : row < rows ? 2 : 3;
    const int h = kind == 0 ? row : kind == 1 ? row - hq : row - hq - hk;
    // the row's loads go out before its token is looked up
    const T* x = nullptr;
    float a[8], b[8];
    if (kind < 3) {
      x = kind == 0 ? head_ptr<T>(p.q, t, h, D) : kind == 1 ? head_ptr<T>(p.k, t, h, D) : head_ptr<T>(p.v, t, h, D);
      load8(x + 8 * l, a);
      load8(x + 8 * (l + L), b);
    }
    const int sq = warp_seq_of_token(p.seq, t, lane);
    if (sq < 0) continue;  // a row of no sequence: nothing is written for it
    const int s0 = p.seq.start(sq);
    const int pos = p.seq.keys(sq) - (p.seq.start(sq + 1) - s0) + (t - s0);
    const bool in_table = !p.cos_sin || (pos >= 0 && pos < p.table_rows);
    const int32_t page = pos >= 0 && pos < p.seq.capacity ? __ldg(p.page_table + (int64_t)sq * p.table_width + pos / p.cache.page_size) : -1;
    const bool in_cache = page >= 0 && page < p.cache.pages;
    if (lane == 0 && (!in_table || !in_cache || __ldg(p.seq.kv_lens + sq) != p.seq.keys(sq)))
      atomicOr(p.status, DT_DEV_ERR_INDEX);
    if (kind < 2 && p.cos_sin && in_table) rotate_row<T, D>(p, x, p.cos_sin + (int64_t)pos * p.rotary, l, a, b);
    if (!in_table) {
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = b[e] = 0.f;
    }
    if (kind == 0) {
      T* y = head_ptr<T>(p.q_out, t, h, D);
      store8(y + 8 * l, a);
      store8(y + 8 * (l + L), b);
    }
    // every lane takes part in the shuffles below
    float la = INFINITY, ha = -INFINITY, lb = INFINITY, hb = -INFINITY;
    if (kind == 1 || kind == 2) {
      la = ha = a[0], lb = hb = b[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        la = min_nan(la, a[e]), ha = max_nan(ha, a[e]);
        lb = min_nan(lb, b[e]), hb = max_nan(hb, b[e]);
      }
    }
    if constexpr (D == 64 && G == 64) {  // both chunks are in the one group
      la = lb = min_nan(la, lb);
      ha = hb = max_nan(ha, hb);
    }
    constexpr int SPAN = (D == 64 && G == 64) ? L : (G / 8 < L ? G / 8 : L);  // lanes of a group
#pragma unroll
    for (int o = SPAN >> 1; o; o >>= 1) {
      la = min_nan(la, __shfl_xor_sync(0xffffffffu, la, o)), ha = max_nan(ha, __shfl_xor_sync(0xffffffffu, ha, o));
      lb = min_nan(lb, __shfl_xor_sync(0xffffffffu, lb, o)), hb = max_nan(hb, __shfl_xor_sync(0xffffffffu, hb, o));
    }
    if (kind != 1 && kind != 2) continue;
    uint32_t wa, wb, pa, pb;
    quantise(la, ha, a, &wa, &pa);
    quantise(lb, hb, b, &wb, &pb);
    if (p.has_stored) {
      T* y = kind == 1 ? head_ptr<T>(p.k_st, t, h, D) : head_ptr<T>(p.v_st, t, h, D);
      store8(y + 8 * l, a);
      store8(y + 8 * (l + L), b);
    }
    if (!in_cache || !in_table) continue;
    uint32_t* rec = reinterpret_cast<uint32_t*>(cache_page(p.cache, page, h)) +
                    (int64_t)(pos % p.cache.page_size) * W;
    uint32_t* codes = rec + (kind == 2 ? D / 8 : 0);
    uint32_t* params = rec + D / 4 + (kind == 2 ? NG : 0);
    codes[l] = wa;
    codes[l + L] = wb;
    if (8 * l % G == 0) params[8 * l / G] = pa;
    if (8 * (l + L) % G == 0) params[8 * (l + L) / G] = pb;
    if (kind == 2 && l < W - D / 4 - 2 * NG) rec[D / 4 + 2 * NG + l] = 0;  // padding
  }
}

template <class T>
void launch_append(const AppendParams& p, int D, int G, cudaStream_t s) {
  const int SG = 32 / (D / 16);
  const int units = (p.q.heads + 2 * p.cache.heads + SG - 1) / SG;
  const int64_t warps = (int64_t)p.seq.tokens * units;
  const int grid = (int)std::min<int64_t>((warps + AP_WARPS - 1) / AP_WARPS, (int64_t)device_sm_count() * 32);
#define DT_AP(d, g) \
  if (D == d && G == g) kv4_append_kernel<T, d, g><<<grid, AP_THREADS, 0, s>>>(p, units)
  DT_AP(64, 32);
  DT_AP(64, 64);
  DT_AP(128, 32);
  DT_AP(128, 64);
  DT_AP(256, 32);
  DT_AP(256, 64);
#undef DT_AP
}

dt_status append_call(const dt_dtensor* k, const dt_dtensor* v, const dt_dtensor* cache, const dt_dtensor* page_table,
                      const dt_dtensor* kv_lens, const dt_dtensor* q_starts, const dt_dtensor* cos_sin,
                      const dt_dtensor* q, const dt_dtensor* q_out, const dt_dtensor* k_stored,
                      const dt_dtensor* v_stored, int D, int G, int interleaved, int tp, int32_t* d_status,
                      cudaStream_t stream) {
  clear_error();
  if (!kv4_format_ok(D, G))
    return fail(DT_ERR_UNSUPPORTED, "head_dim %d in groups of %d (64, 128, 256 in groups of 32 or 64)", D, G);
  if ((q == nullptr) != (q_out == nullptr)) return fail(DT_ERR_INVALID_ARG, "q and q_out go together");
  if ((k_stored == nullptr) != (v_stored == nullptr))
    return fail(DT_ERR_INVALID_ARG, "k_stored and v_stored go together");
  AppendParams p;
  HeadOperand K;
  Layout lk;
  dt_status st = head_operand(k, "k", tp, D, false, &K, &lk);
  if (st != DT_OK) return st;
  struct {
    const dt_dtensor* d;
    const char* name;
    HeadMap* map;
    bool output;
  } rest[] = {{v, "v", &p.v, false},          {q, "q", &p.q, false},           {q_out, "q_out", &p.q_out, true},
              {k_stored, "k_stored", &p.k_st, true}, {v_stored, "v_stored", &p.v_st, true}};
  bool vec = K.vec16;
  int heads_q = 0;
  for (auto& r : rest) {
    r.map->heads = 0;
    r.map->per_slot = 1;
    r.map->mul = 1u << 31;
    if (!r.d && r.map != &p.v) continue;
    HeadOperand o;
    Layout lo;
    if ((st = head_operand(r.d, r.name, tp, D, r.output, &o, &lo)) != DT_OK) return st;
    if ((st = same_mesh(lo, lk, r.name)) != DT_OK) return st;
    if (o.tokens != K.tokens) return fail(DT_ERR_SHAPE, "%s and k have different token counts", r.name);
    if (o.dtype != K.dtype) return fail(DT_ERR_INVALID_ARG, "%s must have the dtype of k", r.name);
    if (r.map == &p.q) heads_q = o.heads;
    const int want = r.map == &p.q ? o.heads : r.map == &p.q_out ? heads_q : K.heads;
    if (o.heads != want) return fail(DT_ERR_SHAPE, "%s has %d heads, %d expected", r.name, o.heads, want);
    vec = vec && o.vec16;
    *r.map = o.map;
  }
  p.k = K.map;
  Kv4Batch B;
  if ((st = kv4_batch(cache, page_table, kv_lens, q_starts, tp, D, G, K.tokens, lk, false, &B)) != DT_OK) return st;
  if (B.cache.heads != K.heads) return fail(DT_ERR_SHAPE, "cache has %d heads, k has %d", B.cache.heads, K.heads);
  p.cos_sin = nullptr;
  p.table_rows = 0;
  p.rotary = 0;
  if (cos_sin) {
    PlainOperand t;
    if ((st = plain_operand(cos_sin, "cos_sin", lk, false, &t)) != DT_OK) return st;
    if (t.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "cos_sin must be fp32");
    if (t.ndim != 2 || t.shape[1] < 16 || t.shape[1] % 16 || t.shape[1] > D)
      return fail(DT_ERR_SHAPE, "cos_sin must be [rows, rotary], rotary a multiple of 16 and at most head_dim");
    if (reinterpret_cast<uintptr_t>(t.ptr) % 16) return fail(DT_ERR_ALIGNMENT, "cos_sin must be 16-byte aligned");
    p.cos_sin = reinterpret_cast<const float*>(t.ptr);
    p.table_rows = t.shape[0];
    p.rotary = (int)t.shape[1];
  }
  if (!vec) return fail(DT_ERR_ALIGNMENT, "k, v, q and the outputs must have 16-byte aligned rows");
  if (K.tokens == 0 || (K.heads == 0 && heads_q == 0) || B.batch == 0) return DT_OK;
  if (B.table_width == 0) return fail(DT_ERR_SHAPE, "page_table has no columns");
  p.cache = B.cache;
  p.page_table = B.page_table;
  p.table_width = B.table_width;
  p.seq = SeqTable{B.q_starts, B.kv_lens, B.batch, B.q_len, (int32_t)K.tokens, B.capacity};
  p.interleaved = interleaved != 0;
  p.has_stored = k_stored != nullptr;
  if ((st = bind_device_of(B.kv_lens)) != DT_OK) return st;
  p.status = device_status_word(d_status);
  if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
  if (K.dtype == DT_BF16) launch_append<__nv_bfloat16>(p, D, G, stream);
  else launch_append<float>(p, D, G, stream);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(DT_ERR_CUDA, "kv4_append launch: %s", cudaGetErrorString(e));
  count_launch();
  return DT_OK;
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" dt_status dt_tp_kv4_append(const dt_dtensor* k, const dt_dtensor* v, const dt_dtensor* cache,
                                      const dt_dtensor* page_table, const dt_dtensor* kv_lens,
                                      const dt_dtensor* q_starts, const dt_dtensor* cos_sin, const dt_dtensor* q,
                                      const dt_dtensor* q_out, const dt_dtensor* k_stored, const dt_dtensor* v_stored,
                                      int32_t head_dim, int32_t group, int32_t interleaved, int32_t tp_mesh_dim,
                                      int32_t* d_status, dt_stream_t stream) {
  return no_throw([&] {
    return append_call(k, v, cache, page_table, kv_lens, q_starts, cos_sin, q, q_out, k_stored, v_stored, head_dim,
                       group, interleaved, tp_mesh_dim, d_status, reinterpret_cast<cudaStream_t>(stream));
  });
}
