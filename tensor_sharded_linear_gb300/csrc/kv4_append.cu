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
// Memory's floor: q, k and v are read once, q and one record per token and kv
// head written once.  Bound: the instructions of the exact quantisation and
// their latency.  Prompts of 9150 tokens together, 32/8 heads of 128 in bf16,
// the stored values returned too: 47.4 us for 240 MB, 5.1 TB/s, 0.75 of a
// copy's rate (with the next row's loads in registers, one block ahead, 54.9;
// with 4 and 5 CTAs an SM 49.3 and 48.3); a decode step of 32 tokens 2.7 us, a
// launch.
//
// Layout.  D/16 lanes hold a head row, two chunks of 8 channels each: chunk
// l and chunk l + D/16, the partners of a full rotation.  The codes of a
// chunk are one word of the record, and a group's minimum and maximum are a
// few shuffles (a group of 64 is 8 neighbouring lanes' chunk).  A block is
// the rows of one kind (q, k or v) that a warp holds at a time; a warp takes
// `inner` blocks of one token, so its sequence, position, page and angles
// are looked up once for them.  Rows come through a ring of asynchronous
// copies, each lane its own chunks, three blocks ahead.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <exception>

#include "heads_sm103.cuh"
#include "kv4.h"

namespace dt {
namespace {

constexpr int AP_THREADS = 128;
constexpr int AP_CTAS = 6;  // per SM
constexpr int AP_WARPS = AP_THREADS / 32;
constexpr int AP_STAGES = 4;

struct AppendParams {
  HeadMap k, v, q, q_out, k_st, v_st;  // q*: heads 0 without queries; *_st: per_slot 0 when not wanted
  CacheMap cache;
  SeqTable seq;
  const int32_t* page_table;
  int32_t table_width;
  uint32_t page_mul, page_shift;  // division by the page size (Kv4Batch)
  const float* cos_sin;  // NULL: no rotation
  int64_t table_rows;
  int32_t rotary, interleaved;
  int32_t has_stored;
  int32_t inner;  // blocks of a warp's unit
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
        rotate_pair(y[2 * e], y[2 * e + 1], load_plain(cs + i), load_plain(cs + R / 2 + i));
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

// Codes and parameters of one chunk of a group with minimum lo and maximum
// hi; y becomes the values as the cache holds them.  A number in [0, 15] is
// rounded to nearest even by adding 1.5 * 2^23, whose sum has it in its low
// bits.
__device__ __forceinline__ void quantise(float lo, float hi, float (&y)[8], uint32_t* word, uint32_t* param) {
  float m = __bfloat162float(__float2bfloat16_rn(lo));
  float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 0.06666667014360428f)));
  float inv = s >= 1.1754943508222875e-38f ? __fdiv_rn(1.f, s) : 0.f;
  if (!isfinite(m) || !isfinite(s)) m = s = __int_as_float(0x7fc00000), inv = 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = fminf(fmaxf(__fmul_rn(__fsub_rn(y[e], m), inv), 0.f), 15.f);  // NaN -> 0
    const float c = __fadd_rn(x, 12582912.f);
    w |= (__float_as_uint(c) & 15u) << (4 * e);
    y[e] = __fadd_rn(__fmul_rn(__fsub_rn(c, 12582912.f), s), m);
  }
  *word = w;
  *param = (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xffff0000u);
}

template <class T, int D, int G>
__global__ void __launch_bounds__(AP_THREADS, AP_CTAS) kv4_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int L = D / 16, SG = 32 / L, W = kv4_words(D, G), NG = D / G;
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / L, l = lane % L;
  const int hk = p.cache.heads, hq = p.q.heads;
  const int nq = (hq + SG - 1) / SG, nk = (hk + SG - 1) / SG;  // blocks of q, of k and of v
  const int blocks = nq + 2 * nk;
  const int per_tok = (blocks + p.inner - 1) / p.inner;  // units of a token
  const int step = gridDim.x * AP_WARPS;
  const int step_tok = step / per_tok, step_blk = step - step_tok * per_tok;
  const bool full_rot = p.cos_sin && !p.interleaved && p.rotary == D;

  // block n: its kind (0 q, 1 k, 2 v) and this lane's head, the last one again where there is none
  auto kind_of = [&](int n) { return n < nq ? 0 : n < nq + nk ? 1 : 2; };
  auto head_of = [&](int n, int kind) { return (n - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * SG + sub; };
  auto row_of = [&](int64_t t, int n) {
    const int kind = kind_of(n), h = head_of(n, kind);
    return kind == 0 ? head_ptr<T>(p.q, t, min(h, hq - 1), D)
                     : head_ptr<T>(kind == 1 ? p.k : p.v, t, min(h, hk - 1), D);
  };

  const int u0 = blockIdx.x * AP_WARPS + warp;
  int t = u0 / per_tok, unit = u0 - t * per_tok;
  // rows come through a ring of asynchronous copies, each lane its own two
  // chunks; (ft, funit, fn) is the block to be fetched next
  constexpr int PIECES = 8 * sizeof(T) / 16, E = 16 / sizeof(T);  // 16-byte pieces of a chunk, elements of a piece
  __shared__ uint4 ring_smem[AP_STAGES * 2 * PIECES * AP_THREADS];
  uint4* ring = ring_smem + threadIdx.x;
  int ft = t, funit = unit, fn = unit * p.inner, fput = 0, fget = 0;
  auto fetch = [&]() {
    if (ft < p.seq.tokens) {
      const T* x = row_of(ft, fn);
      uint4* to = ring + fput * (2 * PIECES * AP_THREADS);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        copy16_async(to + i * AP_THREADS, x + 8 * l + i * E);
        copy16_async(to + (PIECES + i) * AP_THREADS, x + 8 * (l + L) + i * E);
      }
      if (++fn == min((funit + 1) * p.inner, blocks)) {
        ft += step_tok, funit += step_blk;
        if (funit >= per_tok) funit -= per_tok, ++ft;
        fn = funit * p.inner;
      }
    }
    copies_commit();
    if (++fput == AP_STAGES) fput = 0;
  };
  for (int i = 0; i + 1 < AP_STAGES; ++i) fetch();
  while (t < p.seq.tokens) {
    int tn = t + step_tok, un = unit + step_blk;
    if (un >= per_tok) un -= per_tok, ++tn;
    // the token's sequence, position, page and angles
    const int sq = warp_seq_of_token(p.seq, t, lane);
    int pos = -1;
    int32_t page = -1;
    bool in_table = false;
    f2 c2[4], s2[4];
    if (sq >= 0) {
      const int s0 = p.seq.start(sq);
      pos = p.seq.keys(sq) - (p.seq.start(sq + 1) - s0) + (t - s0);
      in_table = !p.cos_sin || (pos >= 0 && pos < p.table_rows);
      if (pos >= 0 && pos < p.seq.capacity) {
        const int pg = __umulhi(2u * (uint32_t)pos, p.page_mul) >> p.page_shift;
        page = load_plain(p.page_table + (int64_t)sq * p.table_width + pg);
      }
      if (full_rot && in_table) {
        Raw8<float> c, s;
        c.load_keep(p.cos_sin + (int64_t)pos * D + 8 * l);
        s.load_keep(p.cos_sin + (int64_t)pos * D + D / 2 + 8 * l);
        c.get2(c2);
        s.get2(s2);
      }
      if (lane == 0 && (!in_table || page < 0 || page >= p.cache.pages || load_plain(p.seq.kv_lens + sq) != p.seq.keys(sq)))
        atomicOr(p.status, DT_DEV_ERR_INDEX);
    }
    const bool to_cache = in_table && page >= 0 && page < p.cache.pages;
    const int last = min((unit + 1) * p.inner, blocks);
    for (int n = unit * p.inner; n < last; ++n) {
      const int kind = kind_of(n), h = head_of(n, kind);
      const bool on = h < (kind == 0 ? hq : hk) && sq >= 0;  // (a row of no sequence: nothing is written for it)
      f2 a2[4], b2[4];
      fetch();
      copies_wait<AP_STAGES - 1>();
      Raw8<T> xa, xb;
      xa.set(ring + fget * (2 * PIECES * AP_THREADS), AP_THREADS);
      xb.set(ring + fget * (2 * PIECES * AP_THREADS) + PIECES * AP_THREADS, AP_THREADS);
      if (++fget == AP_STAGES) fget = 0;
      xa.get2(a2);
      xb.get2(b2);
      if (kind < 2 && full_rot) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          rotate_pair(a2[e].x, b2[e].x, c2[e].x, s2[e].x);
          rotate_pair(a2[e].y, b2[e].y, c2[e].y, s2[e].y);
        }
      }
      float a[8], b[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) a[2 * e] = a2[e].x, a[2 * e + 1] = a2[e].y, b[2 * e] = b2[e].x, b[2 * e + 1] = b2[e].y;
      if (kind < 2 && p.cos_sin && !full_rot && in_table)
        rotate_row<T, D>(p, row_of(t, n), p.cos_sin + (int64_t)pos * p.rotary, l, a, b);
      if (!in_table) {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = b[e] = 0.f;
      }
      if (kind == 0) {
        if (on) {
          T* y = head_ptr<T>(p.q_out, t, h, D);
          store8(y + 8 * l, a);
          store8(y + 8 * (l + L), b);
        }
        continue;
      }
      float la = a[0], ha = a[0], lb = b[0], hb = b[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        la = min_nan(la, a[e]), ha = max_nan(ha, a[e]);
        lb = min_nan(lb, b[e]), hb = max_nan(hb, b[e]);
      }
      if constexpr (D == 64 && G == 64) {  // both chunks are in the one group
        la = lb = min_nan(la, lb);
        ha = hb = max_nan(ha, hb);
      }
      constexpr int SPAN = G / 8 < L ? G / 8 : L;  // lanes of a group
#pragma unroll
      for (int o = SPAN >> 1; o; o >>= 1) {
        la = min_nan(la, __shfl_xor_sync(0xffffffffu, la, o)), ha = max_nan(ha, __shfl_xor_sync(0xffffffffu, ha, o));
        lb = min_nan(lb, __shfl_xor_sync(0xffffffffu, lb, o)), hb = max_nan(hb, __shfl_xor_sync(0xffffffffu, hb, o));
      }
      if (!on) continue;
      uint32_t wa, wb, pa, pb;
      quantise(la, ha, a, &wa, &pa);
      quantise(lb, hb, b, &wb, &pb);
      if (p.has_stored) {
        T* y = head_ptr<T>(kind == 1 ? p.k_st : p.v_st, t, h, D);
        store8(y + 8 * l, a);
        store8(y + 8 * (l + L), b);
      }
      if (!to_cache) continue;
      const int in_page = pos - (int)(__umulhi(2u * (uint32_t)pos, p.page_mul) >> p.page_shift) * p.cache.page_size;
      uint32_t* rec = reinterpret_cast<uint32_t*>(cache_page(p.cache, page, h)) + (int64_t)in_page * W;
      uint32_t* codes = rec + (kind == 2 ? D / 8 : 0);
      uint32_t* params = rec + D / 4 + (kind == 2 ? NG : 0);
      codes[l] = wa;
      codes[l + L] = wb;
      if (8 * l % G == 0) params[8 * l / G] = pa;
      if (8 * (l + L) % G == 0) params[8 * (l + L) / G] = pb;
      if (kind == 2 && l < W - D / 4 - 2 * NG) rec[D / 4 + 2 * NG + l] = 0;  // padding
    }
    t = tn;
    unit = un;
  }
}

template <class T>
cudaError_t launch_append(AppendParams& p, int D, int G, cudaStream_t s) {
  const int SG = 32 / (D / 16);
  const int blocks = (p.q.heads + SG - 1) / SG + 2 * ((p.cache.heads + SG - 1) / SG);
  // as many blocks of a token to a unit as leave four units for every warp of a full device
  const int64_t warps = (int64_t)device_sm_count() * AP_CTAS * AP_WARPS;
  p.inner = 1;
  while (p.inner < blocks && p.seq.tokens * (int64_t)((blocks + 2 * p.inner - 1) / (2 * p.inner)) >= 4 * warps) p.inner *= 2;
  const int64_t units = (int64_t)p.seq.tokens * ((blocks + p.inner - 1) / p.inner);
  const int grid = (int)std::min<int64_t>((units + AP_WARPS - 1) / AP_WARPS, (int64_t)device_sm_count() * AP_CTAS);
#define DT_AP(d, g) \
  if (D == d && G == g) return launch_early(kv4_append_kernel<T, d, g>, dim3(grid), AP_THREADS, 0, s, p)
  DT_AP(64, 32);
  DT_AP(64, 64);
  DT_AP(128, 32);
  DT_AP(128, 64);
  DT_AP(256, 32);
  DT_AP(256, 64);
#undef DT_AP
  return cudaErrorInvalidValue;
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
    if (t.shape[0] == 0 && K.tokens > 0)  // (its pointer may be NULL, which stands for no rotation below)
      return fail(DT_ERR_SHAPE, "cos_sin has no rows: every position would be out of range");
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
  p.page_mul = B.page_mul;
  p.page_shift = B.page_shift;
  p.seq = SeqTable{B.q_starts, B.kv_lens, B.batch, B.q_len, (int32_t)K.tokens, B.capacity};
  p.interleaved = interleaved != 0;
  p.has_stored = k_stored != nullptr;
  if ((st = bind_device_of(B.kv_lens)) != DT_OK) return st;
  p.status = device_status_word(d_status);
  if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
  const cudaError_t e = K.dtype == DT_BF16 ? launch_append<__nv_bfloat16>(p, D, G, stream)
                                           : launch_append<float>(p, D, G, stream);
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
