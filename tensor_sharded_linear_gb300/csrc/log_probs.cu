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

#include "cluster_sm103.cuh"
#include "heads_sm103.cuh"
#include "row_operands.h"

namespace dt {
namespace {

constexpr int LP_MAX_TOP = 32;
constexpr int LP_MAX_GIVEN = 64;
constexpr int LP_WARPS = 8;
constexpr int LP_THREADS = 32 * LP_WARPS;
constexpr int LP_MAX_CLUSTER = 8;
constexpr int64_t LP_MAX_TOP_VOCAB = 1 << 24;
constexpr int LP_MAX_SMEM = 128 * 1024;  // a CTA's list of blocks; on clusters of 8 it holds LP_MAX_TOP_VOCAB
constexpr float LOG2E = 1.44269504088896341f;

// A unit of work is 2 KB of one shard's row, on 16-byte boundaries of memory:
// four vectors a lane, each 512 contiguous bytes over the warp.  Of a row that
// starts off a boundary the first and last units are partly outside it; these
// elements are neither read nor written.
constexpr int LP_VECS = 4;
template <class T>
struct Unit {
  static constexpr int VE = 16 / sizeof(T);      // elements of a vector
  static constexpr int BLOCK = 32 * VE;          // of a vector over the warp
  static constexpr int SIZE = LP_VECS * BLOCK;
};

// Columns [begin, begin + n) of every token.
struct VocabShard {
  char* ptr;
  int64_t ld;  // elements between tokens
  int32_t begin, n;
  int32_t unit, pad;  // units of a row before this shard
};

struct LogProbArgs {
  int32_t shards;
  int32_t units;  // of a row
  int64_t tokens;
  int32_t vocab;
  const int32_t* ids;  // [tokens, given]; NULL: none
  int32_t given, ignore, top;
  float scale;
  float *logp, *lse, *entropy, *top_logp;  // backward: lse and entropy are read
  int32_t* top_ids;
  const float *dlogp, *dentropy;
  int32_t parts;  // CTAs of a row (forward: a cluster)
  int32_t* status;
};
template <int CAP>
struct LogProbParams : LogProbArgs {
  VocabShard z[CAP], dz[CAP];
};
constexpr int LP_SMALL = 8;  // shards of most launches; a parameter block for 64 takes longer to launch

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
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <class T>
struct Vec;  // 16 bytes of logits
template <>
struct Vec<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void get(f2 (&v)[4]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2{__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)};
  }
  __device__ __forceinline__ void put(const f2 (&v)[4]) {
    u = make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y),
                   pack_bf16(v[3].x, v[3].y));
  }
  // the largest of the even and of the odd elements, and what that is as a number
  __device__ __forceinline__ uint32_t most() const {
    return max_nan_bf16x2(max_nan_bf16x2(u.x, u.y), max_nan_bf16x2(u.z, u.w));
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max_nan_bf16x2(a, b); }
  static __device__ __forceinline__ float number(uint32_t m) {
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  // nothing below -1e28 (as bf16); NaN stays
  __device__ __forceinline__ void lift() {
    constexpr uint32_t LOW = 0xee01ee01u;
    u = make_uint4(max_nan_bf16x2(u.x, LOW), max_nan_bf16x2(u.y, LOW), max_nan_bf16x2(u.z, LOW),
                   max_nan_bf16x2(u.w, LOW));
  }
};
template <>
struct Vec<float> {
  uint4 u;
  __device__ __forceinline__ void get(f2 (&v)[2]) const {
    v[0] = f2{__uint_as_float(u.x), __uint_as_float(u.y)}, v[1] = f2{__uint_as_float(u.z), __uint_as_float(u.w)};
  }
  __device__ __forceinline__ void put(const f2 (&v)[2]) {
    u = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  }
  __device__ __forceinline__ float most() const {
    return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                   max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ float larger(float a, float b) { return max_nan(a, b); }
  static __device__ __forceinline__ float number(float m) { return m; }
  __device__ __forceinline__ void lift() {
    auto up = [](uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), -1e28f)); };
    u = make_uint4(up(u.x), up(u.y), up(u.z), up(u.w));
  }
};
__device__ __forceinline__ float element(const Vec<__nv_bfloat16>& v, int i) {
  const uint32_t w = i < 2 ? v.u.x : i < 4 ? v.u.y : i < 6 ? v.u.z : v.u.w;
  return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float element(const Vec<float>& v, int i) {
  return __uint_as_float(i == 0 ? v.u.x : i == 1 ? v.u.y : i == 2 ? v.u.z : v.u.w);
}

// Where a unit lies: the first element of lane 0's first vector is column
// `at` of the shard's row, -VE < at < n.
template <class T>
struct Place {
  const T* row;  // column 0 of the shard's row
  int32_t shard, at, n;
  __device__ __forceinline__ int column(int vec, int lane) const {
    return at + vec * Unit<T>::BLOCK + lane * Unit<T>::VE;
  }
  __device__ __forceinline__ bool inside() const { return at >= 0 && at + Unit<T>::SIZE <= n; }
};
template <class T, class S>
__device__ __forceinline__ Place<T> place(const S* shards, int count, int unit, int64_t t, int& s) {
  while (s + 1 < count && shards[s + 1].unit <= unit) ++s;
  Place<T> p;
  p.row = reinterpret_cast<const T*>(shards[s].ptr) + t * shards[s].ld;
  const int off = (int)(reinterpret_cast<uintptr_t>(p.row) & 15) / (int)sizeof(T);
  p.shard = s;
  p.at = (unit - shards[s].unit) * Unit<T>::SIZE - off;
  p.n = shards[s].n;
  return p;
}
// On to unit `unit`, `step` further.
template <class T, class S>
__device__ __forceinline__ void move_on(Place<T>& p, const S* shards, int count, int unit, int step, int64_t t) {
  int s = p.shard;
  if (s + 1 < count && shards[s + 1].unit <= unit) p = place<T>(shards, count, unit, t, s);
  else p.at += step * Unit<T>::SIZE;
}
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
// The lane's vector `vec` of a unit; -inf for what lies outside the row.
template <class T>
__device__ __forceinline__ Vec<T> load_vec(const Place<T>& p, int vec, int lane) {
  Vec<T> v;
  const int c = p.column(vec, lane);
  if (c >= 0 && c + Unit<T>::VE <= p.n) {
    v.u = load16(p.row + c);
    return v;
  }
  constexpr int N = Unit<T>::VE / 2;
  f2 x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i].x = c + 2 * i >= 0 && c + 2 * i < p.n ? to_f32(p.row[c + 2 * i]) : -INFINITY;
    x[i].y = c + 2 * i + 1 >= 0 && c + 2 * i + 1 < p.n ? to_f32(p.row[c + 2 * i + 1]) : -INFINITY;
  }
  v.put(x);
  return v;
}
template <class T>
__device__ __forceinline__ void load_unit(const Place<T>& p, int lane, Vec<T> (&v)[LP_VECS]) {
  if (p.inside()) {
#pragma unroll
    for (int i = 0; i < LP_VECS; ++i) v[i].u = load16(p.row + p.column(i, lane));
  } else {
#pragma unroll
    for (int i = 0; i < LP_VECS; ++i) v[i] = load_vec(p, i, lane);
  }
}

template <class T, class P>
__device__ __forceinline__ float logit(const P& p, int64_t t, int j) {
  int s = 0;
  while (s + 1 < p.shards && p.z[s + 1].begin <= j) ++s;
  return to_f32(reinterpret_cast<const T*>(p.z[s].ptr)[t * p.z[s].ld + (j - p.z[s].begin)]);
}

// The id at place i: its column, or -1 (and the status bit unless it is the one to be ignored).
__device__ __forceinline__ int given_id(const LogProbArgs& p, int64_t i, bool report) {
  const int32_t id = load_plain(p.ids + i);
  if (id == p.ignore) return -1;  // (which may be a column)
  if (id >= 0 && id < p.vocab) return id;
  if (report) atomicOr(p.status, DT_DEV_ERR_INDEX);
  return -1;
}

// A running softmax in powers of two: the largest logit m, s = sum 2^t and
// e = sum t 2^t over the logits so far, t = c z - fl(c m): one multiply-add a
// logit.  The product's rounding c m - fl(c m) is in every t and drops out at the
// end (`rounding`); it has to stay small, for the largest logit's 2^t is 2 to
// that, and does while |c m| <= 2^22, whose last place is a quarter: an eighth.
// Beyond (m starts there, at the lowest finite number) t = (z - m) c, which has
// no such rounding and does not overflow, and a maximum that goes from one form
// to the other takes the difference of the two roundings along.  Factors stay
// above -1e28, so that 0 times them is 0.
struct Soft {
  float m = -3.402823466e38f, s = 0.f, e = 0.f;
  static __device__ __forceinline__ bool usual(float m, float c) { return fabsf(__fmul_rn(m, c)) <= 0x1p22f; }
  static __device__ __forceinline__ float rounding(float m, float c) {
    return usual(m, c) ? fmaf(m, c, -__fmul_rn(m, c)) : 0.f;
  }
  __device__ __forceinline__ float rounding(float c) const { return rounding(m, c); }
  __device__ __forceinline__ void raise(float to, float c) {  // to >= m, or NaN
    const float from = __fmul_rn(m, c), up = __fmul_rn(to, c);
    float d = __fsub_rn(from, up);
    if (!(fmaxf(fabsf(from), fabsf(up)) <= 0x1p22f)) d = (m - to) * c + (rounding(to, c) - rounding(m, c));
    const float down = fmaxf(d, -1e28f), f = exp2_fast(down);
    e = f * fmaf(down, s, e);
    s *= f;
    m = to;
  }
  template <int N>
  __device__ __forceinline__ void join_lanes(float c) {  // over groups of N lanes
    float top = m;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    raise(top, c);
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
  }
};
// t of two logits under any m
__device__ __forceinline__ f2 difference(f2 z, float m, float c) {
  if (Soft::usual(m, c)) return fma2(z, both(c), both(-__fmul_rn(m, c)));
  return (z + both(-m)) * both(c);
}

template <class T, bool ENT>
__device__ __forceinline__ void soft_unit(Soft& a, Vec<T> (&v)[LP_VECS], float most, float c) {
  most = max_nan(a.m, most);
  if (!(most == a.m)) a.raise(most, c);
  constexpr int N = Unit<T>::VE / 2;
  f2 s[2] = {both(0.f), both(0.f)}, e[2] = {both(0.f), both(0.f)};
  if (__all_sync(0xffffffffu, Soft::usual(a.m, c))) {
    const f2 r2 = both(-__fmul_rn(a.m, c)), c2 = both(c);
#pragma unroll
    for (int i = 0; i < LP_VECS; ++i) {
      if (ENT) v[i].lift();  // (2^t is 0 there either way)
      f2 z[N];
      v[i].get(z);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const f2 t = fma2(z[k], c2, r2), x = f2{exp2_fast(t.x), exp2_fast(t.y)};
        s[k & 1] = s[k & 1] + x;
        if (ENT) e[k & 1] = fma2(x, t, e[k & 1]);
      }
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < LP_VECS; ++i) {
      f2 z[N];
      v[0].get(z);
      v[0] = v[1], v[1] = v[2], v[2] = v[3];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const f2 t = difference(z[k], a.m, c), x = f2{exp2_fast(t.x), exp2_fast(t.y)};
        s[0] = s[0] + x;
        if (ENT) e[0] = fma2(x, f2{fmaxf(t.x, -1e28f), fmaxf(t.y, -1e28f)}, e[0]);
      }
    }
  }
  const f2 s1 = s[0] + s[1], e1 = e[0] + e[1];
  a.s += s1.x + s1.y;
  if (ENT) a.e += e1.x + e1.y;
}

// How many of the n numbers at x (16-byte aligned) are larger.
__device__ __forceinline__ int count_larger(const uint64_t* x, int n, uint64_t mine) {
  int above = 0;
#pragma unroll 4
  for (int i = 0; i + 1 < n; i += 2) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(x + i);
    above += (v.x > mine) + (v.y > mine);
  }
  return n & 1 ? above + (x[n - 1] > mine) : above;
}

// Elements of a vector over the warp whose key is at least `low` and which are
// above `worst`, one lane's vector at a time, an element a lane: body(number)
// with (key, lowest id first) as a number, 0 in lanes without.  Lane 0's first
// element is column `col0` of a shard's row of n, token `begin` + col0.
template <class T, class F>
__device__ __forceinline__ void each_above(const Vec<T>& x, int col0, int n, int begin, uint32_t low, uint64_t worst,
                                           int lane, F&& body) {
  constexpr int VE = Unit<T>::VE;
  auto number = [](uint32_t key, int id) { return (uint64_t)key << 32 | (0xFFFFFFFFu - (uint32_t)id); };
  const uint32_t key = order_key(Vec<T>::number(x.most()));
  unsigned lanes = __ballot_sync(0xffffffffu, key >= low && number(key, max(begin + col0 + lane * VE, 0)) > worst);
#pragma unroll 1
  while (lanes) {
    const int from = __ffs(lanes) - 1;
    lanes &= lanes - 1;
    Vec<T> y;
    y.u.x = __shfl_sync(0xffffffffu, x.u.x, from), y.u.y = __shfl_sync(0xffffffffu, x.u.y, from);
    y.u.z = __shfl_sync(0xffffffffu, x.u.z, from), y.u.w = __shfl_sync(0xffffffffu, x.u.w, from);
    const int col = col0 + from * VE + lane;
    const uint32_t mine = order_key(element(y, lane % VE));
    const bool in = lane < VE && col >= 0 && col < n && mine >= low;
    body(in ? number(mine, begin + col) : 0);
  }
}

// The largest so far, in order over a warp's lanes (lane i: the i-th; 0: none).
struct TopList {
  uint64_t best = 0, worst = 0;  // worst: the k-th
  __device__ __forceinline__ void insert(uint64_t n, int k, int lane) {
    if (n <= worst) return;
    const int pos = __popc(__ballot_sync(0xffffffffu, best > n));
    const uint64_t up = __shfl_up_sync(0xffffffffu, best, 1);
    best = lane < pos ? best : lane == pos ? n : up;
    worst = __shfl_sync(0xffffffffu, best, k - 1);
  }
};

// One cluster of CTAs per token (of one CTA when there are tokens enough): each
// warp takes every so many units, the CTAs' sums meet in the first one's shared
// memory, and that one writes the results.  One pass, each logit read once; two
// units' loads a warp are under way, 32 warps an SM.  With the entropy an element
// costs a multiply-add and a power of two, two sums and its unpacking: 8 warp
// instructions for 32 of them, 0.67 of the issue slots.
//   4096 x 128256 bf16 in 8 shards                153.5 us, 1.01 of a copy's rate; with the entropy 163.0, 0.95
//   64 x 128256 fp32, 5 alternatives               12.8 us: the pass is half of it, then the alternatives' steps
//   777 x 50257 bf16, 10 alternatives              20.2 us, 0.57: the same
//   1 x 128256 bf16, 20 alternatives, entropy       8.7 us: 2 units a warp, then six meetings of the cluster or CTA
// (With 3 CTAs an SM and more registers: 175.7 us with the entropy, 19.1, 19.2 and 8.3.)
//
// Alternatives.  The pass over the row leaves the largest logit of each block
// of 1 KB and of 64 groups of the cluster's lanes (32 in a CTA of one warp).
// The k-th largest of the groups is at most the k-th largest logit, so every
// alternative is in a block that reaches it; these are read again, now from L2,
// and the elements that reach it (hardly more than k when values differ) are
// collected.  Where there are too many, as under a mask that leaves fewer than
// k, the blocks go through a sorted list per warp instead.  What is collected is
// ranked by counting the larger ones.  The order is that of (value, lowest id)
// as one 64-bit number, so the result does not depend on who came first.
constexpr int LP_BLOCK_VECS = 2;
constexpr int LP_UNIT_BLOCKS = LP_VECS / LP_BLOCK_VECS;
constexpr int LP_GROUPS = 64;
constexpr int LP_COLLECT = 256;  // what a CTA collects at most
static_assert(LP_COLLECT >= LP_WARPS * LP_MAX_TOP && LP_COLLECT >= LP_MAX_CLUSTER * LP_MAX_TOP, "lists fit");

template <class T, bool TOP, bool ENT, int CAP>
__global__ void __launch_bounds__(LP_THREADS, 4) log_probs_kernel(const __grid_constant__ LogProbParams<CAP> p) {
  __shared__ Soft soft[LP_WARPS];
  __shared__ Soft meet[LP_MAX_CLUSTER];                                   // in the first CTA
  __shared__ __align__(16) uint64_t recv[LP_MAX_CLUSTER * LP_MAX_TOP];    // in the first CTA
  __shared__ int received[LP_MAX_CLUSTER];                                // in the first CTA
  __shared__ __align__(16) uint64_t cand[LP_COLLECT];
  __shared__ __align__(16) uint32_t group[LP_GROUPS];                     // the cluster's, in every CTA
  __shared__ uint32_t reach;
  __shared__ int listed, found;
  extern __shared__ uint32_t block_key[];  // TOP: [blocks of this CTA], then the list of those to be read again
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int ctas = p.parts, rank = ctas > 1 ? (int)cluster_rank() : 0;
  if (ctas > 1) cluster_arrive();
  const int64_t t = blockIdx.x / ctas;
  const float c = p.scale * LOG2E;
  const int step = ctas * warps, first = rank * warps + warp;
  if (TOP && threadIdx.x == 0) listed = found = 0;
  // the first CTA's threads stand for the given ids (one CTA of one warp: two
  // each): the ids are asked for before the logits, their logits after them
  int32_t id[2] = {-1, -1};
  float z_id[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (rank == 0 && i < p.given) id[j] = load_plain(p.ids + t * p.given + i);
  }
  Soft a;
  int rounds = 0;
  auto work = [&](Vec<T>(&v)[LP_VECS]) {
    auto most = v[0].most();
    if (TOP) {
#pragma unroll
      for (int b = 0; b < LP_UNIT_BLOCKS; ++b) {
        auto m = v[b * LP_BLOCK_VECS].most();
#pragma unroll
        for (int i = 1; i < LP_BLOCK_VECS; ++i) m = Vec<T>::larger(m, v[b * LP_BLOCK_VECS + i].most());
        most = b ? Vec<T>::larger(most, m) : m;
        const uint32_t key = __reduce_max_sync(0xffffffffu, order_key(Vec<T>::number(m)));
        if (lane == 0) block_key[(rounds * warps + warp) * LP_UNIT_BLOCKS + b] = key;
      }
      ++rounds;
    } else {
#pragma unroll
      for (int i = 1; i < LP_VECS; ++i) most = Vec<T>::larger(most, v[i].most());
    }
    soft_unit<T, ENT>(a, v, Vec<T>::number(most), c);
  };
  if (first < p.units) {
    int s = 0;
    Place<T> at = place<T>(p.z, p.shards, first, t, s);
    Vec<T> v[LP_VECS], w[LP_VECS];
    load_unit(at, lane, v);
    for (int u = first;; u += 2 * step) {
      const bool more = u + step < p.units;
      if (more) {
        move_on(at, p.z, p.shards, u + step, step, t);
        load_unit(at, lane, w);
      }
      work(v);
      if (!more) break;
      const bool again = u + 2 * step < p.units;
      if (again) {
        move_on(at, p.z, p.shards, u + 2 * step, step, t);
        load_unit(at, lane, v);
      }
      work(w);
      if (!again) break;
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (rank != 0 || (int)(threadIdx.x + j * blockDim.x) >= p.given) continue;
    if (id[j] >= 0 && id[j] < p.vocab && id[j] != p.ignore) {
      z_id[j] = logit<T>(p, t, id[j]);
    } else {
      if (id[j] != p.ignore) atomicOr(p.status, DT_DEV_ERR_INDEX);
      id[j] = -1;
    }
  }
  // lanes of a group (a power of two, a warp's at most: a cluster's CTAs have 8 warps)
  const int per_group = ctas > 1 ? 32 * LP_WARPS * ctas / LP_GROUPS : max(1, warps / 2);
  const int groups = 32 * warps * ctas / per_group;
  if (ctas > 1) cluster_wait();  // the others are there
  if (TOP) {
    // (no element: below every key; m as it started: at most -inf is known to be there)
    uint32_t g = first < p.units ? order_key(a.m == Soft().m ? -INFINITY : a.m) : 0;
    for (int o = 1; o < per_group; o <<= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
    const int at = (first * 32 + lane) / per_group;
    if (lane % per_group == 0) {
      if (ctas == 1) group[at] = g;
      for (int r = 0; ctas > 1 && r < ctas; ++r) store_cluster(in_cta(&group[at], r), g);
    }
  }
  a.join_lanes<32>(c);
  if (lane == 0) soft[warp] = a;
  __syncthreads();
  a = lane % LP_WARPS < warps ? soft[lane % LP_WARPS] : Soft();
  a.join_lanes<LP_WARPS>(c);
  if (ctas > 1) {
    if (threadIdx.x == 0) {
      store_cluster(in_cta(&meet[rank].m, 0), a.m);
      store_cluster(in_cta(&meet[rank].s, 0), a.s);
      store_cluster(in_cta(&meet[rank].e, 0), a.e);
    }
    cluster_arrive();
    cluster_wait();
    if (!TOP && rank != 0) return;
    if (rank == 0) {
      a = lane % LP_MAX_CLUSTER < ctas ? meet[lane % LP_MAX_CLUSTER] : Soft();
      a.join_lanes<LP_MAX_CLUSTER>(c);
    }
  }
  const bool none = a.s == 0.f;  // no token is possible
  const float ln_s = logf(a.s), ln = fmaf(-0.693147180559945f, a.rounding(c), ln_s);
  auto logp = [&](float z) { return none ? -INFINITY : (z - a.m) * p.scale - ln; };
  if (rank == 0) {
    if (threadIdx.x == 0) {
      if (p.lse) p.lse[t] = none ? -INFINITY : fmaf(a.m, p.scale, ln);
      if (ENT) p.entropy[t] = none ? 0.f : fmaf(-0.693147180559945f, a.e / a.s, ln_s);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i < p.given) p.logp[t * p.given + i] = id[j] >= 0 ? logp(z_id[j]) : 0.f;
    }
  }
  if (!TOP) return;

  {  // a group's number of larger ones: its threads share the others among them
    const int split = 32 * warps / groups, sh = 31 - __clz(split), g = threadIdx.x >> sh;
    const uint32_t mine = group[g];
    int above = 0;
#pragma unroll 4
    for (int i = 4 * (threadIdx.x & (split - 1)); i < groups; i += 4 * split) {
      const uint4 o = *reinterpret_cast<const uint4*>(group + i);
      const int me = g - i;
      above += (o.x > mine || (o.x == mine && 0 < me)) + (o.y > mine || (o.y == mine && 1 < me)) +
               (o.z > mine || (o.z == mine && 2 < me)) + (o.w > mine || (o.w == mine && 3 < me));
    }
    for (int o = split / 2; o; o >>= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (above == p.top - 1) reach = mine;
  }
  __syncthreads();
  const uint32_t low = reach;
  // block i: round i >> shift of the CTA, its warps' units, their blocks
  const int shift = 31 - __clz(warps * LP_UNIT_BLOCKS);
  const int blocks = rank * warps < p.units ? ((p.units - rank * warps + step - 1) / step) << shift : 0;
  uint32_t* list = block_key + blocks;
  auto unit_of = [&](int i) { return rank * warps + (i & ((1 << shift) - 1)) / LP_UNIT_BLOCKS + (i >> shift) * step; };
  for (int i = threadIdx.x; i < blocks; i += blockDim.x)
    if (unit_of(i) < p.units && block_key[i] >= low) list[atomicAdd(&listed, 1)] = i;
  __syncthreads();
  // body(vector, column of lane 0's first element, columns of the shard, its first token)
  auto again = [&](auto&& body) {
#pragma unroll 1
    for (int l = warp; l < listed; l += warps) {
      const int i = (int)list[l];
      int s = 0;
      const Place<T> q = place<T>(p.z, p.shards, unit_of(i), t, s);
      const int vec = i % LP_UNIT_BLOCKS * LP_BLOCK_VECS;
      static_assert(LP_BLOCK_VECS == 2, "x, then y");
      Vec<T> x = load_vec(q, vec, lane);
      const Vec<T> y = load_vec(q, vec + 1, lane);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        body(x, q.column(vec + k, 0), q.n, p.z[q.shard].begin);
        x = y;
      }
    }
  };
  again([&](const Vec<T>& x, int col0, int n, int begin) {
    each_above(x, col0, n, begin, low, 0, lane, [&](uint64_t mine) {
      const unsigned in = __ballot_sync(0xffffffffu, mine != 0);
      if (in == 0) return;
      int base = 0;
      if (lane == 0) base = atomicAdd(&found, __popc(in));
      base = __shfl_sync(0xffffffffu, base, 0) + __popc(in & ((1u << lane) - 1));
      if (mine != 0 && base < LP_COLLECT) cand[base] = mine;
    });
  });
  __syncthreads();
  if (found > LP_COLLECT) {
    TopList best;
    again([&](const Vec<T>& x, int col0, int n, int begin) {
      each_above(x, col0, n, begin, low, best.worst, lane, [&](uint64_t mine) {
        unsigned in = __ballot_sync(0xffffffffu, mine > best.worst);
#pragma unroll 1
        for (; in; in &= in - 1) best.insert(__shfl_sync(0xffffffffu, mine, __ffs(in) - 1), p.top, lane);
      });
    });
    __syncthreads();  // (everyone has read the count)
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    const unsigned have = __ballot_sync(0xffffffffu, lane < p.top && best.best != 0);
    int base = 0;
    if (lane == 0) base = atomicAdd(&found, __popc(have));
    base = __shfl_sync(0xffffffffu, base, 0);
    if (have >> lane & 1) cand[base + __popc(have & ((1u << lane) - 1))] = best.best;
    __syncthreads();
  }
  int total = found;
  if (ctas > 1) {  // what this CTA found, at most its k largest
    for (int i = threadIdx.x; i < total; i += blockDim.x) {
      const int r = total <= p.top ? i : count_larger(cand, total, cand[i]);
      if (r < p.top) store_cluster(in_cta(&recv[rank * p.top + r], 0), cand[i]);
    }
    if (threadIdx.x == 0) store_cluster(in_cta(&received[rank], 0), (uint32_t)min(total, p.top));
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < ctas * LP_MAX_TOP; i += blockDim.x)
      if (i % LP_MAX_TOP < received[i / LP_MAX_TOP])
        cand[atomicAdd(&found, 1)] = recv[i / LP_MAX_TOP * p.top + i % LP_MAX_TOP];
    __syncthreads();
    total = found;
  }
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    const uint64_t mine = cand[i];
    const int r = count_larger(cand, total, mine);
    if (r < p.top) {
      p.top_logp[t * p.top + r] = logp(key_value((uint32_t)(mine >> 32)));
      p.top_ids[t * p.top + r] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine);
    }
  }
}

// l = scale z - lse is as exact as the fp32 lse that the caller has: beyond 2^24 its
// last place is more than 1, and p = exp(l) off by a factor.
//
// A CTA takes a run of units of one token; bound by HBM (4096 x 128256 bf16 in 8
// shards, a tenth of the rows without gradient and not read: 292 us, 1.00 of a
// copy's rate; with the entropy's 312; 301 x 50257 fp32 20.5, 0.87).  The given
// ids' elements are written last, by the threads that stand for them, so that the pass itself
// is the same for all.
template <class T, bool ENT, int CAP>
__global__ void __launch_bounds__(LP_THREADS, 4) log_probs_backward_kernel(const __grid_constant__ LogProbParams<CAP> p) {
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / p.parts;
  const int part = (int)(blockIdx.x - t * p.parts);
  const int u0 = (int)((int64_t)p.units * part / p.parts), u1 = (int)((int64_t)p.units * (part + 1) / p.parts);
  float g = 0.f;
  bool zero = true;
  for (int c = 0; c < p.given; ++c) {
    const int id = given_id(p, t * p.given + c, part == 0 && threadIdx.x == 0);
    const float v = id >= 0 ? load_plain(p.dlogp + t * p.given + c) : 0.f;
    zero = zero && v == 0.f;
    g += v;
  }
  const float lse = load_plain(p.lse + t);
  const float ge = ENT ? load_plain(p.dentropy + t) : 0.f, h = ENT ? load_plain(p.entropy + t) : 0.f;
  zero = (zero && ge == 0.f) || lse == -INFINITY;
  // dlogit = exp(l) (a + b l) with l = scale z - lse, and scale g_c on top at the given ids
  // (below -256 exp(l) is 0, which the other factor, kept finite, does not change)
  const float a = -p.scale * (g + ge * h), b = -p.scale * ge;
  auto value = [&](float z) {
    const float l = fmaf(z, p.scale, -lse), x = exp2_fast(l * LOG2E);
    return x * (ENT ? fmaf(fmaxf(l, -256.f), b, a) : a);
  };
  // the given ids of this CTA's units: their gradients, before the logits may be overwritten
  T* to = nullptr;
  float at_id = 0.f;
  if ((int)threadIdx.x < p.given && !zero) {
    const int id = given_id(p, t * p.given + threadIdx.x, false);
    if (id >= 0) {
      int s = 0;
      while (s + 1 < p.shards && p.z[s + 1].begin <= id) ++s;
      const T* row = reinterpret_cast<const T*>(p.z[s].ptr) + t * p.z[s].ld;
      const int col = id - p.z[s].begin, off = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
      const int u = p.z[s].unit + (col + off) / Unit<T>::SIZE;
      if (u >= u0 && u < u1) {
        float mine = 0.f;
        for (int c = 0; c < p.given; ++c)
          if (load_plain(p.ids + t * p.given + c) == id) mine += load_plain(p.dlogp + t * p.given + c);
        to = reinterpret_cast<T*>(p.dz[s].ptr) + t * p.dz[s].ld + col;
        at_id = fmaf(p.scale, mine, value(to_f32(row[col])));
      }
    }
  }
  __syncthreads();
  constexpr int N = Unit<T>::VE / 2;
  int shard = 0;
  for (int u = u0 + warp; u < u1; u += LP_WARPS) {
    const Place<T> at = place<T>(p.z, p.shards, u, t, shard);
    T* out = reinterpret_cast<T*>(p.dz[at.shard].ptr) + t * p.dz[at.shard].ld;
    // the gradient's row starts as far from a 16-byte boundary as the logits' in all but odd views
    const bool alike = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(at.row)) & 15) == 0;
    Vec<T> v[LP_VECS];
    if (!zero) load_unit(at, lane, v);
#pragma unroll
    for (int i = 0; i < LP_VECS; ++i) {
      f2 x[N];
      if (!zero) {
        v[i].get(x);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const f2 l = fma2(x[k], both(p.scale), both(-lse)), e = l * both(LOG2E);
          const f2 q = f2{exp2_fast(e.x), exp2_fast(e.y)};
          x[k] = q * (ENT ? fma2(f2{fmaxf(l.x, -256.f), fmaxf(l.y, -256.f)}, both(b), both(a)) : both(a));
        }
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = both(0.f);
      }
      v[i].put(x);
      const int c = at.column(i, lane);
      if (alike && c >= 0 && c + Unit<T>::VE <= at.n) {
        __stcs(reinterpret_cast<uint4*>(out + c), v[i].u);
      } else {
#pragma unroll
        for (int k = 0; k < Unit<T>::VE; ++k)
          if (c + k >= 0 && c + k < at.n) from_f32(out + c + k, k & 1 ? x[k / 2].y : x[k / 2].x);
      }
    }
  }
  __syncthreads();
  if (to) from_f32(to, at_id);
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
    out[(*shards)++] = VocabShard{v.ptr, ld, (int32_t)v.goff[last], (int32_t)v.shape[last], 0, 0};
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

dt_status common_checks(const LogProbArgs& p) {
  if (!(p.scale >= 0x1p-20f && p.scale <= 0x1p20f)) return fail(DT_ERR_INVALID_ARG, "scale must be in [2^-20, 2^20]");
  if (p.given > LP_MAX_GIVEN) return fail(DT_ERR_CAPACITY, "%d ids per token (at most %d)", p.given, LP_MAX_GIVEN);
  if (p.tokens > 0 && p.vocab == 0) return fail(DT_ERR_SHAPE, "logits of an empty vocabulary");
  return DT_OK;
}

// The shards' units, for rows that start on 16-byte boundaries or not.
int64_t count_units(VocabShard* z, int shards, int64_t tokens, int esize) {
  int64_t units = 0;
  const int size = LP_VECS * 32 * 16 / esize;
  for (int s = 0; s < shards; ++s) {
    z[s].unit = (int32_t)units;
    const bool even = reinterpret_cast<uintptr_t>(z[s].ptr) % 16 == 0 && (tokens == 1 || z[s].ld * esize % 16 == 0);
    units += ((int64_t)z[s].n + (even ? 0 : 16 / esize - 1) + size - 1) / size;
  }
  return units;
}

template <auto KERNEL, class P>
cudaError_t launch_log_probs(const P& p, int threads, size_t smem, cudaStream_t s) {
  if (smem > 32 * 1024)
    if (cudaError_t e = allow_dynamic_smem<KERNEL, LP_MAX_SMEM>()) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tokens * p.parts));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = p.parts;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, KERNEL, p);
}

template <class T, int CAP>
cudaError_t forward(const LogProbArgs& a, const VocabShard* z, cudaStream_t s) {
  LogProbParams<CAP> p;
  static_cast<LogProbArgs&>(p) = a;
  std::copy(z, z + a.shards, p.z);
  // Few tokens: a cluster for each, as long as all CTAs are resident at once
  // and every warp has a unit.
  const int64_t resident = 4 * (int64_t)device_sm_count();
  p.parts = 1;
  while (p.parts < LP_MAX_CLUSTER && p.tokens * p.parts * 2 <= resident && p.units >= 2 * p.parts * LP_WARPS) p.parts *= 2;
  auto smem = [&] {
    const int64_t step = (int64_t)p.parts * LP_WARPS;
    return a.top ? (size_t)((p.units + step - 1) / step * LP_WARPS * LP_UNIT_BLOCKS * 2 * sizeof(uint32_t)) : 0;
  };
  while (p.parts < LP_MAX_CLUSTER && smem() > LP_MAX_SMEM) p.parts *= 2;
  int warps = 1;
  while (warps < LP_WARPS && warps < p.units) warps *= 2;
  // Many tokens: fewer warps a token, down to 16 units each, as long as the
  // SMs' warps are half busy, for what follows the pass is done by each of them
  // (16384 tokens of 8192 in bf16: 43.0 us, 69.3 with eight warps each; 777 of
  // 50257 with ten alternatives 20.1 and 23.0).
  while (p.parts == 1 && warps > 1 && p.units < 16 * warps && p.tokens * (warps / 2) >= resident * LP_WARPS / 2) warps /= 2;
#define DT_LP(TOP, ENT) \
  if ((a.top > 0) == TOP && (a.entropy != nullptr) == ENT) \
    return launch_log_probs<log_probs_kernel<T, TOP, ENT, CAP>>(p, 32 * warps, smem(), s);
  DT_LP(false, false) DT_LP(false, true) DT_LP(true, false) DT_LP(true, true)
#undef DT_LP
  return cudaErrorInvalidValue;
}

template <class T, int CAP>
cudaError_t backward(const LogProbArgs& a, const VocabShard* z, const VocabShard* dz, cudaStream_t s) {
  LogProbParams<CAP> p;
  static_cast<LogProbArgs&>(p) = a;
  std::copy(z, z + a.shards, p.z);
  std::copy(dz, dz + a.shards, p.dz);
  // parts of at most 8 units a warp, fewer while that leaves CTAs idle
  p.parts = std::max(1, (p.units + 8 * LP_WARPS - 1) / (8 * LP_WARPS));
  while (p.tokens * p.parts < 4 * (int64_t)device_sm_count() && p.units >= 2 * p.parts * LP_WARPS) p.parts *= 2;
  const dim3 grid((unsigned)(p.tokens * p.parts));
  if ((int64_t)grid.x != p.tokens * p.parts) return cudaErrorInvalidValue;
  return a.dentropy ? launch_early(log_probs_backward_kernel<T, true, CAP>, grid, LP_THREADS, 0, s, p)
                    : launch_early(log_probs_backward_kernel<T, false, CAP>, grid, LP_THREADS, 0, s, p);
}

void sizes(const Layout& l, LogProbArgs* p) {
  p->tokens = 1;
  for (int d = 0; d + 1 < l.ndim; ++d) p->tokens *= l.gshape[d];
  p->vocab = (int32_t)l.gshape[l.ndim - 1];
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
    VocabShard z[DT_MAX_SLOTS];
    Layout lz;
    dt_status st;
    if (!logits) return fail(DT_ERR_INVALID_ARG, "logits is NULL");
    if ((st = vocab_operand(logits, "logits", tp_mesh_dim, false, z, &p.shards, &lz)) != DT_OK) return st;
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
      if (k > 0 && p.vocab > LP_MAX_TOP_VOCAB)
        return fail(DT_ERR_CAPACITY, "alternatives from a vocabulary of more than 2^24");
      if (k > 0 && p.vocab > LP_MAX_TOP_VOCAB / 8 && p.tokens > INT32_MAX / LP_MAX_CLUSTER)
        return fail(DT_ERR_CAPACITY, "alternatives of 2^28 tokens from a vocabulary of more than 2^21");
      p.top = (int32_t)k;
      if (k > 0) anchor = ptr;
    }
    if ((st = common_checks(p)) != DT_OK) return st;
    if (p.tokens == 0 || !anchor) return DT_OK;
    if ((st = bind_device_of(anchor)) != DT_OK) return st;
    p.status = device_status_word(d_status);
    if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.units = (int32_t)count_units(z, p.shards, p.tokens, lz.esize);
    const bool small = p.shards <= LP_SMALL;
    const cudaError_t e =
        lz.dtype == DT_BF16 ? (small ? forward<__nv_bfloat16, LP_SMALL>(p, z, s) : forward<__nv_bfloat16, DT_MAX_SLOTS>(p, z, s))
                            : (small ? forward<float, LP_SMALL>(p, z, s) : forward<float, DT_MAX_SLOTS>(p, z, s));
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
    VocabShard z[DT_MAX_SLOTS], dz[DT_MAX_SLOTS];
    int32_t dz_shards = 0;
    Layout lz, ld;
    dt_status st;
    if (!logits || !dlogits) return fail(DT_ERR_INVALID_ARG, "logits or dlogits is NULL");
    if (!lse) return fail(DT_ERR_INVALID_ARG, "lse is NULL");
    if ((ids != nullptr) != (dlogprobs != nullptr)) return fail(DT_ERR_INVALID_ARG, "ids and dlogprobs go together");
    if (!dlogprobs && !dentropy) return fail(DT_ERR_INVALID_ARG, "neither dlogprobs nor dentropy");
    if (dentropy && !entropy) return fail(DT_ERR_INVALID_ARG, "dentropy needs entropy");
    if ((st = vocab_operand(logits, "logits", tp_mesh_dim, false, z, &p.shards, &lz)) != DT_OK) return st;
    if ((st = vocab_operand(dlogits, "dlogits", tp_mesh_dim, true, dz, &dz_shards, &ld)) != DT_OK) return st;
    if ((st = same_mesh(ld, lz, "dlogits")) != DT_OK) return st;
    bool same = ld.ndim == lz.ndim;
    for (int d = 0; same && d < lz.ndim; ++d) same = ld.gshape[d] == lz.gshape[d];
    if (!same) return fail(DT_ERR_SHAPE, "dlogits must have the shape of logits");
    if (ld.dtype != lz.dtype) return fail(DT_ERR_INVALID_ARG, "dlogits must have the dtype of logits");
    if (p.shards != dz_shards) return fail(DT_ERR_PLACEMENT, "dlogits must be placed as logits");
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
    if ((st = common_checks(p)) != DT_OK) return st;
    if (p.tokens == 0) return DT_OK;
    if ((st = bind_device_of(dz[0].ptr)) != DT_OK) return st;
    p.status = device_status_word(d_status);
    if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.units = (int32_t)count_units(z, p.shards, p.tokens, lz.esize);
    const bool small = p.shards <= LP_SMALL;
    const cudaError_t e = lz.dtype == DT_BF16 ? (small ? backward<__nv_bfloat16, LP_SMALL>(p, z, dz, s)
                                                       : backward<__nv_bfloat16, DT_MAX_SLOTS>(p, z, dz, s))
                                              : (small ? backward<float, LP_SMALL>(p, z, dz, s)
                                                       : backward<float, DT_MAX_SLOTS>(p, z, dz, s));
    if (e != cudaSuccess) return fail(DT_ERR_CUDA, "log_probs_backward launch: %s", cudaGetErrorString(e));
    count_launch();
    return DT_OK;
  });
}
