// What lies between the output of one block and the input of the next: the
// partial sums of a row-parallel layer added, a norm, a gate, dropout, the
// scaled residual and the norm before the next block; and its gradients.
//
// Per token (N channels, all arithmetic fp32; what an operand is missing for
// is left out):
//   s = sum of x's parts, in rank order         r(v) = 1 / sqrt(mean(v^2) + eps)
//   u = s r(s) post      f = keep ? u gate / (1 - p) : 0
//   h = a residual + f   y = h r(h) pre
// and for gradients dh of h and dy of y, with z = dy pre and m = mean over channels,
//   g  = dh + r(h) z - r(h)^3 m(h z) h          dresidual = a g
//   e  = keep ? g / (1 - p) : 0                 v = e gate post
//   dx = r(s) v - r(s)^3 m(s v) s               dgate = sum e u
//   dpre = sum dy h r(h)                        dpost = sum e gate s r(s)
// h and y come from the unrounded h; the backward pass computes h again from
// x and the residual, which the forward's caller has, so h is not read and its
// rounding is not in the gradients.
//
// keep of element i = token * N + channel: word i % 4 of Philox4x32-10 (Salmon,
// Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) at
// the counter (i / 4, rng[2], rng[3]) under the key rng[0], rng[1], compared
// with floor(p * 2^32): a function of the element alone, so the mask is the
// same in both passes and on every layout, and is never stored.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "heads_sm103.cuh"
#include "row_operands.h"

namespace dt {
namespace {

// CTAs of a backward launch at most, and so rows of each of its sums in the
// workspace: few channels need more CTAs to fill an SM.
inline int max_backward_blocks(int64_t n) { return n > 2048 ? 320 : n > 1024 ? 640 : 1280; }

struct BlockArgs {
  RowTable x, r, h, y;    // forward: h and y are written; backward: they are dh and dy
  RowTable dx, dr;        // backward
  const void *post, *gate, *pre;
  void *dpost, *dgate, *dpre;
  int32_t post_dtype, gate_dtype, pre_dtype, dpost_dtype, dgate_dtype, dpre_dtype;
  const int32_t* rng;     // NULL: no dropout
  uint32_t drop_below;    // words below this are dropped
  float drop_scale;       // 1 / (1 - p)
  float eps, scale;
  int64_t tokens;
  int32_t n;
  int64_t gate_rows, gate_per;  // rows of the gate, consecutive tokens of each
  // backward: sums per CTA, [CTA][n] for pre and post, [CTA + gate row][n] for the gate
  float *part_pre, *part_post, *part_gate;
  int32_t grid;
};

// The launch's tables of row blocks; most launches need few.
template <int CAP>
struct BlockParams : BlockArgs {
  static constexpr int kCap = CAP;
  RowBlock blocks[CAP];
};
using BlockSmall = BlockParams<40>;
using BlockLarge = BlockParams<6 * DT_MAX_SLOTS>;

__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  return dtype == DT_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == DT_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

// Philox4x32-10: the four words of counter (lo, hi, c2, c3) under key (k0, k1).
__device__ __forceinline__ uint4 philox(uint64_t counter, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
  uint4 c = make_uint4((uint32_t)counter, (uint32_t)(counter >> 32), c2, c3);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  return c;
}

// K sums over a CTA's threads, in an order fixed by its size; the same in
// every thread.  `buf` alternates between two halves, so one barrier is enough.
template <int K, int THREADS>
struct CtaSum {
  float (*buf)[K][THREADS / 32];
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[K]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      for (int o = 16; o; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      if (lane == 0) buf[turn][k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
      for (int w = 0; w < THREADS / 32; ++w) v[k] += buf[turn][k][w];
    }
    turn ^= 1;
  }
};

// ---------------------------------------------------------------- any size and alignment

constexpr int BN_ANY_THREADS = 256;

// One element a thread and step; the later passes over a row come from L1 or L2.
template <class P, bool BWD>
__global__ void __launch_bounds__(BN_ANY_THREADS) block_norm_any_kernel(const __grid_constant__ P p) {
  __shared__ float buf[2][5][BN_ANY_THREADS / 32];
  wait_for_previous_kernel();
  CtaSum<5, BN_ANY_THREADS> cta_sum{buf};
  const int n = p.n;
  const float inv_n = 1.f / (float)n;
  uint32_t rng[4] = {0, 0, 0, 0};
  if (p.rng)
    for (int i = 0; i < 4; ++i) rng[i] = (uint32_t)load_plain(p.rng + i);
  // forward: tokens one after the other over the CTAs; backward: a run of consecutive tokens per CTA
  const int64_t t0 = BWD ? (int64_t)blockIdx.x * p.tokens / gridDim.x : blockIdx.x;
  const int64_t t1 = BWD ? (int64_t)(blockIdx.x + 1) * p.tokens / gridDim.x : p.tokens;
  int ax = 0, ar = 0, ah = 0, ay = 0, adx = 0, adr = 0;
  for (int64_t t = t0; t < t1; t += BWD ? 1 : gridDim.x) {
    const int bx = row_block(p.blocks, p.x, t, ax);
    const int64_t seg = p.gate ? t / p.gate_per : 0;
    const RowBlock* none = nullptr;
    auto at = [&](const RowTable& r, int& a) { return r.count ? &p.blocks[row_block(p.blocks, r, t, a)] : none; };
    const RowBlock *R = at(p.r, ar), *H = at(p.h, ah), *Y = at(p.y, ay);
    const int ex = p.x.dtype == DT_BF16 ? 2 : 4, er = p.r.dtype == DT_BF16 ? 2 : 4, eh = p.h.dtype == DT_BF16 ? 2 : 4;
    const char* r = R ? row_at(*R, t, er) : nullptr;
    char *h = H ? row_at(*H, t, eh) : nullptr, *y = Y ? row_at(*Y, t, ex) : nullptr;
    auto sum_x = [&](int c) {
      float s = 0.f;
      for (int k = 0; k < p.x.parts; ++k) {
        const float v = load_any(row_at(p.blocks[bx + k * p.x.count], t, ex), p.x.dtype, c);
        s = k ? s + v : v;
      }
      return s;
    };
    auto kept = [&](int c) {
      if (!p.rng) return true;
      const uint64_t i = (uint64_t)t * n + c;
      const uint4 w = philox(i >> 2, rng[2], rng[3], rng[0], rng[1]);
      const int j = (int)(i & 3);
      return (j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w) >= p.drop_below;
    };
    auto post = [&](int c) { return p.post ? load_any(p.post, p.post_dtype, c) : 1.f; };
    auto gate = [&](int c) { return p.gate ? load_any(p.gate, p.gate_dtype, seg * n + c) : 1.f; };
    auto pre = [&](int c) { return load_any(p.pre, p.pre_dtype, c); };
    float rx = 1.f, rh = 1.f;
    if (p.post) {
      float v[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = threadIdx.x; c < n; c += BN_ANY_THREADS) {
        const float s = sum_x(c);
        v[0] += s * s;
      }
      cta_sum(v);
      rx = rsqrtf(v[0] * inv_n + p.eps);
    }
    auto value = [&](int c, float s, bool keep) {  // h
      const float f = keep ? s * rx * post(c) * gate(c) * p.drop_scale : 0.f;
      return r ? fmaf(p.scale, load_any(r, p.r.dtype, c), f) : f;
    };
    if (!BWD) {
      if (p.pre) {
        float v[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
        for (int c = threadIdx.x; c < n; c += BN_ANY_THREADS) {
          const float a = value(c, sum_x(c), kept(c));
          v[0] += a * a;
        }
        cta_sum(v);
        rh = rsqrtf(v[0] * inv_n + p.eps);
      }
      for (int c = threadIdx.x; c < n; c += BN_ANY_THREADS) {
        const float a = value(c, sum_x(c), kept(c));
        if (h) store_any(h, p.h.dtype, c, a);
        if (y) store_any(y, p.y.dtype, c, a * rh * pre(c));
      }
      continue;
    }
    float kh = 0.f, kx = 0.f;  // r(h)^3 m(h z), r(s)^3 m(s v)
    auto grad = [&](int c, float a) {  // g, for a value a of h
      const float z = y ? load_any(y, p.y.dtype, c) * pre(c) : 0.f;
      return (h ? load_any(h, p.h.dtype, c) : 0.f) + rh * z - kh * a;
    };
    if (p.pre) {
      float v[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = threadIdx.x; c < n; c += BN_ANY_THREADS) {
        const float a = value(c, sum_x(c), kept(c));
        v[0] += a * a;
        v[1] += a * load_any(y, p.y.dtype, c) * pre(c);
      }
      cta_sum(v);
      rh = rsqrtf(v[0] * inv_n + p.eps);
      kh = rh * rh * rh * (v[1] * inv_n);
    }
    if (p.post) {
      float v[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = threadIdx.x; c < n; c += BN_ANY_THREADS) {
        const float s = sum_x(c);
        const bool keep = kept(c);
        if (keep) v[0] += s * grad(c, value(c, s, true)) * p.drop_scale * gate(c) * post(c);
      }
      cta_sum(v);
      kx = rx * rx * rx * (v[0] * inv_n);
    }
    const RowBlock *DX = at(p.dx, adx), *DR = at(p.dr, adr);
    char *dx = DX ? row_at(*DX, t, ex) : nullptr, *dr = DR ? row_at(*DR, t, er) : nullptr;
    const bool first = t == t0, first_gate = first || t % p.gate_per == 0;
    for (int c = threadIdx.x; c < n; c += BN_ANY_THREADS) {
      const float s = sum_x(c);
      const bool keep = kept(c);
      const float a = value(c, s, keep), g = grad(c, a);
      if (dr) store_any(dr, p.dr.dtype, c, p.scale * g);
      auto add = [&](float* to, bool begin, float v) { *to = begin ? v : *to + v; };
      if (p.pre) add(p.part_pre + (int64_t)blockIdx.x * n + c, first, load_any(y, p.y.dtype, c) * a * rh);
      const float e = keep ? g * p.drop_scale : 0.f, w = e * gate(c);
      if (p.gate) {
        const float d = keep ? e * s * rx * post(c) : 0.f;
        if (p.gate_per == 1) store_any(p.dgate, p.dgate_dtype, t * n + c, d);
        else add(p.part_gate + ((int64_t)blockIdx.x + seg) * n + c, first_gate, d);
      }
      if (p.post) add(p.part_post + (int64_t)blockIdx.x * n + c, first, keep ? w * s * rx : 0.f);
      if (dx) store_any(dx, p.dx.dtype, c, p.post ? rx * w * post(c) - kx * s : w);
    }
  }
}

// dpre, dpost and the gate's rows from the CTAs' sums: 32 channels a block,
// each warp every 32nd CTA's, then the warps'; a fixed order.
constexpr int BN_SUM_THREADS = 1024;
__global__ void __launch_bounds__(BN_SUM_THREADS) block_norm_sums_kernel(const __grid_constant__ BlockArgs p) {
  __shared__ float acc[32][33];
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = p.gate && p.gate_per != 1 ? p.gate_rows : 0;
  for (int64_t which = blockIdx.y; which < 2 + rows; which += gridDim.y) {
    void* out = which == 0 ? p.dpre : which == 1 ? p.dpost : p.dgate;
    if (!out) continue;
    const int dtype = which == 0 ? p.dpre_dtype : which == 1 ? p.dpost_dtype : p.dgate_dtype;
    const float* part = which == 0 ? p.part_pre : which == 1 ? p.part_post : p.part_gate;
    int64_t b0 = 0, b1 = p.tokens ? p.grid : 0, row = 0;
    if (which >= 2) {  // the CTAs that hold tokens of this row, and their sums' places
      row = which - 2;
      if (p.tokens) {
        b0 = ((row * p.gate_per + 1) * p.grid - 1) / p.tokens + row;
        b1 = ((row + 1) * p.gate_per * p.grid - 1) / p.tokens + 1 + row;
      }
    }
    int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < p.n) {
#pragma unroll 4
      for (int64_t b = b0 + warp; b < b1; b += 32) s += part[b * p.n + c];
    }
    acc[warp][lane] = s;
    __syncthreads();
    s = acc[lane][warp];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    c = (int64_t)blockIdx.x * 32 + warp;
    if (lane == 0 && c < p.n) store_any(out, dtype, row * p.n + c, s);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- channels in vectors of 8

// Rows of a multiple of 8 channels on 16-byte boundaries: a CTA per row, a
// thread holds VPT vectors of 8 channels of it, `blockDim.x` vectors apart.
constexpr int row_threads(int vpt) { return vpt == 1 ? 1024 : 512; }

// The sum over a CTA, in an order fixed by its size; the same in every thread.
// `buf` [2][K][32] is zero behind the CTA's warps.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*buf)[K][32], int& turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (lane == 0 && warps > 1) buf[turn][k][warp] = v[k];
  }
  if (warps == 1) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = 0.f;
    for (int w = 0; w < warps; w += 4) {
      const float4 x = *reinterpret_cast<const float4*>(&buf[turn][k][w]);
      v[k] += (x.x + x.y) + (x.z + x.w);
    }
  }
  turn ^= 1;
}
template <int K>
__device__ __forceinline__ void clear_sums(float (*buf)[K][32]) {
  for (int i = threadIdx.x; i < 2 * K * 32; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
  __syncthreads();
}

// 8 channels of a vector over channels (bf16 or fp32, 16-byte aligned).
__device__ __forceinline__ void load_w8(const void* w, int dtype, int64_t c, f2 (&v)[4]) {
  if (dtype == DT_BF16) {
    Raw8<__nv_bfloat16> x;
    x.u = load_plain(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c));
    x.get2(v);
  } else {
    Raw8<float> x;
    x.load_keep(static_cast<const float*>(w) + c);
    x.get2(v);
  }
}

// Dropout of 8 channels from channel c of token t: bit i keeps channel c + i.
struct Dropout {
  uint32_t key[4], below;
  bool on;
  __device__ __forceinline__ explicit Dropout(const BlockArgs& p) : below(p.drop_below), on(p.rng != nullptr) {
    for (int i = 0; i < 4; ++i) key[i] = on ? (uint32_t)load_plain(p.rng + i) : 0;
  }
  __device__ __forceinline__ uint32_t bits(int64_t t, int n, int c) const {
    const uint64_t i = ((uint64_t)t * n + c) >> 2;
    const uint4 a = philox(i, key[2], key[3], key[0], key[1]), b = philox(i + 1, key[2], key[3], key[0], key[1]);
    return (a.x >= below) | (a.y >= below) << 1 | (a.z >= below) << 2 | (a.w >= below) << 3 | (b.x >= below) << 4 |
           (b.y >= below) << 5 | (b.z >= below) << 6 | (b.w >= below) << 7;
  }
};
__device__ __forceinline__ f2 kept(f2 v, uint32_t bits, int i, float scale) {  // pair i of the 8
  return f2{bits >> (2 * i) & 1 ? v.x * scale : 0.f, bits >> (2 * i + 1) & 1 ? v.y * scale : 0.f};
}

template <class T>
struct Pieces {
  static constexpr int N = sizeof(T) / 2;  // 16-byte pieces of 8 elements
};
// A row's vector into a stage of the ring (`to`: this thread's first piece, `step` apart).
template <class T>
__device__ __forceinline__ void fetch8(uint4* to, const char* row, int c, int step) {
  const T* from = reinterpret_cast<const T*>(row) + c;
#pragma unroll
  for (int i = 0; i < Pieces<T>::N; ++i) copy16_async(to + i * step, reinterpret_cast<const uint4*>(from) + i);
}

// RING: x (one part) and the residual come through a ring of asynchronous
// copies of STAGES rows, each thread its own pieces, so that the next rows are
// on their way without taking registers or barriers.  Else (parts to be added,
// rows too large for a ring) plain loads, all of a row at once.
constexpr int BN_STAGES = 3;

template <class XT, class RT, int VPT, bool RING, class P>
__global__ void __launch_bounds__(row_threads(VPT), VPT == 2 ? 2 : 1) block_norm_row_kernel(const __grid_constant__ P p) {
  __shared__ __align__(16) float buf[2][1][32];
  extern __shared__ uint4 ring[];
  wait_for_previous_kernel();
  clear_sums(buf);
  int turn = 0;
  const int n = p.n, nt = blockDim.x, tid = threadIdx.x;
  const float inv_n = 1.f / (float)n;
  const Dropout drop(p);
  constexpr int PX = Pieces<XT>::N, PR = Pieces<RT>::N, PIECES = VPT * (PX + PR);
  const bool res = p.r.count > 0, out_h = p.h.count > 0, out_y = p.y.count > 0;
  int ax = 0, ar = 0, ah = 0, ay = 0;
  auto channel = [&](int v) { return (v * nt + tid) * 8; };
  uint4* const mine = ring + tid;
  int put = 0, get = 0;
  auto fetch = [&](int64_t t) {
    if (t < p.tokens) {
      const char* x = row_at(p.blocks[row_block(p.blocks, p.x, t, ax)], t, sizeof(XT));
      const char* r = res ? row_at(p.blocks[row_block(p.blocks, p.r, t, ar)], t, sizeof(RT)) : nullptr;
      uint4* to = mine + put * PIECES * nt;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = channel(v);
        if (c >= n) break;
        fetch8<XT>(to + v * PX * nt, x, c, nt);
        if (res) fetch8<RT>(to + (VPT * PX + v * PR) * nt, r, c, nt);
      }
    }
    copies_commit();
    if (++put == BN_STAGES) put = 0;
  };
  if (RING)
    for (int i = 0; i + 1 < BN_STAGES; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x);
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    f2 u[VPT][4], h[VPT][4];
    Raw8<RT> r[VPT];
    if constexpr (RING) {
      fetch(t + (int64_t)(BN_STAGES - 1) * gridDim.x);
      copies_wait<BN_STAGES - 1>();
      const uint4* from = mine + get * PIECES * nt;
      if (++get == BN_STAGES) get = 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        Raw8<XT> x;
        x.zero(), r[v].zero();
        if (channel(v) < n) {
          x.set(from + v * PX * nt, nt);
          if (res) r[v].set(from + (VPT * PX + v * PR) * nt, nt);
        }
        x.get2(u[v]);
      }
    } else {
      const int bx = row_block(p.blocks, p.x, t, ax);
      const char* rr = res ? row_at(p.blocks[row_block(p.blocks, p.r, t, ar)], t, sizeof(RT)) : nullptr;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        r[v].zero();
        if (res && channel(v) < n) r[v].load(reinterpret_cast<const RT*>(rr) + channel(v));
#pragma unroll
        for (int i = 0; i < 4; ++i) u[v][i] = both(0.f);
      }
#pragma unroll 4
      for (int k = 0; k < p.x.parts; ++k) {
        const XT* x = reinterpret_cast<const XT*>(row_at(p.blocks[bx + k * p.x.count], t, sizeof(XT)));
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          Raw8<XT> w;
          w.zero();
          if (channel(v) < n) w.load(x + channel(v));
          f2 s[4];
          w.get2(s);
#pragma unroll
          for (int i = 0; i < 4; ++i) u[v][i] = u[v][i] + s[i];
        }
      }
    }
    float sum[1];
    auto total = [&](const f2(&a)[VPT][4]) {
      f2 s = both(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(a[v][i], a[v][i], s);
      sum[0] = s.x + s.y;
      row_sum(sum, buf, turn);
      return rsqrtf(sum[0] * inv_n + p.eps);
    };
    const float rx = p.post ? total(u) : 1.f;
    const int64_t seg = p.gate ? (uint32_t)t / (uint32_t)p.gate_per : 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = channel(v);
      if (c < n) {
        f2 w[4];
        if (p.post) {
          load_w8(p.post, p.post_dtype, c, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) u[v][i] = u[v][i] * both(rx) * w[i];
        }
        if (p.gate) {
          load_w8(p.gate, p.gate_dtype, seg * n + c, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) u[v][i] = u[v][i] * w[i];
        }
        if (drop.on) {
          const uint32_t bits = drop.bits(t, n, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) u[v][i] = kept(u[v][i], bits, i, p.drop_scale);
        }
      }
      r[v].get2(h[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[v][i] = res ? fma2(both(p.scale), h[v][i], u[v][i]) : u[v][i];
    }
    if (out_h) {
      RT* o = reinterpret_cast<RT*>(row_at(p.blocks[row_block(p.blocks, p.h, t, ah)], t, sizeof(RT)));
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (channel(v) < n) store8(o + channel(v), h[v]);
    }
    if (out_y) {
      const float rh = total(h);
      XT* o = reinterpret_cast<XT*>(row_at(p.blocks[row_block(p.blocks, p.y, t, ay)], t, sizeof(XT)));
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = channel(v);
        if (c >= n) break;
        f2 w[4];
        load_w8(p.pre, p.pre_dtype, c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = h[v][i] * both(rh) * w[i];
        store8(o + c, w);
      }
    }
  }
  if (RING) copies_wait<0>();
}

// Gradients.  A CTA takes a run of consecutive tokens and keeps the sums over
// them in registers; x, the residual, dh and dy come through the ring and are
// read from it twice, before and after the means, instead of being held.  The
// means' sums are taken at once: with a = gate post keep x / (1 - p), h =
// scale residual + r(x) a and g = dh + r(h) z - k h, the sum of a g is that of
// a dh, a z and a h, so one meeting of the CTA does after that of r(x).
constexpr int bwd_stages(int pieces) { return pieces > 8 ? 2 : 3; }

template <class XT, class RT, int VPT, class P>
__global__ void __launch_bounds__(VPT == 1 ? 256 : 512, VPT == 1 ? 2 : 1)
    block_norm_row_backward_kernel(const __grid_constant__ P p) {
  __shared__ __align__(16) float buf[2][5][32];
  extern __shared__ uint4 ring[];
  wait_for_previous_kernel();
  clear_sums(buf);
  int turn = 0;
  const int n = p.n, nt = blockDim.x, tid = threadIdx.x;
  const float inv_n = 1.f / (float)n;
  const Dropout drop(p);
  constexpr int PX = Pieces<XT>::N, PR = Pieces<RT>::N, PIECES = 2 * VPT * (PX + PR);
  constexpr int STAGES = bwd_stages(PIECES / VPT);
  const bool res = p.r.count > 0, has_h = p.h.count > 0, has_y = p.y.count > 0;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens / gridDim.x, t1 = (int64_t)(blockIdx.x + 1) * p.tokens / gridDim.x;
  int ax = 0, ar = 0, ah = 0, ay = 0, adx = 0, adr = 0;
  auto channel = [&](int v) { return (v * nt + tid) * 8; };
  uint4* const mine = ring + tid;
  int put = 0, get = 0;
  auto fetch = [&](int64_t t) {
    if (t < t1) {
      auto row = [&](const RowTable& r, int& a, int es) {
        return r.count ? row_at(p.blocks[row_block(p.blocks, r, t, a)], t, es) : nullptr;
      };
      const char *x = row(p.x, ax, sizeof(XT)), *r = row(p.r, ar, sizeof(RT)), *h = row(p.h, ah, sizeof(RT)),
                 *y = row(p.y, ay, sizeof(XT));
      uint4* to = mine + put * PIECES * nt;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = channel(v);
        if (c >= n) break;
        fetch8<XT>(to + v * PX * nt, x, c, nt);
        if (has_y) fetch8<XT>(to + (VPT + v) * PX * nt, y, c, nt);
        if (res) fetch8<RT>(to + (2 * VPT * PX + v * PR) * nt, r, c, nt);
        if (has_h) fetch8<RT>(to + (2 * VPT * PX + (VPT + v) * PR) * nt, h, c, nt);
      }
    }
    copies_commit();
    if (++put == STAGES) put = 0;
  };
  for (int i = 0; i + 1 < STAGES; ++i) fetch(t0 + i);
  f2 s_pre[VPT][4], s_post[VPT][4], s_gate[VPT][4];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_pre[v][i] = s_post[v][i] = s_gate[v][i] = both(0.f);
  auto write_sums = [&](float* to, const f2(&s)[VPT][4]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (channel(v) < n) {
        float4* o = reinterpret_cast<float4*>(to + channel(v));
        o[0] = make_float4(s[v][0].x, s[v][0].y, s[v][1].x, s[v][1].y);
        o[1] = make_float4(s[v][2].x, s[v][2].y, s[v][3].x, s[v][3].y);
      }
  };
  int64_t seg = p.gate ? (uint32_t)t0 / (uint32_t)p.gate_per : 0, seg_end = (seg + 1) * p.gate_per;
  for (int64_t t = t0; t < t1; ++t) {
    fetch(t + STAGES - 1);
    copies_wait<STAGES - 1>();
    const uint4* from = mine + get * PIECES * nt;
    if (++get == STAGES) get = 0;
    if (t == seg_end) {
      ++seg;
      seg_end += p.gate_per;
    }
    auto load_x = [&](int v, f2(&x)[4]) {
      Raw8<XT> w;
      w.set(from + v * PX * nt, nt);
      w.get2(x);
    };
    float rx = 1.f, rh = 1.f, kh = 0.f, kx = 0.f;
    if (p.post) {
      f2 s = both(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (channel(v) >= n) break;
        f2 x[4];
        load_x(v, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(x[i], x[i], s);
      }
      float sum[5] = {s.x + s.y, 0.f, 0.f, 0.f, 0.f};
      row_sum(sum, buf, turn);
      rx = rsqrtf(sum[0] * inv_n + p.eps);
    }
    uint32_t bits[VPT];
    // a vector's x, a, h, z and dh
    auto values = [&](int v, f2(&x)[4], f2(&a)[4], f2(&h)[4], f2(&z)[4], f2(&dy)[4], f2(&dh)[4], f2(&post)[4],
                      f2(&gate)[4]) {
      const int c = channel(v);
      load_x(v, x);
      if (p.post) load_w8(p.post, p.post_dtype, c, post);
      if (p.gate) load_w8(p.gate, p.gate_dtype, seg * n + c, gate);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = x[i];
        if (p.post) a[i] = a[i] * post[i];
        if (p.gate) a[i] = a[i] * gate[i];
        if (drop.on) a[i] = kept(a[i], bits[v], i, p.drop_scale);
      }
      if (res) {
        Raw8<RT> w;
        w.set(from + (2 * VPT * PX + v * PR) * nt, nt);
        w.get2(h);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 f = a[i] * both(rx);
        h[i] = res ? fma2(both(p.scale), h[i], f) : f;
        dh[i] = dy[i] = z[i] = both(0.f);
      }
      if (has_h) {
        Raw8<RT> w;
        w.set(from + (2 * VPT * PX + (VPT + v) * PR) * nt, nt);
        w.get2(dh);
      }
      if (has_y) {
        Raw8<XT> w;
        w.set(from + (VPT + v) * PX * nt, nt);
        w.get2(dy);
        load_w8(p.pre, p.pre_dtype, c, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = z[i] * dy[i];
      }
    };
    f2 q[5] = {both(0.f), both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (channel(v) >= n) break;
      if (drop.on) bits[v] = drop.bits(t, n, channel(v));
      if (!has_y && !p.post) continue;
      f2 x[4], a[4], h[4], z[4], dy[4], dh[4], post[4], gate[4];
      values(v, x, a, h, z, dy, dh, post, gate);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[0] = fma2(h[i], h[i], q[0]);
        q[1] = fma2(h[i], z[i], q[1]);
        q[2] = fma2(a[i], dh[i], q[2]);
        q[3] = fma2(a[i], z[i], q[3]);
        q[4] = fma2(a[i], h[i], q[4]);
      }
    }
    if (has_y || p.post) {
      float sum[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) sum[i] = q[i].x + q[i].y;
      row_sum(sum, buf, turn);
      if (has_y) {
        rh = rsqrtf(sum[0] * inv_n + p.eps);
        kh = rh * rh * rh * (sum[1] * inv_n);
      }
      kx = p.post ? rx * rx * rx * ((sum[2] + rh * sum[3] - kh * sum[4]) * inv_n) : 0.f;
    }
    char* dx = p.dx.count ? row_at(p.blocks[row_block(p.blocks, p.dx, t, adx)], t, sizeof(XT)) : nullptr;
    char* dr = p.dr.count ? row_at(p.blocks[row_block(p.blocks, p.dr, t, adr)], t, sizeof(RT)) : nullptr;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = channel(v);
      if (c >= n) break;
      f2 x[4], a[4], h[4], z[4], dy[4], dh[4], post[4], gate[4];
      values(v, x, a, h, z, dy, dh, post, gate);
      f2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2 g = dh[i];
        if (has_y) {
          g = fma2(z[i], both(rh), fma2(h[i], both(-kh), g));
          s_pre[v][i] = fma2(dy[i], h[i] * both(rh), s_pre[v][i]);
        }
        dh[i] = g * both(p.scale);
        const f2 e = drop.on ? kept(g, bits[v], i, p.drop_scale) : g;
        f2 xr = p.post ? x[i] * both(rx) : x[i];
        if (drop.on) xr = kept(xr, bits[v], i, 1.f);  // (what is dropped may be NaN)
        f2 w = e;
        if (p.gate) {
          a[i] = e * (p.post ? xr * post[i] : xr);
          s_gate[v][i] = s_gate[v][i] + a[i];
          w = e * gate[i];
        }
        if (p.post) {
          s_post[v][i] = fma2(w, xr, s_post[v][i]);
          o[i] = fma2(w * post[i], both(rx), x[i] * both(-kx));
        } else {
          o[i] = w;
        }
      }
      if (dr) store8(reinterpret_cast<RT*>(dr) + c, dh);
      if (dx) store8(reinterpret_cast<XT*>(dx) + c, o);
      if (p.gate && p.gate_per == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          store_any(p.dgate, p.dgate_dtype, t * n + c + 2 * i, a[i].x);
          store_any(p.dgate, p.dgate_dtype, t * n + c + 2 * i + 1, a[i].y);
        }
      }
    }
    if (p.gate && p.gate_per != 1 && (t + 1 == t1 || t + 1 == seg_end)) {
      write_sums(p.part_gate + ((int64_t)blockIdx.x + seg) * n, s_gate);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_gate[v][i] = both(0.f);
    }
  }
  if (p.pre) write_sums(p.part_pre + (int64_t)blockIdx.x * n, s_pre);
  if (p.post) write_sums(p.part_post + (int64_t)blockIdx.x * n, s_post);
  copies_wait<0>();
}

// ---------------------------------------------------------------- host

struct BlockCall {
  const dt_dtensor *x, *residual, *post, *gate, *pre, *rng;
  const dt_dtensor *h, *y;                              // outputs; backward: their gradients
  const dt_dtensor *dx, *dresidual, *dpost, *dgate, *dpre;  // backward
  float eps, scale, dropout;
  int32_t tp;
};

dt_status channel_vector(const dt_dtensor* w, const char* what, const Layout& of, int64_t n, bool output,
                         const void** ptr, int32_t* dtype, int64_t* rows) {
  PlainOperand o;
  dt_status st = plain_operand(w, what, of, output, &o);
  if (st != DT_OK) return st;
  if (o.shape[o.ndim - 1] != n || (!rows && o.ndim != 1))
    return fail(DT_ERR_SHAPE, "%s must be %s", what, rows ? "[channels] or [..., channels]" : "[channels]");
  if (o.dtype != DT_BF16 && o.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "%s must be bf16 or fp32", what);
  *ptr = o.ptr;
  *dtype = o.dtype;
  if (rows) {
    *rows = 1;
    for (int d = 0; d + 1 < o.ndim; ++d) *rows *= o.shape[d];
  }
  return DT_OK;
}

// Rows of the gate's sums in the workspace beyond one per CTA.
int64_t gate_part_rows(int64_t tokens, int64_t gate_rows) { return gate_rows == tokens ? 0 : gate_rows; }

// How a launch covers its rows.
struct Shape {
  int threads = 0, vpt = 0, grid = 0;  // vpt 0: the kernels for any size
  bool ring = false;
  size_t smem = 0;
};

int round_up(int64_t a, int b) { return (int)((a + b - 1) / b * b); }

Shape forward_shape(const BlockArgs& p, bool vec, bool small) {
  Shape s;
  const int sms = device_sm_count();
  const int64_t vectors = p.n / 8;
  if (!vec || vectors > 4 * 512) {
    s.grid = (int)std::min<int64_t>(p.tokens, (int64_t)sms * 8);
    return s;
  }
  // a vector a thread where there are few tokens (the shortest way through a
  // row) or few channels; else two, four for the widest
  s.vpt = vectors <= 256 || (p.tokens <= sms && vectors <= 1024) ? 1 : vectors <= 1024 ? 2 : 4;
  s.threads = round_up((vectors + s.vpt - 1) / s.vpt, 32);
  const size_t stage = (size_t)s.threads * s.vpt * 8 * (dtype_size(p.x.dtype) + dtype_size(p.h.dtype));
  s.ring = small && p.x.parts == 1 && stage * BN_STAGES <= 200 * 1024;
  s.smem = s.ring ? stage * BN_STAGES : 0;
  int ctas = std::max(1, std::min(32, 1024 / s.threads));
  if (s.ring) ctas = std::max(1, std::min<int>(ctas, (int)(220 * 1024 / (s.smem + 1280))));
  s.grid = (int)std::min<int64_t>(p.tokens, (int64_t)sms * ctas);
  return s;
}

Shape backward_shape(const BlockArgs& p, bool vec, bool small) {
  Shape s;
  const int sms = device_sm_count();
  const int64_t vectors = p.n / 8;
  int64_t most = 2 * sms;
  const int pieces = 2 * (dtype_size(p.x.dtype) + dtype_size(p.h.dtype)) / 2;  // 16-byte pieces of a vector
  if (vec && small && p.x.parts == 1 && vectors <= 1024) {
    s.vpt = vectors <= 256 ? 1 : 2;
    s.threads = round_up((vectors + s.vpt - 1) / s.vpt, 32);
    s.smem = (size_t)s.threads * s.vpt * pieces * 16 * bwd_stages(pieces);
    s.ring = true;
    if (s.smem > 220 * 1024) s = Shape();
    else most = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(512 / s.threads, 220 * 1024 / (s.smem + 2048)), 8)) * sms;
  }
  // four tokens a CTA at least, for its sums are written and read again
  most = std::min<int64_t>(most, std::max<int64_t>(sms, (p.tokens + 3) / 4));
  s.grid = (int)std::max<int64_t>(1, std::min<int64_t>({p.tokens, most, max_backward_blocks(p.n)}));
  return s;
}

template <class K, class P>
cudaError_t launch_rows(K kernel, const P& p, const Shape& s, cudaStream_t stream) {
  if (s.smem > 40 * 1024)
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s.smem)) return e;
  return launch_early(kernel, dim3(s.grid), s.threads, s.smem, stream, p);
}

template <class XT, class RT, class P>
cudaError_t launch_typed(const P& p, bool bwd, const Shape& s, cudaStream_t stream) {
  constexpr bool SMALL = P::kCap == BlockSmall::kCap;
  if constexpr (SMALL) {
    if (bwd)
      return s.vpt == 1 ? launch_rows(block_norm_row_backward_kernel<XT, RT, 1, P>, p, s, stream)
                        : launch_rows(block_norm_row_backward_kernel<XT, RT, 2, P>, p, s, stream);
    if (s.ring)
      return s.vpt == 1   ? launch_rows(block_norm_row_kernel<XT, RT, 1, true, P>, p, s, stream)
             : s.vpt == 2 ? launch_rows(block_norm_row_kernel<XT, RT, 2, true, P>, p, s, stream)
                          : launch_rows(block_norm_row_kernel<XT, RT, 4, true, P>, p, s, stream);
  }
  return s.vpt == 1   ? launch_rows(block_norm_row_kernel<XT, RT, 1, false, P>, p, s, stream)
         : s.vpt == 2 ? launch_rows(block_norm_row_kernel<XT, RT, 2, false, P>, p, s, stream)
                      : launch_rows(block_norm_row_kernel<XT, RT, 4, false, P>, p, s, stream);
}

template <class P>
cudaError_t launch_block(const P& p, bool bwd, const Shape& s, cudaStream_t stream) {
  if (!s.vpt)
    return bwd ? launch_early(block_norm_any_kernel<P, true>, dim3(s.grid), BN_ANY_THREADS, 0, stream, p)
               : launch_early(block_norm_any_kernel<P, false>, dim3(s.grid), BN_ANY_THREADS, 0, stream, p);
  if (p.x.dtype == DT_FP32) return launch_typed<float, float>(p, bwd, s, stream);
  if (p.h.dtype == DT_FP32) return launch_typed<__nv_bfloat16, float>(p, bwd, s, stream);
  return launch_typed<__nv_bfloat16, __nv_bfloat16>(p, bwd, s, stream);
}

dt_status block_call(bool bwd, const BlockCall& A, void* ws, size_t ws_bytes, int32_t* d_status, cudaStream_t stream) {
  clear_error();
  if (!(A.eps >= 0.f) || A.eps > 1.f) return fail(DT_ERR_INVALID_ARG, "eps must be in [0, 1]");
  if (!(A.dropout >= 0.f) || !(A.dropout < 1.f)) return fail(DT_ERR_INVALID_ARG, "dropout must be in [0, 1)");
  if (!std::isfinite(A.scale)) return fail(DT_ERR_INVALID_ARG, "residual_scale must be finite");
  if (!A.x) return fail(DT_ERR_INVALID_ARG, "x is NULL");
  if (A.dropout > 0.f && !A.rng) return fail(DT_ERR_INVALID_ARG, "dropout needs rng");
  if (!bwd && (A.pre != nullptr) != (A.y != nullptr)) return fail(DT_ERR_INVALID_ARG, "pre_weight and y go together");
  if (!A.h && !A.y) return fail(DT_ERR_INVALID_ARG, bwd ? "neither dh nor dy" : "neither h nor y");
  if (bwd) {
    if ((A.pre != nullptr) != (A.y != nullptr)) return fail(DT_ERR_INVALID_ARG, "pre_weight and dy go together");
    if ((A.pre != nullptr) != (A.dpre != nullptr))
      return fail(DT_ERR_INVALID_ARG, "pre_weight and dpre_weight go together");
    if ((A.post != nullptr) != (A.dpost != nullptr))
      return fail(DT_ERR_INVALID_ARG, "post_weight and dpost_weight go together");
    if ((A.gate != nullptr) != (A.dgate != nullptr)) return fail(DT_ERR_INVALID_ARG, "gate and dgate go together");
    if (A.dresidual && !A.residual) return fail(DT_ERR_INVALID_ARG, "dresidual without a residual");
  }
  static thread_local BlockLarge p;
  static_cast<BlockArgs&>(p) = BlockArgs{};
  dt_status st;
  Layout lx, lo;
  int used = 0;
  RowOperand X;
  const void* anchor = nullptr;  // something that the call writes
  bool vec = true;
  auto add = [&](const RowOperand& o, RowTable* t) {
    *t = RowTable{(int16_t)used, (int16_t)o.count, (int16_t)o.parts, (int16_t)o.dtype};
    std::copy(o.block, o.block + o.count * o.parts, p.blocks + used);
    used += o.count * o.parts;
    vec = vec && o.vec16;
  };
  if ((st = row_operand(A.x, "x", A.tp, false, true, &X, &lx)) != DT_OK) return st;
  add(X, &p.x);
  // the others: of x's shape; dtype of the residual stream (-1: not known yet) or of x
  int stream_dtype = -1;
  auto rows = [&](const dt_dtensor* in, const char* what, bool output, bool of_stream, RowTable* t) {
    if (!in) {
      *t = RowTable{};
      return DT_OK;
    }
    RowOperand o;
    dt_status s = row_operand(in, what, A.tp, output, false, &o, &lo);
    if (s != DT_OK) return s;
    if ((s = same_mesh(lo, lx, what)) != DT_OK) return s;
    bool shape = lo.ndim == lx.ndim;
    for (int d = 0; shape && d < lo.ndim; ++d) shape = lo.gshape[d] == lx.gshape[d];
    if (!shape) return fail(DT_ERR_SHAPE, "%s must have the shape of x", what);
    if (of_stream && stream_dtype < 0) stream_dtype = o.dtype;
    if (o.dtype != (of_stream ? stream_dtype : X.dtype))
      return fail(DT_ERR_INVALID_ARG, "%s must have the dtype of %s", what, of_stream ? "the residual stream" : "x");
    if (of_stream && X.dtype == DT_FP32 && o.dtype == DT_BF16)
      return fail(DT_ERR_UNSUPPORTED, "%s: a bf16 residual stream with fp32 x", what);
    add(o, t);
    if (output && o.count) anchor = o.block[0].ptr;
    return DT_OK;
  };
  if ((st = rows(A.residual, "residual", false, true, &p.r)) != DT_OK) return st;
  if ((st = rows(A.h, bwd ? "dh" : "h", !bwd, true, &p.h)) != DT_OK) return st;
  if ((st = rows(A.y, bwd ? "dy" : "y", !bwd, false, &p.y)) != DT_OK) return st;
  if (bwd) {
    if ((st = rows(A.dx, "dx", true, false, &p.dx)) != DT_OK) return st;
    if ((st = rows(A.dresidual, "dresidual", true, true, &p.dr)) != DT_OK) return st;
  }
  // what is not there has the type of what is like it
  for (RowTable* t : {&p.r, &p.h, &p.dr}) t->dtype = (int16_t)(stream_dtype < 0 ? X.dtype : stream_dtype);
  for (RowTable* t : {&p.y, &p.dx}) t->dtype = (int16_t)X.dtype;
  p.tokens = X.tokens;
  p.n = (int32_t)X.n;
  p.gate_rows = 1;
  const void* w = nullptr;
  if (A.post && (st = channel_vector(A.post, "post_weight", lx, X.n, false, &p.post, &p.post_dtype, nullptr)) != DT_OK)
    return st;
  if (A.pre && (st = channel_vector(A.pre, "pre_weight", lx, X.n, false, &p.pre, &p.pre_dtype, nullptr)) != DT_OK)
    return st;
  if (A.gate) {
    if ((st = channel_vector(A.gate, "gate", lx, X.n, false, &p.gate, &p.gate_dtype, &p.gate_rows)) != DT_OK) return st;
    if (p.gate_rows < 1 ? p.tokens > 0 : p.tokens % p.gate_rows != 0)
      return fail(DT_ERR_SHAPE, "gate: %lld rows for %lld tokens", (long long)p.gate_rows, (long long)p.tokens);
  }
  p.gate_per = p.gate_rows > 0 && p.tokens > 0 ? p.tokens / p.gate_rows : 1;
  if (p.tokens == 0) p.gate_per = 2;  // (no token: the gate's gradient is written by the sums)
  if (A.dpost) {
    if ((st = channel_vector(A.dpost, "dpost_weight", lx, X.n, true, &w, &p.dpost_dtype, nullptr)) != DT_OK) return st;
    p.dpost = const_cast<void*>(w);
  }
  if (A.dpre) {
    if ((st = channel_vector(A.dpre, "dpre_weight", lx, X.n, true, &w, &p.dpre_dtype, nullptr)) != DT_OK) return st;
    p.dpre = const_cast<void*>(w);
  }
  if (A.dgate) {
    int64_t r = 0;
    if ((st = channel_vector(A.dgate, "dgate", lx, X.n, true, &w, &p.dgate_dtype, &r)) != DT_OK) return st;
    if (r != p.gate_rows) return fail(DT_ERR_SHAPE, "dgate must have the rows of gate");
    p.dgate = const_cast<void*>(w);
  }
  p.drop_scale = 1.f;
  if (A.rng) {
    PlainOperand o;
    if ((st = plain_operand(A.rng, "rng", lx, false, &o)) != DT_OK) return st;
    if (o.dtype != DT_INT32 || o.numel != 4) return fail(DT_ERR_INVALID_ARG, "rng must be int32 [4]");
    if (A.dropout > 0.f) {
      p.rng = reinterpret_cast<const int32_t*>(o.ptr);
      p.drop_below = (uint32_t)((double)A.dropout * 4294967296.0);
      p.drop_scale = (float)(1.0 / (1.0 - (double)A.dropout));
    }
  }
  p.eps = A.eps;
  p.scale = A.scale;
  const bool sums = bwd && (p.dpre || p.dpost || (p.dgate && p.gate_per != 1)) && X.n > 0;
  for (const void* c : {(const void*)p.dpre, (const void*)p.dpost, (const void*)p.dgate})
    if (!anchor && sums) anchor = c;
  if (!anchor && p.dgate && X.n > 0 && p.tokens > 0) anchor = p.dgate;
  if (X.n == 0 || !anchor) return DT_OK;
  if ((st = bind_device_of(anchor)) != DT_OK) return st;
  vec = vec && X.n % 8 == 0;
  for (const void* v : {p.post, p.gate, p.pre}) vec = vec && reinterpret_cast<uintptr_t>(v) % 16 == 0;
  const bool small = used <= BlockSmall::kCap;
  const Shape shape = bwd ? backward_shape(p, vec, small) : forward_shape(p, vec, small);
  p.grid = shape.grid;
  if (sums) {
    const int64_t rows_pre = p.dpre ? p.grid : 0, rows_post = p.dpost ? p.grid : 0;
    const int64_t rows_gate = p.dgate && p.gate_per != 1 ? p.grid + p.gate_rows : 0;
    const size_t need = (size_t)(rows_pre + rows_post + rows_gate) * X.n * sizeof(float);
    if (!ws || ws_bytes < need)
      return fail(DT_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(DT_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    p.part_pre = static_cast<float*>(ws);
    p.part_post = p.part_pre + rows_pre * X.n;
    p.part_gate = p.part_post + rows_post * X.n;
  }
  cudaError_t e = cudaSuccess;
  if (p.tokens > 0) {
    if (small) {
      BlockSmall s;
      static_cast<BlockArgs&>(s) = p;
      std::copy(p.blocks, p.blocks + used, s.blocks);
      std::fill(s.blocks + used, s.blocks + BlockSmall::kCap, RowBlock{});
      e = launch_block(s, bwd, shape, stream);
    } else {
      e = launch_block(p, bwd, shape, stream);
    }
    if (e != cudaSuccess) return fail(DT_ERR_CUDA, "block_norm launch: %s", cudaGetErrorString(e));
    count_launch();
  }
  if (sums) {
    const int64_t which = 2 + (p.dgate && p.gate_per != 1 ? p.gate_rows : 0);
    e = launch_early(block_norm_sums_kernel, dim3((unsigned)((X.n + 31) / 32), (unsigned)std::min<int64_t>(which, 4096)),
                     BN_SUM_THREADS, 0, stream, static_cast<const BlockArgs&>(p));
    if (e != cudaSuccess) return fail(DT_ERR_CUDA, "block_norm sums launch: %s", cudaGetErrorString(e));
    count_launch();
  }
  return DT_OK;
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" dt_status dt_tp_block_norm(const dt_dtensor* x, const dt_dtensor* residual, const dt_dtensor* post_weight,
                                      const dt_dtensor* gate, const dt_dtensor* pre_weight, const dt_dtensor* rng,
                                      const dt_dtensor* h, const dt_dtensor* y, float eps, float residual_scale,
                                      float dropout, int32_t tp_mesh_dim, int32_t* d_status, dt_stream_t stream) {
  return no_throw([&] {
    BlockCall a{x, residual, post_weight, gate, pre_weight, rng, h, y, nullptr, nullptr, nullptr, nullptr, nullptr,
                eps, residual_scale, dropout, tp_mesh_dim};
    return block_call(false, a, nullptr, 0, d_status, reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" dt_status dt_tp_block_norm_backward(const dt_dtensor* dh, const dt_dtensor* dy, const dt_dtensor* x,
                                               const dt_dtensor* residual, const dt_dtensor* post_weight,
                                               const dt_dtensor* gate, const dt_dtensor* pre_weight,
                                               const dt_dtensor* rng, const dt_dtensor* dx, const dt_dtensor* dresidual,
                                               const dt_dtensor* dpost_weight, const dt_dtensor* dgate,
                                               const dt_dtensor* dpre_weight, float eps, float residual_scale,
                                               float dropout, int32_t tp_mesh_dim, void* workspace,
                                               size_t workspace_bytes, int32_t* d_status, dt_stream_t stream) {
  return no_throw([&] {
    BlockCall a{x, residual, post_weight, gate, pre_weight, rng, dh, dy, dx, dresidual, dpost_weight, dgate,
                dpre_weight, eps, residual_scale, dropout, tp_mesh_dim};
    return block_call(true, a, workspace, workspace_bytes, d_status, reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" dt_status dt_tp_block_norm_backward_workspace_size(int64_t tokens, int64_t channels, int64_t gate_rows,
                                                              size_t* bytes) {
  clear_error();
  if (!bytes) return fail(DT_ERR_INVALID_ARG, "bytes is NULL");
  if (tokens < 0 || channels < 0 || gate_rows < 0 || channels > (1 << 30) || tokens >= MAX_ROWS)
    return fail(DT_ERR_INVALID_ARG, "tokens %lld, channels %lld, gate_rows %lld", (long long)tokens,
                (long long)channels, (long long)gate_rows);
  if (gate_rows > std::max<int64_t>(tokens, 1)) return fail(DT_ERR_SHAPE, "more gate rows than tokens");
  *bytes = (size_t)(3 * max_backward_blocks(channels) + gate_part_rows(tokens, gate_rows)) * channels * sizeof(float);
  return DT_OK;
}
