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

// Rows of a multiple of 8 channels on 16-byte boundaries: a CTA takes a run of
// consecutive rows, one at a time; a thread holds VPT vectors of 8 channels of
// it, `blockDim.x` vectors apart.
constexpr int BN_MAX_WARPS = 32;

// The sum over a CTA, in an order fixed by its size; the same in every thread.
// `buf` is zero behind the CTA's warps.  It alternates between two halves, so
// one meeting of the CTA is enough.
__device__ __forceinline__ float row_sum(float v, float (*buf)[BN_MAX_WARPS], int& turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  if (lane == 0) buf[turn][warp] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < warps; w += 4) {
    const float4 x = *reinterpret_cast<const float4*>(&buf[turn][w]);
    v += (x.x + x.y) + (x.z + x.w);
  }
  turn ^= 1;
  return v;
}

// Eight sums over a CTA of at most 16 warps at once: the lanes split the
// values among them on the way (fifteen exchanges instead of forty), lane l
// ends up with value l / 4 of the warp, and then of the CTA.
__device__ __forceinline__ void row_sums(float (&v)[8], float (*buf)[8][16], int& turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16, k = 4; k; o >>= 1, k >>= 1) {
    const bool high = lane & o;
#pragma unroll
    for (int i = 0; i < k; ++i) {
      const float keep = high ? v[i + k] : v[i], send = high ? v[i] : v[i + k];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float x = v[0];
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  if (warps > 1) {
    if ((lane & 3) == 0) buf[turn][lane >> 2][warp] = x;
    __syncthreads();
    const float4 y = *reinterpret_cast<const float4*>(&buf[turn][lane >> 2][4 * (lane & 3)]);
    x = (y.x + y.y) + (y.z + y.w);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    turn ^= 1;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, x, 4 * i);
}
__device__ __forceinline__ void clear(float* buf, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) buf[i] = 0.f;
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
  __device__ __forceinline__ void words(int64_t t, int n, int c, uint4& a, uint4& b) const {
    const uint64_t i = ((uint64_t)t * (uint32_t)n + (uint32_t)c) >> 2;
    a = philox(i, key[2], key[3], key[0], key[1]), b = philox(i + 1, key[2], key[3], key[0], key[1]);
  }
  __device__ __forceinline__ uint32_t bits(int64_t t, int n, int c) const {
    uint4 a, b;
    words(t, n, c, a, b);
    return (a.x >= below) | (a.y >= below) << 1 | (a.z >= below) << 2 | (a.w >= below) << 3 | (b.x >= below) << 4 |
           (b.y >= below) << 5 | (b.z >= below) << 6 | (b.w >= below) << 7;
  }
};
__device__ __forceinline__ f2 kept(f2 v, uint32_t bits, int i) {  // pair i of the 8
  return f2{bits & (1u << (2 * i)) ? v.x : 0.f, bits & (2u << (2 * i)) ? v.y : 0.f};
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

// Rows of K tensors, one token after the other: all blocks are looked up again
// where one of them ends.  Steps between rows fit 31 bits (else the kernels for
// any size run).
template <int K>
struct RowCursors {
  char* ptr[K];  // NULL: no such tensor
  int32_t step[K];
  int32_t left;  // tokens from this one to the end of a block
  template <class P>
  __device__ __forceinline__ void find(const P& p, const RowTable* const (&tables)[K], int64_t t, int64_t end) {
    int64_t until = end;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const RowTable& r = *tables[k];
      ptr[k] = nullptr;
      step[k] = 0;
      if (!r.count || t >= end) continue;
      int at = 0;
      const RowBlock& b = p.blocks[row_block(p.blocks, r, t, at)];
      const int esize = r.dtype == DT_BF16 ? 2 : 4;
      ptr[k] = row_at(b, t, esize);
      step[k] = (int32_t)b.ld * esize;
      if (at + 1 < r.count) until = min(until, p.blocks[r.first + at + 1].begin);
    }
    left = (int32_t)(until - t);
  }
  // to token t, the next one
  template <class P>
  __device__ __forceinline__ void next(const P& p, const RowTable* const (&tables)[K], int64_t t, int64_t end) {
    if (--left > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) ptr[k] += step[k];
    } else if (t < end) {
      find(p, tables, t, end);
    }
  }
};

// body(w, v): v's vectors of a weight's channels; the type is looked at once, so
// that the loads of all vectors can be on their way together.
template <int VPT, class C, class F>
__device__ __forceinline__ void each_w8(const void* weight, int dtype, C&& channel, F&& body) {
  f2 w[4];
  if (dtype == DT_BF16) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      Raw8<__nv_bfloat16> x;
      x.u = load_plain(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(weight) + channel(v)));
      x.get2(w);
      body(w, v);
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      Raw8<float> x;
      x.load_keep(static_cast<const float*>(weight) + channel(v));
      x.get2(w);
      body(w, v);
    }
  }
}

// Threads of forward CTAs that an SM's registers are shared among, measured
// together with the vectors a thread at 8192 x 4096 with dropout: four vectors
// and 640 threads 51.6 us, two and 768 57.7, eight and 512 64.7.
constexpr int forward_resident(int vpt, bool ahead, int er) {
  return vpt == 1 ? 1024 : vpt == 2 ? (ahead ? 768 : 1024) : ahead ? (er == 4 ? 512 : 640) : 768;
}

// Forward.  AHEAD (x in one part): the next row's loads are on their way while
// a row is worked on, x's from where it has been unpacked, the residual's from
// where it has been added.  Else the parts' loads go out four at a time.
// Threads without a last vector load the row's first one instead and drop it.
template <class XT, class RT, int VPT, bool AHEAD, class P>
__global__ void __launch_bounds__(forward_resident(VPT, AHEAD, sizeof(RT)))
    block_norm_row_kernel(const __grid_constant__ P p) {
  __shared__ __align__(16) float buf[2][BN_MAX_WARPS];
  clear(&buf[0][0], 2 * BN_MAX_WARPS);
  int turn = 0;
  const int n = p.n, nt = blockDim.x, tid = threadIdx.x;
  const float inv_n = 1.f / (float)n;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens / gridDim.x, t1 = (int64_t)(blockIdx.x + 1) * p.tokens / gridDim.x;
  // x alone (its parts are looked up where they are read), the residual alone
  // (its loads go out later), the outputs
  const RowTable *const tx[1] = {&p.x}, *const tr[1] = {&p.r}, *const to[2] = {&p.h, &p.y};
  RowCursors<1> cx, cr;
  RowCursors<2> out;
  cx.find(p, tx, t0, t1);
  cr.find(p, tr, t0, t1);
  out.find(p, to, t0, t1);
  const int parts = p.x.parts;
  int at = 0;
  // vectors below the last two are there in every thread
  const bool last = tid + (VPT - 1) * nt < n / 8, last_but_one = tid + (VPT - 2) * nt < n / 8;
  auto has = [&](int v) { return v < VPT - 2 || (v == VPT - 1 ? last : last_but_one); };
  auto channel = [&](int v) { return has(v) ? (tid + v * nt) * 8 : 0; };
  const bool res = p.r.count > 0;
  wait_for_previous_kernel();  // (until here: parameters and shared memory alone)
  const Dropout drop(p);
  Raw8<XT> x[VPT];
  Raw8<RT> r[VPT];
  auto load_x = [&](const char* row) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) x[v].load(reinterpret_cast<const XT*>(row) + channel(v));
  };
  auto load_r = [&] {
    if (!res) return;
#pragma unroll
    for (int v = 0; v < VPT; ++v) r[v].load(reinterpret_cast<const RT*>(cr.ptr[0]) + channel(v));
  };
  if (AHEAD && t0 < t1) {
    load_x(cx.ptr[0]);
    load_r();
  }
  const int64_t seg0 = p.gate ? (uint32_t)t0 / (uint32_t)p.gate_per : 0;
  int64_t seg_end = (seg0 + 1) * p.gate_per;
  const char* gate = static_cast<const char*>(p.gate);
  const int64_t gate_step = (int64_t)n * (p.gate_dtype == DT_BF16 ? 2 : 4);
  if (gate) gate += seg0 * gate_step;
  // a vector a thread: its weights stay in registers
  constexpr bool KEEP = VPT == 1;
  f2 w_post[4], w_gate[4], w_pre[4];
  if (KEEP) {
    if (p.post) load_w8(p.post, p.post_dtype, channel(0), w_post);
    if (gate) load_w8(gate, p.gate_dtype, channel(0), w_gate);
    if (p.pre) load_w8(p.pre, p.pre_dtype, channel(0), w_pre);
  }
  auto weigh = [&](const void* weight, int dtype, const f2(&w)[4], auto&& body) {
    if constexpr (KEEP) body(w, 0);
    else each_w8<VPT>(weight, dtype, channel, body);
  };
  for (int64_t t = t0; t < t1; ++t) {
    f2 h[VPT][4];
    auto unpack = [&](int v, f2(&w)[4]) {
      x[v].get2(w);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = has(v) ? w[i] : both(0.f);
    };
    if constexpr (AHEAD) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) unpack(v, h[v]);
      if (t + 1 < t1) {
        cx.next(p, tx, t + 1, t1);
        load_x(cx.ptr[0]);
      }
    } else {
      load_r();
      const int block = row_block(p.blocks, p.x, t, at);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = both(0.f);
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        load_x(k ? row_at(p.blocks[block + k * p.x.count], t, sizeof(XT)) : cx.ptr[0]);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          f2 w[4];
          unpack(v, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[v][i] = k ? h[v][i] + w[i] : w[i];
        }
      }
      cx.next(p, tx, t + 1, t1);
    }
    auto total = [&] {
      f2 s = both(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(h[v][i], h[v][i], s);
      return rsqrtf(row_sum(s.x + s.y, buf, turn) * inv_n + p.eps);
    };
    if (p.post) {
      const f2 rx = both(total());
      weigh(p.post, p.post_dtype, w_post, [&](const f2(&w)[4], int v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = h[v][i] * rx * w[i];
      });
    }
    if (gate) {
      if (t == seg_end) {
        gate += gate_step;
        seg_end += p.gate_per;
        if (KEEP) load_w8(gate, p.gate_dtype, channel(0), w_gate);
      }
      weigh(gate, p.gate_dtype, w_gate, [&](const f2(&w)[4], int v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = h[v][i] * w[i];
      });
    }
    if (drop.on) {
      // the words in a loop of two vectors a round: unrolled, the code does not stay in the instruction cache
      uint64_t keep = 0;
#pragma unroll 2
      for (int v = 0; v < VPT; ++v) keep |= (uint64_t)drop.bits(t, n, (tid + v * nt) * 8) << (8 * v);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = kept(h[v][i] * both(p.drop_scale), (uint32_t)(keep >> (8 * v)), i);
    }
    if (res) {
      const f2 scale = both(p.scale);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        f2 w[4];
        r[v].get2(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = has(v) ? fma2(scale, w[i], h[v][i]) : h[v][i];
      }
      cr.next(p, tr, t + 1, t1);
      if (AHEAD && t + 1 < t1) load_r();
    }
    if (out.ptr[0]) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (has(v)) store8(reinterpret_cast<RT*>(out.ptr[0]) + channel(v), h[v]);
    }
    if (out.ptr[1]) {
      const f2 rh = both(total());
      weigh(p.pre, p.pre_dtype, w_pre, [&](const f2(&w)[4], int v) {
        f2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = h[v][i] * rh * w[i];
        if (has(v)) store8(reinterpret_cast<XT*>(out.ptr[1]) + channel(v), y);
      });
    }
    out.next(p, to, t + 1, t1);
  }
}

// Gradients.  A CTA keeps the sums over its tokens and the weights in
// registers; x, dy, the residual and dh come through a ring of S rows.  Three
// things keep the work per element small.
//  - The means' sums are taken at once: with a = w s (w = gate post / (1 - p),
//    0 where dropped), h = scale residual + r(s) a and g = dh + r(h) z - k h,
//    the sum of a g is made of those of a dh, a z and a h; and (S > 1) the next
//    row's sum of s^2 goes with them, so the CTA meets once a row.
//  - dgate and dpost are one sum: with q = sum over the tokens of a gate row
//    of g s r(s) (kept elements), dgate = post q / (1 - p), and dpost adds up
//    gate q / (1 - p).
//  - What an operand is missing for is 0 (or, of w, 1) and computed all the same.
template <class XT, class RT, int VPT, int S, class P>
__global__ void __launch_bounds__(512) block_norm_row_backward_kernel(const __grid_constant__ P p) {
  __shared__ __align__(16) float buf[2][8][16];
  extern __shared__ uint4 ring[];
  clear(&buf[0][0][0], 2 * 8 * 16);
  int turn = 0;
  const int n = p.n, nt = blockDim.x, tid = threadIdx.x;
  const float inv_n = 1.f / (float)n;
  constexpr int PX = Pieces<XT>::N, PR = Pieces<RT>::N, STAGE = 2 * VPT * (PX + PR);
  constexpr bool HOLD = VPT == 1;  // a row's values stay in registers between the two looks at it
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens / gridDim.x, t1 = (int64_t)(blockIdx.x + 1) * p.tokens / gridDim.x;
  const RowTable *const tin[4] = {&p.x, &p.y, &p.r, &p.h}, *const tout[2] = {&p.dx, &p.dr};
  RowCursors<4> in;
  RowCursors<2> out;
  in.find(p, tin, t0, t1);
  out.find(p, tout, t0, t1);
  const bool has_y = p.y.count > 0, res = p.r.count > 0, has_h = p.h.count > 0, post = p.post, gate = p.gate;
  wait_for_previous_kernel();  // (until here: parameters and shared memory alone)
  const Dropout drop(p);
  auto channel = [&](int v) { return (v * nt + tid) * 8; };
  uint4* const mine = ring + tid;
  int64_t tf = t0;
  auto fetch = [&](uint4* to) {
    if (tf < t1) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = channel(v);
        if (c >= n) break;
        fetch8<XT>(to + v * PX * nt, in.ptr[0], c, nt);
        if (has_y) fetch8<XT>(to + (VPT + v) * PX * nt, in.ptr[1], c, nt);
        if (res) fetch8<RT>(to + (2 * VPT * PX + v * PR) * nt, in.ptr[2], c, nt);
        if (has_h) fetch8<RT>(to + (2 * VPT * PX + (VPT + v) * PR) * nt, in.ptr[3], c, nt);
      }
      ++tf;
      in.next(p, tin, tf, t1);
    }
    copies_commit();
  };
  for (int i = 0; i < S; ++i) {  // places that no copy fills are 0
    uint4* to = mine + i * STAGE * nt;
#pragma unroll
    for (int k = 0; k < STAGE; ++k) {
      const int v = k < 2 * VPT * PX ? k / PX % VPT : (k - 2 * VPT * PX) / PR % VPT;
      const bool there = k < VPT * PX ? true : k < 2 * VPT * PX ? has_y : k < 2 * VPT * PX + VPT * PR ? res : has_h;
      if (!there || channel(v) >= n) to[k * nt] = make_uint4(0, 0, 0, 0);
    }
  }
  for (int i = 0; i < S; ++i) fetch(mine + i * STAGE * nt);
  f2 s_pre[VPT][4], s_post[VPT][4], q_gate[VPT][4], w_pre[VPT][4], w[VPT][4];
  int64_t seg = gate ? (uint32_t)t0 / (uint32_t)p.gate_per : 0, seg_end = (seg + 1) * p.gate_per;
  auto weights = [&] {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = channel(v);
      if (c >= n) break;
      f2 a[4], b[4];
      if (post) load_w8(p.post, p.post_dtype, c, a);
      if (gate) load_w8(p.gate, p.gate_dtype, seg * n + c, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[v][i] = both(p.drop_scale);
        if (post) w[v][i] = w[v][i] * a[i];
        if (gate) w[v][i] = w[v][i] * b[i];
      }
    }
  };
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_pre[v][i] = s_post[v][i] = q_gate[v][i] = w_pre[v][i] = w[v][i] = both(0.f);
  weights();
  if (has_y) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (channel(v) < n) load_w8(p.pre, p.pre_dtype, channel(v), w_pre[v]);
  }
  auto write_sums = [&](float* to, int v, const f2(&s)[4]) {
    float4* o = reinterpret_cast<float4*>(to + channel(v));
    o[0] = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
    o[1] = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
  };
  // the end of a gate row's tokens (or, without a gate, of the CTA's)
  auto close = [&] {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = channel(v);
      if (c >= n) break;
      f2 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = b[i] = both(1.f);
        q_gate[v][i] = q_gate[v][i] * both(p.drop_scale);
      }
      if (post) load_w8(p.post, p.post_dtype, c, a);
      if (gate) load_w8(p.gate, p.gate_dtype, seg * n + c, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = a[i] * q_gate[v][i];
        s_post[v][i] = fma2(b[i], q_gate[v][i], s_post[v][i]);
        q_gate[v][i] = both(0.f);
      }
      if (!gate) continue;
      if (p.gate_per != 1) write_sums(p.part_gate + ((int64_t)blockIdx.x + seg) * n, v, a);
      else if (p.dgate_dtype == DT_BF16) store8(static_cast<__nv_bfloat16*>(p.dgate) + seg * n + c, a);
      else store8(static_cast<float*>(p.dgate) + seg * n + c, a);
    }
  };
  auto square = [&](const uint4* from) {  // this thread's share of the sum of s^2
    f2 s = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      Raw8<XT> r;
      r.set(from + v * PX * nt, nt);
      f2 x[4];
      r.get2(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(x[i], x[i], s);
    }
    return s.x + s.y;
  };
  float rx = 1.f;
  int slot = 0;
  const f2 scale = both(p.scale);
  for (int64_t t = t0; t < t1; ++t) {
    uint4* const from = mine + slot * STAGE * nt;
    if (++slot == S) slot = 0;
    copies_wait<(S > 1 ? S - 2 : 0)>();  // this row and (S > 1) the next
    float q[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (post && (S == 1 || t == t0)) {
      q[0] = square(from);
      row_sums(q, buf, turn);
      rx = rsqrtf(q[0] * inv_n + p.eps);
    }
    uint32_t bits[VPT];
    f2 x[4], h[4], dy[4], dh[4];  // of one vector
    auto values = [&](int v) {
      Raw8<XT> xw, yw;
      Raw8<RT> rw, hw;
      xw.set(from + v * PX * nt, nt);
      yw.set(from + (VPT + v) * PX * nt, nt);
      rw.set(from + (2 * VPT * PX + v * PR) * nt, nt);
      hw.set(from + (2 * VPT * PX + (VPT + v) * PR) * nt, nt);
      xw.get2(x), yw.get2(dy), rw.get2(h), hw.get2(dh);
    };
    auto branch = [&](int v, int i) {  // a
      const f2 a = x[i] * w[v][i];
      return drop.on ? kept(a, bits[v], i) : a;
    };
    f2 sum[5] = {both(0.f), both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (drop.on) bits[v] = drop.bits(t, n, channel(v));
      values(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 a = branch(v, i), z = dy[i] * w_pre[v][i];
        h[i] = fma2(scale, h[i], a * both(rx));
        sum[0] = fma2(h[i], h[i], sum[0]);
        sum[1] = fma2(h[i], z, sum[1]);
        sum[2] = fma2(a, dh[i], sum[2]);
        sum[3] = fma2(a, z, sum[3]);
        sum[4] = fma2(a, h[i], sum[4]);
      }
    }
    float rh = 0.f, kh = 0.f, kx = 0.f, next_rx = 1.f;
    if (has_y || post) {
#pragma unroll
      for (int i = 0; i < 5; ++i) q[i] = sum[i].x + sum[i].y;
      q[5] = q[6] = q[7] = 0.f;
      if (S > 1 && post && t + 1 < t1) q[5] = square(mine + slot * STAGE * nt);
      row_sums(q, buf, turn);
      if (has_y) {
        rh = rsqrtf(q[0] * inv_n + p.eps);
        kh = rh * rh * rh * (q[1] * inv_n);
      }
      if (post) {
        kx = rx * rx * rx * ((q[2] + rh * q[3] - kh * q[4]) * inv_n);
        next_rx = rsqrtf(q[5] * inv_n + p.eps);
      }
    }
    const f2 rx2 = both(rx), rh2 = both(rh), kh2 = both(-kh), kx2 = both(-kx);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = channel(v);
      if (!HOLD) {
        values(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = fma2(scale, h[i], branch(v, i) * rx2);
      }
      f2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2 g = dh[i], xr = x[i] * rx2;
        if (has_y) {  // (a choice: kh may not be finite where h is 0)
          g = fma2(dy[i] * w_pre[v][i], rh2, fma2(h[i], kh2, g));
          s_pre[v][i] = fma2(dy[i], h[i] * rh2, s_pre[v][i]);
        }
        dh[i] = g * scale;
        if (drop.on) g = kept(g, bits[v], i), xr = kept(xr, bits[v], i);  // (what is dropped may be NaN)
        q_gate[v][i] = fma2(g, xr, q_gate[v][i]);
        o[i] = g * w[v][i];
        if (post) o[i] = fma2(o[i], rx2, x[i] * kx2);
      }
      if (c < n) {
        if (out.ptr[1]) store8(reinterpret_cast<RT*>(out.ptr[1]) + c, dh);
        if (out.ptr[0]) store8(reinterpret_cast<XT*>(out.ptr[0]) + c, o);
      }
    }
    out.next(p, tout, t + 1, t1);
    fetch(from);
    if (S > 1) rx = next_rx;
    if (t + 1 == t1) {
      close();
    } else if (gate && t + 1 == seg_end) {
      close();
      ++seg;
      seg_end += p.gate_per;
      weights();
    }
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (channel(v) >= n) break;
    if (has_y) write_sums(p.part_pre + (int64_t)blockIdx.x * n, v, s_pre[v]);
    if (post) write_sums(p.part_post + (int64_t)blockIdx.x * n, v, s_post[v]);
  }
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
  int stages = 0;  // backward: rows of the ring
  bool ahead = false;  // forward: the next row's loads go out early
  size_t smem = 0;
};

int round_up(int64_t a, int b) { return (int)((a + b - 1) / b * b); }
constexpr int64_t BN_SMEM = 224 * 1024;  // of an SM, for rings
constexpr int64_t BN_STATIC = 2048;      // a CTA's other shared memory, at most

Shape forward_shape(const BlockArgs& p, bool vec, bool small) {
  Shape s;
  const int sms = device_sm_count();
  const int64_t vectors = p.n / 8;
  if (!vec || vectors > 4 * 512) {
    s.grid = (int)std::min<int64_t>(p.tokens, (int64_t)sms * 8);
    return s;
  }
  // Few tokens: a vector a thread, the shortest way through a row.  Else four,
  // for what a row costs besides its vectors is paid by each warp, or two where
  // that leaves a fifth fewer threads idle.
  auto threads = [&](int vpt) { return round_up((vectors + vpt - 1) / vpt, 32); };
  s.vpt = 4;
  if (p.tokens <= 2 * sms && vectors <= 1024) s.vpt = 1;
  else if (vectors <= 64 || (vectors <= 1024 && 8 * threads(2) < 13 * threads(4))) s.vpt = vectors <= 32 ? 1 : 2;
  s.threads = threads(s.vpt);
  s.ahead = small && p.x.parts == 1 && p.tokens > 2 * sms;
  const int ctas = std::max(1, std::min(32, forward_resident(s.vpt, s.ahead, dtype_size(p.h.dtype)) / s.threads));
  s.grid = (int)std::min<int64_t>(p.tokens, (int64_t)sms * ctas);
  return s;
}

Shape backward_shape(const BlockArgs& p, bool vec, bool small) {
  Shape s;
  const int sms = device_sm_count();
  const int64_t vectors = p.n / 8;
  int64_t most = 2 * sms;
  if (vec && small && p.x.parts == 1 && vectors <= 1024) {
    s.vpt = vectors <= 256 ? 1 : 2;  // (8192 x 4096: two vectors 85.9 us, one 91.0)
    s.threads = round_up((vectors + s.vpt - 1) / s.vpt, 32);
    const int64_t stage = (int64_t)s.threads * s.vpt * 16 * (dtype_size(p.x.dtype) + dtype_size(p.h.dtype));
    const int64_t ctas = std::min(8, 512 / s.threads);
    s.stages = s.vpt == 1 && (5 * stage + BN_STATIC) * ctas <= BN_SMEM ? 5 : (3 * stage + BN_STATIC) * ctas <= BN_SMEM ? 3 : 1;
    s.smem = stage * s.stages;
    most = std::max<int64_t>(1, std::min<int64_t>(ctas, BN_SMEM / (int64_t)(s.smem + BN_STATIC))) * sms;
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
#define DT_BN_BACK(VPT, S) \
  if (s.vpt == VPT && s.stages == S) return launch_rows(block_norm_row_backward_kernel<XT, RT, VPT, S, P>, p, s, stream);
  if constexpr (P::kCap == BlockSmall::kCap) {
    if (bwd) {
      DT_BN_BACK(1, 5) DT_BN_BACK(1, 3) DT_BN_BACK(2, 3) DT_BN_BACK(2, 1)
      return cudaErrorInvalidValue;
    }
    if (s.ahead)
      return s.vpt == 1   ? launch_rows(block_norm_row_kernel<XT, RT, 1, true, P>, p, s, stream)
             : s.vpt == 2 ? launch_rows(block_norm_row_kernel<XT, RT, 2, true, P>, p, s, stream)
                          : launch_rows(block_norm_row_kernel<XT, RT, 4, true, P>, p, s, stream);
  }
  return s.vpt == 1   ? launch_rows(block_norm_row_kernel<XT, RT, 1, false, P>, p, s, stream)
         : s.vpt == 2 ? launch_rows(block_norm_row_kernel<XT, RT, 2, false, P>, p, s, stream)
                      : launch_rows(block_norm_row_kernel<XT, RT, 4, false, P>, p, s, stream);
#undef DT_BN_BACK
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
  for (int i = 0; i < used; ++i) vec = vec && p.blocks[i].ld < (1 << 29);  // steps between rows in 31 bits
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
