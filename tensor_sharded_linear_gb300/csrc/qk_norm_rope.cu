// Norms of queries and keys for each head with the position rotation in the
// same pass, and their backward pass.
//
// Per head of D channels and token t (all sums in fp32):
//   r = 1 / sqrt(mean(x^2) + eps)        z = x * r * w        y = R(pos_t) z
// and, for a gradient dy of y,
//   dz = R(pos_t)^T dy      dw = sum over tokens and heads of dz * x * r
//   g = dz * w              dx = r * (g - x r * mean(g * x r))
// R(pos) turns the pairs (i, i + R/2), or (2i, 2i + 1) when interleaved, of
// the first R channels by the angles of row pos of the cos/sin table.
//
// Both passes are bound by memory: the forward reads and writes each element
// once, the backward reads x and dy and writes dx.  8192 tokens, 32 + 32 heads
// of 128 in bf16: forward 44.8 us for 273 MB, 6.1 TB/s, 0.90 of a copy's rate;
// backward 64.6 us for 407 MB, 6.3 TB/s, 0.93.  8 tokens take 2.6 us, a launch.
//
// Layout.  A head's channels are cut into chunks of 8.  A lane holds two
// chunks of a head -- the two partners of a rotation, chunk l and chunk
// l + R/16, so a pair never crosses lanes -- and D/16 lanes hold the head:
// each access is 16 bytes (bf16), 128 contiguous bytes per 8 lanes.  A warp
// takes heads of ONE token, so its cos/sin vectors are loaded once, with the
// weight folded in (forward: y = r (P x + Q partner)), and a CTA takes one
// tensor (q or k), so the weights stay in registers.  The next heads' loads
// are in flight while the present ones are worked on.  The arithmetic runs on
// register pairs (fp32x2): with one channel per instruction the forward
// needs more instructions a byte than an SM issues.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "heads_sm103.cuh"

namespace dt {
namespace {

constexpr int NR_THREADS = 128;
constexpr int NR_WARPS = NR_THREADS / 32;
constexpr int NR_MAX_D = 1024;

struct NormParams {
  HeadMap x[2];         // q and k as they came
  HeadMap y[2];         // forward: the outputs; backward: dx
  HeadMap g[2];         // backward: dy
  const void* w[2];     // NULL: no norm
  void* dw[2];
  int32_t w_dtype[2], dw_dtype[2];
  const float* cos_sin;  // [table_rows, rotary]: cosines then sines; NULL: no rotation
  const int32_t* pos;
  int64_t table_rows;
  int64_t tokens;
  int32_t D, rotary, interleaved;
  int32_t blocks_q;  // CTAs [0, blocks_q) work on q, the others on k
  int32_t inner[2];  // blocks of heads of a warp's unit
  float eps;
  float* part;  // backward: [CTA][D] sums of dw
  int32_t* status;
};

__device__ __forceinline__ float load_w(const void* w, int dtype, int i) {
  return dtype == DT_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                          : static_cast<const float*>(w)[i];
}

// Row of the cos/sin table for token t, or -1 (and the status bit) when its
// position lies outside the table.
__device__ __forceinline__ int64_t table_row(const NormParams& p, int64_t t, bool report) {
  const int32_t r = load_plain(p.pos + t);
  if (r >= 0 && r < p.table_rows) return r;
  if (report) atomicOr(p.status, DT_DEV_ERR_INDEX);
  return -1;
}

// Adds the CTA's sums of dw (acc: [NR_WARPS][D] in shared memory) in warp
// order and writes them to this CTA's row of the workspace.
__device__ __forceinline__ void write_dw_part(const NormParams& p, const float* acc) {
  __syncthreads();
  for (int c = threadIdx.x; c < p.D; c += NR_THREADS) {
    float s = acc[c];
    for (int w = 1; w < NR_WARPS; ++w) s += acc[w * p.D + c];
    p.part[(int64_t)blockIdx.x * p.D + c] = s;
  }
}

// D and rotary multiples of 16, D <= 512, 16-byte aligned heads.  A unit of
// work is `inner` blocks of heads (SG * U heads each) of one token.
// CTAs per SM: 5 forward, 4 backward (128 registers for its sums of dw);
// measured at 8192 tokens x 64 heads against 3..5 CTAs (backward with 5: 97.7
// us, with 4: 64.6; bf16: fp32 takes the same numbers, without a measurement
// of its own).
__host__ __device__ constexpr int norm_ctas(bool bwd) { return bwd ? 4 : 5; }

template <class T, bool BWD>
struct NormVec {
  static constexpr int U = sizeof(T) == 2 && !BWD ? 2 : 1;  // heads per lane and step
  // bf16 backward: x and dy come through a ring of asynchronous copies, each
  // lane its own four chunks, so three steps are on their way without taking
  // registers: 64.6 us where the next step's loads in registers, one step
  // ahead, took 79.3 (8192 tokens x 64 heads); the forward is the other way
  // round, 46.3 and 44.8.  In fp32 a stage takes twice the room: a ring of
  // two took 13.0 us where loads in registers took 11.4 (1531 tokens x 16
  // heads of 64; today 10.7); deeper ones were not tried.
  static constexpr int STAGES = BWD && sizeof(T) == 2 ? 4 : 0;
  static constexpr int RING = STAGES * 64 * NR_THREADS;
};

// LANES: D / 16 where that is 4, 8 or 16 (all lanes hold channels and the
// sums' steps are known), else 0.
template <class T, bool BWD, bool INTER, int LANES>
__global__ void __launch_bounds__(NR_THREADS, norm_ctas(BWD)) qk_norm_vec_kernel(const __grid_constant__ NormParams p) {
  wait_for_previous_kernel();
  constexpr int U = NormVec<T, BWD>::U;
  extern __shared__ __align__(16) float nr_acc[];  // backward: [NR_WARPS][D] sums; forward: [D] weights
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = LANES ? 16 * LANES : p.D, L = D / 16;
  int LP = LANES;
  if (!LANES) {
    LP = 1;
    while (LP < L) LP <<= 1;
  }
  const int SG = 32 / LP, sub = lane / LP, l = lane & (LP - 1);
  const bool act = LANES || l < L;
  // the sum over a head's lanes
  auto head_sum = [&](float v) {
    if constexpr (LANES) {
#pragma unroll
      for (int o = LANES >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
      v = act ? v : 0.f;
      for (int o = LP >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
  };
  const int which = blockIdx.x >= p.blocks_q;
  const HeadMap &X = p.x[which], &Y = p.y[which], &G = p.g[which];
  const int rl = p.cos_sin ? p.rotary / 16 : 0;  // lanes that hold rotated pairs
  const bool rot = l < rl;
  // first channels of the lane's two chunks; a pair's partner is in the other
  // chunk, or (INTER) the neighbour channel.  2 rl chunks are rotated, so the
  // rest starts at chunk 2 l.
  const int ca = !act ? 0 : rot && !INTER ? 8 * l : 16 * l;
  const int cb = rot && !INTER ? 8 * (l + rl) : ca + 8;
  const bool norm = p.w[which] != nullptr;
  f2 wa[4], wb[4], da[4], db[4];
  if (BWD) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wa[i] = wb[i] = both(1.f), da[i] = db[i] = both(0.f);
      if (norm && act) {
        wa[i] = f2{load_w(p.w[which], p.w_dtype[which], ca + 2 * i), load_w(p.w[which], p.w_dtype[which], ca + 2 * i + 1)};
        wb[i] = f2{load_w(p.w[which], p.w_dtype[which], cb + 2 * i), load_w(p.w[which], p.w_dtype[which], cb + 2 * i + 1)};
      }
    }
  } else {
    for (int c = threadIdx.x; c < p.D; c += NR_THREADS) nr_acc[c] = norm ? load_w(p.w[which], p.w_dtype[which], c) : 1.f;
    __syncthreads();
  }
  const int inner = p.inner[which];
  const int64_t tokens = X.heads ? p.tokens : 0;
  const int per_tok = max(1, ((X.heads + SG * U - 1) / (SG * U) + inner - 1) / inner);  // units of a token
  const int step = (which ? gridDim.x - p.blocks_q : p.blocks_q) * NR_WARPS;
  const int step_tok = step / per_tok, step_blk = step - step_tok * per_tok;  // a stride of units, without a division
  const float inv_d = 1.f / (float)D;

  Raw8<T> xa[U], xb[U], ga[U], gb[U];
  using V = NormVec<T, BWD>;
  constexpr bool RING = V::STAGES > 0;
  auto load = [&](int64_t t, int block, Raw8<T>(&a)[U], Raw8<T>(&b)[U], Raw8<T>(&c)[U], Raw8<T>(&d)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = min((block * U + i) * SG + sub, X.heads - 1);  // past the last head: that one again, not stored
      const T* x = head_ptr<T>(X, t, h, D);
      a[i].load(x + ca);
      b[i].load(x + cb);
      if (BWD) {
        const T* g = head_ptr<T>(G, t, h, D);
        c[i].load(g + ca);
        d[i].load(g + cb);
      }
    }
  };
  const int u0 = (which ? blockIdx.x - p.blocks_q : blockIdx.x) * NR_WARPS + warp;
  int64_t t = u0 / per_tok;
  int blk = u0 - (int)t * per_tok;  // unit blk of token t
  int64_t row_next = 0;
  // the ring, and the step to be fetched into it next
  uint4* ring = reinterpret_cast<uint4*>(nr_acc + NR_WARPS * D) + threadIdx.x;
  int64_t ft = t;
  int fblk = blk, fin = 0, fput = 0, fget = 0;
  auto fetch = [&]() {
    if constexpr (RING) {
      if (ft < tokens) {
        const int h = min((fblk * inner + fin) * SG + sub, X.heads - 1);
        const T *x = head_ptr<T>(X, ft, h, D), *g = head_ptr<T>(G, ft, h, D);
        uint4* to = ring + fput * (4 * NR_THREADS);
        copy16_async(to, x + ca);
        copy16_async(to + NR_THREADS, x + cb);
        copy16_async(to + 2 * NR_THREADS, g + ca);
        copy16_async(to + 3 * NR_THREADS, g + cb);
        if (++fin == inner) {
          fin = 0;
          ft += step_tok, fblk += step_blk;
          if (fblk >= per_tok) fblk -= per_tok, ++ft;
        }
      }
      copies_commit();
      if (++fput == V::STAGES) fput = 0;
    }
  };
  auto take = [&]() {
    if constexpr (RING) {
      copies_wait<V::STAGES - 1>();
      const uint4* from = ring + fget * (4 * NR_THREADS);
      xa[0].u = from[0], xb[0].u = from[NR_THREADS], ga[0].u = from[2 * NR_THREADS], gb[0].u = from[3 * NR_THREADS];
      if (++fget == V::STAGES) fget = 0;
    }
  };
  if constexpr (RING)
    for (int i = 0; i + 1 < V::STAGES; ++i) fetch();
  if (t < tokens) {
    if (!RING) load(t, blk * inner, xa, xb, ga, gb);
    if (p.cos_sin) row_next = table_row(p, t, lane == 0);
  }
  while (t < tokens) {
    const int64_t row = row_next;
    const bool ok = row >= 0;
    f2 c2[4], s2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c2[i] = both(1.f), s2[i] = both(0.f);
    if (rot && ok) {
      Raw8<float> c, s;
      c.load_keep(p.cos_sin + row * p.rotary + 8 * l);
      s.load_keep(p.cos_sin + row * p.rotary + p.rotary / 2 + 8 * l);
      c.get2(c2);
      s.get2(s2);
    }
    int64_t tn = t + step_tok;
    int bn = blk + step_blk;
    if (bn >= per_tok) bn -= per_tok, ++tn;
    if (tn < tokens && p.cos_sin) row_next = table_row(p, tn, lane == 0);
    // pair e of chunk a has the cosines cosa(e), of chunk b cosb(e)
    auto at = [](const f2(&v)[4], int e) { return e & 1 ? v[e >> 1].y : v[e >> 1].x; };
    auto cosa = [&](int e) { return INTER ? both(at(c2, e)) : c2[e]; };
    auto cosb = [&](int e) { return INTER ? both(at(c2, 4 + e)) : c2[e]; };
    auto sina = [&](int e) { return INTER ? both(at(s2, e)) : s2[e]; };
    auto sinb = [&](int e) { return INTER ? both(at(s2, 4 + e)) : s2[e]; };
    auto swap = [](f2 v) { return f2{v.y, v.x}; };
    // forward: y = P x + Q partner with the weights in P and Q
    f2 pa[4], pb[4], qa[4], qb[4];
    if (!BWD) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 va = act ? *reinterpret_cast<const f2*>(nr_acc + ca + 2 * e) : both(0.f);
        const f2 vb = act ? *reinterpret_cast<const f2*>(nr_acc + cb + 2 * e) : both(0.f);
        pa[e] = cosa(e) * va, pb[e] = cosb(e) * vb;
        qa[e] = INTER ? sina(e) * f2{-va.y, va.x} : sina(e) * vb * both(-1.f);
        qb[e] = INTER ? sinb(e) * f2{-vb.y, vb.x} : sinb(e) * va;
      }
    }
#pragma unroll(BWD && !RING ? 2 : 1)
    for (int in = 0; in < inner; ++in) {
      const int block = blk * inner + in;
      Raw8<T> nxa[U], nxb[U], nga[U], ngb[U];
      if constexpr (RING) {
        fetch();
        take();
      } else {
        if (in + 1 < inner) load(t, block + 1, nxa, nxb, nga, ngb);
        else if (tn < tokens) load(tn, bn * inner, nxa, nxb, nga, ngb);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int h = (block * U + i) * SG + sub;
        f2 a[4], b[4], ya[4], yb[4];
        xa[i].get2(a);
        xb[i].get2(b);
        float r = 1.f;
        if (norm) {
          f2 ss = a[0] * a[0];
#pragma unroll
          for (int e = 1; e < 4; ++e) ss = fma2(a[e], a[e], ss);
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = fma2(b[e], b[e], ss);
          r = rsqrtf(head_sum(ss.x + ss.y) * inv_d + p.eps);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = a[e] * both(r), b[e] = b[e] * both(r);
        }
        if (!BWD) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ya[e] = a[e] * pa[e], yb[e] = b[e] * pb[e];
            if (rot) {  // (a choice, not a sine of 0: the other channel may be infinite)
              ya[e] = fma2(INTER ? swap(a[e]) : b[e], qa[e], ya[e]);
              yb[e] = fma2(INTER ? swap(b[e]) : a[e], qb[e], yb[e]);
            }
          }
        } else {
          f2 dya[4], dyb[4];  // dz = R^T dy
          ga[i].get2(dya);
          gb[i].get2(dyb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ya[e] = dya[e] * cosa(e), yb[e] = dyb[e] * cosb(e);
            if (rot) {
              ya[e] = fma2(INTER ? f2{dya[e].y, -dya[e].x} : dyb[e], sina(e), ya[e]);
              yb[e] = fma2(INTER ? f2{dyb[e].y, -dyb[e].x} : dya[e] * both(-1.f), sinb(e), yb[e]);
            }
          }
          if (norm) {
            const bool on = ok && h < X.heads;  // (a choice, not a factor: what is left out may be NaN)
            f2 gx = both(0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const f2 ta = ya[e] * a[e], tb = yb[e] * b[e];
              if (on) da[e] = fma2(ya[e], a[e], da[e]), db[e] = fma2(yb[e], b[e], db[e]);
              gx = fma2(ta, wa[e], gx), gx = fma2(tb, wb[e], gx);
            }
            const float k = head_sum(gx.x + gx.y) * -r * inv_d;  // - r * mean(g * x r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ya[e] = fma2(a[e], both(k), ya[e] * (wa[e] * both(r)));
              yb[e] = fma2(b[e], both(k), yb[e] * (wb[e] * both(r)));
            }
          }
        }
        if (!act || h >= X.heads) continue;
        if (!ok) {  // no such position: the row is zero, as an embedding row of a bad id
#pragma unroll
          for (int e = 0; e < 4; ++e) ya[e] = yb[e] = both(0.f);
        }
        T* y = head_ptr<T>(Y, t, h, D);
        store8(y + ca, ya);
        store8(y + cb, yb);
      }
#pragma unroll
      for (int i = 0; i < U && !RING; ++i) {
        xa[i] = nxa[i], xb[i] = nxb[i];
        if (BWD) ga[i] = nga[i], gb[i] = ngb[i];
      }
    }
    t = tn;
    blk = bn;
  }
  if (BWD && p.part) {
    // the subgroups' sums, then the warps', in a fixed order: the same
    // inputs give the same bits
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      for (int o = LP; o < 32; o <<= 1) {
        da[e].x += __shfl_xor_sync(0xffffffffu, da[e].x, o), da[e].y += __shfl_xor_sync(0xffffffffu, da[e].y, o);
        db[e].x += __shfl_xor_sync(0xffffffffu, db[e].x, o), db[e].y += __shfl_xor_sync(0xffffffffu, db[e].y, o);
      }
    }
    if (act && sub == 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<f2*>(nr_acc + warp * p.D + ca + 2 * e) = da[e];
        *reinterpret_cast<f2*>(nr_acc + warp * p.D + cb + 2 * e) = db[e];
      }
    }
    write_dw_part(p, nr_acc);
  }
}

// Any even rotary <= D <= NR_MAX_D and any alignment: a warp per head, a lane
// per pair of channels, 32 pairs a step (the second look at the head comes
// from L1).
template <class T, bool BWD>
__global__ void __launch_bounds__(NR_THREADS) qk_norm_any_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float nr_acc[];
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = blockIdx.x >= p.blocks_q;
  const HeadMap &X = p.x[which], &Y = p.y[which], &G = p.g[which];
  const bool norm = p.w[which] != nullptr;
  float* acc = nr_acc + warp * p.D;
  if (BWD && p.part)
    for (int c = lane; c < p.D; c += 32) acc[c] = 0.f;
  __syncwarp();
  const int half = p.cos_sin ? p.rotary / 2 : 0;
  const int pairs = (p.D + 1) / 2;  // rotated pairs first; of the rest, channels 2j and 2j + 1
  const float inv_d = 1.f / (float)p.D;
  const int64_t units = p.tokens * X.heads;
  const int64_t first = (int64_t)(which ? blockIdx.x - p.blocks_q : blockIdx.x) * NR_WARPS + warp;
  const int64_t step = (int64_t)(which ? gridDim.x - p.blocks_q : p.blocks_q) * NR_WARPS;
  for (int64_t u = first; u < units; u += step) {
    const int64_t t = u / X.heads;
    const int h = (int)(u - t * X.heads);
    const T* x = head_ptr<T>(X, t, h, p.D);
    const T* g = BWD ? head_ptr<T>(G, t, h, p.D) : nullptr;
    T* y = head_ptr<T>(Y, t, h, p.D);
    const int64_t row = p.cos_sin ? table_row(p, t, lane == 0) : 0;
    const bool ok = row >= 0;
    const float* cs = p.cos_sin ? p.cos_sin + (ok ? row : 0) * p.rotary : nullptr;
    float ss = 0.f, gx = 0.f, r = 1.f, k = 0.f;
    for (int pass = norm ? 0 : 1; pass < 2; ++pass) {
      for (int j = lane; j < pairs; j += 32) {
        const bool rot = j < half;
        const int ia = rot && !p.interleaved ? j : 2 * j, ib = rot && !p.interleaved ? j + half : 2 * j + 1;
        const bool two = ib < p.D;
        float a = to_f32(x[ia]), b = two ? to_f32(x[ib]) : 0.f, ya = 0.f, yb = 0.f;
        const float wa = norm ? load_w(p.w[which], p.w_dtype[which], ia) : 1.f;
        const float wb = norm && two ? load_w(p.w[which], p.w_dtype[which], ib) : 1.f;
        if (BWD) {
          ya = to_f32(g[ia]), yb = two ? to_f32(g[ib]) : 0.f;
          if (rot && ok) rotate_pair(ya, yb, load_plain(cs + j), -load_plain(cs + half + j));
        }
        if (pass == 0) {
          ss += a * a + b * b;
          if (BWD) gx += ya * wa * a + yb * wb * b;
          continue;
        }
        const float na = a * r, nb = b * r;
        if (BWD) {
          if (norm && ok && p.part) {
            acc[ia] += ya * na;
            if (two) acc[ib] += yb * nb;
          }
          a = norm ? r * (ya * wa - na * k) : ya;
          b = norm ? r * (yb * wb - nb * k) : yb;
        } else {
          if (norm) a = na * wa, b = nb * wb;
          if (rot && ok) rotate_pair(a, b, load_plain(cs + j), load_plain(cs + half + j));
        }
        from_f32(y + ia, ok ? a : 0.f);
        if (two) from_f32(y + ib, ok ? b : 0.f);
      }
      if (pass == 0) {
        for (int o = 16; o; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (BWD) gx += __shfl_xor_sync(0xffffffffu, gx, o);
        }
        r = rsqrtf(ss * inv_d + p.eps);
        k = gx * r * inv_d;
      }
    }
  }
  if (BWD && p.part) write_dw_part(p, nr_acc);
}

// dw of q (blockIdx.y 0) and k (1): the CTAs' sums of 32 channels, each warp
// every 32nd row of them, then the warps' sums; a fixed order.
constexpr int DW_THREADS = 1024;
__global__ void __launch_bounds__(DW_THREADS) qk_norm_dw_kernel(const __grid_constant__ NormParams p, int nblocks) {
  __shared__ float acc[32][33];
  wait_for_previous_kernel();
  const int which = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!p.dw[which]) return;
  const int b0 = which ? p.blocks_q : 0, b1 = which ? nblocks : p.blocks_q;
  int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < p.D) {
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += 32) s += p.part[(int64_t)b * p.D + c];
  }
  acc[warp][lane] = s;
  __syncthreads();
  s = acc[lane][warp];
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  c = blockIdx.x * 32 + warp;
  if (lane == 0 && c < p.D) {
    if (p.dw_dtype[which] == DT_BF16) static_cast<__nv_bfloat16*>(p.dw[which])[c] = __float2bfloat16_rn(s);
    else static_cast<float*>(p.dw[which])[c] = s;
  }
}

// ---------------------------------------------------------------- host

constexpr int NR_MAX_BLOCKS = 2048;  // rows of the backward's workspace at most

struct NormArgs {
  const dt_dtensor *dy_q, *dy_k;  // backward only
  const dt_dtensor *q, *k, *q_weight, *k_weight, *cos_sin, *positions, *q_out, *k_out;
  const dt_dtensor *dq_weight, *dk_weight;  // backward only
};

dt_status norm_weight(const dt_dtensor* w, const char* what, const Layout& of, int D, bool output, const void** ptr,
                      int32_t* dtype) {
  PlainOperand o;
  dt_status st = plain_operand(w, what, of, output, &o);
  if (st != DT_OK) return st;
  if (o.ndim != 1 || o.shape[0] != D) return fail(DT_ERR_SHAPE, "%s must be [head_dim]", what);
  if (o.dtype != DT_BF16 && o.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "%s must be bf16 or fp32", what);
  *ptr = o.ptr;
  *dtype = o.dtype;
  return DT_OK;
}

// CTAs of a launch over tokens * heads head rows: enough to fill the device,
// fewer when there are not that many units of work.
int norm_blocks(int64_t units, bool bwd) {
  const int64_t full = std::min<int64_t>((int64_t)device_sm_count() * norm_ctas(bwd), NR_MAX_BLOCKS / 2);
  return (int)std::max<int64_t>(1, std::min<int64_t>((units + NR_WARPS - 1) / NR_WARPS, full));
}

int vec_lanes(int D) { return D == 64 || D == 128 || D == 256 ? D / 16 : 0; }

template <class T, bool BWD>
cudaError_t launch_norm(const NormParams& p, bool vec, int grid, cudaStream_t s) {
  constexpr int RING = NormVec<T, BWD>::RING;
  size_t smem = (size_t)p.D * sizeof(float) * (!BWD ? 1 : p.part || (vec && RING) ? NR_WARPS : 0);
  if (vec) smem += RING;  // (at most 40 KB)
#define DT_NR(inter, lanes)                                              \
  if (vec && (p.interleaved != 0) == inter && vec_lanes(p.D) == lanes) \
    return launch_early(qk_norm_vec_kernel<T, BWD, inter, lanes>, dim3(grid), NR_THREADS, smem, s, p);
  DT_NR(false, 4) DT_NR(false, 8) DT_NR(false, 16) DT_NR(false, 0)
  DT_NR(true, 4) DT_NR(true, 8) DT_NR(true, 16) DT_NR(true, 0)
#undef DT_NR
  return launch_early(qk_norm_any_kernel<T, BWD>, dim3(grid), NR_THREADS, smem, s, p);
}

dt_status norm_call(bool bwd, const NormArgs& A, int D, float eps, int interleaved, int tp, void* ws, size_t ws_bytes,
                    int32_t* d_status, cudaStream_t stream) {
  clear_error();
  if (D < 2 || D > NR_MAX_D) return fail(DT_ERR_UNSUPPORTED, "head_dim %d (2 .. %d)", D, NR_MAX_D);
  if (!(eps >= 0.f) || eps > 1.f) return fail(DT_ERR_INVALID_ARG, "eps must be in [0, 1]");
  if (!A.q) return fail(DT_ERR_INVALID_ARG, "q is NULL");
  if (!A.k && (A.k_weight || A.k_out || A.dy_k || A.dk_weight))
    return fail(DT_ERR_INVALID_ARG, "k is NULL but another k operand is not");
  if (!A.q_weight && !A.k_weight && !A.cos_sin) return fail(DT_ERR_INVALID_ARG, "neither a norm nor a rotation");
  if ((A.cos_sin == nullptr) != (A.positions == nullptr))
    return fail(DT_ERR_INVALID_ARG, "cos_sin and positions go together");
  NormParams p;
  HeadOperand x[2], y[2], g[2];
  Layout lq, lx;
  dt_status st;
  const int n = A.k ? 2 : 1;
  const dt_dtensor* xs[2] = {A.q, A.k};
  const dt_dtensor* ys[2] = {A.q_out, A.k_out};
  const dt_dtensor* gs[2] = {A.dy_q, A.dy_k};
  const dt_dtensor* wts[2] = {A.q_weight, A.k_weight};
  const dt_dtensor* dws[2] = {A.dq_weight, A.dk_weight};
  static const char* const names[2][4] = {{"q", "dq_out", "q_weight", "dq_weight"},
                                          {"k", "dk_out", "k_weight", "dk_weight"}};
  const char* const ynames[2] = {bwd ? "dq" : "q_out", bwd ? "dk" : "k_out"};
  bool vec = D % 16 == 0 && D <= 512, any_dw = false;
  for (int i = 0; i < n; ++i) {
    if ((st = head_operand(xs[i], names[i][0], tp, D, false, &x[i], i ? &lx : &lq)) != DT_OK) return st;
    if (i && (st = same_mesh(lx, lq, names[i][0])) != DT_OK) return st;
    if (x[i].tokens != x[0].tokens) return fail(DT_ERR_SHAPE, "q and k have different token counts");
    if (x[i].dtype != x[0].dtype) return fail(DT_ERR_INVALID_ARG, "q and k must have one dtype");
    for (int r = 0; r < (bwd ? 2 : 1); ++r) {
      HeadOperand& o = r ? g[i] : y[i];
      const char* nm = r ? names[i][1] : ynames[i];
      Layout lo;
      if ((st = head_operand(r ? gs[i] : ys[i], nm, tp, D, r == 0, &o, &lo)) != DT_OK) return st;
      if ((st = same_mesh(lo, lq, nm)) != DT_OK) return st;
      if (o.heads != x[i].heads || o.tokens != x[i].tokens)
        return fail(DT_ERR_SHAPE, "%s must have the shape of %s", nm, names[i][0]);
      if (o.dtype != x[i].dtype) return fail(DT_ERR_INVALID_ARG, "%s must have the dtype of %s", nm, names[i][0]);
      vec = vec && o.vec16;
    }
    vec = vec && x[i].vec16;
    p.x[i] = x[i].map;
    p.y[i] = y[i].map;
    if (bwd) p.g[i] = g[i].map;
    p.w[i] = p.dw[i] = nullptr;
    if (wts[i]) {
      const void* w;
      if ((st = norm_weight(wts[i], names[i][2], lq, D, false, &w, &p.w_dtype[i])) != DT_OK) return st;
      p.w[i] = w;
    }
    if (bwd && (wts[i] == nullptr) != (dws[i] == nullptr))
      return fail(DT_ERR_INVALID_ARG, "%s and %s go together", names[i][2], names[i][3]);
    if (bwd && dws[i]) {
      const void* w;
      if ((st = norm_weight(dws[i], names[i][3], lq, D, true, &w, &p.dw_dtype[i])) != DT_OK) return st;
      p.dw[i] = const_cast<void*>(w);
      any_dw = true;
    }
  }
  p.cos_sin = nullptr;
  p.pos = nullptr;
  p.table_rows = 0;
  p.rotary = 0;
  if (A.cos_sin) {
    PlainOperand t, pos;
    if ((st = plain_operand(A.cos_sin, "cos_sin", lq, false, &t)) != DT_OK) return st;
    if ((st = plain_operand(A.positions, "positions", lq, false, &pos)) != DT_OK) return st;
    if (t.ndim != 2 || t.shape[1] < 2 || t.shape[1] % 2 || t.shape[1] > D)
      return fail(DT_ERR_SHAPE, "cos_sin must be [rows, rotary], rotary even and at most head_dim");
    if (t.dtype != DT_FP32) return fail(DT_ERR_INVALID_ARG, "cos_sin must be fp32");
    if (pos.dtype != DT_INT32) return fail(DT_ERR_INVALID_ARG, "positions must be int32");
    if (pos.numel != x[0].tokens) return fail(DT_ERR_SHAPE, "positions must have one entry per token");
    if (t.shape[0] == 0 && x[0].tokens > 0)
      return fail(DT_ERR_SHAPE, "cos_sin has no rows: every position would be out of range");
    p.cos_sin = reinterpret_cast<const float*>(t.ptr);
    p.pos = reinterpret_cast<const int32_t*>(pos.ptr);
    p.table_rows = t.shape[0];
    p.rotary = (int)t.shape[1];
    vec = vec && p.rotary % 16 == 0 && reinterpret_cast<uintptr_t>(t.ptr) % 16 == 0;
  }
  p.D = D;
  p.eps = eps;
  p.interleaved = interleaved != 0;
  p.tokens = x[0].tokens;
  p.part = nullptr;
  const int heads_k = n == 2 ? x[1].heads : 0;
  const bool nothing = p.tokens == 0 || x[0].heads + heads_k == 0;
  if (nothing && !any_dw) return DT_OK;
  // A warp's unit is as many blocks of heads of one token as leave four
  // units for every warp of a full device: the token's angles are fetched
  // once for them (measured at 8192 tokens x 64 heads, backward: 139.8 us
  // with one block a unit where four took 90.8 us).
  int LP = 1;
  while (LP < D / 16) LP <<= 1;
  const int U = x[0].dtype == DT_BF16 && !bwd ? NormVec<__nv_bfloat16, false>::U : NormVec<float, true>::U;
  const int per_block = vec ? 32 / LP * U : 1;
  const int64_t all = std::max<int64_t>(1, (int64_t)x[0].heads + heads_k);
  int64_t units[2];
  for (int i = 0; i < 2; ++i) {
    const int heads = i ? heads_k : x[0].heads, blocks = std::max(1, (heads + per_block - 1) / per_block);
    const int64_t warps = (int64_t)device_sm_count() * norm_ctas(bwd) * NR_WARPS * heads / all;
    p.inner[i] = 1;
    while (vec && p.inner[i] < blocks && p.tokens * ((blocks + 2 * p.inner[i] - 1) / (2 * p.inner[i])) >= 4 * warps)
      p.inner[i] *= 2;
    units[i] = heads ? p.tokens * ((blocks + p.inner[i] - 1) / p.inner[i]) : 0;
  }
  // CTAs in proportion to the heads
  const int total = norm_blocks(units[0] + units[1], bwd);
  int bq = (int)((double)total * (double)x[0].heads / (double)all + 0.5);
  bq = std::max(1, std::min(bq, total));
  const int bk = units[1] > 0 ? std::max(1, total - bq) : 0;
  p.blocks_q = bq;
  const int grid = bq + bk;
  if (any_dw) {
    const size_t need = (size_t)grid * D * sizeof(float);
    if (!ws || ws_bytes < need)
      return fail(DT_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(DT_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    p.part = static_cast<float*>(ws);
  }
  if ((st = bind_device_of(x[0].heads && p.tokens ? p.y[0].slot[0].ptr : any_dw ? p.dw[0] ? p.dw[0] : p.dw[1] : nullptr)) !=
      DT_OK)
    return st;
  p.status = device_status_word(d_status);
  if (!p.status) return fail(DT_ERR_CUDA, "no device status word");
  cudaError_t e = x[0].dtype == DT_BF16 ? (bwd ? launch_norm<__nv_bfloat16, true>(p, vec, grid, stream)
                                               : launch_norm<__nv_bfloat16, false>(p, vec, grid, stream))
                                        : (bwd ? launch_norm<float, true>(p, vec, grid, stream)
                                               : launch_norm<float, false>(p, vec, grid, stream));
  if (e != cudaSuccess) return fail(DT_ERR_CUDA, "qk_norm_rope launch: %s", cudaGetErrorString(e));
  count_launch();
  if (any_dw) {
    e = launch_early(qk_norm_dw_kernel, dim3((D + 31) / 32, n), DW_THREADS, 0, stream, p, grid);
    if (e != cudaSuccess) return fail(DT_ERR_CUDA, "qk_norm_rope dw launch: %s", cudaGetErrorString(e));
    count_launch();
  }
  return DT_OK;
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" dt_status dt_tp_qk_norm_rope(const dt_dtensor* q, const dt_dtensor* k, const dt_dtensor* q_weight,
                                        const dt_dtensor* k_weight, const dt_dtensor* cos_sin,
                                        const dt_dtensor* positions, const dt_dtensor* q_out, const dt_dtensor* k_out,
                                        int32_t head_dim, float eps, int32_t interleaved, int32_t tp_mesh_dim,
                                        int32_t* d_status, dt_stream_t stream) {
  return no_throw([&] {
    NormArgs a{nullptr, nullptr, q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, nullptr, nullptr};
    return norm_call(false, a, head_dim, eps, interleaved, tp_mesh_dim, nullptr, 0, d_status,
                     reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" dt_status dt_tp_qk_norm_rope_backward(const dt_dtensor* dq_out, const dt_dtensor* dk_out,
                                                 const dt_dtensor* q, const dt_dtensor* k, const dt_dtensor* q_weight,
                                                 const dt_dtensor* k_weight, const dt_dtensor* cos_sin,
                                                 const dt_dtensor* positions, const dt_dtensor* dq,
                                                 const dt_dtensor* dk, const dt_dtensor* dq_weight,
                                                 const dt_dtensor* dk_weight, int32_t head_dim, float eps,
                                                 int32_t interleaved, int32_t tp_mesh_dim, void* workspace,
                                                 size_t workspace_bytes, int32_t* d_status, dt_stream_t stream) {
  return no_throw([&] {
    NormArgs a{dq_out, dk_out, q, k, q_weight, k_weight, cos_sin, positions, dq, dk, dq_weight, dk_weight};
    return norm_call(true, a, head_dim, eps, interleaved, tp_mesh_dim, workspace, workspace_bytes, d_status,
                     reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" dt_status dt_tp_qk_norm_rope_backward_workspace_size(int32_t head_dim, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(DT_ERR_INVALID_ARG, "bytes is NULL");
  if (head_dim < 2 || head_dim > NR_MAX_D) return fail(DT_ERR_UNSUPPORTED, "head_dim %d (2 .. %d)", head_dim, NR_MAX_D);
  *bytes = (size_t)NR_MAX_BLOCKS * head_dim * sizeof(float);
  return DT_OK;
}
