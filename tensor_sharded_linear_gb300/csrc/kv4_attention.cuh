// Attention of a few queries per sequence over the paged 4-bit cache: decode
// steps, drafts, and any other call (long prompts in slices of rows).
//
// Mathematics.  With codes c, steps s and minima m of a key's groups,
//   q . k  = sum over groups of  s_g (q_g . c_g) + m_g sum(q_g)
//   O      = sum over keys of    (p s'_g) c'_g  +  p m'_g
// so the matrix products run on the integer codes and the parameters enter
// as one multiply-add per key, row and group.  A code becomes a bf16 number
// by putting its nibble into the mantissa of 128 (a shift and a logic
// operation for two codes): 128 + c.  For q . k the products see that, and
// 128 sum(q_g) comes off in the multiply-add.  For O one subtraction per two
// codes makes it c - 8 and the minimum m + 8 s: the products are then centred
// like the values they stand for, where an offset of 128 (or codes of mean
// 7.5) would cancel against the sum of all p s' and lose what a long sequence
// averages to (measured at 131071 keys: 1.0% off with 128 + c).  fp32
// activations enter as three bf16 parts (24 bits), with centred codes on both
// sides; each tile's product is then added to the sums in the ordinary fp32
// adder, which rounds to nearest where the matrix unit's own accumulation
// truncates.
//
// The softmax runs in one pass with a running maximum and sum in fp32.  The
// products are S^T = K Q^T (16 keys x 8 rows x 16 channels) and
// O^T = V^T P^T, so 8 (query, head) rows fill the narrow side: the 4 or 8
// query heads that share a kv head are the rows, and the accumulators of S^T
// turn into the operand of O^T with one 8 x 8 transpose (movmatrix).
//
// Work.  A unit is (sequence, kv head, block of rows); its keys come in
// blocks of 128.  The device adds up all units' blocks from kv_lens and gives
// every CTA an equal, contiguous share, whatever the lengths: no host
// knowledge of them, no idle SM for one long sequence.  A share that ends
// inside a unit leaves its sums in the workspace, and the join kernel adds
// them.  Inside a CTA each of the four warps takes every fourth tile of 32
// keys with its own ring of bulk copies (a page's records of a head are
// contiguous: one copy per page and tile), so no warp waits for another
// until the unit ends.
//
// Bound: HBM for 1 to 8 rows (every record is read once), instruction issue
// close behind it.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "kv4_attention.h"
#include "ptx_sm103.cuh"

namespace dt {
namespace kv4 {

template <int D>
constexpr int kStages = D <= 128 ? 4 : 3;

template <int D, int G, int NT, int NP>
struct Shape {
  static constexpr int W = kv4_words(D, G);
  static constexpr int NG = D / G;
  static constexpr int WPG = G / 32;        // key code words of a lane in a group
  static constexpr int WL = D / 32;         // key code words of a lane
  static constexpr int MT = G / 16;         // 16-channel tiles of O^T in a group
  static constexpr int RB = 8 * NT;         // rows of a unit
  static constexpr int STAGES = kStages<D>;
  static constexpr int TILE_BYTES = TILE * W * 4;
  static constexpr int RING = WARPS * STAGES * TILE_BYTES;
  static constexpr int QF = NT * NP * WL * 32 * 16;
  static constexpr int MERGE = WARPS * RB * D * 4;
  static constexpr int RING_OR_MERGE = RING > MERGE ? RING : MERGE;
  static constexpr int OFF_QF = RING_OR_MERGE;
  static constexpr int OFF_QS = OFF_QF + QF;
  static constexpr int OFF_ML = OFF_QS + RB * NG * 4;
  static constexpr int OFF_BAR = OFF_ML + WARPS * RB * 8;
  static constexpr int OFF_VM = OFF_BAR + WARPS * STAGES * 8;
  static constexpr int OFF_SCAN = (OFF_VM + WARPS * STAGES * 4 + 15) / 16 * 16;
  static constexpr int SMEM = OFF_SCAN + THREADS * 8 + 16;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Nibble I of both halves of w as bf16 128 + code; CENTRED: code - 8.
template <int I, bool CENTRED>
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
  uint32_t r = ((w >> (4 * I)) & 0x000f000fu) | 0x43004300u;
  if (CENTRED) {
    const __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(&r);
    const __nv_bfloat162 y = __hsub2(x, __floats2bfloat162_rn(136.f, 136.f));
    r = *reinterpret_cast<const uint32_t*>(&y);
  }
  return r;
}

__device__ __forceinline__ float step_of(uint32_t param) { return __uint_as_float(param << 16); }
__device__ __forceinline__ float min_of(uint32_t param) { return __uint_as_float(param & 0xffff0000u); }

// x as NP bf16 parts whose sum is x (to 8 NP bits).
template <int NP>
__device__ __forceinline__ void parts_of(float x, float (&y)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    y[i] = __bfloat162float(__float2bfloat16_rn(x));
    x -= y[i];
  }
}

// One sequence's share of the schedule.
struct Seq {
  int q0, rows, kv, off;  // first token, (query, head) rows per kv head, keys, position of the first query
  int nrb, nblk, klo;     // row blocks, key blocks, first key of the first block
};

template <int RB>
__device__ __forceinline__ Seq seq_info(const AttnParams& p, int b) {
  Seq s;
  s.q0 = p.seq.start(b);
  const int ql = max(0, p.seq.start(b + 1) - s.q0);
  s.kv = p.seq.keys(b);
  s.rows = ql * p.g;
  s.off = s.kv - ql;
  s.nrb = (s.rows + RB - 1) / RB;
  s.klo = p.window ? max(0, s.off - p.window + 1) / TILE * TILE : 0;
  s.nblk = max(1, (s.kv - s.klo + BLOCK - 1) / BLOCK);  // an empty sequence still writes its rows
  return s;
}

__device__ __forceinline__ int64_t cost(const AttnParams& p, const Seq& s) {
  return (int64_t)s.nrb * s.nblk * p.cache.heads;
}

template <int D, int G, int NT, int NP>
__global__ void __launch_bounds__(THREADS) kv4_attention_kernel(const __grid_constant__ AttnParams p) {
  using S = Shape<D, G, NT, NP>;
  using T = typename std::conditional<NP == 1, __nv_bfloat16, float>::type;
  constexpr int W = S::W, NG = S::NG, WPG = S::WPG, WL = S::WL, MT = S::MT, RB = S::RB, STAGES = S::STAGES;
  constexpr bool FULL = NP > 1;  // fp32 activations
  constexpr float KOFF = FULL ? 8.f : -128.f;  // what the key products' codes are offset by, negated
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, ql = lane & 3;
  uint8_t* ring = smem + warp * STAGES * S::TILE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR) + warp * STAGES;
  volatile uint32_t* vmask = reinterpret_cast<volatile uint32_t*>(smem + S::OFF_VM) + warp * STAGES;
  float* qs = reinterpret_cast<float*>(smem + S::OFF_QS);
  float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + S::OFF_SCAN);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(scan + THREADS);
  if (lane == 0)
    for (int i = 0; i < STAGES; ++i) mbar_init(&bars[i], 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  fence_mbar_init();

  // ---- the schedule: this CTA's share [g0, g1) of all units' key blocks
  const int per = (p.seq.batch + THREADS - 1) / THREADS;
  {
    int64_t sum = 0;
    const int b0 = threadIdx.x * per;
    for (int b = b0; b < min(b0 + per, p.seq.batch); ++b) {
      sum += cost(p, seq_info<RB>(p, b));
      if (blockIdx.x == 0 && __ldg(p.seq.kv_lens + b) != p.seq.keys(b)) atomicOr(p.status, DT_DEV_ERR_INDEX);
    }
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    scan[threadIdx.x] = x;  // inclusive within the warp
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += scan[32 * w + 31];
    __syncthreads();
    scan[threadIdx.x] = x + before;
  }
  __syncthreads();
  const int64_t total = scan[THREADS - 1];
  if (threadIdx.x == 0) p.split[blockIdx.x].unit = -1;
  // CTAs that share the work: with fewer blocks than CTAs, one block each (so
  // that every CTA between a split unit's first and last holds a piece)
  const int64_t ncta = min((int64_t)gridDim.x, total);
  if (blockIdx.x >= ncta) return;
  const int64_t g0 = total * blockIdx.x / ncta, g1 = total * (blockIdx.x + 1) / ncta;
  int b = 0;
  int64_t base = 0;
  {
    int lo = 0, hi = THREADS - 1;  // first thread whose inclusive sum exceeds g0
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (scan[mid] > g0) hi = mid;
      else lo = mid + 1;
    }
    b = lo * per;
    base = lo ? scan[lo - 1] : 0;
  }

  uint32_t put = 0, got = 0;  // tiles issued to and taken from this warp's ring
  bool dead = false;          // a wait ran out: load and compute nothing more
  for (int64_t at = g0; at < g1;) {
    Seq s = seq_info<RB>(p, b);
    while (at >= base + cost(p, s)) {
      base += cost(p, s);
      s = seq_info<RB>(p, ++b);
    }
    const int64_t rem = at - base;
    const int unit = (int)(rem / s.nblk), blk0 = (int)(rem - (int64_t)unit * s.nblk);
    const int nb = (int)min((int64_t)(s.nblk - blk0), g1 - at);
    const int hk = unit / s.nrb, row0 = (unit - hk * s.nrb) * RB;
    const int rows = min(RB, s.rows - row0);
    // positions of the block's first and last query, and the keys any of them sees
    const int pos_a = s.off + row0 / p.g, pos_z = s.off + (row0 + rows - 1) / p.g;
    const int khi = p.causal ? min(s.kv, pos_z + 1) : s.kv;
    const int klo = p.window ? max(0, pos_a - p.window + 1) : 0;
    const int32_t* pages = p.page_table + (int64_t)b * p.table_width;
    const int key0 = s.klo + (blk0 * WARPS + warp) * TILE;

    auto issue = [&](int i) {
      const int stage = put % STAGES, j0 = key0 + i * BLOCK, j = j0 + lane;
      ++put;
      bool ok = j < khi && j0 + TILE > klo && !dead;
      const int pg = j / p.cache.page_size, in_pg = j - pg * p.cache.page_size;
      int32_t page = 0;
      if (ok) {
        page = __ldg(pages + pg);
        if (page < 0 || page >= p.cache.pages) {
          ok = false;
          atomicOr(p.status, DT_DEV_ERR_INDEX);
        }
      }
      const uint32_t vm = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) {
        vmask[stage] = vm;
        if (!dead) mbar_expect_tx(&bars[stage], __popc(vm) * W * 4);
      }
      __syncwarp();
      if (ok && (lane == 0 || in_pg == 0)) {
        const int n = min(min(p.cache.page_size - in_pg, TILE - lane), khi - j);
        bulk_load(ring + stage * S::TILE_BYTES + lane * (W * 4),
                  cache_page(p.cache, page, hk) + (int64_t)in_pg * W, n * W * 4, &bars[stage]);
      }
      __syncwarp();
    };
    const int ahead = min(nb, STAGES - 1);
    for (int i = 0; i < ahead; ++i) issue(i);

    // ---- the queries as matrix operands, and their sums per group
    for (int e = warp; e < NT * NG; e += WARPS) {
      const int nt = e / NG, grp = e - nt * NG;
      const int row = row0 + nt * 8 + r;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < WPG; ++j) {
        float x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = 0.f;
        if (nt * 8 + r < rows) {
          const T* q = head_ptr<T>(p.q, s.q0 + row / p.g, hk * p.g + row % p.g, D);
          load8(q + grp * G + 8 * (ql * WPG + j), x);
        }
        float y[8][NP];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          parts_of<NP>(x[c], y[c]);
          sum += x[c];
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          uint4 f;
          f.x = pack_bf16(y[0][n], y[4][n]);
          f.y = pack_bf16(y[1][n], y[5][n]);
          f.z = pack_bf16(y[2][n], y[6][n]);
          f.w = pack_bf16(y[3][n], y[7][n]);
          reinterpret_cast<uint4*>(smem + S::OFF_QF)[((nt * NP + n) * WL + grp * WPG + j) * 32 + lane] = f;
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (ql == 0) qs[(nt * 8 + r) * NG + grp] = sum;
    }
    __syncthreads();
    float qsum[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int e = 0; e < 2; ++e) qsum[nt][grp][e] = qs[(nt * 8 + 2 * ql + e) * NG + grp];

    float o[NT][NG][MT][4], om[NT][NG][2], mx[NT][2], den[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][grp][m][e] = 0.f;
        om[nt][grp][0] = om[nt][grp][1] = 0.f;
      }
      mx[nt][0] = mx[nt][1] = -INFINITY;
      den[nt][0] = den[nt][1] = 0.f;
    }

    for (int i = 0; i < nb; ++i) {
      if (i + ahead < nb) issue(i + ahead);
      const int stage = got % STAGES;
      if (!dead && !mbar_wait_warp(&bars[stage], (got / STAGES) & 1, abort_flag, p.wait_limit_ns)) {
        dead = true;
        if (lane == 0) {
          *abort_flag = 1;
          atomicOr(p.status, DT_DEV_ERR_TIMEOUT);
        }
      }
      ++got;
      const uint32_t vm = vmask[stage];
      if (dead || vm == 0) continue;
      const int j0 = key0 + i * BLOCK;
      const uint32_t* tile = reinterpret_cast<const uint32_t*>(ring + stage * S::TILE_BYTES);

      // ---- S^T for 32 keys: lane holds keys r, r + 8, r + 16, r + 24 and rows 2 ql, 2 ql + 1
      float sv[NT][4][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t* ka = tile + (16 * h + r) * W;
        const uint32_t* kb = ka + 8 * W;
        float acc[NT][NG][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][grp][e] = 0.f;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          uint32_t wa[WPG], wb[WPG];
          if constexpr (WPG == 2) {
            const uint2 a2 = *reinterpret_cast<const uint2*>(ka + grp * 8 + 2 * ql);
            const uint2 b2 = *reinterpret_cast<const uint2*>(kb + grp * 8 + 2 * ql);
            wa[0] = a2.x, wa[1] = a2.y, wb[0] = b2.x, wb[1] = b2.y;
          } else {
            wa[0] = ka[grp * 4 + ql], wb[0] = kb[grp * 4 + ql];
          }
#pragma unroll
          for (int j = 0; j < WPG; ++j) {
            const uint32_t a0 = nibbles<0, FULL>(wa[j]), a1 = nibbles<0, FULL>(wb[j]);
            const uint32_t a2 = nibbles<1, FULL>(wa[j]), a3 = nibbles<1, FULL>(wb[j]);
            const uint32_t a4 = nibbles<2, FULL>(wa[j]), a5 = nibbles<2, FULL>(wb[j]);
            const uint32_t a6 = nibbles<3, FULL>(wa[j]), a7 = nibbles<3, FULL>(wb[j]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int n = 0; n < NP; ++n) {
                const uint4 f = reinterpret_cast<const uint4*>(
                    smem + S::OFF_QF)[((nt * NP + n) * WL + grp * WPG + j) * 32 + lane];
                mma16816(acc[nt][grp], a0, a1, a2, a3, f.x, f.y);
                mma16816(acc[nt][grp], a4, a5, a6, a7, f.z, f.w);
              }
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) sv[nt][2 * h + k][0] = sv[nt][2 * h + k][1] = 0.f;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          const uint32_t pa = ka[D / 4 + grp], pb = kb[D / 4 + grp];
          const float sa = step_of(pa), sb = step_of(pb);
          const float ma = fmaf(KOFF, sa, min_of(pa)), mb = fmaf(KOFF, sb, min_of(pb));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sv[nt][2 * h][e] += fmaf(sa, acc[nt][grp][e], ma * qsum[nt][grp][e]);
              sv[nt][2 * h + 1][e] += fmaf(sb, acc[nt][grp][2 + e], mb * qsum[nt][grp][e]);
            }
        }
      }

      // ---- mask, running maximum, p = 2^(S * scale - maximum)
      const bool masked = vm != 0xffffffffu || (p.causal && j0 + TILE - 1 > pos_a) ||
                          (p.window && j0 <= pos_z - p.window);
      uint32_t hidden = 0;  // bit nt * 8 + k * 2 + e: key k is not seen by row e
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int pos = s.off + (row0 + nt * 8 + 2 * ql + e) / p.g;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = j0 + 8 * k + r;
              if (!((vm >> (8 * k + r)) & 1) || (p.causal && j > pos) || (p.window && j <= pos - p.window)) {
                hidden |= 1u << (nt * 8 + k * 2 + e);
                sv[nt][k][e] = -INFINITY;
              }
            }
          }
      }
      bool grew = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(fmaxf(sv[nt][0][e], sv[nt][1][e]), fmaxf(sv[nt][2][e], sv[nt][3][e])) * p.scale_log2;
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          top[nt][e] = fmaxf(mx[nt][e], t);
          grew = grew || top[nt][e] > mx[nt][e];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = top[nt][e] > mx[nt][e] ? ex2(mx[nt][e] - top[nt][e]) : 1.f;
            mx[nt][e] = top[nt][e];
            den[nt][e] *= f;
#pragma unroll
            for (int grp = 0; grp < NG; ++grp) {
              om[nt][grp][e] *= f;
#pragma unroll
              for (int m = 0; m < MT; ++m) o[nt][grp][m][e] *= f, o[nt][grp][m][2 + e] *= f;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = mx[nt][e] == -INFINITY ? 0.f : mx[nt][e];  // a row that has seen nothing yet
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sv[nt][k][e] = ex2(fmaf(sv[nt][k][e], p.scale_log2, -ref));
            den[nt][e] += sv[nt][k][e];
          }
        }

      // ---- O^T += V^T P^T, 16 keys at a time
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t* va = tile + (16 * h + r) * W + D / 4 + NG;  // parameters of keys r and r + 8
        const uint32_t* vb = va + 8 * W;
        const uint32_t* vw = tile + (16 * h + 2 * ql) * W + D / 8 + (WPG == 2 ? r : r & 3);
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          const float st[2] = {step_of(va[grp]), step_of(vb[grp])};
          const float mid[2] = {fmaf(8.f, st[0], min_of(va[grp])), fmaf(8.f, st[1], min_of(vb[grp]))};
          uint32_t bf[NT][NP][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[2][2];  // [key r / r + 8][row]
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float pe = sv[nt][2 * h + k][e];
                float ps = pe * st[k], pm = pe * mid[k];
                if (masked && (hidden >> (nt * 8 + (2 * h + k) * 2 + e) & 1)) ps = pm = 0.f;  // not 0 * NaN
                x[k][e] = ps;
                om[nt][grp][e] += pm;
              }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y0[NP], y1[NP];
              parts_of<NP>(x[k][0], y0);
              parts_of<NP>(x[k][1], y1);
#pragma unroll
              for (int n = 0; n < NP; ++n) bf[nt][n][k] = transpose8x8(pack_bf16(y0[n], y1[n]));
            }
          }
          const uint32_t* w = vw + grp * (G / 8);
          const uint32_t w0 = w[0], w1 = w[W], w2 = w[8 * W], w3 = w[9 * W];
          const uint32_t sel = WPG == 2 || r < 4 ? 0x5410u : 0x7632u;
#pragma unroll
          for (int half = 0; half < WPG; ++half) {
            const uint32_t x01 = __byte_perm(w0, w1, half ? 0x7632u : sel);
            const uint32_t x23 = __byte_perm(w2, w3, half ? 0x7632u : sel);
            const uint32_t a0 = nibbles<0, true>(x01), a1 = nibbles<1, true>(x01);
            const uint32_t a2 = nibbles<0, true>(x23), a3 = nibbles<1, true>(x23);
            const uint32_t a4 = nibbles<2, true>(x01), a5 = nibbles<3, true>(x01);
            const uint32_t a6 = nibbles<2, true>(x23), a7 = nibbles<3, true>(x23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (FULL) {
                float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int n = NP - 1; n >= 0; --n) {  // small parts first
                  mma16816(t0, a0, a1, a2, a3, bf[nt][n][0], bf[nt][n][1]);
                  mma16816(t1, a4, a5, a6, a7, bf[nt][n][0], bf[nt][n][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][grp][2 * half][e] += t0[e], o[nt][grp][2 * half + 1][e] += t1[e];
              } else {
                mma16816(o[nt][grp][2 * half], a0, a1, a2, a3, bf[nt][0][0], bf[nt][0][1]);
                mma16816(o[nt][grp][2 * half + 1], a4, a5, a6, a7, bf[nt][0][0], bf[nt][0][1]);
              }
            }
          }
        }
      }
      __syncwarp();  // the stage may be refilled
    }

    // ---- the four warps' sums meet in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          den[nt][e] += __shfl_xor_sync(0xffffffffu, den[nt][e], x);
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) om[nt][grp][e] += __shfl_xor_sync(0xffffffffu, om[nt][grp][e], x);
        }
        if (r == 0) ml[warp * RB + nt * 8 + 2 * ql + e] = make_float2(mx[nt][e], den[nt][e]);
      }
    __syncthreads();  // every warp is done with its ring
    float* os = reinterpret_cast<float*>(smem) + warp * RB * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float add = om[nt][grp][e];
            const int ch = grp * G + (WPG == 2 ? 8 * r : 8 * (r & 3) + 4 * (r >> 2)) + 2 * m;
            *reinterpret_cast<float2*>(os + (nt * 8 + 2 * ql + e) * D + ch) =
                make_float2(o[nt][grp][m][e] + add, o[nt][grp][m][2 + e] + add);
          }
    __syncthreads();
    const bool whole = blk0 == 0 && nb == s.nblk;
    const bool first = blk0 == 0;  // of the pieces of a split unit
    const int64_t piece = 2 * (int64_t)blockIdx.x + (first ? 1 : 0);
    for (int x = threadIdx.x; x < rows * (D / 4); x += THREADS) {
      const int row = x / (D / 4), c4 = x - row * (D / 4);
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) m = fmaxf(m, ml[w * RB + row].x);
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 mlw = ml[w * RB + row];
        const float f = ex2(mlw.x - ref);
        const float4 v = reinterpret_cast<const float4*>(smem)[(w * RB + row) * (D / 4) + c4];
        l += mlw.y * f;
        a.x += v.x * f, a.y += v.y * f, a.z += v.z * f, a.w += v.w * f;
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // nothing seen: zeros; NaN stays
        const int qr = row0 + row;
        const int tok = s.q0 + qr / p.g, head = hk * p.g + qr % p.g;
        T* y = head_ptr<T>(p.out, tok, head, D) + 4 * c4;
        if constexpr (NP == 1)
          *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
        else
          *reinterpret_cast<float4*>(y) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        if (p.want_lse && c4 == 0) *head_ptr<float>(p.lse, tok, head, 1) = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      } else {
        float* out = p.part + (piece * RB + row) * (D + 4);
        reinterpret_cast<float4*>(out)[c4] = a;
        if (c4 == 0) out[D] = m, out[D + 1] = l;
      }
    }
    if (threadIdx.x == 0 && first && !whole) {
      // the CTA whose share holds the unit's last block
      const int64_t end = base + (int64_t)(unit + 1) * s.nblk - 1;
      Split sp;
      sp.unit = unit;
      sp.q_row = row0;
      sp.rows = rows;
      sp.q0 = s.q0;
      sp.head = hk;
      sp.last = (int32_t)(((end + 1) * ncta - 1) / total);
      p.split[blockIdx.x] = sp;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring was written by plain stores
    __syncthreads();
    at += nb;
  }
  if (dead) {  // copies issued before a wait gave up: a bounded time to land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 20000000ull) {
    }
  }
}

// Adds the pieces of the units that were split, one CTA per unit and quarter
// of the channels, in the order of the keys.
template <int D, int G, int NT, int NP>
__global__ void __launch_bounds__(THREADS) kv4_join_kernel(const __grid_constant__ AttnParams p) {
  using S = Shape<D, G, NT, NP>;
  using T = typename std::conditional<NP == 1, __nv_bfloat16, float>::type;
  constexpr int RB = S::RB, C4 = D / 16;  // float4s of a quarter
  const Split sp = p.split[blockIdx.x];
  if (sp.unit < 0) return;
  for (int x = threadIdx.x; x < sp.rows * C4; x += THREADS) {
    const int row = x / C4, c4 = blockIdx.y * C4 + x % C4;
    float m = -INFINITY;
    for (int c = blockIdx.x; c <= sp.last; ++c) {
      const int64_t piece = 2 * (int64_t)c + (c == (int)blockIdx.x ? 1 : 0);
      m = fmaxf(m, p.part[(piece * RB + row) * (D + 4) + D]);
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = blockIdx.x; c <= sp.last; ++c) {
      const int64_t piece = 2 * (int64_t)c + (c == (int)blockIdx.x ? 1 : 0);
      const float* in = p.part + (piece * RB + row) * (D + 4);
      const float f = ex2(in[D] - ref);
      const float4 v = reinterpret_cast<const float4*>(in)[c4];
      l += in[D + 1] * f;
      a.x += v.x * f, a.y += v.y * f, a.z += v.z * f, a.w += v.w * f;
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    const int qr = sp.q_row + row;
    const int tok = sp.q0 + qr / p.g, head = sp.head * p.g + qr % p.g;
    T* y = head_ptr<T>(p.out, tok, head, D) + 4 * c4;
    if constexpr (NP == 1)
      *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    else
      *reinterpret_cast<float4*>(y) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if (p.want_lse && c4 == 0)
      *head_ptr<float>(p.lse, tok, head, 1) = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, int G, int NT, int NP>
cudaError_t variant_of(Variant* out) {
  using S = Shape<D, G, NT, NP>;
  static int per_sm[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!per_sm[dev]) {
    e = cudaFuncSetAttribute(kv4_attention_kernel<D, G, NT, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv4_attention_kernel<D, G, NT, NP>, THREADS, S::SMEM);
    if (e != cudaSuccess) return e;
    per_sm[dev] = n > 0 ? n : 1;
  }
  out->grid = device_sm_count() * per_sm[dev];
  out->rows = S::RB;
  const size_t splits = ((size_t)out->grid * sizeof(Split) + 255) / 256 * 256;
  out->bytes = splits + (size_t)2 * out->grid * S::RB * (D + 4) * sizeof(float);
  return cudaSuccess;
}

template <int D, int G, int NT, int NP>
cudaError_t launch_of(const AttnParams& p, int grid, cudaStream_t s) {
  kv4_attention_kernel<D, G, NT, NP><<<grid, THREADS, Shape<D, G, NT, NP>::SMEM, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kv4_join_kernel<D, G, NT, NP><<<dim3(grid, 4), THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

// Rows of a unit: 8 for fp32 (three parts per operand) and for up to 8 rows
// per sequence and kv head; 16 beyond that where the accumulators fit
// (head_dim 64 and 128).
template <int D>
cudaError_t variant(int G, bool fp32, int64_t rows_per_seq, Variant* out) {
  constexpr int NTMAX = D <= 128 ? 2 : 1;
  if (fp32) return G == 32 ? variant_of<D, 32, 1, 3>(out) : variant_of<D, 64, 1, 3>(out);
  if (rows_per_seq <= 8) return G == 32 ? variant_of<D, 32, 1, 1>(out) : variant_of<D, 64, 1, 1>(out);
  return G == 32 ? variant_of<D, 32, NTMAX, 1>(out) : variant_of<D, 64, NTMAX, 1>(out);
}

template <int D>
cudaError_t launch(const AttnParams& p, int G, bool fp32, int64_t rows_per_seq, int grid, cudaStream_t s) {
  constexpr int NTMAX = D <= 128 ? 2 : 1;
  if (fp32) return G == 32 ? launch_of<D, 32, 1, 3>(p, grid, s) : launch_of<D, 64, 1, 3>(p, grid, s);
  if (rows_per_seq <= 8) return G == 32 ? launch_of<D, 32, 1, 1>(p, grid, s) : launch_of<D, 64, 1, 1>(p, grid, s);
  return G == 32 ? launch_of<D, 32, NTMAX, 1>(p, grid, s) : launch_of<D, 64, NTMAX, 1>(p, grid, s);
}

}  // namespace kv4
}  // namespace dt
