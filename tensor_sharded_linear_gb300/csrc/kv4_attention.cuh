// Attention of a few queries per sequence over the paged 4-bit cache: decode
// steps, drafts, and any other call (long prompts in slices of rows).
//
// Mathematics.  With codes c, steps s and minima m of a key's groups,
//   q . k  = sum over groups of  s_g (q_g . c_g) + m_g sum(q_g)
//   O      = sum over keys of    (p s'_g) c'_g  +  p m'_g
// so the matrix products run on the integer codes and the parameters enter
// as a multiply-add per key, row and group, and as one small product with the
// parameter words as they lie in memory.
// bf16 activations: fp16 products.  An fp16 number below 2^-13 is its bit
// pattern times 2^-24, subnormal or not, so a masked nibble IS code * 2^-24
// (bits 0..3) or 16 * code * 2^-24 (bits 4..7): two codes cost one logic
// operation and a quarter of a shift.  Queries are scaled per row by a power
// of two to [2^10, 2^11), where a bf16 number fits fp16 exactly unless it is
// 2^-25 of the row's largest.  p s' is scaled by the power of two that keeps
// the largest step seen below 2^12: eleven bits for whatever is within 2^-26
// of it.
// The accumulators of a long sequence have to be centred: a code's mean of
// 7.5 would cancel against the sum of all p m' and take the low bits along
// (the matrix unit truncates; an offset of 128 cost 1.0% at 131071 keys in
// runs of 2900).  So each tile adds -8 times its sum of p s' as rounded, which
// one more product per 16 keys and group forms in fp32 (a sum taken in fp16
// instead cost an error of 2^-10 of the result), and m' becomes m' + 8 s'.
// fp32 activations: three bf16 parts (24 bits) times codes - 8 made from the
// nibble in the mantissa of 128; each tile's product is added to the sums in
// the ordinary fp32 adder, which rounds to nearest.
//
// The softmax runs in one pass with a running maximum and sum in fp32.  The
// products are S^T = K Q^T (16 keys x 8 rows x 16 channels) and
// O^T = V^T P^T, so 8 (query, head) rows fill the narrow side: the 4 or 8
// query heads that share a kv head are the rows, and the accumulators of S^T
// turn into the operand of O^T with one 8 x 8 transpose (movmatrix).
//
// Work.  A unit is (sequence, kv head, block of rows); its keys come in
// blocks of four tiles.  The device adds up all units' blocks from kv_lens
// and gives every CTA an equal, contiguous share, whatever the lengths: no
// host knowledge of them, no idle SM for one long sequence.  A share that ends
// inside a unit leaves its sums in the workspace, and the join kernel adds
// them.  Inside a CTA each of the four warps takes every fourth tile of 64
// keys (32 at head_dim 256) with its own ring of bulk copies (a page's records
// of a head are contiguous: one copy per page and tile), so no warp waits for
// another until the unit ends.
//
// Bound: the instructions and their latency at the 12 warps an SM has room for
// (168 registers each), HBM next.  48 sequences of up to 8192 keys, 32/8 heads
// of 128: 68.2 us for 252 MB of records, 3.7 TB/s; the same loads without the
// arithmetic 48.3, the arithmetic without the loads 63.8.  Five sequences of
// 131071: 94.2 us for 436 MB, 4.6 TB/s (73.6 and 91.5).  One sequence of 4097:
// 11.9 us (9.5 and 11.5), launches and latency.  Tiles of 32 keys with up to
// five CTAs an SM: 81 to 153 us where these take 68.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "kv4_attention.h"
#include "kv4_join.cuh"
#include "ptx_sm103.cuh"

namespace dt {
namespace kv4 {

template <int D, int G, int NT, int NP>
struct Shape {
  static constexpr int W = kv4_words(D, G);
  static constexpr int NG = D / G;
  static constexpr int WPG = G / 32;        // key code words of a lane in a group
  static constexpr int WL = D / 32;         // key code words of a lane
  static constexpr int MT = G / 16;         // 16-channel tiles of O^T in a group
  static constexpr int RB = 8 * NT;         // rows of a unit
  static constexpr int TILE = D <= 128 ? 64 : 32;  // keys of a warp's tile
  static constexpr int HT = TILE / 16;
  static constexpr int BLOCK = TILE * WARPS;       // keys of a step of the schedule
  static constexpr int STAGES = 2;
  // products that carry the parameters' share of q . k: 3 parts of each
  // group's sum(q), 8 pairs (step, minimum) a product
  static constexpr int PM = (3 * NG + 7) / 8;
  static constexpr int TILE_BYTES = TILE * W * 4;
  static constexpr int RING = WARPS * STAGES * TILE_BYTES;
  static constexpr int QF = NT * NP * WL * 32 * 16;
  static_assert(RB * D * 4 <= TILE_BYTES, "a warp's sums fit one stage of its ring");
  static constexpr int OFF_QF = RING;
  static constexpr int OFF_QS = OFF_QF + QF;
  static constexpr int OFF_ML = OFF_QS + RB * (NG + 1) * 4;
  static constexpr int OFF_BAR = OFF_ML + WARPS * RB * 8;
  static constexpr int OFF_VM = OFF_BAR + WARPS * STAGES * 8;
  static constexpr int OFF_ABORT = OFF_VM + WARPS * STAGES * 8;
  static constexpr int SMEM = OFF_ABORT + 16;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// fp16 operands; accumulators d = c + a b.
__device__ __forceinline__ void mma16816_h(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_h_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Nibbles 0..3 of both halves of w as four operand registers.
// FULL: bf16 code - 8.  `one` is 0x43004300 in a register that the compiler
// does not see through: mask and exponent go in with one LOP3, where two
// immediates would take two.  Else fp16: code * 2^-24 (0 and 2) and 16 times
// that (1 and 3).
template <bool FULL>
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t one, uint32_t (&n)[4]) {
  if constexpr (FULL) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(n[i]) : "r"(w >> (4 * i)), "r"(one));  // (a & b) | c
      const __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(&n[i]);
      const __nv_bfloat162 y = __hsub2(x, __floats2bfloat162_rn(136.f, 136.f));
      n[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
  } else {
    const uint32_t h = w >> 8;
    n[0] = w & 0x000f000fu, n[1] = w & 0x00f000f0u, n[2] = h & 0x000f000fu, n[3] = h & 0x00f000f0u;
  }
}
__device__ __forceinline__ uint32_t exponent_of_128() {
  uint32_t r;
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(r));
  return r;
}

// N consecutive words of shared memory, as wide as their number allows (the
// callers' addresses are aligned to that).
template <int N>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p + i);
      w[i] = v.x, w[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = p[i];
  }
}

__device__ __forceinline__ float step_of(uint32_t param) { return __uint_as_float(param << 16); }
__device__ __forceinline__ float min_of(uint32_t param) { return __uint_as_float(param & 0xffff0000u); }

// x as NP bf16 parts whose sum is x (to 8 NP bits).
template <int NP>
__device__ __forceinline__ void parts_of(float x, float (&y)[NP]) {
  if constexpr (NP == 1) {
    y[0] = x;  // rounded where it is packed
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      y[i] = __bfloat162float(__float2bfloat16_rn(x));
      x -= y[i];
    }
  }
}

// One sequence's share of the schedule.
struct Seq {
  int q0, rows, kv, off;  // first token, (query, head) rows per kv head, keys, position of the first query
  int nrb, nblk, klo;     // row blocks, key blocks, first key of the first block
};

// Besides its blocks of keys a unit counts one more in the schedule, after
// them, for its start and end (measured at 48 sequences of 800 to 8192 keys:
// without it the busiest SM worked 22% longer than the average).
constexpr int UNIT_EXTRA = 1;

template <int RB, int TILE>
__device__ __forceinline__ Seq seq_info(const AttnParams& p, int b) {
  Seq s;
  s.q0 = p.seq.start(b);
  const int ql = max(0, p.seq.start(b + 1) - s.q0);
  s.kv = p.seq.keys(b);
  s.rows = ql * p.g;
  s.off = s.kv - ql;
  s.nrb = (s.rows + RB - 1) / RB;
  s.klo = window_begin(s.off, p.window) / TILE * TILE;
  s.nblk = max(1, (s.kv - s.klo + TILE * WARPS - 1) / (TILE * WARPS));  // an empty sequence still writes its rows
  return s;
}

__device__ __forceinline__ int64_t cost(const AttnParams& p, const Seq& s) {
  return (int64_t)s.nrb * (s.nblk + UNIT_EXTRA) * p.cache.heads;
}

template <int D, int G, int NT, int NP>
__global__ void __launch_bounds__(THREADS, NP == 1 && NT * D <= 128 ? 3 : 2)
    kv4_attention_kernel(const __grid_constant__ AttnParams p) {
  using S = Shape<D, G, NT, NP>;
  using T = typename std::conditional<NP == 1, __nv_bfloat16, float>::type;
  constexpr int W = S::W, NG = S::NG, WPG = S::WPG, MT = S::MT, RB = S::RB, STAGES = S::STAGES;
  constexpr int WL = S::WL, TILE = S::TILE, HT = S::HT, BLOCK = S::BLOCK, PM = S::PM;
  constexpr bool FULL = NP > 1;  // fp32 activations
  constexpr float KOFF = FULL ? 8.f : 0.f;  // what the key products' codes are offset by, negated
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, ql = lane & 3;
  uint8_t* ring = smem + warp * STAGES * S::TILE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR) + warp * STAGES;
  volatile uint64_t* vmask = reinterpret_cast<volatile uint64_t*>(smem + S::OFF_VM) + warp * STAGES;
  float* qs = reinterpret_cast<float*>(smem + S::OFF_QS);
  float* rsc = qs + RB * NG;
  float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);
  int64_t* scan = reinterpret_cast<int64_t*>(smem);  // before the ring is in use
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::OFF_ABORT);
  const uint32_t one = exponent_of_128();
  if (lane == 0)
    for (int i = 0; i < STAGES; ++i) mbar_init(&bars[i], 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  fence_mbar_init();
  wait_for_previous_kernel();

  // ---- the schedule: this CTA's share [g0, g1) of all units' key blocks
  const int per = (p.seq.batch + THREADS - 1) / THREADS;
  {
    int64_t sum = 0;
    const int b0 = threadIdx.x * per;
    for (int b = b0; b < min(b0 + per, p.seq.batch); ++b) {
      sum += cost(p, seq_info<RB, TILE>(p, b));
      if (blockIdx.x == 0 && load_plain(p.seq.kv_lens + b) != p.seq.keys(b)) atomicOr(p.status, DT_DEV_ERR_INDEX);
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
  if (blockIdx.x >= ncta) return;  // (a CTA that leaves allows the next kernel too)
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
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring was written by plain stores
  __syncthreads();

  uint32_t put = 0, got = 0;  // tiles issued to and taken from this warp's ring
  bool dead = false;          // a wait ran out: load and compute nothing more
  const int ps = p.cache.page_size;

  // A unit's part within this CTA's share.
  struct Segment {
    int q0, off, row0, rows;   // first token of the sequence, its first query's position; rows of the unit
    int hk, unit, nb;          // kv head; the unit's number within the sequence; key blocks here
    int key0, klo, khi;        // this warp's first key; the keys any row sees
    int pos_a, pos_z;          // positions of the first and last query
    bool first, whole;         // holds the unit's first block; all of them
    int last;                  // CTA with the unit's last block (set where first)
    const int32_t *pages, *base;  // the sequence's page table row; the head's records in page 0
    int64_t page_stride;
  };
  int64_t at = g0;
  // The next segment of the share and true, or false at its end.
  auto advance = [&](Segment& x) {
    while (at < g1) {
      Seq s = seq_info<RB, TILE>(p, b);
      while (at >= base + cost(p, s)) {
        base += cost(p, s);
        s = seq_info<RB, TILE>(p, ++b);
      }
      const int64_t rem = at - base;
      const int width = s.nblk + UNIT_EXTRA;
      x.unit = (int)(rem / width);
      const int blk0 = (int)(rem - (int64_t)x.unit * width);
      at = min(g1, base + (int64_t)(x.unit + 1) * width);
      if (blk0 >= s.nblk) continue;  // only the unit's extra
      x.nb = (int)min((int64_t)(s.nblk - blk0), at - rem - base);
      x.hk = x.unit / s.nrb;
      x.row0 = (x.unit - x.hk * s.nrb) * RB;
      x.rows = min(RB, s.rows - x.row0);
      x.q0 = s.q0;
      x.off = s.off;
      x.pos_a = s.off + x.row0 / p.g;
      x.pos_z = s.off + (x.row0 + x.rows - 1) / p.g;
      x.khi = p.causal ? min(s.kv, x.pos_z + 1) : s.kv;
      x.klo = window_begin(x.pos_a, p.window);
      x.key0 = s.klo + (blk0 * WARPS + warp) * TILE;
      x.first = blk0 == 0;
      x.whole = x.first && x.nb == s.nblk;
      x.last = (int)(((base + (int64_t)x.unit * width + s.nblk) * ncta - 1) / total);
      x.pages = p.page_table + (int64_t)b * p.table_width;
      const int slot = x.hk / p.cache.per_slot;
      x.page_stride = p.cache.page_stride[slot];
      x.base = p.cache.ptr[slot] + (int64_t)(x.hk - slot * p.cache.per_slot) * p.cache.head_stride[slot];
      return true;
    }
    return false;
  };

  // A tile's keys lie in runs of consecutive records, one per page: lane n
  // copies run n.  Its page is looked up a tile ahead (`ready`).  Keys of the
  // first tile that no row sees (behind the window) are left out: their pages
  // need not exist.
  auto first_page = [&](int j0) { return (int)(__umulhi(2u * (uint32_t)j0, p.page_mul) >> p.page_shift); };
  auto look_up = [&](const Segment& x, int i) {
    const int j0 = x.key0 + i * BLOCK, pg = first_page(max(j0, x.klo)) + lane;
    return i < x.nb && (int64_t)pg * ps < min(j0 + TILE, x.khi) ? load_plain(x.pages + pg) : -1;
  };
  int32_t ready;
  auto issue = [&](const Segment& x, int i) {
    const int stage = put % STAGES, j0 = x.key0 + i * BLOCK;
    ++put;
    const int begin = max(j0, x.klo), end = dead ? begin : min(j0 + TILE, x.khi);
    const int pg0 = first_page(begin), n_keys = max(0, end - begin);
    uint64_t vm = n_keys >= 64 ? ~0ull : ((1ull << n_keys) - 1) << ((begin - j0) & 63);
    const int nruns = n_keys ? first_page(end - 1) - pg0 + 1 : 0;
    uint32_t* dst = reinterpret_cast<uint32_t*>(ring + stage * S::TILE_BYTES);
    for (int n0 = 0; n0 < nruns; n0 += 32) {
      const int n = n0 + lane;
      const int32_t page = n0 == 0 ? ready : n < nruns ? load_plain(x.pages + pg0 + n) : 0;
      const bool ok = n >= nruns || (page >= 0 && page < p.cache.pages);
      if (!__all_sync(0xffffffffu, ok)) {  // pages that are none: their keys are hidden
        if (lane == 0) atomicOr(p.status, DT_DEV_ERR_INDEX);
        uint64_t bad = 0;
        if (!ok) {
          const int a = max(begin, (pg0 + n) * ps) - j0, z = min(end, (pg0 + n + 1) * ps) - j0;
          bad = (z - a >= 64 ? ~0ull : (1ull << (z - a)) - 1) << a;
        }
        for (int o = 16; o; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
        vm &= ~bad;
      }
    }
    if (lane == 0) {
      vmask[stage] = vm;
      if (!dead) mbar_expect_tx(&bars[stage], __popcll(vm) * W * 4 + (put > p.starve ? 16 : 0));
    }
    __syncwarp();
    for (int n = lane; n < nruns; n += 32) {
      const int32_t page = n < 32 ? ready : load_plain(x.pages + pg0 + n);
      if (page < 0 || page >= p.cache.pages) continue;
      const int a = max(begin, (pg0 + n) * ps), z = min(end, (pg0 + n + 1) * ps);
      bulk_load(dst + (a - j0) * W, x.base + page * x.page_stride + (int64_t)(a - (pg0 + n) * ps) * W,
                (z - a) * W * 4, &bars[stage]);
    }
    ready = look_up(x, i + 1);
    __syncwarp();
  };
  // The queries of a segment as loaded (warp nt holds 8 rows).
  Raw8<T> qraw[WL];
  auto load_queries = [&](const Segment& x) {
    const int row = x.row0 + warp * 8 + r;
    if (warp < NT && warp * 8 + r < x.rows) {
      const T* q = head_ptr<T>(p.q, x.q0 + row / p.g, x.hk * p.g + row % p.g, D);
#pragma unroll
      for (int w = 0; w < WL; ++w) qraw[w].load(q + w / WPG * G + 8 * (ql * WPG + w % WPG));
    } else {
#pragma unroll
      for (int w = 0; w < WL; ++w) qraw[w].zero();
    }
  };

  allow_next_kernel();  // the join's CTAs find room as this kernel's leave
  Segment next;
  if (!advance(next)) return;
  ready = look_up(next, 0);
  load_queries(next);
  issue(next, 0);
  while (true) {
    const Segment s = next;
    const int nb = s.nb, hk = s.hk, row0 = s.row0, rows = s.rows, pos_a = s.pos_a, pos_z = s.pos_z, key0 = s.key0;

    // ---- the queries as matrix operands, and their sums per group: warp nt takes 8 rows
    if (warp < NT) {
      const int nt = warp;
      float x[WL][8];
#pragma unroll
      for (int w = 0; w < WL; ++w) qraw[w].get(x[w]);
      float mult = 1.f;
      if constexpr (!FULL) {
        float top = 0.f;
#pragma unroll
        for (int w = 0; w < WL; ++w)
#pragma unroll
          for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(x[w][c]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = __float_as_uint(top) >> 23;  // 2^10 / 2^(exponent of top), within the normal numbers
        mult = __uint_as_float((uint32_t)max(10, min(254, 264 - ex)) << 23);
      }
      // (never 0: a hidden key's -inf times it has to stay -inf)
      if (ql == 0) rsc[nt * 8 + r] = FULL ? p.scale_log2 : fmaxf(p.scale_log2 * 16777216.f / mult, LEAST_SCALE);
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < WPG; ++j) {
          const int w = grp * WPG + j;
          float y[8][NP];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            x[w][c] *= mult;
            sum += x[w][c];
            if (!FULL && (c & 1)) x[w][c] *= 0.0625f;  // the odd nibbles come out 16 times as large
            parts_of<NP>(x[w][c], y[c]);
          }
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            uint4 f;
            if constexpr (FULL)
              f = make_uint4(pack_bf16(y[0][n], y[4][n]), pack_bf16(y[1][n], y[5][n]), pack_bf16(y[2][n], y[6][n]),
                             pack_bf16(y[3][n], y[7][n]));
            else
              f = make_uint4(pack_f16(y[0][n], y[4][n]), pack_f16(y[1][n], y[5][n]), pack_f16(y[2][n], y[6][n]),
                             pack_f16(y[3][n], y[7][n]));
            reinterpret_cast<uint4*>(smem + S::OFF_QF)[((nt * NP + n) * WL + w) * 32 + lane] = f;
          }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // beside fp16 products of codes * 2^-24
        if (ql == 0) qs[(nt * 8 + r) * NG + grp] = FULL ? sum : sum * 5.9604644775390625e-8f;
      }
    }
    __syncthreads();
    float sc[NT][2];  // softmax scale * log2(e) of the lane's rows, their queries' scaling undone
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = rsc[nt * 8 + 2 * ql], sc[nt][1] = rsc[nt * 8 + 2 * ql + 1];
    // The parameters' share of S as products: row k of the narrow operand is
    // KOFF sum(q_g) beside a step and sum(q_g) beside a minimum, in three
    // bf16 parts; the wide operand is the keys' parameter words as they are.
    // Pair n of the products' 8 PM is part n / NG of group n % NG.
    uint32_t qm[NT][PM][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mm = 0; mm < PM; ++mm)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = mm * 8 + h * 4 + ql, part = n / NG;
          float x = qs[(nt * 8 + r) * NG + n % NG], y[3];
          parts_of<3>(x, y);
          x = part == 0 ? y[0] : part == 1 ? y[1] : part == 2 ? y[2] : 0.f;
          qm[nt][mm][h] = pack_bf16(KOFF * x, x);
        }

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
    // 2^12 over the power of two above the largest value step that some row has seen (one for all rows: a row's own
    // takes 73.1 and 96.6 us where this takes 67.9 and 93.9)
    uint32_t step_ex = 0;  // its exponent field
    float vmult = __uint_as_float(254u << 23);

    for (int i = 0; i < nb; ++i) {
      if (i + 1 < nb) issue(s, i + 1);
      const int stage = got % STAGES;
      if (!dead && !mbar_wait_warp(&bars[stage], (got / STAGES) & 1, abort_flag, p.wait_limit_ns)) {
        dead = true;
        if (lane == 0) {
          *abort_flag = 1;
          atomicOr(p.status, DT_DEV_ERR_TIMEOUT);
        }
      }
      ++got;
      const uint64_t vm = vmask[stage];
      if (dead || vm == 0) {
        __syncwarp();
        continue;
      }
      const int j0 = key0 + i * BLOCK;
      const uint32_t* tile = reinterpret_cast<const uint32_t*>(ring + stage * S::TILE_BYTES);

      // ---- S^T: of every 16 keys a lane holds keys r and r + 8, rows 2 ql and 2 ql + 1
      float sv[NT][2 * HT][2];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const uint32_t* ka = tile + (16 * h + r) * W;
        const uint32_t* kb = ka + 8 * W;
        float acc[NT][NG][4], base_[NT][4];
        {
          const uint32_t a0 = ka[D / 4 + ql % NG], a1 = kb[D / 4 + ql % NG];
          const uint32_t a2 = NG == 8 ? ka[D / 4 + 4 + ql] : a0, a3 = NG == 8 ? kb[D / 4 + 4 + ql] : a1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mm = 0; mm < PM; ++mm) {
              if (mm == 0) mma16816_first(base_[nt], a0, a1, a2, a3, qm[nt][mm][0], qm[nt][mm][1]);
              else mma16816(base_[nt], a0, a1, a2, a3, qm[nt][mm][0], qm[nt][mm][1]);
            }
        }
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          uint32_t wa[WPG], wb[WPG];
          load_words<WPG>(ka + grp * (G / 8) + WPG * ql, wa);
          load_words<WPG>(kb + grp * (G / 8) + WPG * ql, wb);
#pragma unroll
          for (int j = 0; j < WPG; ++j) {
            uint32_t ca[4], cb[4];
            nibbles<FULL>(wa[j], one, ca);
            nibbles<FULL>(wb[j], one, cb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int n = 0; n < NP; ++n) {
                const uint4 f = reinterpret_cast<const uint4*>(
                    smem + S::OFF_QF)[((nt * NP + n) * WL + grp * WPG + j) * 32 + lane];
                if constexpr (FULL) {
                  if (j == 0 && n == 0) mma16816_first(acc[nt][grp], ca[0], cb[0], ca[1], cb[1], f.x, f.y);
                  else mma16816(acc[nt][grp], ca[0], cb[0], ca[1], cb[1], f.x, f.y);
                  mma16816(acc[nt][grp], ca[2], cb[2], ca[3], cb[3], f.z, f.w);
                } else {
                  if (j == 0) mma16816_h_first(acc[nt][grp], ca[0], cb[0], ca[1], cb[1], f.x, f.y);
                  else mma16816_h(acc[nt][grp], ca[0], cb[0], ca[1], cb[1], f.x, f.y);
                  mma16816_h(acc[nt][grp], ca[2], cb[2], ca[3], cb[3], f.z, f.w);
                }
              }
            }
          }
        }
        uint32_t pa[NG], pb[NG];
        load_words<NG>(ka + D / 4, pa);
        load_words<NG>(kb + D / 4, pb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = base_[nt][e], y = base_[nt][2 + e];
#pragma unroll
            for (int grp = 0; grp < NG; ++grp) {
              x = fmaf(step_of(pa[grp]), acc[nt][grp][e], x);
              y = fmaf(step_of(pb[grp]), acc[nt][grp][2 + e], y);
            }
            sv[nt][2 * h][e] = x, sv[nt][2 * h + 1][e] = y;
          }
      }

      // ---- mask, running maximum, p = 2^(S * scale - maximum)
      constexpr uint64_t ALL = TILE == 64 ? ~0ull : (1ull << TILE) - 1;
      const bool masked = vm != ALL || (p.causal && j0 + TILE - 1 > pos_a) || j0 < window_begin(pos_z, p.window);
      uint32_t hidden[NT];  // bit 2 k + e: key 8 k + r is not seen by row 2 ql + e
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) hidden[nt] = 0;
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int pos = s.off + (row0 + nt * 8 + 2 * ql + e) / p.g, lo = window_begin(pos, p.window);
#pragma unroll
            for (int k = 0; k < 2 * HT; ++k) {
              const int j = j0 + 8 * k + r;
              if (!((vm >> (8 * k + r)) & 1) || (p.causal && j > pos) || j < lo) {
                hidden[nt] |= 1u << (k * 2 + e);
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
          float t = sv[nt][0][e];
#pragma unroll
          for (int k = 1; k < 2 * HT; ++k) t = fmaxf(t, sv[nt][k][e]);
          t *= sc[nt][e];
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
      for (int nt = 0; nt < NT; ++nt) {
        f2 less, sum = both(0.f);  // (0 for a row that has seen nothing yet)
        less.x = mx[nt][0] == -INFINITY ? 0.f : -mx[nt][0];
        less.y = mx[nt][1] == -INFINITY ? 0.f : -mx[nt][1];
#pragma unroll
        for (int k = 0; k < 2 * HT; ++k) {
          const f2 y = fma2(f2{sv[nt][k][0], sv[nt][k][1]}, f2{sc[nt][0], sc[nt][1]}, less);
          sv[nt][k][0] = ex2(y.x), sv[nt][k][1] = ex2(y.y);
          sum = sum + f2{sv[nt][k][0], sv[nt][k][1]};
        }
        den[nt][0] += sum.x, den[nt][1] += sum.y;
      }

      // ---- O^T += V^T P^T, 16 keys at a time
      float csum[NT][NG][4];  // -8 (even nibbles) and -128 (odd ones, 16 times as large) times 2^-24 times the sums of p s'
      uint32_t vp[HT][2][NG];  // value parameters of keys r and r + 8
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) load_words<NG>(tile + (16 * h + 8 * k + r) * W + D / 4 + NG, vp[h][k]);
      if (masked) {  // what lies where no key is counts as zero
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int grp = 0; grp < NG; ++grp)
              if (!((vm >> (16 * h + 8 * k + r)) & 1)) vp[h][k][grp] = 0;
      }
      if constexpr (!FULL) {
        uint32_t big = 0;
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int grp = 0; grp < NG; ++grp) big = max(big, vp[h][k][grp] << 16);
        if (__any_sync(0xffffffffu, (big >> 23) > step_ex)) {
          // steps that are not finite (a sign bit or an exponent of ones) do not count
          big = 0;
#pragma unroll
          for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int grp = 0; grp < NG; ++grp) {
                const uint32_t st = vp[h][k][grp] << 16;
                if (st < 0x7f800000u) big = max(big, st);
              }
          const uint32_t ex = max(step_ex, __reduce_max_sync(0xffffffffu, big) >> 23);
          if (ex > step_ex) {
            const float m2 = __uint_as_float(min(254u, 265u - ex) << 23), f = m2 / vmult;
            vmult = m2, step_ex = ex;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int grp = 0; grp < NG; ++grp)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[nt][grp][m][e] *= f;
          }
        }
      }
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const uint32_t* vw = tile + (16 * h + 2 * ql) * W + D / 8 + (WPG == 2 ? r : r & 3);
        float x[NT][NG][2][2];  // p * step of [key r / r + 8][row]
        if (masked) {           // a hidden key adds nothing, not 0 * NaN
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float st = step_of(vp[h][k][grp]);
              const float mid = fmaf(8.f, st, min_of(vp[h][k][grp]));
              if (!FULL) st *= vmult;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const bool hide = hidden[nt] >> ((2 * h + k) * 2 + e) & 1;
                  x[nt][grp][k][e] = hide ? 0.f : sv[nt][2 * h + k][e] * st;
                  om[nt][grp][e] += hide ? 0.f : sv[nt][2 * h + k][e] * mid;
                }
            }
        } else {
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float st = step_of(vp[h][k][grp]);
              const float mid = fmaf(8.f, st, min_of(vp[h][k][grp]));
              if (!FULL) st *= vmult;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  x[nt][grp][k][e] = sv[nt][2 * h + k][e] * st;
                  om[nt][grp][e] = fmaf(sv[nt][2 * h + k][e], mid, om[nt][grp][e]);
                }
            }
        }
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          uint32_t bf[NT][NP][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if constexpr (FULL) {
                float y0[NP], y1[NP];
                parts_of<NP>(x[nt][grp][k][0], y0);
                parts_of<NP>(x[nt][grp][k][1], y1);
#pragma unroll
                for (int n = 0; n < NP; ++n) bf[nt][n][k] = transpose8x8(pack_bf16(y0[n], y1[n]));
              } else {
                bf[nt][0][k] = transpose8x8(pack_f16(x[nt][grp][k][0], x[nt][grp][k][1]));
              }
            }
          if constexpr (!FULL) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (h == 0)
                mma16816_h_first(csum[nt][grp], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, bf[nt][0][0], bf[nt][0][1]);
              else
                mma16816_h(csum[nt][grp], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, bf[nt][0][0], bf[nt][0][1]);
            }
          }
          const uint32_t* w = vw + grp * (G / 8);
          const uint32_t w0 = w[0], w1 = w[W], w2 = w[8 * W], w3 = w[9 * W];
          const uint32_t sel = WPG == 2 || r < 4 ? 0x5410u : 0x7632u;
#pragma unroll
          for (int half = 0; half < WPG; ++half) {
            uint32_t ca[4], cb[4];  // keys 2 ql and 2 ql + 1; the same + 8
            nibbles<FULL>(__byte_perm(w0, w1, half ? 0x7632u : sel), one, ca);
            nibbles<FULL>(__byte_perm(w2, w3, half ? 0x7632u : sel), one, cb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float(&t0)[4] = o[nt][grp][2 * half];
              float(&t1)[4] = o[nt][grp][2 * half + 1];
              if constexpr (FULL) {
                float u0[4], u1[4];
                mma16816_first(u0, ca[0], ca[1], cb[0], cb[1], bf[nt][NP - 1][0], bf[nt][NP - 1][1]);  // small parts first
                mma16816_first(u1, ca[2], ca[3], cb[2], cb[3], bf[nt][NP - 1][0], bf[nt][NP - 1][1]);
#pragma unroll
                for (int n = NP - 2; n >= 0; --n) {
                  mma16816(u0, ca[0], ca[1], cb[0], cb[1], bf[nt][n][0], bf[nt][n][1]);
                  mma16816(u1, ca[2], ca[3], cb[2], cb[3], bf[nt][n][0], bf[nt][n][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) t0[e] += u0[e], t1[e] += u1[e];
              } else {
                mma16816_h(t0, ca[0], ca[1], cb[0], cb[1], bf[nt][0][0], bf[nt][0][1]);
                mma16816_h(t1, ca[2], ca[3], cb[2], cb[3], bf[nt][0][0], bf[nt][0][1]);
              }
            }
          }
        }
      }
      if constexpr (!FULL) {  // centre
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][grp][m][e] += csum[nt][grp][e];
      }
      __syncwarp();  // the stage may be refilled
    }

    // ---- the next segment's first tile and queries are under way before this one is finished
    const bool more = advance(next);
    if (more) {
      ready = look_up(next, 0);
      issue(next, 0);
    }

    // ---- the four warps' sums meet in shared memory, each in the stage of its ring that no copy is on its way to
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
    const int spare = put % STAGES * S::TILE_BYTES;
    float* os = reinterpret_cast<float*>(ring + spare);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float add = om[nt][grp][e], inv = FULL ? 1.f : 1.f / vmult;
            const float even = FULL ? 1.f : 16777216.f, odd = FULL ? 1.f : 1048576.f;
            const int ch = grp * G + (WPG == 2 ? 8 * r : 8 * (r & 3) + 4 * (r >> 2)) + 2 * m;
            *reinterpret_cast<float2*>(os + (nt * 8 + 2 * ql + e) * D + ch) =
                make_float2(fmaf(o[nt][grp][m][e] * even, inv, add), fmaf(o[nt][grp][m][2 + e] * odd, inv, add));
          }
    if (more) load_queries(next);
    __syncthreads();
    const int64_t piece = 2 * (int64_t)blockIdx.x + (s.first ? 1 : 0);
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
        const float4 v = reinterpret_cast<const float4*>(smem + w * STAGES * S::TILE_BYTES + spare)[x];
        l += mlw.y * f;
        a.x += v.x * f, a.y += v.y * f, a.z += v.z * f, a.w += v.w * f;
      }
      if (s.whole) {
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // nothing seen: zeros; NaN stays
        const int qr = row0 + row;
        const int tok = s.q0 + qr / p.g, head = hk * p.g + qr % p.g;
        T* y = head_ptr<T>(p.out, tok, head, D) + 4 * c4;
        if constexpr (NP == 1)
          *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
        else
          *reinterpret_cast<float4*>(y) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        if (p.want_lse && c4 == 0)
          *head_ptr<float>(p.lse, tok, head, 1) = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      } else {
        float* out = p.part + (piece * RB + row) * (D + 4);
        reinterpret_cast<float4*>(out)[c4] = a;
        if (c4 == 0) out[D] = m, out[D + 1] = l;
      }
    }
    if (threadIdx.x == 0 && s.first && !s.whole)
      p.split[blockIdx.x] = Split{s.unit, row0, rows, s.q0, hk, s.last};
    if (!more) break;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring was written by plain stores
    __syncthreads();
  }
  if (dead) {  // copies issued before a wait gave up: a bounded time to land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 20000000ull) {
    }
  }
}

template <int D, int G, int NT, int NP>
cudaError_t variant_of(Variant* out) {
  using S = Shape<D, G, NT, NP>;
  static std::atomic<int> per_sm[64];  // by device; calls come from any thread
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int resident = per_sm[dev].load(std::memory_order_acquire);
  if (!resident) {
    e = cudaFuncSetAttribute(kv4_attention_kernel<D, G, NT, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv4_attention_kernel<D, G, NT, NP>, THREADS, S::SMEM);
    if (e != cudaSuccess) return e;
    resident = n > 0 ? n : 1;
    per_sm[dev].store(resident, std::memory_order_release);
  }
  out->grid = device_sm_count() * resident;
  out->rows = S::RB;
  const size_t splits = ((size_t)out->grid * sizeof(Split) + 255) / 256 * 256;
  out->bytes = splits + (size_t)2 * out->grid * S::RB * (D + 4) * sizeof(float);
  return cudaSuccess;
}

template <int D, int G, int NT, int NP>
cudaError_t launch_of(const AttnParams& p, int grid, cudaStream_t s) {
  cudaError_t e = launch_early(kv4_attention_kernel<D, G, NT, NP>, dim3(grid), THREADS, Shape<D, G, NT, NP>::SMEM, s, p);
  if (e != cudaSuccess) return e;
  using T = typename std::conditional<NP == 1, __nv_bfloat16, float>::type;
  return launch_early(kv4_join_kernel<T, D>, join_grid(grid, p.rb, D), 32 * JOIN_WARPS, 0, s, p);
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
