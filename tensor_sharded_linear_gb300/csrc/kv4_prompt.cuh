// Attention of many queries per sequence over the paged 4-bit cache: prompts
// and chunks of prompts (bf16 activations, head_dim 64 or 128).
//
// The same mathematics as kv4_attention.cuh, in the form that feeds
// tcgen05: a CTA takes 256 (query, head) rows of one sequence and kv head as
// two tiles of 128, and steps through the keys 128 at a time.
//   S = Q K^T   both operands in shared memory, S in tensor memory
//   P = 2^(S * scale - reference), fp16, over S's columns in tensor memory
//   O += P V    P from tensor memory, V from shared memory
// The codes are unpacked once per CTA and step, for 256 rows: a number
// minimum + step * code is one fp16 multiply-add, correctly rounded to 11
// bits (with bf16's 8, keys, values and probabilities would each add as much
// error as the output's own rounding).  fp16's range is met by powers of
// two: per row for the queries, per step of 128 keys for K (undone in the
// softmax's multiplier), and for V the largest so far, with O rescaled where
// it grows.
//
// Roles, 14 warps: two softmax groups of four warps (one row of one tile per
// thread), four unpacking warps (one key per thread), one warp that issues
// the bulk copies of the packed records, one that issues the matrix products.
// While one tile's softmax runs, the tensor core works on the other's
// products.  A row's reference for the exponential follows its maximum only
// when that has grown by more than 2^8, so O, which stays in tensor memory,
// is rescaled rarely.
//
// Bound: the tensor core (4 D flops a pair of row and key) for contexts of
// any length; per step of 256 rows x 128 keys the products take about 2050
// cycles, the softmax 3400 and the unpacking 2200 of 8200 issue slots.
//
// The schedule, the pieces of units that a CTA's share cuts and the join are
// those of kv4_attention.cuh, with each row block's own number of key blocks.
#pragma once

#include <cuda_fp16.h>

#include "gemm_sm103.cuh"
#include "kv4_attention.h"
#include "kv4_join.cuh"
#include "ptx_sm103.cuh"

namespace dt {
namespace kv4 {

constexpr int PROMPT_ROWS = 256;
constexpr int PROMPT_KEYS = 128;
constexpr int PROMPT_WARPS = 14;
constexpr int PROMPT_EXTRA = 1;  // key blocks a unit counts for its start and end

template <int D, int G>
struct PromptShape {
  static constexpr int W = kv4_words(D, G);
  static constexpr int NG = D / G;
  static constexpr int PANELS = D / 64;                   // 64 channels: one 128-byte row
  static constexpr int TILE_BYTES = 128 * D * 2;          // 128 rows or keys, fp16
  static constexpr int PACKED_BYTES = PROMPT_KEYS * W * 4;
  static constexpr int OFF_K = 2 * TILE_BYTES, OFF_V = 4 * TILE_BYTES, OFF_PACKED = 6 * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_PACKED + PACKED_BYTES;  // barriers, flags
  static constexpr int SMEM = OFF_BAR + 512 + 1024;          // and alignment to 1024
  static constexpr int TMEM_S = 0, TMEM_O = 256;             // columns: S (and P) of tile t at t * 128; O at 256 + t * D
};

struct PromptBars {
  uint64_t packed_full, packed_empty;
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t sfull[2], pready[2], qready[2], ofull[2];
  uint32_t valid[4];      // keys of the packed step that exist
  uint32_t svalid[2][4];  // the same of the step in a V stage
  float kmul[2];       // what S of a K stage is to be multiplied by
  float vgrow[2];      // what O is to be multiplied by before a V stage's product
  float vscale[2];     // what O is to be multiplied by in the end
  uint32_t top[2][2][4];  // the unpacking warps' largest magnitudes (step parity; K, V)
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(PromptBars) <= 512, "barriers and flags");

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::
          "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// fp16 instruction descriptor, fp32 accumulator, A K-major.
__host__ __device__ constexpr uint32_t prompt_idesc(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// Two codes of w (nibble I of both halves) times the step plus the minimum.
template <int I>
__device__ __forceinline__ uint32_t unpack2(uint32_t w, uint32_t magic, __half2 s, __half2 m) {
  uint32_t r;
  if constexpr (I == 0) asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(r) : "r"(w), "r"(magic));
  else asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(r) : "r"(w), "r"(magic));
  __half2 x = *reinterpret_cast<__half2*>(&r);  // 1024 + code, or 1024 + 16 code
  x = I == 0 ? __hsub2(x, __float2half2_rn(1024.f)) : __hfma2(x, __float2half2_rn(0.0625f), __float2half2_rn(-64.f));
  x = __hfma2(x, s, m);
  return *reinterpret_cast<uint32_t*>(&x);
}

template <int D, int G>
__global__ void __launch_bounds__(32 * PROMPT_WARPS, 1) kv4_prompt_kernel(const __grid_constant__ AttnParams p) {
  using S = PromptShape<D, G>;
  constexpr int W = S::W, NG = S::NG, RB = PROMPT_ROWS, KB = PROMPT_KEYS;
  extern __shared__ uint8_t prompt_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(prompt_smem_raw) + 1023) & ~uintptr_t(1023));
  PromptBars& B = *reinterpret_cast<PromptBars*>(smem + S::OFF_BAR);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  volatile int* abort_flag = &B.abort;

  if (threadIdx.x == 0) {
    mbar_init(&B.packed_full, 1);
    mbar_init(&B.packed_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.kfull[i], 4);
      mbar_init(&B.kempty[i], 1);
      mbar_init(&B.vfull[i], 4);
      mbar_init(&B.vempty[i], 1);
      mbar_init(&B.sfull[i], 1);
      mbar_init(&B.pready[i], 4);
      mbar_init(&B.qready[i], 4);
      mbar_init(&B.ofull[i], 1);
    }
    B.abort = 0;
    fence_mbar_init();
  }
  if (warp == PROMPT_WARPS - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- the schedule: this CTA's share [g0, g1) of all units' key blocks
  struct Part {
    int q0, rows, kv, off, nrb;
  };
  auto seq_at = [&](int b) {
    Part s;
    s.q0 = p.seq.start(b);
    const int ql = max(0, p.seq.start(b + 1) - s.q0);
    s.kv = p.seq.keys(b);
    s.rows = ql * p.g;
    s.off = s.kv - ql;
    s.nrb = (s.rows + RB - 1) / RB;
    return s;
  };
  // keys [lo, hi) that row block rb sees, and its number of key blocks
  auto span = [&](const Part& s, int rb, int* lo, int* hi) {
    const int row0 = rb * RB, row1 = min(s.rows, row0 + RB) - 1;
    *lo = p.window ? max(0, s.off + row0 / p.g - p.window + 1) : 0;
    *hi = p.causal ? min(s.kv, s.off + row1 / p.g + 1) : s.kv;
    return max(1, (*hi - *lo + KB - 1) / KB);
  };
  auto head_cost = [&](const Part& s) {
    int64_t c = 0;
    int lo, hi;
    for (int rb = 0; rb < s.nrb; ++rb) c += span(s, rb, &lo, &hi) + PROMPT_EXTRA;
    return c;
  };
  constexpr int SCAN = 128;
  int64_t* scan = reinterpret_cast<int64_t*>(smem);  // before the tiles are in use
  const int per = (p.seq.batch + SCAN - 1) / SCAN;
  if (threadIdx.x < SCAN) {
    int64_t sum = 0;
    for (int b = threadIdx.x * per; b < min((int)(threadIdx.x + 1) * per, p.seq.batch); ++b) {
      sum += head_cost(seq_at(b)) * p.cache.heads;
      if (blockIdx.x == 0 && __ldg(p.seq.kv_lens + b) != p.seq.keys(b)) atomicOr(p.status, DT_DEV_ERR_INDEX);
    }
    scan[threadIdx.x] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t x[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += scan[4 * lane + i], x[i] = sum;
    int64_t y = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    y -= sum;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) scan[4 * lane + i] = y + x[i];
  }
  gemm::tc_fence_before();
  __syncthreads();
  gemm::tc_fence_after();
  const uint32_t tmem = B.tmem;
  const int64_t total = scan[SCAN - 1];
  if (threadIdx.x == 0) p.split[blockIdx.x].unit = -1;
  const int64_t ncta = min((int64_t)gridDim.x, total);
  const bool working = blockIdx.x < ncta;
  allow_next_kernel();
  int64_t at = working ? total * blockIdx.x / ncta : 0;
  const int64_t g1 = working ? total * (blockIdx.x + 1) / ncta : 0;
  int b = 0;
  int64_t base = 0;
  if (working) {
    int lo = 0, hi = SCAN - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (scan[mid] > at) hi = mid;
      else lo = mid + 1;
    }
    b = lo * per;
    base = lo ? scan[lo - 1] : 0;
  }
  __syncthreads();
  fence_async_smem();  // the tiles' memory was written by plain stores
  __syncthreads();

  struct Segment {
    int q0, off, row0, rows, hk, unit, nb;
    int key0, khi;      // first key of this part; end of the keys any row sees
    int b;
    bool first, whole;
    int last;
  };
  // The next segment of the share, or false at its end (every role walks the
  // same list on its own).
  int64_t cost_b = -1;  // cost of one kv head of sequence b
  auto advance = [&](Segment& x) {
    while (at < g1) {
      Part s = seq_at(b);
      if (cost_b < 0) cost_b = head_cost(s);
      while (at >= base + cost_b * p.cache.heads) {
        base += cost_b * p.cache.heads;
        s = seq_at(++b);
        cost_b = head_cost(s);
      }
      int64_t rem = at - base;
      x.hk = (int)(rem / cost_b);
      rem -= (int64_t)x.hk * cost_b;
      int rb = 0, lo, hi, n = span(s, 0, &lo, &hi);
      while (rem >= n + PROMPT_EXTRA) {
        rem -= n + PROMPT_EXTRA;
        n = span(s, ++rb, &lo, &hi);
      }
      const int64_t start = at - rem, was = at;  // of the unit
      at = min(g1, start + n + PROMPT_EXTRA);
      if (rem >= n) continue;  // only the unit's extra
      x.nb = (int)min((int64_t)n - rem, at - was);
      x.unit = x.hk * s.nrb + rb;
      x.row0 = rb * RB;
      x.rows = min(RB, s.rows - x.row0);
      x.q0 = s.q0;
      x.off = s.off;
      x.khi = hi;
      x.key0 = lo + (int)rem * KB;
      x.b = b;
      x.first = rem == 0;
      x.whole = x.first && x.nb == n;
      x.last = (int)(((start + n) * ncta - 1) / total);
      return true;
    }
    return false;
  };
  // Bounded wait of a whole warp; false: give up everywhere.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait_warp(bar, parity, abort_flag, p.wait_limit_ns)) return true;
    if (lane == 0) {
      atomicExch(&B.abort, 1);
      atomicOr(p.status, DT_DEV_ERR_TIMEOUT);
    }
    return false;
  };

  if (warp < 8) {
    // ================================================= softmax: tile t, one row per thread
    const int t = warp >> 2, row_in = t * 128 + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + S::TMEM_S + t * 128, to = tmem + lanes + S::TMEM_O + t * D;
    uint8_t* qtile = smem + t * S::TILE_BYTES;
    uint32_t steps = 0, vsteps = 0;  // S tiles taken so far (this tile's; all of the share's steps)
    Segment s;
    uint32_t nseg = 0;
    bool ok = true;
    while (ok && advance(s)) {
      const bool tile_on = t == 0 || s.rows > 128;  // else this tile has no rows
      if (!tile_on) {
        vsteps += s.nb;
        continue;
      }
      const bool on = row_in < s.rows;
      const int qr = s.row0 + row_in, tok = s.q0 + qr / p.g, head = s.hk * p.g + qr % p.g;
      const int pos = s.off + qr / p.g;
      // ---- the row's query: fp16, scaled to [2^10, 2^11) at its largest
      float mult = 1.f;
      {
        Raw8<__nv_bfloat16> raw[D / 8];
        float top = 0.f;
        if (on) {
          const __nv_bfloat16* q = head_ptr<__nv_bfloat16>(p.q, tok, head, D);
#pragma unroll
          for (int w = 0; w < D / 8; ++w) raw[w].load(q + 8 * w);
        } else {
#pragma unroll
          for (int w = 0; w < D / 8; ++w) raw[w].zero();
        }
#pragma unroll
        for (int w = 0; w < D / 8; ++w) {
          float x[8];
          raw[w].get(x);
#pragma unroll
          for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(x[c]));
        }
        mult = __uint_as_float((uint32_t)max(10, min(254, 264 - (int)(__float_as_uint(top) >> 23))) << 23);
#pragma unroll
        for (int w = 0; w < D / 8; ++w) {
          float x[8];
          raw[w].get(x);
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] *= mult;
          // the order of channels in which a word's nibble pairs come apart
          auto pk = [](float lo, float hi) {
            const __half2 h = __floats2half2_rn(lo, hi);
            return *reinterpret_cast<const uint32_t*>(&h);
          };
          const int r = row_in & 127;
          *reinterpret_cast<uint4*>(qtile + (w >> 3) * 16384 + r * 128 + (((w & 7) ^ (r & 7)) << 4)) =
              make_uint4(pk(x[0], x[4]), pk(x[1], x[5]), pk(x[2], x[6]), pk(x[3], x[7]));
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.qready[t]);
      const float row_scale = p.scale_log2 / mult;
      float ref = -INFINITY, den = 0.f, vs = 1.f;  // P = 2^(S - ref + 6)
      for (int i = 0; i < s.nb; ++i, ++steps, ++vsteps) {
        if (!(ok = wait(&B.sfull[t], steps & 1))) break;
        gemm::tc_fence_after();
        const int stage = vsteps & 1;
        const float sc = row_scale * B.kmul[stage], vgrow = B.vgrow[stage];
        vs = B.vscale[stage];
        const int j0 = s.key0 + i * KB;
        // columns [lo, hi) of the step are seen by this row
        int lo = 0, hi = min(KB, s.khi - j0);
        if (p.causal) hi = min(hi, pos + 1 - j0);
        if (p.window) lo = max(0, pos - p.window + 1 - j0);
        uint32_t see[4];
        bool masked = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int a = max(lo - 32 * c, 0), z = min(hi - 32 * c, 32);  // bits [a, z)
          see[c] = z > a ? (0xffffffffu >> (32 - (z - a))) << a : 0;
          see[c] &= B.svalid[stage][c];
          masked = masked || see[c] != 0xffffffffu;
        }
        masked = __any_sync(0xffffffffu, masked);
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          gemm::tmem_ld32(ts + 32 * c, v);
          gemm::tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see[c] >> e & 1)) v[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(v[e]));
        }
        top *= sc;
        float f = 1.f;
        if (i == 0) {
          ref = top;
        } else if (top > ref + 8.f) {
          f = ex2(ref - top);
          ref = top;
        }
        den *= f;
        f *= vgrow;
        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[16], w[16];
            tmem_ld16(to + 32 * c, v);
            tmem_ld16(to + 32 * c + 16, w);
            gemm::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
              w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
            }
            tmem_st16(to + 32 * c, v);
            tmem_st16(to + 32 * c + 16, w);
          }
        }
        const float add = ref == -INFINITY ? 0.f : 6.f - ref;  // a row that has seen nothing yet
        f2 sum = both(0.f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32], w[16];
          gemm::tmem_ld32(ts + 32 * c, v);
          gemm::tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see[c] >> e & 1)) v[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            f2 x = fma2(f2{__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])}, both(sc), both(add));
            x = f2{ex2(x.x), ex2(x.y)};
            sum = sum + x;
            const __half2 h = __floats2half2_rn(x.x, x.y);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tmem_st16(ts + 16 * c, w);  // over columns that have been read
        }
        den += sum.x + sum.y;
        tmem_st_wait();
        gemm::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.pready[t]);
      }
      if (!ok || !(ok = wait(&B.ofull[t], nseg & 1))) break;
      ++nseg;
      gemm::tc_fence_after();
      // ---- the row's result (channels back in order), or this share's piece of it
      const float inv = den > 0.f ? vs / den : den == 0.f ? 0.f : den;
      const int64_t piece = 2 * (int64_t)blockIdx.x + (s.first ? 1 : 0);
      __nv_bfloat16* y = on && s.whole ? head_ptr<__nv_bfloat16>(p.out, tok, head, D) : nullptr;
      float* out = p.part + (piece * RB + row_in) * (D + 4);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        gemm::tmem_ld32(to + 32 * c, v);
        gemm::tmem_ld_wait();
        if (!on) continue;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float x[8];
          const float mul = s.whole ? inv : vs;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[(e >> 1) + 4 * (e & 1)] = __uint_as_float(v[8 * w + e]) * mul;
          if (s.whole) {
            *reinterpret_cast<uint4*>(y + 32 * c + 8 * w) =
                make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
          } else {
            *reinterpret_cast<float4*>(out + 32 * c + 8 * w) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(out + 32 * c + 8 * w + 4) = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
      }
      gemm::tc_fence_before();  // before the next products into O
      if (on) {
        const float m = den == 0.f ? -INFINITY : ref - 6.f;
        if (!s.whole) out[D] = m, out[D + 1] = den;
        else if (p.want_lse)
          *head_ptr<float>(p.lse, tok, head, 1) = den == 0.f ? -INFINITY : (m + log2f(den)) * 0.6931471805599453f;
      }
      if (threadIdx.x == 0 && s.first && !s.whole)
        p.split[blockIdx.x] = Split{s.unit, s.row0, s.rows, s.q0, s.hk, s.last};
    }
  } else if (warp < 12) {
    // ================================================= unpacking: one key per thread
    const int key = threadIdx.x - 256, w4 = warp - 8;
    uint32_t magic;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
    uint32_t steps = 0;
    Segment s;
    bool ok = true;
    while (ok && advance(s)) {
      int vex = 0;  // exponent field that V's scaling is made for
      for (int i = 0; i < s.nb; ++i, ++steps) {
        const int stage = steps & 1;
        if (!(ok = wait(&B.packed_full, steps & 1))) break;
        uint32_t rec[W];
        const uint32_t* src = reinterpret_cast<const uint32_t*>(smem + S::OFF_PACKED) + key * W;
#pragma unroll
        for (int x = 0; x < W; x += 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + x);
          rec[x] = v.x, rec[x + 1] = v.y, rec[x + 2] = v.z, rec[x + 3] = v.w;
        }
        const bool have = B.valid[key >> 5] >> (key & 31) & 1;
        // the largest magnitudes of the step's keys and values
        uint32_t top[2] = {0, 0};
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) {
            uint32_t& w = rec[D / 4 + kv * NG + grp];
            if (!have) w = 0;
            const float st = __uint_as_float(w << 16), m = __uint_as_float(w & 0xffff0000u);
            const uint32_t a = __float_as_uint(fmaxf(fabsf(m), fabsf(fmaf(15.f, st, m))));
            if (a < 0x7f800000u) top[kv] = max(top[kv], a);
          }
          top[kv] = __reduce_max_sync(0xffffffffu, top[kv]);
        }
        uint32_t(&tops)[2][4] = B.top[stage];  // (the other step's may still be read)
        if (lane == 0) tops[0][w4] = top[0], tops[1][w4] = top[1];
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (key == 0) mbar_arrive(&B.packed_empty);  // every record is in registers
        const uint32_t kt = max(max(tops[0][0], tops[0][1]), max(tops[0][2], tops[0][3])) >> 23;
        const uint32_t vt = max(max(tops[1][0], tops[1][1]), max(tops[1][2], tops[1][3])) >> 23;
        // K: below 2^15; V: the largest so far in [2^12, 2^13)
        const float kmul = kt > 141 ? __uint_as_float((268u - kt) << 23) : 1.f;  // 2^(14 - (kt - 127))
        const int vex2 = max(max(vex, (int)vt), 13);
        const float vmul = __uint_as_float((uint32_t)min(254, 266 - vex2) << 23);  // 2^(12 - (vex2 - 127))
        if (!(ok = wait(&B.vempty[stage], ((steps >> 1) & 1) ^ 1))) break;  // (its scales are still in use until then)
        const uint32_t there = __ballot_sync(0xffffffffu, have);
        if (lane == 0) B.svalid[stage][w4] = there;
        if (key == 0) {
          B.kmul[stage] = 1.f / kmul;
          const int d = i == 0 ? 0 : vex - vex2;  // by which power of two O shrinks
          B.vgrow[stage] = d > -126 ? __uint_as_float((uint32_t)(127 + d) << 23) : 0.f;
          B.vscale[stage] = 1.f / vmul;
        }
        vex = vex2;
        if (!(ok = wait(&B.kempty[stage], ((steps >> 1) & 1) ^ 1))) break;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint8_t* dst = smem + (kv ? S::OFF_V : S::OFF_K) + stage * S::TILE_BYTES + key * 128;
          const float mul = kv ? vmul : kmul;
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) {
            const uint32_t pw = rec[D / 4 + kv * NG + grp];
            const __half2 st = __float2half2_rn(__uint_as_float(pw << 16) * mul);
            __half2 m = __float2half2_rn(__uint_as_float(pw & 0xffff0000u) * mul);
            if (kv == 0) {  // a value that is NaN reaches the queries that see its key, through S
              const uint32_t vw = rec[D / 4 + NG + grp];
              if ((vw & 0x7f80u) == 0x7f80u || (vw & 0x7f800000u) == 0x7f800000u) m = __float2half2_rn(__int_as_float(0x7fc00000));
            }
            const bool bad = kv && ((pw & 0x7f80u) == 0x7f80u || (pw & 0x7f800000u) == 0x7f800000u);
#pragma unroll
            for (int x = 0; x < G / 8; ++x) {
              const int word = grp * (G / 8) + x;
              const uint32_t cw = rec[kv * (D / 8) + word], ch = cw >> 8;
              uint4 o = make_uint4(unpack2<0>(cw, magic, st, m), unpack2<1>(cw, magic, st, m),
                                   unpack2<0>(ch, magic, st, m), unpack2<1>(ch, magic, st, m));
              if (kv && bad) o = make_uint4(0, 0, 0, 0);  // 0 * NaN must not reach the others
              *reinterpret_cast<uint4*>(dst + (word >> 3) * 16384 + (((word & 7) ^ (key & 7)) << 4)) = o;
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv ? &B.vfull[stage] : &B.kfull[stage]);
        }
      }
    }
  } else if (warp == 12) {
    // ================================================= bulk copies of the packed records
    uint32_t steps = 0;
    Segment s;
    bool ok = true;
    const int ps = p.cache.page_size;
    auto first_page = [&](int j) { return (int)(__umulhi(2u * (uint32_t)j, p.page_mul) >> p.page_shift); };
    while (ok && advance(s)) {
      const int32_t* pages = p.page_table + (int64_t)s.b * p.table_width;
      const int slot = s.hk / p.cache.per_slot;
      const int64_t page_stride = p.cache.page_stride[slot];
      const int32_t* head_base = p.cache.ptr[slot] + (int64_t)(s.hk - slot * p.cache.per_slot) * p.cache.head_stride[slot];
      for (int i = 0; i < s.nb; ++i, ++steps) {
        const int j0 = s.key0 + i * KB, end = max(j0, min(j0 + KB, s.khi));
        const int pg0 = first_page(j0), nruns = end > j0 ? first_page(end - 1) - pg0 + 1 : 0;
        if (!(ok = wait(&B.packed_empty, (steps & 1) ^ 1))) break;
        // keys that exist: those before `end` whose page is one
        uint32_t vm[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = end - j0 - 32 * c;
          vm[c] = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1 : 0;
        }
        int bytes = (end - j0) * W * 4;
        for (int n0 = 0; n0 < nruns; n0 += 32) {
          const int n = n0 + lane;
          const int32_t page = n < nruns ? __ldg(pages + pg0 + n) : 0;
          const bool good = page >= 0 && page < p.cache.pages;
          unsigned badm = __ballot_sync(0xffffffffu, !good);
          if (badm) {
            if (lane == 0) atomicOr(p.status, DT_DEV_ERR_INDEX);
            while (badm) {
              const int m = n0 + __ffs(badm) - 1;
              badm &= badm - 1;
              const int a = max(j0, (pg0 + m) * ps) - j0, z = min(end, (pg0 + m + 1) * ps) - j0;
              for (int k = a; k < z; ++k) vm[k >> 5] &= ~(1u << (k & 31));
              bytes -= (z - a) * W * 4;
            }
          }
        }
        if (lane == 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) B.valid[c] = vm[c];
          mbar_expect_tx(&B.packed_full, bytes);
        }
        __syncwarp();
        for (int n = lane; n < nruns; n += 32) {
          const int32_t page = __ldg(pages + pg0 + n);
          if (page < 0 || page >= p.cache.pages) continue;
          const int a = max(j0, (pg0 + n) * ps), z = min(end, (pg0 + n + 1) * ps);
          bulk_load(smem + S::OFF_PACKED + (a - j0) * (W * 4),
                    head_base + page * page_stride + (int64_t)(a - (pg0 + n) * ps) * W, (z - a) * W * 4, &B.packed_full);
        }
        __syncwarp();
      }
    }
  } else {
    // ================================================= matrix products
    const bool leader = elect_one();
    const uint32_t qa = smem_u32(smem), ka = qa + S::OFF_K, va = qa + S::OFF_V;
    constexpr uint32_t idesc_s = prompt_idesc(KB, false), idesc_o = prompt_idesc(D, true);
    auto product_s = [&](int t, int stage) {
      if (leader) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16_ss(tmem + S::TMEM_S + t * 128,
                     gemm::smem_desc(qa + t * S::TILE_BYTES + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024),
                     gemm::smem_desc(ka + stage * S::TILE_BYTES + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024), idesc_s,
                     k > 0);
        mma_commit(&B.sfull[t]);
      }
      __syncwarp();
    };
    uint32_t steps = 0, nseg = 0, pcount[2] = {0, 0}, qcount[2] = {0, 0};
    Segment s;
    bool ok = true;
    while (ok && advance(s)) {
      const int tiles = s.rows > 128 ? 2 : 1;
      if (!(ok = wait(&B.kfull[steps & 1], (steps >> 1) & 1))) break;
      for (int t = 0; t < tiles && ok; ++t) {
        if (!(ok = wait(&B.qready[t], qcount[t]++ & 1))) break;
        gemm::tc_fence_after();
        product_s(t, steps & 1);
      }
      if (!ok) break;
      if (leader) mma_commit(&B.kempty[steps & 1]);
      __syncwarp();
      for (int i = 0; i < s.nb && ok; ++i, ++steps) {
        const int stage = steps & 1, next = stage ^ 1;
        if (!(ok = wait(&B.vfull[stage], (steps >> 1) & 1))) break;
        for (int t = 0; t < tiles; ++t) {
          if (!(ok = wait(&B.pready[t], pcount[t]++ & 1))) break;
          gemm::tc_fence_after();
          if (leader) {
#pragma unroll
            for (int k = 0; k < KB / 16; ++k)
              mma_f16_ts(tmem + S::TMEM_O + t * D, tmem + S::TMEM_S + t * 128 + 8 * k,
                         gemm::smem_desc(va + stage * S::TILE_BYTES + k * 2048, 16384, 1024), idesc_o,
                         i > 0 || k > 0);
            if (i + 1 == s.nb) mma_commit(&B.ofull[t]);
            if (t + 1 == tiles) mma_commit(&B.vempty[stage]);
          }
          __syncwarp();
          if (i + 1 < s.nb) {
            if (t == 0 && !(ok = wait(&B.kfull[next], ((steps + 1) >> 1) & 1))) break;
            gemm::tc_fence_after();
            product_s(t, next);
            if (t + 1 == tiles) {
              if (leader) mma_commit(&B.kempty[next]);
              __syncwarp();
            }
          }
        }
      }
      ++nseg;
    }
  }
  // ---- everything issued is done (or, given up, has had its time); free tensor memory
  __syncwarp();
  if (*abort_flag) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 20000000ull) {
    }
  }
  gemm::tc_fence_before();
  __syncthreads();
  gemm::tc_fence_after();
  if (warp == PROMPT_WARPS - 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

}  // namespace kv4
}  // namespace dt
