// Attention of many queries per sequence over the paged 4-bit cache: prompts
// and chunks of prompts (bf16 activations).
//
// The same mathematics as kv4_attention.cuh, in the form that feeds
// tcgen05: a CTA takes 256 (query, head) rows of one sequence and kv head as
// two tiles of 128 (head_dim 256: one tile), and steps through the keys 64 at
// a time.
//   S = Q K^T   both operands in shared memory, S in tensor memory
//   P = 2^(S * scale - reference), fp16, over S's columns in tensor memory
//   O += P V    P from tensor memory, V from shared memory
// The codes are unpacked once per CTA and step, for 256 rows: a number
// minimum + step * code is one fp16 multiply-add, correctly rounded to 11
// bits (with bf16's 8, keys, values and probabilities would each add as much
// error as the output's own rounding).  fp16's range is met by powers of
// two: per row for the queries, per step of 64 keys for K (the largest to
// [2^14, 2^15), undone in the softmax's multiplier), and for V the largest so
// far, with O rescaled where it grows.  The error of the chunks below against
// 64 bits is that of the output's rounding, 0.0017 of the norm.
//
// Roles, 15 warps: two softmax groups of four warps (one row of one tile per
// thread), four unpacking warps (two for K, two for V, one key per thread), one
// warp that issues the bulk copies of the packed records, one per tile that
// issues its matrix products.  Everything goes in steps of 64 keys through
// rings: four packed, three unpacked, two S per tile.  While the softmax of a
// step runs, the tensor core forms P V of the step before and S of the step
// after, for both tiles in turn, and the records of the next steps are on
// their way.
// A row's reference for the exponential follows its maximum only when a step's
// sum passes 2^14, so ordinary steps take no maximum, and O, which stays in
// tensor memory, is rescaled rarely.
//
// Bound: three chunks of up to 1024 tokens on up to 8000 keys, 32/8 heads of
// 128, take 240 us for 239 GFLOP, 1.00 PFLOP/s; 256 rows against 128 keys take
// 3710 cycles, of which the products need 2050 at the tensor core's rate.  An S
// of 64 keys takes 372 cycles instead of 256, since it reads the queries' tile
// from shared memory each time; without exponentials, tensor-memory loads and
// unpacking's stores 3395 are left, with half of each S 2650, without products
// 2300, the round trips between the roles.  Tensor memory is full (two O, four
// S), so an S of 128 keys has one buffer a tile: 5370 cycles, the softmax then
// waits for every product.  A second loader warp, four unpacked stages and
// longer or shorter sleeps in the waits changed nothing.  Heads of 256 have room
// for one tile, two unpacked stages and one packed: 184 us for three chunks of
// up to 512 tokens on up to 8000 keys, 16/2 heads, 0.67 PFLOP/s (958 us in
// passes of 16 rows).
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

constexpr int PROMPT_KEYS = 64;  // of a step
constexpr int PROMPT_WARPS = 15;
// Steps that a unit counts for its start and end when the work is shared out
// (4: 281 us, 12: 267 us for three chunks of up to 1024 tokens on up to 8000
// keys; with shorter steps since, 12: 244, 16: 241, 22: 244).
constexpr int PROMPT_EXTRA = 16;
constexpr int PROMPT_PACKED = 4, PROMPT_STAGES = 3, PROMPT_INFO = 8;  // rings at most: packed, unpacked, scales

template <int D, int G>
struct PromptShape {
  static constexpr int W = kv4_words(D, G);
  static constexpr int NG = D / G;
  static constexpr int TILES = D <= 128 ? 2 : 1, ROWS = 128 * TILES;  // (a tile's O of 256 channels fills half of
                                                                      // tensor memory, its queries 64 KB)
  static constexpr int PACKED = D <= 128 ? PROMPT_PACKED : 1, STAGES = D <= 128 ? PROMPT_STAGES : 2;  // what fits
  static constexpr int PANELS = D / 64;                    // 64 channels: one 128-byte row
  static constexpr int Q_BYTES = 128 * D * 2;              // a tile of 128 rows, fp16
  static constexpr int KV_BYTES = PROMPT_KEYS * D * 2;     // a step's keys or values, fp16
  static constexpr int KV_PANEL = PROMPT_KEYS * 128;
  static constexpr int PACKED_BYTES = PROMPT_KEYS * W * 4;
  static constexpr int OFF_K = TILES * Q_BYTES, OFF_V = OFF_K + STAGES * KV_BYTES;
  static constexpr int OFF_PACKED = OFF_V + STAGES * KV_BYTES;
  static constexpr int OFF_BAR = OFF_PACKED + PACKED * PACKED_BYTES;  // barriers, flags
  static constexpr int SMEM = OFF_BAR + 1024 + 1024;                         // and alignment to 1024
  static constexpr int TMEM_S = 0, TMEM_O = 256;  // columns: S (and P) of tile t, step n at t * 128 + (n & 1) * 64; O
};

// What the softmax has to know of a step.  A slot is written again eight
// steps later; no role is more than five steps ahead of another.
struct alignas(16) StepInfo {
  float kmul;         // S is to be multiplied by this
  float vgrow;        // O is to be multiplied by this before the step's product
  float vscale;       // O is to be multiplied by this in the end
  uint32_t all;       // all 64 keys exist
  uint32_t valid[2];  // which do
};

struct PromptBars {
  uint64_t packed_full[PROMPT_PACKED], packed_empty[PROMPT_PACKED];
  uint64_t kfull[PROMPT_STAGES], kempty[PROMPT_STAGES], vfull[PROMPT_STAGES], vempty[PROMPT_STAGES];
  uint64_t sfull[2][2], pready[2][2];  // [tile][step & 1]
  uint64_t pdone[2], ofull[2], qready[2];  // [tile]
  StepInfo info[PROMPT_INFO];
  uint32_t valid[PROMPT_PACKED][2];    // keys of a packed step that exist
  uint32_t top[2][2][2];               // [step & 1][K, V][warp]: largest magnitudes
  uint32_t there[2][2];                // [step & 1][warp]: keys that exist
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(PromptBars) <= 1024, "barriers and flags");

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bounded wait of a whole warp that sleeps in the barrier unit (up to the
// hint per try) instead of spinning.
__device__ __forceinline__ bool mbar_try_wait_hint(uint64_t* bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_sleep_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                unsigned long long limit_ns) {
  if (__all_sync(0xffffffffu, mbar_try_wait_hint(bar, parity, 20000))) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait_hint(bar, parity, 20000))) return true;
    const int give_up = (*abort_flag != 0) || (globaltimer() - t0 > limit_ns);
    if (__any_sync(0xffffffffu, give_up)) return false;
  }
}

// Four products of 16 deep each: operands advance by fixed steps of their
// descriptors (16-byte units) and tensor-memory columns, so that a product
// costs the issuing warp a few instructions.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
      "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
      "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u64 b, %2, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.u32 a, %1, 16;\n\tadd.u64 b, %2, 256;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
      "add.u32 a, %1, 24;\n\tadd.u64 b, %2, 384;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t}" ::"r"(d),
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
  constexpr int W = S::W, NG = S::NG, RB = S::ROWS, KB = PROMPT_KEYS;
  extern __shared__ uint8_t prompt_smem_raw[];
  uint8_t* smem = prompt_smem_raw + ((1024 - (smem_u32(prompt_smem_raw) & 1023)) & 1023);
  PromptBars& B = *reinterpret_cast<PromptBars*>(smem + S::OFF_BAR);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  volatile int* abort_flag = &B.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < PROMPT_PACKED; ++i) mbar_init(&B.packed_full[i], 1), mbar_init(&B.packed_empty[i], 4);
    for (int i = 0; i < PROMPT_STAGES; ++i) {
      mbar_init(&B.kfull[i], 2);
      mbar_init(&B.kempty[i], S::TILES);
      mbar_init(&B.vfull[i], 2);
      mbar_init(&B.vempty[i], S::TILES);
    }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) mbar_init(&B.sfull[i][j], 1), mbar_init(&B.pready[i][j], 4);
      mbar_init(&B.pdone[i], 1);
      mbar_init(&B.ofull[i], 1);
      mbar_init(&B.qready[i], 4);
    }
    B.abort = 0;
    fence_mbar_init();
  }

  wait_for_previous_kernel();
  // Tensor memory is taken after that: a CTA that held it while it waits could keep one of the kernel before, set up
  // on the same SM but not yet at its own allocation, from ending.
  if (warp == 13) {
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
    *lo = window_begin(s.off + row0 / p.g, p.window);
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
      if (blockIdx.x == 0 && load_plain(p.seq.kv_lens + b) != p.seq.keys(b)) atomicOr(p.status, DT_DEV_ERR_INDEX);
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
    if (mbar_sleep_warp(bar, parity, abort_flag, p.wait_limit_ns)) return true;
    if (lane == 0) {
      atomicExch(&B.abort, 1);
      atomicOr(p.status, DT_DEV_ERR_TIMEOUT);
    }
    return false;
  };

  if (warp < 4 * S::TILES) {
    // ================================================= softmax: tile t, one row per thread
    const int t = warp >> 2, row_in = t * 128 + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + S::TMEM_S + t * 128, to = tmem + lanes + S::TMEM_O + t * D;
    uint8_t* qtile = smem + t * S::Q_BYTES;
    uint32_t mine = 0, all = 0, nseg = 0;  // steps so far in which this tile has rows; of the whole share; units
    uint32_t vstage = 0, vphase = 0;       // ring position of step `all`
    auto skip = [&](uint32_t n) {
      all += n, vstage += n;
      while (vstage >= S::STAGES) vstage -= S::STAGES, vphase ^= 1;
    };
    Segment s;
    bool ok = true;
    while (ok && advance(s)) {
      if (t == 1 && s.rows <= 128) {  // no rows in this tile
        skip(s.nb);
        continue;
      }
      const bool on = row_in < s.rows;
      const int qr = s.row0 + row_in, tok = s.q0 + qr / p.g, head = s.hk * p.g + qr % p.g;
      const int pos = s.off + qr / p.g;
      // ---- the row's query: fp16, scaled to [2^10, 2^11) at its largest.  (The last S of the unit before
      // has been taken, so its queries are done with.)
      float row_scale;
      {
        // (256 channels would not stay in registers: they are read twice)
        constexpr int HELD = D <= 128 ? D / 8 : 0;
        const __nv_bfloat16* q = on ? head_ptr<__nv_bfloat16>(p.q, tok, head, D) : nullptr;
        Raw8<__nv_bfloat16> raw[HELD ? HELD : 1];
        auto fetch = [&](int w) {
          Raw8<__nv_bfloat16> x;
          if (on) x.load(q + 8 * w);
          else x.zero();
          return x;
        };
#pragma unroll
        for (int w = 0; w < HELD; ++w) raw[w] = fetch(w);
        float top = 0.f;
#pragma unroll(HELD ? HELD : 8)
        for (int w = 0; w < D / 8; ++w) {
          float x[8];
          (HELD ? raw[HELD ? w : 0] : fetch(w)).get(x);
#pragma unroll
          for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(x[c]));
        }
        const float mult = __uint_as_float((uint32_t)max(10, min(254, 264 - (int)(__float_as_uint(top) >> 23))) << 23);
        row_scale = p.scale_log2 / mult;
#pragma unroll(HELD ? HELD : 8)
        for (int w = 0; w < D / 8; ++w) {
          float x[8];
          (HELD ? raw[HELD ? w : 0] : fetch(w)).get(x);
          // the order of channels in which a word's nibble pairs come apart
          auto pk = [&](float lo, float hi) {
            const __half2 h = __floats2half2_rn(lo * mult, hi * mult);
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
      float ref = -INFINITY, den = 0.f, vs = 1.f;  // P = 2^(S - ref + 6)
      // (The loop stays a loop: unrolled, the roles' code misses the instruction cache all the time.)
#pragma unroll 1
      for (int i = 0; i < s.nb; ++i) {
        const uint32_t place = mine & 1, tb = ts + 64 * place;
        // (V's barrier second: its phase is told by its parity, so the step before has to have come, as it has
        // when there is an S.  Both in one look: a wait that need not wait costs 150 cycles.)
        const bool s_there = mbar_test(&B.sfull[t][place], (mine >> 1) & 1), v_there = mbar_test(&B.vfull[vstage], vphase);
        if (!__all_sync(0xffffffffu, s_there && v_there) &&
            !(ok = wait(&B.sfull[t][place], (mine >> 1) & 1) && wait(&B.vfull[vstage], vphase)))
          break;
        gemm::tc_fence_after();
        const StepInfo& I = B.info[all % PROMPT_INFO];
        const float sc = fmaxf(row_scale * I.kmul, LEAST_SCALE);
        vs = I.vscale;
        const int j0 = s.key0 + i * KB;
        // columns [lo, hi) of the step are seen by this row
        int lo = 0, hi = min(KB, s.khi - j0);
        if (p.causal) hi = min(hi, pos + 1 - j0);
        if (p.window) lo = max(0, window_begin(pos, p.window) - j0);
        const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < KB || !I.all);
        float f = I.vgrow;  // what O is to be multiplied by
        // The reference stays while the row's sum of this step is at most 2^14, so no maximum is taken; else (and
        // where there is none yet) the step is taken once more with its maximum.
        bool look = __any_sync(0xffffffffu, ref == -INFINITY);
        uint32_t w[32];
        f2 sum;
#pragma unroll 1
        while (true) {
          uint32_t u[32], v[32];
          gemm::tmem_ld32(tb, u);
          gemm::tmem_ld32(tb + 32, v);
          gemm::tmem_ld_wait();
          if (masked) {
            auto see = [&](int c) {  // bit e: column 32 c + e
              const int a = max(lo - 32 * c, 0), z = min(hi - 32 * c, 32);
              return (z > a ? (0xffffffffu >> (32 - (z - a))) << a : 0u) & I.valid[c];
            };
            const uint32_t su = see(0), sv = see(1);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(su >> e & 1)) u[e] = 0xff800000u;
              if (!(sv >> e & 1)) v[e] = 0xff800000u;
            }
          }
          if (look) {
            float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (four short chains)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              t4[e & 2] = fmaxf(t4[e & 2], fmaxf(__uint_as_float(u[e]), __uint_as_float(u[e + 1])));
              t4[1 + (e & 2)] = fmaxf(t4[1 + (e & 2)], fmaxf(__uint_as_float(v[e]), __uint_as_float(v[e + 1])));
            }
            const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * sc;
            if (top > ref) {
              const float g = ex2(ref - top);  // (0 from no reference: O and the sum are zero there, or not yet begun)
              ref = top;
              den *= g;
              f *= g;
            }
          }
          const float add = ref == -INFINITY ? 0.f : 6.f - ref;  // a row that has seen nothing yet
          sum = both(0.f);
          auto half = [&](const uint32_t(&x)[32], int at) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              f2 y = fma2(f2{__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])}, both(sc), both(add));
              y = f2{ex2(y.x), ex2(y.y)};
              sum = sum + y;
              const __half2 h = __floats2half2_rn(y.x, y.y);
              w[at + e] = *reinterpret_cast<const uint32_t*>(&h);
            }
          };
          half(u, 0);
          half(v, 16);
          if (look || __all_sync(0xffffffffu, sum.x + sum.y <= 16384.f)) break;
          look = true;
        }
        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
          // every product before is in O (S of this step followed all but the last)
          if (!(ok = wait(&B.pdone[t], (mine - 1) & 1))) break;
          gemm::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t x[16];
            tmem_ld16(to + 16 * c, x);
            gemm::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
            tmem_st16(to + 16 * c, x);
          }
        }
        tmem_st16(tb, *reinterpret_cast<uint32_t(*)[16]>(w));  // over columns that have been read
        tmem_st16(tb + 16, *reinterpret_cast<uint32_t(*)[16]>(w + 16));
        den += sum.x + sum.y;
        tmem_st_wait();
        gemm::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.pready[t][place]);
        ++mine;
        skip(1);
      }
      if (!ok || !(ok = wait(&B.ofull[t], nseg & 1))) break;  // the unit's last product (a barrier of its own: of
      ++nseg;                                                 // pdone's two may be outstanding here)
      gemm::tc_fence_after();
      // ---- the row's result (channels back in order), or this share's piece of it
      const float inv = den > 0.f ? vs / den : den == 0.f ? 0.f : den;
      const int64_t piece = 2 * (int64_t)blockIdx.x + (s.first ? 1 : 0);
      __nv_bfloat16* y = on && s.whole ? head_ptr<__nv_bfloat16>(p.out, tok, head, D) : nullptr;
      float* out = p.part + (piece * RB + row_in) * (D + 4);
      const float mul = s.whole ? inv : vs;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        gemm::tmem_ld32(to + 32 * c, v);
        gemm::tmem_ld_wait();
        if (!on) continue;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float x[8];
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
  } else if (warp >= 8 && warp < 12) {
    // ================================================= unpacking: warps 8, 9 keys, 10, 11 values; one key per thread
    const int kv = (warp - 8) >> 1, half = warp & 1, key = half * 32 + lane;
    uint32_t magic;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
    uint32_t n = 0, stage = 0, phase = 0;  // step of the share, its place in the rings
    Segment s;
    bool ok = true;
    int left = 0;  // of the unit's meetings, where a wait gave up
    while (ok && advance(s)) {
      int vex = 0;  // exponent field that V's scaling is made for
      for (int i = 0; i < s.nb; ++i, ++n) {
        const uint32_t slot = n % S::PACKED, par = n & 1;
        if (!(ok = wait(&B.packed_full[slot], n / S::PACKED & 1))) {
          left = s.nb - i;
          break;
        }
        const uint32_t* rec = reinterpret_cast<const uint32_t*>(smem + S::OFF_PACKED + slot * S::PACKED_BYTES) + key * W;
        uint32_t word[D / 8], prm[2 * NG];
#pragma unroll
        for (int x = 0; x < D / 8; x += 4) {
          const uint4 q = *reinterpret_cast<const uint4*>(rec + kv * (D / 8) + x);
          word[x] = q.x, word[x + 1] = q.y, word[x + 2] = q.z, word[x + 3] = q.w;
        }
#pragma unroll
        for (int x = 0; x < 2 * NG; x += 2) {
          const uint2 q = *reinterpret_cast<const uint2*>(rec + D / 4 + x);
          prm[x] = q.x, prm[x + 1] = q.y;
        }
        const bool have = B.valid[slot][half] >> lane & 1;
        // the largest magnitude of the step's keys (values), and where values are not finite
        uint32_t top = 0, nan = 0, mine[NG];
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          mine[grp] = !have ? 0 : kv ? prm[NG + grp] : prm[grp];
          const float st = __uint_as_float(mine[grp] << 16), m = __uint_as_float(mine[grp] & 0xffff0000u);
          const uint32_t a = __float_as_uint(fmaxf(fabsf(m), fabsf(fmaf(15.f, st, m))));
          if (a < 0x7f800000u) top = max(top, a);
          // (not finite: minimum, step or the largest value that they make)
          const uint32_t vw = prm[NG + grp];
          const float vt = fmaf(15.f, __uint_as_float(vw << 16), __uint_as_float(vw & 0xffff0000u));
          if (have && !(fabsf(vt) < INFINITY)) nan |= 1u << grp;
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const uint32_t there = __ballot_sync(0xffffffffu, have);
        if (lane == 0) {
          mbar_arrive(&B.packed_empty[slot]);  // (the warp's records are in its registers)
          B.top[par][kv][half] = top;
          if (kv == 0) B.there[par][half] = there;
        }
        asm volatile("bar.sync %0, 64;" ::"r"(1 + kv) : "memory");
        const int ex = (int)(max(B.top[par][kv][0], B.top[par][kv][1]) >> 23);
        StepInfo& I = B.info[n % PROMPT_INFO];
        float mul;
        if (kv == 0) {  // the step's largest in [2^14, 2^15), however small it is
          const int kex = max(ex, 15);
          mul = __uint_as_float((268u - kex) << 23);  // 2^(14 - (kex - 127))
          if (key == 0) {
            I.kmul = __uint_as_float((kex - 14u) << 23);  // 1 / mul
            I.valid[0] = B.there[par][0], I.valid[1] = B.there[par][1];
            I.all = (B.there[par][0] & B.there[par][1]) == 0xffffffffu;
          }
        } else {  // the largest so far in [2^12, 2^13)
          const int vex2 = max(max(vex, ex), 13);
          mul = __uint_as_float((uint32_t)min(254, 266 - vex2) << 23);  // 2^(12 - (vex2 - 127))
          if (key == 0) {
            const int d = i == 0 ? 0 : vex - vex2;  // by which power of two O shrinks
            I.vgrow = d > -126 ? __uint_as_float((uint32_t)(127 + d) << 23) : 0.f;
            I.vscale = __uint_as_float((uint32_t)max(0, vex2 - 12) << 23);  // 1 / mul
          }
          vex = vex2;
        }
        if (!(ok = wait(kv ? &B.vempty[stage] : &B.kempty[stage], phase ^ 1))) {
          left = s.nb - i - 1;
          break;
        }
        uint8_t* dst = smem + (kv ? S::OFF_V : S::OFF_K) + stage * S::KV_BYTES + key * 128;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          __half2 st = __float2half2_rn(__uint_as_float(mine[grp] << 16) * mul);
          __half2 m = __float2half2_rn(__uint_as_float(mine[grp] & 0xffff0000u) * mul);
          if (nan) {  // a value that is not finite makes NaN of the queries that see its key, through S; its group
                      // of V is zeros, as 0 * NaN must not reach the others
            if (kv == 0) m = __float2half2_rn(__int_as_float(0x7fc00000));
            else if (nan >> grp & 1) st = m = __float2half2_rn(0.f);
          }
#pragma unroll
          for (int x = 0; x < G / 8; ++x) {
            const int c = grp * (G / 8) + x;
            const uint32_t cw = word[c], ch = cw >> 8;
            *reinterpret_cast<uint4*>(dst + (c >> 3) * S::KV_PANEL + (((c & 7) ^ (key & 7)) << 4)) =
                make_uint4(unpack2<0>(cw, magic, st, m), unpack2<1>(cw, magic, st, m), unpack2<0>(ch, magic, st, m),
                           unpack2<1>(ch, magic, st, m));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv ? &B.vfull[stage] : &B.kfull[stage]);
        if (++stage == S::STAGES) stage = 0, phase ^= 1;
      }
    }
    // A warp that gave up still comes to every meeting of the share, so that its partner, which may see the same
    // barrier complete or learn of the end a step later, never waits there for good.
    while (!ok) {
      for (; left > 0; --left) asm volatile("bar.sync %0, 64;" ::"r"(1 + kv) : "memory");
      if (!advance(s)) break;
      left = s.nb;
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
      // lane n copies the step's run n of records, one per page, looked up a step ahead
      auto look_up = [&](int i) {
        const int j0 = s.key0 + i * KB, pg = first_page(j0) + lane;
        return i < s.nb && (int64_t)pg * ps < min(j0 + KB, s.khi) ? load_plain(pages + pg) : -1;
      };
      int32_t ready = look_up(0);
      for (int i = 0; i < s.nb; ++i, ++steps) {
        const uint32_t ring = steps % S::PACKED;
        const int j0 = s.key0 + i * KB, end = max(j0, min(j0 + KB, s.khi));
        const int pg0 = first_page(j0), nruns = end > j0 ? first_page(end - 1) - pg0 + 1 : 0;
        // keys that exist: those before `end` whose page is one
        uint64_t vm = end - j0 >= 64 ? ~0ull : (1ull << (end - j0)) - 1;
        for (int n0 = 0; n0 < nruns; n0 += 32) {
          const int n = n0 + lane;
          const int32_t page = n0 == 0 ? ready : n < nruns ? load_plain(pages + pg0 + n) : 0;
          const bool good = n >= nruns || (page >= 0 && page < p.cache.pages);
          if (!__all_sync(0xffffffffu, good)) {
            if (lane == 0) atomicOr(p.status, DT_DEV_ERR_INDEX);
            uint64_t bad = 0;
            if (!good) {
              const int a = max(j0, (pg0 + n) * ps) - j0, z = min(end, (pg0 + n + 1) * ps) - j0;
              bad = (z - a >= 64 ? ~0ull : (1ull << (z - a)) - 1) << a;
            }
            for (int o = 16; o; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
            vm &= ~bad;
          }
        }
        if (!(ok = wait(&B.packed_empty[ring], (steps / S::PACKED & 1) ^ 1))) break;
        if (lane == 0) {
          B.valid[ring][0] = (uint32_t)vm, B.valid[ring][1] = (uint32_t)(vm >> 32);
          const uint32_t starve = steps >= p.starve ? 16 : 0;  // (more bytes than will come)
          mbar_expect_tx(&B.packed_full[ring], __popcll(vm) * W * 4 + starve);
        }
        __syncwarp();
        for (int n = lane; n < nruns; n += 32) {
          const int32_t page = n < 32 ? ready : load_plain(pages + pg0 + n);
          if (page < 0 || page >= p.cache.pages) continue;
          const int a = max(j0, (pg0 + n) * ps), z = min(end, (pg0 + n + 1) * ps);
          bulk_load(smem + S::OFF_PACKED + ring * S::PACKED_BYTES + (a - j0) * (W * 4),
                    head_base + page * page_stride + (int64_t)(a - (pg0 + n) * ps) * W, (z - a) * W * 4,
                    &B.packed_full[ring]);
        }
        ready = look_up(i + 1);
        __syncwarp();
      }
    }
  } else if (warp >= 13 && warp < 13 + S::TILES) {
    // ================================================= matrix products of tile t
    const int t = warp - 13;
    const bool leader = elect_one();
    const uint32_t qa = smem_u32(smem) + t * S::Q_BYTES, ka = smem_u32(smem) + S::OFF_K, va = smem_u32(smem) + S::OFF_V;
    const uint32_t ds = tmem + S::TMEM_S + t * 128, dout = tmem + S::TMEM_O + t * D;
    constexpr uint32_t idesc_s = prompt_idesc(KB, false), idesc_o = prompt_idesc(D, true);
    uint32_t kst = 0, kph = 0, vst = 0, vph = 0;  // ring positions of the next K and V
    uint32_t done = 0, units = 0;                 // this tile's steps and units so far
    auto next_k = [&]() {
      if (++kst == S::STAGES) kst = 0, kph ^= 1;
    };
    auto next_v = [&]() {
      if (++vst == S::STAGES) vst = 0, vph ^= 1;
    };
    auto product_s = [&](uint32_t place) {
      if (leader) {
#pragma unroll
        for (int pn = 0; pn < S::PANELS; ++pn)
          mma4_ss(ds + 64 * place, gemm::smem_desc(qa + pn * 16384, 16, 1024),
                  gemm::smem_desc(ka + kst * S::KV_BYTES + pn * S::KV_PANEL, 16, 1024), idesc_s, pn > 0);
        mma_commit(&B.sfull[t][place]);
        mma_commit(&B.kempty[kst]);
      }
      __syncwarp();
      next_k();
    };
    Segment s;
    bool ok = true;
    while (ok && advance(s)) {
      if (t == 1 && s.rows <= 128) {  // no rows in this tile: its share in the rings' barriers all the same
        for (int i = 0; i < s.nb && ok; ++i) {
          if (!(ok = wait(&B.kfull[kst], kph))) break;
          if (lane == 0) mbar_arrive(&B.kempty[kst]);
          next_k();
          if (!(ok = wait(&B.vfull[vst], vph))) break;
          if (lane == 0) mbar_arrive(&B.vempty[vst]);
          next_v();
        }
        continue;
      }
      ok = wait(&B.qready[t], units++ & 1);
      for (int i = 0; i < min(2, s.nb) && ok; ++i) {  // S of the first two steps
        if (!(ok = wait(&B.kfull[kst], kph))) break;
        gemm::tc_fence_after();
        product_s((done + i) & 1);
      }
      for (int i = 0; i < s.nb && ok; ++i) {
        const uint32_t place = done & 1;
        if (!(ok = wait(&B.vfull[vst], vph) && wait(&B.pready[t][place], (done >> 1) & 1))) break;
        gemm::tc_fence_after();
        if (leader) {
          mma4_ts(dout, ds + 64 * place, gemm::smem_desc(va + vst * S::KV_BYTES, S::KV_PANEL, 1024), idesc_o, i > 0);
          mma_commit(&B.pdone[t]);
          if (i + 1 == s.nb) mma_commit(&B.ofull[t]);
          mma_commit(&B.vempty[vst]);
        }
        __syncwarp();
        next_v();
        ++done;
        if (i + 2 < s.nb) {  // S two steps on, where this step's P was
          if (!(ok = wait(&B.kfull[kst], kph))) break;
          gemm::tc_fence_after();
          product_s(place);
        }
      }
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
  if (warp == 13)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

}  // namespace kv4
}  // namespace dt
