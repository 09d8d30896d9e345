// Kernels of the block norms on vectors of 8 channels (block_norm.cu has the
// mathematics).
//
// A CTA takes a run of consecutive rows, one at a time; a thread holds VPT
// vectors of 8 channels of it, `blockDim.x` vectors apart.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_norm.h"
#include "cluster_sm103.cuh"
#include "heads_sm103.cuh"

namespace dt {
namespace {

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

// How rows lie: of a multiple of 8 channels on 16-byte boundaries (EVEN), or
// not: wide accesses and shifts (WIDE), or element by element (SINGLE), which
// takes fewer registers and so is what the gradients do.  4000 rows of 8191
// channels, both norms: wide 151 us in bf16 and 176 in fp32, element by element
// 202 and 307; their gradients 412 and 421, 350 and 413.
enum class Rows { EVEN, WIDE, SINGLE };

// Words of a run of bytes that starts o bytes (a multiple of 2) into w.
template <int N, int M>
__device__ __forceinline__ void shifted(uint32_t (&w)[M], int o, uint32_t (&out)[N]) {
  if (o & 8) {
#pragma unroll
    for (int i = 0; i + 2 < M; ++i) w[i] = w[i + 2];
  }
  if (o & 4) {
#pragma unroll
    for (int i = 0; i + 1 < M; ++i) w[i] = w[i + 1];
  }
  const int bits = (o & 2) * 8;
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(w[i], i + 1 < M ? w[i + 1] : 0, bits);
}

// 8 channels of a row of n, in fp32 or as loaded, with 0 behind the row's end.
template <class T>
__device__ __forceinline__ void load8_single(const T* row, int c, int n, Raw8<T>& r) {
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = c + i < n ? load_plain(row + c + i) : T(0.f);
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __bfloat16_as_ushort(e[2 * i]) | (uint32_t)__bfloat16_as_ushort(e[2 * i + 1]) << 16;
    r.u = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    r.a = make_float4(e[0], e[1], e[2], e[3]), r.b = make_float4(e[4], e[5], e[6], e[7]);
  }
}
// The same by 16-byte accesses, one more than on their boundaries, where these
// do not reach beyond the row.
template <class T>
__device__ __forceinline__ void load8_wide(const T* row, int c, int n, Raw8<T>& r) {
  constexpr int P = sizeof(T) / 2, E = 16 / sizeof(T);
  const int o = (int)(reinterpret_cast<uintptr_t>(row) & 15), before = o / (int)sizeof(T);
  if (c < before || c - before + (P + 1) * E > n) {
    load8_single(row, c, n, r);
    return;
  }
  uint32_t w[4 * P + 4], out[4 * P];
  const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row + c) - o);
#pragma unroll
  for (int i = 0; i <= P; ++i) {
    const uint4 u = load_plain(from + i);
    w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
  }
  shifted(w, o, out);
  if constexpr (P == 1) {
    r.u = make_uint4(out[0], out[1], out[2], out[3]);
  } else {
    r.a = make_float4(__uint_as_float(out[0]), __uint_as_float(out[1]), __uint_as_float(out[2]), __uint_as_float(out[3]));
    r.b = make_float4(__uint_as_float(out[4]), __uint_as_float(out[5]), __uint_as_float(out[6]), __uint_as_float(out[7]));
  }
}
template <Rows ROWS, class T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* row, int c, int n) {
  if constexpr (ROWS == Rows::EVEN) r.load(row + c);
  else if constexpr (ROWS == Rows::WIDE) load8_wide(row, c, n, r);
  else load8_single(row, c, n, r);
}
// Off 16-byte boundaries: a lane writes the 16 bytes that its last channels and
// the next lane's first ones share, and (fp32) those that are its own; what has
// no such neighbour goes element by element.  All lanes of the warp come here,
// lane l for channel c of lane 0 + 8 l; those with c >= n write nothing.
template <class T>
__device__ __forceinline__ void store8_wide(T* row, int c, int n, const f2 (&v)[4]) {
  constexpr int P = sizeof(T) / 2, E = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, o = (int)(reinterpret_cast<uintptr_t>(row) & 15);
  uint32_t w[4 * P + 4], out[4 * P];
#pragma unroll
  for (int i = 0; i < 4 * P; ++i) {
    if constexpr (P == 1) w[i] = pack_bf16(v[i].x, v[i].y);
    else w[i] = __float_as_uint(i & 1 ? v[i >> 1].y : v[i >> 1].x);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[4 * P + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
  // elements below `head` share 16 bytes with the lane before, those from `tail` on with the next
  const int head = o ? E - o / (int)sizeof(T) : 0, tail = head + (P - 1) * E;
  const bool full = c + 8 <= n, shared = o ? lane < 31 && c + 16 <= n : full;
  shifted(w, o ? 16 - o : 0, out);
  char* to = reinterpret_cast<char*>(row + c) + (o ? 16 - o : 0);
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (i + 1 < P ? full : shared)
      __stcs(reinterpret_cast<uint4*>(to) + i, make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]));
  const bool mine = !(full && lane > 0);
  if ((mine && head > 0) || !shared) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n && (i < head ? mine : i < tail ? !full : !shared))
        from_f32(row + c + i, i & 1 ? v[i >> 1].y : v[i >> 1].x);
  }
}
// KEEP: without the hint that it is not read again soon.  y is, by the next
// block's product (13403 x 1152: 30.4 us instead of 32.4; h, dx and dr with it
// make 8192 x 4096 slower).
template <Rows ROWS, bool KEEP = false, class T>
__device__ __forceinline__ void store8(T* row, int c, int n, const f2 (&v)[4]) {
  if constexpr (ROWS == Rows::EVEN && KEEP && sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y),
                                                    pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
  } else if constexpr (ROWS == Rows::EVEN) {
    dt::store8(row + c, v);
  } else if constexpr (ROWS == Rows::WIDE) {
    store8_wide(row, c, n, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) from_f32(row + c + i, i & 1 ? v[i >> 1].y : v[i >> 1].x);
  }
}
// of a vector over channels, bf16 or fp32
template <Rows ROWS>
__device__ __forceinline__ void load_w8(const void* w, int dtype, int c, int n, f2 (&v)[4]) {
  if (dtype == DT_BF16) {
    Raw8<__nv_bfloat16> x;
    if constexpr (ROWS == Rows::EVEN) x.u = load_plain(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c));
    else load8<ROWS>(x, static_cast<const __nv_bfloat16*>(w), c, n);
    x.get2(v);
  } else {
    Raw8<float> x;
    if constexpr (ROWS == Rows::EVEN) x.load_keep(static_cast<const float*>(w) + c);
    else load8<ROWS>(x, static_cast<const float*>(w), c, n);
    x.get2(v);
  }
}
// body(w, v): v's vectors of a weight's channels; the type is looked at once, so
// that the loads of all vectors can be on their way together.
template <int VPT, Rows ROWS, class C, class F>
__device__ __forceinline__ void each_w8(const void* weight, int dtype, int n, C&& channel, F&& body) {
  f2 w[4];
  if (dtype == DT_BF16) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      load_w8<ROWS>(weight, DT_BF16, channel(v), n, w);
      body(w, v);
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      load_w8<ROWS>(weight, DT_FP32, channel(v), n, w);
      body(w, v);
    }
  }
}

// Dropout of 8 channels from channel c of token t: bit i keeps channel c + i.
struct Dropout {
  uint32_t key[4], below;
  bool on;
  __device__ __forceinline__ explicit Dropout(const BlockArgs& p) : below(p.drop_below), on(p.rng != nullptr) {
    for (int i = 0; i < 4; ++i) key[i] = on ? (uint32_t)load_plain(p.rng + i) : 0;
  }
  __device__ __forceinline__ uint32_t bits4(uint64_t i) const {
    const uint4 a = philox(i, key[2], key[3], key[0], key[1]);
    return (a.x >= below) | (a.y >= below) << 1 | (a.z >= below) << 2 | (a.w >= below) << 3;
  }
  template <bool EVEN>  // (EVEN: the 8 channels are two whole counters)
  __device__ __forceinline__ uint32_t bits(int64_t t, int n, int c) const {
    const uint64_t e = (uint64_t)t * (uint32_t)n + (uint32_t)c, i = e >> 2;
    const uint32_t b = bits4(i) | bits4(i + 1) << 4;
    return EVEN ? b : (b | bits4(i + 2) << 8) >> (e & 3) & 0xff;
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
template <class T, bool EVEN>
__device__ __forceinline__ void fetch8(uint4* to, const char* row, int c, int n, int step) {
  const T* from = reinterpret_cast<const T*>(row);
  if constexpr (EVEN) {
#pragma unroll
    for (int i = 0; i < Pieces<T>::N; ++i) copy16_async(to + i * step, reinterpret_cast<const uint4*>(from + c) + i);
  } else {
    Raw8<T> r;
    load8<Rows::SINGLE>(r, from, c, n);
    const uint4* w = reinterpret_cast<const uint4*>(&r);
#pragma unroll
    for (int i = 0; i < Pieces<T>::N; ++i) to[i * step] = w[i];
  }
}

// Rows of K tensors, one token after the other: all blocks are looked up again
// where one of them ends.  Steps between rows fit 31 bits (else the kernels for
// any size run).
template <int K>
struct RowCursors {
  char* ptr[K];  // NULL: no such tensor
  int32_t step[K];
  int32_t left = 0;  // tokens from this one to the end of a block
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
  // to token t, the first one or the one behind the present one
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

// Forward.  Bound by HBM; what keeps it from a copy's rate is the time between a
// row's loads and its stores, with two sums over the CTA in it.  AHEAD (x in one
// part): the next row's loads are on their way while a row is worked on, x's from
// where it has been unpacked, the residual's from where it has been added (a ring
// of rows in shared memory, which takes the weights' L1, 53 us instead of 51.6 at
// the first size below).  Else the parts' loads go out four at a time.  Threads
// without a last vector work on the row's first one instead, with its weights,
// and leave it out of sums and stores (whatever it holds then, NaN too).
//   8192 x 4096 bf16, dropout, residual, norm     50.7 us, 0.78 of a copy's rate
//     (42.8 us without dropout's arithmetic, ten rounds for four elements)
//   2048 x 8192 bf16 in 8 parts, both norms       66.2 us, 0.82 (waits for the parts)
//   13403 x 1152 bf16, fp32 residual stream, gate 30.0 us, 0.91
//   8192 x 4096 bf16 in an fp32 stream, both norms 70.0 us, 0.85; fp32 95.1 us, 0.83
//   8 x 4096 bf16 in 4 parts, both norms           4.1 us, one row's latency
template <class XT, class RT, int VPT, bool AHEAD, bool EVEN, class P>
__global__ void __launch_bounds__(block_forward_resident(VPT, AHEAD, sizeof(RT)))
    block_norm_row_kernel(const __grid_constant__ P p) {
  constexpr Rows ROWS = EVEN ? Rows::EVEN : Rows::WIDE;
  __shared__ __align__(16) float buf[2][BN_MAX_WARPS];
  clear(&buf[0][0], 2 * BN_MAX_WARPS);
  int turn = 0;
  const int n = p.n, nt = blockDim.x, tid = threadIdx.x;
  const float inv_n = 1.f / (float)n;
  const int64_t t0 = run_begin(p, blockIdx.x), t1 = run_begin(p, blockIdx.x + 1);
  // x alone (its parts are looked up where they are read), the residual alone
  // (its loads go out later), the outputs
  const RowTable *const tx[1] = {&p.x}, *const tr[1] = {&p.r}, *const to[2] = {&p.h, &p.y};
  RowCursors<1> cx, cr;
  RowCursors<2> out;
  const int parts = p.x.parts;
  int at = 0;
  // vectors below the last two are there in every thread
  const int vectors = (n + 7) / 8;
  const bool last = tid + (VPT - 1) * nt < vectors, last_but_one = tid + (VPT - 2) * nt < vectors;
  auto has = [&](int v) { return v < VPT - 2 || (v == VPT - 1 ? last : last_but_one); };
  auto channel = [&](int v) { return has(v) ? (tid + v * nt) * 8 : 0; };
  const bool res = p.r.count > 0;
  wait_for_previous_kernel();  // (until here: parameters and shared memory alone)
  const Dropout drop(p);
  Raw8<XT> x[VPT];
  Raw8<RT> r[VPT];
  auto load_x = [&](const char* row) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) load8<ROWS>(x[v], reinterpret_cast<const XT*>(row), channel(v), n);
  };
  auto load_r = [&](int64_t t) {
    if (!res) return;
    cr.next(p, tr, t, t1);
#pragma unroll
    for (int v = 0; v < VPT; ++v) load8<ROWS>(r[v], reinterpret_cast<const RT*>(cr.ptr[0]), channel(v), n);
  };
  const char* gate = static_cast<const char*>(p.gate);
  int64_t gate_end = t0;  // of the tokens of the gate's present row
  // a vector a thread: its weights stay in registers
  constexpr bool KEEP = VPT == 1;
  f2 w_post[4], w_gate[4], w_pre[4];
  if (KEEP) {
    if (p.post) load_w8<ROWS>(p.post, p.post_dtype, channel(0), n, w_post);
    if (p.pre) load_w8<ROWS>(p.pre, p.pre_dtype, channel(0), n, w_pre);
  }
  auto weigh = [&](const void* weight, int dtype, const f2(&w)[4], auto&& body) {
    if constexpr (KEEP) body(w, 0);
    else each_w8<VPT, ROWS>(weight, dtype, n, channel, body);
  };
  if (AHEAD) {
    cx.next(p, tx, t0, t1);
    load_x(cx.ptr[0]);
    load_r(t0);
  }
  for (int64_t t = t0; t < t1; ++t) {
    f2 h[VPT][4];
    if (gate && t >= gate_end) {
      const int64_t row = (uint32_t)t / (uint32_t)p.gate_per;
      gate = static_cast<const char*>(p.gate) + row * n * (p.gate_dtype == DT_BF16 ? 2 : 4);
      gate_end = (row + 1) * p.gate_per;
      if (KEEP) load_w8<ROWS>(gate, p.gate_dtype, channel(0), n, w_gate);
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) x[v].get2(h[v]);
      if (t + 1 < t1) {
        cx.next(p, tx, t + 1, t1);
        load_x(cx.ptr[0]);
      }
    } else {
      load_r(t);
      cx.next(p, tx, t, t1);
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
          x[v].get2(w);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[v][i] = k ? h[v][i] + w[i] : w[i];
        }
      }
    }
    auto total = [&] {
      f2 s = both(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (!has(v)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(h[v][i], h[v][i], s);
      }
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
      weigh(gate, p.gate_dtype, w_gate, [&](const f2(&w)[4], int v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = h[v][i] * w[i];
      });
    }
    if (drop.on) {
      uint64_t keep = 0;  // 8 bits a vector
#pragma unroll
      for (int v = 0; v < VPT; ++v) keep |= (uint64_t)drop.bits<EVEN>(t, n, (tid + v * nt) * 8) << (8 * v);
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
        for (int i = 0; i < 4; ++i) h[v][i] = fma2(scale, w[i], h[v][i]);
      }
    }
    if (AHEAD && t + 1 < t1) load_r(t + 1);
    out.next(p, to, t, t1);
    if (out.ptr[0]) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (!EVEN || has(v)) store8<ROWS>(reinterpret_cast<RT*>(out.ptr[0]), (tid + v * nt) * 8, n, h[v]);
    }
    if (out.ptr[1]) {
      const f2 rh = both(total());
      weigh(p.pre, p.pre_dtype, w_pre, [&](const f2(&w)[4], int v) {
        f2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = h[v][i] * rh * w[i];
        if (!EVEN || has(v)) store8<ROWS, true>(reinterpret_cast<XT*>(out.ptr[1]), (tid + v * nt) * 8, n, y);
      });
    }
  }
}

// Gradients.  A CTA (or a cluster of two, each with half of the channels) keeps
// the sums over its tokens and the weights in registers; x, dy, the residual
// and dh come through a ring of S rows.  Three things keep the work per element
// small.
//  - The means' sums are taken at once: with a = w s (w = gate post / (1 - p),
//    0 where dropped), h = scale residual + r(s) a and g = dh + r(h) z - k h,
//    the sum of a g is made of those of a dh, a z and a h; and (S > 1) the next
//    row's sum of s^2 goes with them, so the CTA meets once a row.
//  - dgate and dpost are one sum: with q = sum over the tokens of a gate row
//    of g s r(s) (kept elements), dgate = post q / (1 - p), and dpost adds up
//    gate q / (1 - p).
//  - What an operand is missing for is 0 (or, of w, 1) and computed all the same,
//    but for what may not be finite: h without a norm of it, dh in dropped places.
// What bounds it: latency at 16 warps an SM (its sums and weights fill the
// registers); 0.58 of the issue slots and 0.61 of the DRAM cycles are used.
//   8192 x 4096 bf16, both norms, a gate          76.8 us with the sums' kernel, 0.77 of a copy's rate
//   1533 x 1000 fp32, both, gates, dropout        18.9 us, four rows a CTA one after the other
//   1600 x 16384 bf16, both norms, pairs of CTAs  93.1 us, 3.4 TB/s
// Parts of x (ONE false) are added up in the ring, in fp32, over the first of
// them.  Rows off 16-byte boundaries (EVEN false) come by plain loads.  Both go
// with S = 1, as do rows of which three do not fit: the next row's loads go out
// after the present one's stores, and nothing overlaps within a CTA.
//   744 x 4096 bf16 in 8 parts, both norms        28.6 us, 0.41
//   8192 x 4096 bf16 in an fp32 stream, both     132 us, 0.67; fp32 201 us, 0.59
// DROP false: no code for dropout (8192 x 4096: 79.4 us, with it 83.5).
template <class XT, class RT, int VPT, int S, int CLUSTER, bool ONE, bool EVEN, bool DROP, class P>
__global__ void __launch_bounds__(512) block_norm_row_backward_kernel(const __grid_constant__ P p) {
  constexpr Rows ROWS = EVEN ? Rows::EVEN : Rows::SINGLE;
  static_assert(S == 1 || (ONE && EVEN), "parts and rows off 16-byte boundaries: one row at a time");
  __shared__ __align__(16) float buf[2][8][16];
  __shared__ float meet[2][2][8];  // the cluster's CTAs' sums
  extern __shared__ uint4 ring[];
  clear(&buf[0][0][0], 2 * 8 * 16);
  const int rank = CLUSTER > 1 ? (int)cluster_rank() : 0, run = blockIdx.x / CLUSTER;
  if (CLUSTER > 1) {  // both are there
    cluster_arrive();
    cluster_wait();
  }
  int turn = 0, meet_turn = 0;
  const int n = p.n, nt = blockDim.x, tid = threadIdx.x, parts = ONE ? 1 : p.x.parts;
  const float inv_n = 1.f / (float)n;
  constexpr int PX = Pieces<XT>::N, PR = Pieces<RT>::N;
  constexpr bool HOLD = VPT == 1;  // a row's values stay in registers between the two looks at it (else h alone)
  // pieces of a stage: x's parts, dy, the residual, dh
  const int at_y = parts * VPT * PX * nt, at_r = at_y + VPT * PX * nt, at_h = at_r + VPT * PR * nt,
            stage = at_h + VPT * PR * nt;
  const int64_t t0 = run_begin(p, run), t1 = run_begin(p, run + 1);
  const RowTable *const tin[4] = {&p.x, &p.y, &p.r, &p.h}, *const tout[2] = {&p.dx, &p.dr};
  RowCursors<4> in;
  RowCursors<2> out;
  in.find(p, tin, t0, t1);
  out.find(p, tout, t0, t1);
  const bool has_y = p.y.count > 0, res = p.r.count > 0, has_h = p.h.count > 0, post = p.post, gate = p.gate;
  wait_for_previous_kernel();  // (until here: parameters and shared memory alone)
  const Dropout drop(p);
  const bool dropout = DROP && drop.on;
  auto channel = [&](int v) { return ((rank * VPT + v) * nt + tid) * 8; };
  uint4* const mine = ring + tid;
  int64_t tf = t0;
  int at = 0;
  auto fetch = [&](uint4* to) {
    if (tf < t1) {
      const int block = parts > 1 ? row_block(p.blocks, p.x, tf, at) : 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = channel(v);
        if (c >= n) break;
        fetch8<XT, EVEN>(to + v * PX * nt, in.ptr[0], c, n, nt);
        for (int k = 1; k < parts; ++k)
          fetch8<XT, EVEN>(to + (k * VPT + v) * PX * nt, row_at(p.blocks[block + k * p.x.count], tf, sizeof(XT)), c, n, nt);
        if (has_y) fetch8<XT, EVEN>(to + at_y + v * PX * nt, in.ptr[1], c, n, nt);
        if (res) fetch8<RT, EVEN>(to + at_r + v * PR * nt, in.ptr[2], c, n, nt);
        if (has_h) fetch8<RT, EVEN>(to + at_h + v * PR * nt, in.ptr[3], c, n, nt);
      }
      ++tf;
      in.next(p, tin, tf, t1);
    }
    if (EVEN) copies_commit();
  };
  for (int i = 0; i < S; ++i) {  // places that no copy fills are 0
    uint4* to = mine + i * stage;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const bool none = channel(v) >= n;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      for (int k = 0; none && k < parts * PX; ++k) to[(k / PX * VPT + v) * PX * nt + k % PX * nt] = zero;
      for (int k = 0; (none || !has_y) && k < PX; ++k) to[at_y + (v * PX + k) * nt] = zero;
      for (int k = 0; (none || !res) && k < PR; ++k) to[at_r + (v * PR + k) * nt] = zero;
      for (int k = 0; (none || !has_h) && k < PR; ++k) to[at_h + (v * PR + k) * nt] = zero;
    }
  }
  for (int i = 0; i < S; ++i) fetch(mine + i * stage);
  f2 s_pre[VPT][4], q_gate[VPT][4], w_pre[VPT][4], w[VPT][4];
  bool closed = false;  // a sum of this run's is in the workspace
  int64_t seg = gate ? (uint32_t)t0 / (uint32_t)p.gate_per : 0, seg_end = (seg + 1) * p.gate_per;
  auto gate_row = [&] { return static_cast<const char*>(p.gate) + seg * n * (p.gate_dtype == DT_BF16 ? 2 : 4); };
  auto weights = [&] {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = channel(v);
      if (c >= n) break;
      f2 a[4], b[4];
      if (post) load_w8<ROWS>(p.post, p.post_dtype, c, n, a);
      if (gate) load_w8<ROWS>(gate_row(), p.gate_dtype, c, n, b);
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
    for (int i = 0; i < 4; ++i) s_pre[v][i] = q_gate[v][i] = w_pre[v][i] = w[v][i] = both(0.f);
  weights();
  if (has_y) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (channel(v) < n) load_w8<ROWS>(p.pre, p.pre_dtype, channel(v), n, w_pre[v]);
  }
  auto write_sums = [&](float* to, int v, const f2(&s)[4]) {  // (rows of a multiple of 8 numbers)
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
      if (post) load_w8<ROWS>(p.post, p.post_dtype, c, n, a);
      if (gate) load_w8<ROWS>(gate_row(), p.gate_dtype, c, n, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = a[i] * q_gate[v][i];
        b[i] = b[i] * q_gate[v][i];
        q_gate[v][i] = both(0.f);
      }
      if (post) {  // (this thread's own place)
        float* to = p.part_post + (int64_t)run * p.pitch;
        if (closed) {
          f2 had[4];
          load_w8<Rows::EVEN>(to, DT_FP32, c, n, had);
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = b[i] + had[i];
        }
        write_sums(to, v, b);
      }
      if (!gate) continue;
      if (p.gate_per != 1) write_sums(p.part_gate + ((int64_t)run + seg) * p.pitch, v, a);
      else if (p.dgate_dtype == DT_BF16) store8<ROWS>(static_cast<__nv_bfloat16*>(p.dgate) + seg * n, c, n, a);
      else store8<ROWS>(static_cast<float*>(p.dgate) + seg * n, c, n, a);
    }
    closed = true;
  };
  auto load_x = [&](const uint4* from, int v, f2(&x)[4]) {
    if (parts == 1) {
      Raw8<XT> r;
      r.set(from + v * PX * nt, nt);
      r.get2(x);
    } else {  // the sum: in fp32 over the first part (bf16: the first two)
      Raw8<float> r;
      r.set(from + v * PX * nt, (PX == 1 ? VPT : 1) * nt);
      r.get2(x);
    }
  };
  auto add_parts = [&](uint4* from) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      f2 x[4], y[4];
      Raw8<XT> r;
      r.set(from + v * PX * nt, nt);
      r.get2(x);
      for (int k = 1; k < parts; ++k) {
        r.set(from + (k * VPT + v) * PX * nt, nt);
        r.get2(y);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = x[i] + y[i];
      }
      float4* to = reinterpret_cast<float4*>(from + v * PX * nt);
      to[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
      to[(PX == 1 ? VPT : 1) * nt] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
  };
  auto square = [&](const uint4* from) {  // this thread's share of the sum of s^2
    f2 s = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      f2 x[4];
      load_x(from, v, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(x[i], x[i], s);
    }
    return s.x + s.y;
  };
  auto row_totals = [&](float(&q)[8]) {
    row_sums(q, buf, turn);
    if (CLUSTER == 1) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (tid == i) {
        store_cluster(in_cta(&meet[meet_turn][rank][i], rank ^ 1), q[i]);
        meet[meet_turn][rank][i] = q[i];
      }
    cluster_arrive();
    cluster_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = meet[meet_turn][0][i] + meet[meet_turn][1][i];
    meet_turn ^= 1;
  };
  float rx = 1.f;
  int slot = 0;
  const f2 scale = both(p.scale);
  for (int64_t t = t0; t < t1; ++t) {
    uint4* const from = mine + slot * stage;
    if (++slot == S) slot = 0;
    uint4* const next = mine + slot * stage;
    if (EVEN) copies_wait<(S > 1 ? S - 2 : 0)>();  // this row and (S > 1) the next
    if (parts > 1) add_parts(from);
    float q[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (post && (S == 1 || t == t0)) {
      q[0] = square(from);
      row_totals(q);
      rx = rsqrtf(q[0] * inv_n + p.eps);
    }
    uint32_t bits[VPT] = {};
    f2 x[4], h[VPT][4], dy[4], dh[4];  // x, dy and dh of one vector
    auto values = [&](int v) {
      load_x(from, v, x);
      Raw8<XT> yw;
      Raw8<RT> hw;
      yw.set(from + at_y + v * PX * nt, nt);
      hw.set(from + at_h + v * PR * nt, nt);
      yw.get2(dy), hw.get2(dh);
    };
    auto branch = [&](int v, int i) {  // a
      const f2 a = x[i] * w[v][i];
      return dropout ? kept(a, bits[v], i) : a;
    };
    f2 sum[5] = {both(0.f), both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (dropout) bits[v] = drop.bits<EVEN>(t, n, channel(v));
      values(v);
      Raw8<RT> rw;
      rw.set(from + at_r + v * PR * nt, nt);
      rw.get2(h[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 a = branch(v, i), z = dy[i] * w_pre[v][i];
        h[v][i] = fma2(scale, h[v][i], a * both(rx));
        sum[0] = fma2(h[v][i], h[v][i], sum[0]);
        sum[1] = fma2(h[v][i], z, sum[1]);
        sum[2] = fma2(a, dropout ? kept(dh[i], bits[v], i) : dh[i], sum[2]);  // (0 times what is dropped)
        sum[3] = fma2(a, z, sum[3]);
        sum[4] = fma2(a, h[v][i], sum[4]);
      }
    }
    float rh = 0.f, kh = 0.f, kx = 0.f, next_rx = 1.f;
    if (has_y || post) {
#pragma unroll
      for (int i = 0; i < 5; ++i) q[i] = sum[i].x + sum[i].y;
      q[5] = q[6] = q[7] = 0.f;
      if (S > 1 && post && t + 1 < t1) q[5] = square(next);
      row_totals(q);
      if (has_y) {
        rh = rsqrtf(q[0] * inv_n + p.eps);
        kh = rh * rh * rh * (q[1] * inv_n);
      }
      if (post) {
        // (h may hold anything where there is no norm of it)
        kx = rx * rx * rx * ((has_y ? q[2] + rh * q[3] - kh * q[4] : q[2]) * inv_n);
        next_rx = rsqrtf(q[5] * inv_n + p.eps);
      }
    }
    const f2 rx2 = both(rx), rh2 = both(rh), kh2 = both(-kh), kx2 = both(-kx);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = channel(v);
      if (!HOLD) values(v);
      f2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2 g = dh[i], xr = x[i] * rx2;
        if (has_y) {  // (a choice: kh may not be finite where h is 0)
          g = fma2(dy[i] * w_pre[v][i], rh2, fma2(h[v][i], kh2, g));
          s_pre[v][i] = fma2(dy[i], h[v][i] * rh2, s_pre[v][i]);
        }
        dh[i] = g * scale;
        if (dropout) g = kept(g, bits[v], i), xr = kept(xr, bits[v], i);  // (what is dropped may be NaN)
        q_gate[v][i] = fma2(g, xr, q_gate[v][i]);
        o[i] = g * w[v][i];
        if (post) o[i] = fma2(o[i], rx2, x[i] * kx2);
      }
      if (c < n) {
        if (out.ptr[1]) store8<ROWS>(reinterpret_cast<RT*>(out.ptr[1]), c, n, dh);
        if (out.ptr[0]) store8<ROWS>(reinterpret_cast<XT*>(out.ptr[0]), c, n, o);
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
    if (has_y) write_sums(p.part_pre + (int64_t)run * p.pitch, v, s_pre[v]);
  }
  if (EVEN) copies_wait<0>();
}

// ---------------------------------------------------------------- launches

template <auto KERNEL, class P>
cudaError_t launch_rows(const BlockShape& s, cudaStream_t stream, const P& p) {
  if (s.smem > 40 * 1024)
    if (cudaError_t e = allow_dynamic_smem<KERNEL, BN_SMEM - BN_STATIC>()) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.grid);
  cfg.blockDim = dim3(s.threads);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = s.cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = s.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, KERNEL, p);
}

template <class XT, class RT, bool AHEAD, bool EVEN, class P>
cudaError_t forward_rows(const P& p, const BlockShape& s, cudaStream_t stream) {
  return s.vpt == 1   ? launch_rows<block_norm_row_kernel<XT, RT, 1, AHEAD, EVEN, P>>(s, stream, p)
         : s.vpt == 2 ? launch_rows<block_norm_row_kernel<XT, RT, 2, AHEAD, EVEN, P>>(s, stream, p)
                      : launch_rows<block_norm_row_kernel<XT, RT, 4, AHEAD, EVEN, P>>(s, stream, p);
}
template <class XT, class RT>
cudaError_t block_rows(const BlockSmall& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  if (!bwd)
    return !s.even   ? forward_rows<XT, RT, false, false>(p, s, stream)
           : s.ahead ? forward_rows<XT, RT, true, true>(p, s, stream)
                     : forward_rows<XT, RT, false, true>(p, s, stream);
#define DT_BN_BACK(VPT, S, CLUSTER, ONE, EVEN, DROP)                                                       \
  if (s.vpt == VPT && s.stages == S && s.cluster == CLUSTER && (!ONE || p.x.parts == 1) && s.even == EVEN && \
      (DROP || !p.rng))                                                                                    \
    return launch_rows<block_norm_row_backward_kernel<XT, RT, VPT, S, CLUSTER, ONE, EVEN, DROP, BlockSmall>>(s, stream, p);
  DT_BN_BACK(1, 5, 1, true, true, false) DT_BN_BACK(1, 5, 1, true, true, true)
  DT_BN_BACK(1, 3, 1, true, true, false) DT_BN_BACK(1, 3, 1, true, true, true)
  DT_BN_BACK(2, 3, 1, true, true, false) DT_BN_BACK(2, 3, 1, true, true, true)
  DT_BN_BACK(2, 1, 1, true, true, false) DT_BN_BACK(2, 1, 1, true, true, true)
  DT_BN_BACK(2, 3, 2, true, true, false) DT_BN_BACK(2, 3, 2, true, true, true)
  DT_BN_BACK(2, 1, 2, true, true, false) DT_BN_BACK(2, 1, 2, true, true, true)
  DT_BN_BACK(1, 1, 1, false, true, true)
  DT_BN_BACK(2, 1, 1, false, true, true)
  DT_BN_BACK(2, 1, 2, false, true, true)
  DT_BN_BACK(1, 1, 1, false, false, true)
  DT_BN_BACK(2, 1, 1, false, false, true)
  DT_BN_BACK(2, 1, 2, false, false, true)
#undef DT_BN_BACK
  return cudaErrorInvalidValue;
}
template <class XT, class RT>
cudaError_t block_rows(const BlockLarge& p, bool, const BlockShape& s, cudaStream_t stream) {
  return forward_rows<XT, RT, false, true>(p, s, stream);
}

}  // namespace
}  // namespace dt
