// The join of units that were split over CTAs (see kv4_attention.cuh).
#pragma once

#include <cuda_bf16.h>

#include "kv4_attention.h"

namespace dt {
namespace kv4 {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Adds the pieces of the units that were split, in an order fixed by the
// schedule.  A warp takes C float4 of the channels of 32 / C rows or pieces:
// of a few pieces each lane adds all (C = 32 or what a row has); of many, C = 8
// lanes lie across the channels and four across the pieces (a decode step of
// one long sequence has tens of pieces of 8 rows; measured there, one lane a
// float4 waits for every piece in turn, 22 us instead of 12; a prompt's two
// or three pieces of 256 rows take 38 us with four lanes a float4).
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_FEW = 6;

template <class T, int D, int C>
__device__ __forceinline__ void join_rows(const AttnParams& p, const Split& sp, int n) {
  constexpr bool FEW = C > 8;
  constexpr int SEG = D / 4 / C, PL = 32 / C;  // parts of a row; lanes across rows (FEW) or pieces
  const int lane = threadIdx.x & 31, c4 = lane % C, pl = lane / C;
  const int per_warp = FEW ? PL : 1;           // rows
  const int tasks = (sp.rows + per_warp - 1) / per_warp * SEG;
  for (int w = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5); w < tasks; w += gridDim.y * JOIN_WARPS) {
    const int row = w / SEG * per_warp + (FEW ? pl : 0), col = (w % SEG) * C + c4;
    const bool on = row < sp.rows;
    auto at = [&](int i) {
      const int64_t piece = 2 * (int64_t)(blockIdx.x + i) + (i == 0 ? 1 : 0);
      return p.part + (piece * p.rb + (on ? row : 0)) * (D + 4);
    };
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float mi, float li, float4 v) {
      const float top = fmaxf(m, mi), ref = top == -INFINITY ? 0.f : top;
      const float f0 = ex2(m - ref), f1 = ex2(mi - ref);
      m = top;
      l = l * f0 + li * f1;
      a.x = a.x * f0 + v.x * f1, a.y = a.y * f0 + v.y * f1, a.z = a.z * f0 + v.z * f1, a.w = a.w * f0 + v.w * f1;
    };
    const int step = FEW ? 1 : PL;
    for (int i = FEW ? 0 : pl; i < n; i += 2 * step) {
      const float* x = at(i);
      const float* y = at(min(i + step, n - 1));
      const float2 mx = *reinterpret_cast<const float2*>(x + D), my = *reinterpret_cast<const float2*>(y + D);
      const float4 vx = reinterpret_cast<const float4*>(x)[col], vy = reinterpret_cast<const float4*>(y)[col];
      add(mx.x, mx.y, vx);
      if (i + step < n) add(my.x, my.y, vy);
    }
    if constexpr (!FEW) {
#pragma unroll
      for (int o = C; o < 32; o <<= 1) {
        const float mi = __shfl_xor_sync(0xffffffffu, m, o), li = __shfl_xor_sync(0xffffffffu, l, o);
        float4 v;
        v.x = __shfl_xor_sync(0xffffffffu, a.x, o), v.y = __shfl_xor_sync(0xffffffffu, a.y, o);
        v.z = __shfl_xor_sync(0xffffffffu, a.z, o), v.w = __shfl_xor_sync(0xffffffffu, a.w, o);
        add(mi, li, v);
      }
      if (pl) continue;
    }
    if (!on) continue;
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    const int qr = sp.q_row + row;
    const int tok = sp.q0 + qr / p.g, head = sp.head * p.g + qr % p.g;
    T* out = head_ptr<T>(p.out, tok, head, D) + 4 * col;
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    else
      *reinterpret_cast<float4*>(out) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if (p.want_lse && col == 0)
      *head_ptr<float>(p.lse, tok, head, 1) = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <class T, int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kv4_join_kernel(const __grid_constant__ AttnParams p) {
  wait_for_previous_kernel();
  const Split sp = p.split[blockIdx.x];
  if (sp.unit < 0) return;
  const int n = sp.last - (int)blockIdx.x + 1;
  if (n <= JOIN_FEW) join_rows<T, D, D / 4 < 32 ? D / 4 : 32>(p, sp, n);
  else join_rows<T, D, 8>(p, sp, n);
}

// Grid of the join: one column of CTAs per CTA of the first kernel, as many
// rows as give each warp of a split unit two tasks (64 at most).
inline dim3 join_grid(int grid, int rows, int D) {
  const int tasks = rows * (D / 32), y = (tasks + 2 * JOIN_WARPS - 1) / (2 * JOIN_WARPS);
  return dim3(grid, y < 64 ? y : 64);
}

}  // namespace kv4
}  // namespace dt
