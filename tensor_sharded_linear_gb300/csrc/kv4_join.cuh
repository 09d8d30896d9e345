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
// schedule.  A warp takes a row and up to 32 float4 of its channels: C lanes
// across the channels, 32 / C lanes across the pieces, two pieces in flight
// per lane.
constexpr int JOIN_WARPS = 8;

template <class T, int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kv4_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int C = 8, SEG = D / 4 / C, PL = 32 / C;
  wait_for_previous_kernel();
  const Split sp = p.split[blockIdx.x];
  if (sp.unit < 0) return;
  const int lane = threadIdx.x & 31, c4 = lane % C, pl = lane / C;
  for (int w = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5); w < sp.rows * SEG; w += gridDim.y * JOIN_WARPS) {
    const int row = w / SEG, col = (w % SEG) * C + c4;
    const int n = sp.last - (int)blockIdx.x + 1;
    auto at = [&](int i) {
      const int64_t piece = 2 * (int64_t)(blockIdx.x + i) + (i == 0 ? 1 : 0);
      return p.part + (piece * p.rb + row) * (D + 4);
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
    for (int i = pl; i < n; i += 2 * PL) {
      const float* x = at(i);
      const float* y = at(min(i + PL, n - 1));
      const float2 mx = *reinterpret_cast<const float2*>(x + D), my = *reinterpret_cast<const float2*>(y + D);
      const float4 vx = reinterpret_cast<const float4*>(x)[col], vy = reinterpret_cast<const float4*>(y)[col];
      add(mx.x, mx.y, vx);
      if (i + PL < n) add(my.x, my.y, vy);
    }
#pragma unroll
    for (int o = C; o < 32; o <<= 1) {
      const float mi = __shfl_xor_sync(0xffffffffu, m, o), li = __shfl_xor_sync(0xffffffffu, l, o);
      float4 v;
      v.x = __shfl_xor_sync(0xffffffffu, a.x, o), v.y = __shfl_xor_sync(0xffffffffu, a.y, o);
      v.z = __shfl_xor_sync(0xffffffffu, a.z, o), v.w = __shfl_xor_sync(0xffffffffu, a.w, o);
      add(mi, li, v);
    }
    if (pl) continue;
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

// Grid of the join: one column of CTAs per CTA of the first kernel, as many
// rows as give each warp of a split unit's two tasks (16 at most).
inline dim3 join_grid(int grid, int rows, int D) {
  const int tasks = rows * (D / 32), y = (tasks + 2 * JOIN_WARPS - 1) / (2 * JOIN_WARPS);
  return dim3(grid, y < 16 ? y : 16);
}

}  // namespace kv4
}  // namespace dt
