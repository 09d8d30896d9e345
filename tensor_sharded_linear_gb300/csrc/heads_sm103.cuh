// Device helpers shared by the kernels on attention heads: bf16 and fp32
// vectors of 8 channels, the rotation of one pair, and the sequence that a
// token of a ragged batch belongs to.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "head_operands.h"
#include "ptx_sm103.cuh"

namespace dt {

// Two fp32 numbers in a register pair, and the arithmetic that takes both in
// one instruction.
struct f2 {
  float x, y;
};
__device__ __forceinline__ uint64_t f2_bits(f2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ f2 f2_of(uint64_t r) {
  f2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ f2 operator*(f2 a, f2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ f2 operator+(f2 a, f2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_of(r);
}
__device__ __forceinline__ f2 both(float a) { return f2{a, a}; }

// Asynchronous copies of 16 bytes, and waits for all but a thread's last N groups.
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <class T>
__device__ __forceinline__ T load_plain(const T* p) {
  return *p;
}
// 8 consecutive channels (16-byte aligned) as fp32, and back with one
// rounding.  Activations are read once and outputs written once, so both
// use the streaming cache hint.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                 pack_bf16(v[6], v[7])));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
template <class T>
struct Raw8;  // 8 channels as loaded, to be unpacked where they are used
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void set(const uint4* p, int) { u = p[0]; }  // from 16-byte pieces, `step` apart
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get2(f2 (&v)[4]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2{__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void set(const uint4* p, int step) {
    a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + step);
  }
  __device__ __forceinline__ void load_keep(const float* p) {  // what other warps re-read
    a = load_plain(reinterpret_cast<const float4*>(p)), b = load_plain(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get2(f2 (&v)[4]) const {
    v[0] = f2{a.x, a.y}, v[1] = f2{a.z, a.w}, v[2] = f2{b.x, b.y}, v[3] = f2{b.z, b.w};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const f2 (&v)[4]) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y),
                                                 pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y)));
}
__device__ __forceinline__ void store8(float* p, const f2 (&v)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
}

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  Raw8<T> x;
  x.load(p);
  x.get(v);
}
// 8 fp32 values of a table that many warps re-read.
__device__ __forceinline__ void load8_keep(const float* p, float (&v)[8]) {
  const float4 a = load_plain(reinterpret_cast<const float4*>(p)), b = load_plain(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The pair (a, b) turned by the angle with cosine c and sine s.  Products
// and sums round one by one, never fused: the 4-bit codes of a rotated key
// are then a function of the formula alone, not of the compiler's choice of
// fused multiply-adds.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// Kernels here are launched early: their CTAs are set up while the last ones of
// the stream's kernel before run (once each of those has left, or allowed it),
// and wait for its end, and its writes, before they touch memory.  Every
// thread waits, first thing, so that a kernel's end implies that of all before
// it.  Loads are plain ones: what the kernel before may have written is not
// read-only for this one's duration.
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A batch of sequences with new tokens: sequence b's are rows
// [q_starts[b], q_starts[b + 1]) of the activations (without q_starts, each
// sequence has q_len of them) and its keys, the new ones included, number
// kv_lens[b].  Every value read from the device is clamped to what the
// operands hold, so no length can send a kernel out of bounds.
struct SeqTable {
  const int32_t* q_starts;  // NULL: q_len rows each
  const int32_t* kv_lens;
  int32_t batch, q_len, tokens;
  int32_t capacity;  // keys one page table row can address

  __device__ __forceinline__ int start(int b) const {
    if (!q_starts) return b * q_len;
    return min(max(load_plain(q_starts + b), 0), tokens);
  }
  __device__ __forceinline__ int keys(int b) const { return min(max(load_plain(kv_lens + b), 0), capacity); }
};

// Sequence of token t (all lanes of a converged warp call this with one t):
// the last b with start(b) <= t, found 32 candidates a step.  Returns -1 for
// tokens before the first or after the last sequence.
__device__ __forceinline__ int warp_seq_of_token(const SeqTable& s, int t, int lane) {
  if (!s.q_starts) {
    const int b = t / s.q_len;
    return b < s.batch ? b : -1;
  }
  int lo = 0, n = s.batch + 1;  // candidates lo .. lo + n - 1 (entry `batch` is the end)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && s.start(lo + at) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return -1;
    const int top = 31 - __clz(m);
    lo += top * step;
    n = min(step, n - top * step);
  }
  return (lo < s.batch && s.start(lo) <= t) ? lo : -1;
}

}  // namespace dt
