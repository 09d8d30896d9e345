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

#include "block_norm.h"
#include "block_norm.cuh"

namespace dt {
namespace {

// Runs of tokens of a backward launch at most, and so rows of each of its sums
// in the workspace: few channels need more CTAs to fill an SM.
inline int max_backward_blocks(int64_t n) { return n > 2048 ? 320 : n > 1024 ? 640 : 1280; }

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

// For more than 16384 channels; steps between rows of 2^29 elements and more; more
// than 64 row blocks in all operands (gradients, and forward off 16-byte
// boundaries); gradients with parts of x whose row does not fit the shared memory
// of two SMs.  One element a thread and step; the later passes over a row come
// from L1 or L2 and compute its values again (1600 x 20000 bf16, both norms:
// 452 us, gradients 2.9 ms).
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
  const int64_t t0 = BWD ? run_begin(p, blockIdx.x) : blockIdx.x;
  const int64_t t1 = BWD ? run_begin(p, blockIdx.x + 1) : p.tokens;
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
      const float d = h ? load_any(h, p.h.dtype, c) : 0.f;
      return y ? d + rh * (load_any(y, p.y.dtype, c) * pre(c)) - kh * a : d;
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
      auto add = [&](float* to, bool begin, float v) { *to = begin ? v : *to + v; };
      if (p.pre) add(p.part_pre + (int64_t)blockIdx.x * p.pitch + c, first, load_any(y, p.y.dtype, c) * a * rh);
      const float e = keep ? g * p.drop_scale : 0.f, w = e * gate(c);
      if (p.gate) {
        const float d = keep ? e * s * rx * post(c) : 0.f;
        if (p.gate_per == 1) store_any(p.dgate, p.dgate_dtype, t * n + c, d);
        else add(p.part_gate + ((int64_t)blockIdx.x + seg) * p.pitch + c, first_gate, d);
      }
      if (p.post) add(p.part_post + (int64_t)blockIdx.x * p.pitch + c, first, keep ? w * s * rx : 0.f);
      if (dr) store_any(dr, p.dr.dtype, c, p.scale * g);
      if (dx) store_any(dx, p.dx.dtype, c, p.post ? rx * w * post(c) - kx * s : w);
    }
  }
}

// dpre, dpost and the gate's rows from the sums of the runs of tokens: a few MB
// that are still in L2, bound by latency.  A block takes 32 channels, four a
// lane; its 64 groups of eight lanes take every 64th run's sums, six of them at
// once (all of 384 runs), and theirs are added at the end; a fixed order.
// (8192 x 4096, 304 runs, with the kernel before: 77.0 us; 64 channels and 32
// groups with six at once 77.4, with eight 79.3.  1533 x 1000: 18.8, 19.1, 21.6.)
constexpr int BN_SUM_THREADS = 512, BN_SUM_CHANNELS = 32, BN_SUM_LOADS = 6;
constexpr int BN_SUM_LANES = BN_SUM_CHANNELS / 4, BN_SUM_GROUPS = BN_SUM_THREADS / BN_SUM_LANES;
constexpr int BN_SUM_SHARE = BN_SUM_THREADS / BN_SUM_CHANNELS;  // threads a channel at the end
__global__ void __launch_bounds__(BN_SUM_THREADS) block_norm_sums_kernel(const __grid_constant__ BlockArgs p) {
  __shared__ float acc[BN_SUM_GROUPS][BN_SUM_CHANNELS + 1];
  wait_for_previous_kernel();
  const int lane = threadIdx.x % BN_SUM_LANES, group = threadIdx.x / BN_SUM_LANES;
  const int64_t rows = p.gate && p.gate_per != 1 ? p.gate_rows : 0;
  const int64_t c0 = (int64_t)blockIdx.x * BN_SUM_CHANNELS;
  for (int64_t which = blockIdx.y; which < 2 + rows; which += gridDim.y) {
    void* out = which == 0 ? p.dpre : which == 1 ? p.dpost : p.dgate;
    if (!out) continue;
    const int dtype = which == 0 ? p.dpre_dtype : which == 1 ? p.dpost_dtype : p.dgate_dtype;
    int64_t b0 = 0, b1 = p.tokens ? p.runs : 0, row = 0;
    if (which >= 2) {  // the runs that hold tokens of this row, and their sums' places
      row = which - 2;
      if (p.tokens) {
        b0 = run_of(p, row * p.gate_per) + row;
        b1 = run_of(p, (row + 1) * p.gate_per - 1) + 1 + row;
      }
    }
    const int64_t c = c0 + lane * 4;
    const float* part = (which == 0 ? p.part_pre : which == 1 ? p.part_post : p.part_gate) + b0 * p.pitch + c;
    const int count = c < p.n ? (int)(b1 - b0) : 0;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = group; b < count; b += BN_SUM_GROUPS * BN_SUM_LOADS) {
      float4 v[BN_SUM_LOADS];
#pragma unroll
      for (int k = 0; k < BN_SUM_LOADS; ++k) {
        const int at = b + BN_SUM_GROUPS * k;
        v[k] = at < count ? load_plain(reinterpret_cast<const float4*>(part + at * (int64_t)p.pitch))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < BN_SUM_LOADS; ++k) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
    }
    float* const mine = acc[group] + lane * 4;
    mine[0] = s.x, mine[1] = s.y, mine[2] = s.z, mine[3] = s.w;
    __syncthreads();
    const int ch = threadIdx.x / BN_SUM_SHARE, k0 = threadIdx.x % BN_SUM_SHARE;
    static_assert(BN_SUM_GROUPS == 4 * BN_SUM_SHARE, "four sums a thread");
    float v = (acc[k0][ch] + acc[k0 + BN_SUM_SHARE][ch]) +
              (acc[k0 + 2 * BN_SUM_SHARE][ch] + acc[k0 + 3 * BN_SUM_SHARE][ch]);
#pragma unroll
    for (int o = BN_SUM_SHARE / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (k0 == 0 && c0 + ch < p.n) store_any(out, dtype, row * p.n + c0 + ch, v);
    __syncthreads();
  }
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

int round_up(int64_t a, int b) { return (int)((a + b - 1) / b * b); }

// vec: no step between rows is beyond what the kernels on vectors count in;
// even: rows of a multiple of 8 channels on 16-byte boundaries; small: few row blocks.
BlockShape forward_shape(const BlockArgs& p, bool vec, bool even, bool small) {
  BlockShape s;
  const int sms = device_sm_count();
  const int64_t vectors = ((int64_t)p.n + 7) / 8;
  if (!vec || vectors > 4 * 512 || (!even && !small)) {
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
  s.even = even;
  s.ahead = small && even && p.x.parts == 1 && p.tokens > 2 * sms;
  const int ctas = std::max(1, std::min(32, block_forward_resident(s.vpt, s.ahead, dtype_size(p.h.dtype)) / s.threads));
  s.grid = (int)std::min<int64_t>(p.tokens, (int64_t)sms * ctas);
  return s;
}

BlockShape backward_shape(const BlockArgs& p, bool vec, bool even, bool small, int* runs) {
  BlockShape s;
  const int sms = device_sm_count();
  const int64_t vectors = ((int64_t)p.n + 7) / 8;
  int64_t most = 2 * sms;
  // one CTA a row, or a pair where there are more channels than a CTA takes, or parts of x that do not fit an SM
  // (744 x 8192 fp32 in 4 parts: 105 us, the kernel for any size 682)
  for (int cluster = vectors <= 1024 ? 1 : 2; vec && small && vectors <= 2048 && !s.vpt && cluster <= 2; ++cluster) {
    const int vpt = cluster == 1 && vectors <= 256 ? 1 : 2;  // (8192 x 4096: two vectors 79.0 us, one 88.9)
    const int threads = round_up((vectors + vpt * cluster - 1) / (vpt * cluster), 32);
    const int64_t stage = (int64_t)threads * vpt * 8 *
                          ((p.x.parts + 1) * dtype_size(p.x.dtype) + 2 * dtype_size(p.h.dtype));
    if (stage + BN_STATIC > BN_SMEM) continue;
    const int64_t ctas = std::min(8, 512 / threads);
    s.cluster = cluster;
    s.vpt = vpt;
    s.threads = threads;
    s.even = even;
    s.stages = !even || p.x.parts > 1                                    ? 1
               : vpt == 1 && (5 * stage + BN_STATIC) * ctas <= BN_SMEM ? 5
               : (3 * stage + BN_STATIC) * ctas <= BN_SMEM             ? 3
                                                                       : 1;
    s.smem = stage * s.stages;
    most = std::min<int64_t>(ctas, BN_SMEM / (int64_t)(s.smem + BN_STATIC)) * sms / cluster;
  }
  // four tokens a run at least, for its sums are written and read again
  most = std::min<int64_t>(most, std::max<int64_t>(sms / s.cluster, (p.tokens + 3) / 4));
  *runs = (int)std::max<int64_t>(1, std::min<int64_t>({p.tokens, most, max_backward_blocks(p.n)}));
  s.grid = *runs * s.cluster;
  return s;
}

template <class P>
cudaError_t launch_block(const P& p, bool bwd, const BlockShape& s, cudaStream_t stream) {
  if (!s.vpt)
    return bwd ? launch_early(block_norm_any_kernel<P, true>, dim3(s.grid), BN_ANY_THREADS, 0, stream, p)
               : launch_early(block_norm_any_kernel<P, false>, dim3(s.grid), BN_ANY_THREADS, 0, stream, p);
  if (p.x.dtype == DT_FP32) return block_rows_fp32(p, bwd, s, stream);
  if (p.h.dtype == DT_FP32) return block_rows_mixed(p, bwd, s, stream);
  return block_rows_bf16(p, bwd, s, stream);
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
  bool even = true;
  auto add = [&](const RowOperand& o, RowTable* t) {
    *t = RowTable{(int16_t)used, (int16_t)o.count, (int16_t)o.parts, (int16_t)o.dtype};
    std::copy(o.block, o.block + o.count * o.parts, p.blocks + used);
    used += o.count * o.parts;
    even = even && o.vec16;
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
  even = even && X.n % 8 == 0;
  for (const void* v : {p.post, p.gate, p.pre}) even = even && reinterpret_cast<uintptr_t>(v) % 16 == 0;
  even = even && (p.gate_per != 1 || reinterpret_cast<uintptr_t>(p.dgate) % 16 == 0);
  bool vec = true;
  for (int i = 0; i < used; ++i) vec = vec && p.blocks[i].ld < (1 << 29);  // steps between rows in 31 bits
  const bool small = used <= BlockSmall::kCap;
  const BlockShape shape = bwd ? backward_shape(p, vec, even, small, &p.runs) : forward_shape(p, vec, even, small);
  if (!bwd) p.runs = shape.grid;
  p.pitch = round_up(X.n, 8);
  p.run_tokens = (int32_t)(p.tokens / std::max(p.runs, 1));
  p.run_more = (int32_t)(p.tokens % std::max(p.runs, 1));
  if (sums) {
    const int64_t rows_pre = p.dpre ? p.runs : 0, rows_post = p.dpost ? p.runs : 0;
    const int64_t rows_gate = p.dgate && p.gate_per != 1 ? p.runs + p.gate_rows : 0;
    const size_t need = (size_t)(rows_pre + rows_post + rows_gate) * p.pitch * sizeof(float);
    if (!ws || ws_bytes < need)
      return fail(DT_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(DT_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    p.part_pre = static_cast<float*>(ws);
    p.part_post = p.part_pre + rows_pre * p.pitch;
    p.part_gate = p.part_post + rows_post * p.pitch;
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
    const dim3 grid((unsigned)((X.n + BN_SUM_CHANNELS - 1) / BN_SUM_CHANNELS), (unsigned)std::min<int64_t>(which, 4096));
    e = launch_early(block_norm_sums_kernel, grid, BN_SUM_THREADS, 0, stream, static_cast<const BlockArgs&>(p));
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
  if (tokens > 0 && gate_rows > tokens) return fail(DT_ERR_SHAPE, "more gate rows than tokens");
  *bytes = (size_t)(3 * max_backward_blocks(channels) + gate_part_rows(tokens, gate_rows)) * ((channels + 7) / 8 * 8) *
           sizeof(float);
  return DT_OK;
}
