// qknorm.cu -- fa_qk_norm_rope and fa_qk_norm_rope_bwd: q and k normalised for
// each head by their root mean square, weighted, and rotated by their positions,
// in one pass over the data, and the gradients of that.
//
// Forward: with r = (mean(x^2) + eps)^(-1/2) over a head's d columns,
//     y = R(p) (w x r).
// Backward: g = R(p)^T dy is the gradient of the weighted row, and with the
// unit row u = x r
//     dx = r (g w - u mean(g w u)),   dw = sum over rows and heads of g u.
// r is computed again from x, which the backward pass reads anyway.
//
// Bound: HBM; 4 bytes an element forward, 6 backward, about 7 and 16 flop.  A
// thread takes 16 columns of a head (two 16-byte loads), the d / 16 lanes of a
// head sum its squares by shuffles, and all arithmetic is fp32 with one rounding
// at the store.  A warp works alone on one token's heads, 32 / (d / 16) at a time (a
// round), and makes the token's (cos, sin) once; its lanes hold the turns and
// weights of their columns in registers.  Forward, a warp has four rounds of q or k, all
// loads under way before the turns are made.  The backward pass is one wave of warps,
// each with an even share of the rounds, three of them ahead by cp.async; a lane
// holds its columns' dw in registers over all of them, a CTA's sum goes to the
// workspace and a second kernel adds the CTAs' in their order: no atomics, and the
// result does not depend on scheduling.  A lane's and a CTA's sums are fp32 (a lane has a term
// for each round of its warp, 27 for q of the layer below), the second kernel's two fp32 words.
//
// Measured (8192 tokens, 32 + 8 heads, d 128, bf16, all columns rotated): forward 32.6 us
// (5.2 TB/s), backward 53 us (4.7 TB/s), of it 4 for dw; one token 4 .. 6 us.  The issue
// slots are two thirds full at that rate; what helped: turns once per token and warp (with
// eight tokens' turns to a CTA of 256 threads, between barriers, 48 and 98 us), pairs of
// fp32 to an instruction, whole sectors for interleaved pairs (backward, no rotation: 69 us to 43).
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "norm_rows.cuh"

using namespace mfa;

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kFwdBlocks = 5;  // CTAs per SM
constexpr int kBwdBlocks = 4;
constexpr int kAhead = 4;      // rounds whose loads are under way, forward
constexpr int kStages = 4;     // rounds in shared memory, backward
constexpr int kDwThreads = 1024;
constexpr int kMaxParts = 1024;  // CTAs of the backward pass
static_assert(FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES >= kWsHeadBytes + (size_t)kMaxParts * 2 * 128 * 4, "partials of dw");

// q or k.
struct NormRows {
  const uint16_t* x;
  const uint16_t* dy;  // backward
  uint16_t* out;       // y, or dx
  int64_t x_sb, x_ss, x_sh, dy_sb, dy_ss, dy_sh, out_sb, out_ss, out_sh;
  HeadWeight w;
  float* dw;  // nullable
  int32_t heads;
  int32_t rounds;  // of a token
  int64_t share, more;  // backward: every warp's rounds, and the number of warps with one more
};

struct NormParams {
  NormRows t[2];  // q, k
  int64_t rows;
  int32_t S;
  const int32_t* positions;
  int64_t pos_sb, pos_ss;
  const double* inv_freq;
  int32_t half;  // pairs; 0: no rotation
  float mscale, eps;
  int32_t units, span;  // forward: warps of a token, and rounds of a warp
  float* part;  // backward: [CTAs][2][D], null without weight gradients
  int32_t n_parts;
};

__device__ __forceinline__ int position_of(const NormParams& p, int b, int i) {
  return p.positions ? __ldg(p.positions + b * p.pos_sb + i * p.pos_ss) : i;
}

template <int D, bool F16, int LAYOUT>
__global__ void __launch_bounds__(kThreads, kFwdBlocks) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes per head; heads of a round
  __shared__ __align__(16) float2 s_cs[kWarps][D / 2];
  __shared__ Weights<kLanes> s_w;
  __shared__ float s_row[LAYOUT == kHalfOdd ? kWarps * kHeads * D : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLanes, slot = lane / kLanes, half = p.half;
  const uint32_t group = blockIdx.x / (uint32_t)p.units;
  const int r0 = (int)(blockIdx.x - group * p.units) * p.span, rq = p.t[0].rounds, r1 = min(r0 + p.span, rq + p.t[1].rounds);
  const int64_t at_row = (int64_t)group * kWarps + warp;
  const bool live = at_row < p.rows;
  const int b = live ? (int)at_row / p.S : 0, i = live ? (int)at_row - b * p.S : 0;
  const Columns at = lane_columns<D, LAYOUT>(c, half);
  const uint16_t* const src[2] = {p.t[0].x + b * p.t[0].x_sb + i * p.t[0].x_ss, p.t[1].x + b * p.t[1].x_sb + i * p.t[1].x_ss};
  auto load = [&](int r, uint4& va, uint4& vb) {
    const int n = r >= rq, h = (n ? r - rq : r) * kHeads + slot;
    va = vb = make_uint4(0, 0, 0, 0);
    if (live && r < r1 && h < p.t[n].heads) {
      const uint16_t* from = (n ? src[1] : src[0]) + h * p.t[n].x_sh;
      va = *reinterpret_cast<const uint4*>(from + at.xa);
      vb = *reinterpret_cast<const uint4*>(from + at.xb);
    }
  };
  uint4 va[kAhead], vb[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(r0 + k, va[k], vb[k]);
  uint64_t u[2] = {0, 0};
  int pos = 0;
  if (half > 0) {
    if (live) pos = position_of(p, b, i);
    turn_steps(p.inv_freq, half, lane, u);
  }
  stage_weights<F16, LAYOUT, kLanes>(p.t[0].w, p.t[1].w, half, s_w);
  if (!live) return;
  Turns tw;
  if (half > 0) {
    make_turns<LAYOUT>(pos, u, half, p.mscale, false, lane, s_cs[warp]);
    load_turns<D, LAYOUT>(s_cs[warp], c, tw);
  }
  uint16_t* const dst[2] = {p.t[0].out + b * p.t[0].out_sb + i * p.t[0].out_ss, p.t[1].out + b * p.t[1].out_sb + i * p.t[1].out_ss};
  // (the lanes of a warp stay together through the shuffles: those without a head
  // compute on zeros and store nothing)
#pragma unroll 1
  for (int r = r0; r < r1; r += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (r + k >= r1) break;
      const int n = r + k >= rq, h = (n ? r + k - rq : r + k) * kHeads + slot;
      Pairs x = unpack_pairs<F16, LAYOUT>(va[k], vb[k]);
      load(r + k + kAhead, va[k], vb[k]);
      const float inv = rsqrtf(fmaf(dot<kLanes>(x, x), 1.f / D, p.eps));
      scale_by(x, inv);
      multiply(x, weight_of<kLanes>(s_w, n, c));
      rotate<D, LAYOUT>(x, tw, s_cs[warp], c, half, s_row + (LAYOUT == kHalfOdd ? (warp * kHeads + slot) * D : 0));
      if (h < p.t[n].heads) {
        uint16_t* to = (n ? dst[1] : dst[0]) + h * p.t[n].out_sh;
        uint4 ya, yb;
        pack_pairs<F16, LAYOUT>(x, ya, yb);
        *reinterpret_cast<uint4*>(to + at.xa) = ya;
        *reinterpret_cast<uint4*>(to + at.xb) = yb;
      }
    }
  }
}

// A warp's rounds of the backward pass: an even share of q's, then one of k's.
struct Walk {
  int n, left, b, i, round;
  __device__ __forceinline__ void start(const NormParams& p, int tensor) {
    n = tensor;
    const NormRows& r = p.t[n];
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), lo = w * r.share + min(w, r.more);
    left = (int)(r.share + (w < r.more));
    if (left == 0) return;
    // (a 64-bit division takes a microsecond)
    const int64_t row = lo <= UINT32_MAX ? (uint32_t)lo / (uint32_t)r.rounds : lo / r.rounds;
    round = (int)(lo - row * r.rounds);
    b = (int)((uint32_t)row / (uint32_t)p.S);
    i = (int)row - b * p.S;
  }
  __device__ __forceinline__ void begin(const NormParams& p) {
    start(p, 0);
    if (left == 0) start(p, 1);
  }
  // To the next round; true if its token is another (or its tensor).
  __device__ __forceinline__ bool next(const NormParams& p) {
    if (--left == 0) {
      if (n == 0) start(p, 1);
      return true;
    }
    if (++round < p.t[n].rounds) return false;
    round = 0;
    if (++i == p.S) {
      i = 0;
      ++b;
    }
    return true;
  }
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;  // (0: the rest is zeros, and nothing is read)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes)
               : "memory");
}

template <int D, bool F16, int LAYOUT>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
  __shared__ uint4 s_in[kWarps][kStages][4][32];  // a lane reads what it copied: x and dy, 32 bytes each
  __shared__ __align__(16) float2 s_cs[kWarps][D / 2];
  __shared__ int s_pos[kWarps][kStages];
  __shared__ float s_sum[2][kWarps][D];
  __shared__ Weights<kLanes> s_w;
  __shared__ float s_row[LAYOUT == kHalfOdd ? kWarps * kHeads * D : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLanes, slot = lane / kLanes, half = p.half;
  const Columns at = lane_columns<D, LAYOUT>(c, half);
  float* row = s_row + (LAYOUT == kHalfOdd ? (warp * kHeads + slot) * D : 0);
  uint64_t u[2] = {0, 0};
  if (half > 0) turn_steps(p.inv_freq, half, lane, u);
  Pairs dw;
#pragma unroll
  for (int k = 0; k < 4; ++k) dw.a[k] = dw.b[k] = both(0.f);
#pragma unroll
  for (int n = 0; n < 2; ++n)
    for (int col = lane; col < D; col += 32) s_sum[n][warp][col] = 0.f;
  __syncwarp();

  // the warp's sums of dw, over its heads by shuffles
  auto flush = [&](int n) {
    if (!p.part) return;
    float sums[16];
    columns_from<LAYOUT>(dw, sums);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = sums[e];
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < kLanes) s_sum[n][warp][e < 8 ? at.xa + e : at.xb + e - 8] = v;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) dw.a[k] = dw.b[k] = both(0.f);
  };
  // (the next round's x and dy of this lane)
  const uint16_t *f_x = nullptr, *f_dy = nullptr;
  const int apart = at.xb - at.xa;
  auto issue = [&](const Walk& f, bool fresh, int stage) {
    const NormRows& r = p.t[f.n];
    if (fresh) {
      const int h = f.round * kHeads + slot;
      f_x = r.x + f.b * r.x_sb + f.i * r.x_ss + h * r.x_sh + at.xa;
      f_dy = r.dy + f.b * r.dy_sb + f.i * r.dy_ss + h * r.dy_sh + at.xa;
    }
    const bool valid = f.round * kHeads + slot < r.heads;
    uint4* to = &s_in[warp][stage][0][lane];
    const uint16_t *src = valid ? f_x : r.x, *grad = valid ? f_dy : r.dy;
    copy16(to, src, valid);
    copy16(to + 32, src + apart, valid);
    copy16(to + 64, grad, valid);
    copy16(to + 96, grad + apart, valid);
    f_x += kHeads * r.x_sh;
    f_dy += kHeads * r.dy_sh;
    if (half > 0 && lane == 0) {
      int* at_pos = &s_pos[warp][stage];
      if (p.positions)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(at_pos)),
                     "l"(p.positions + f.b * p.pos_sb + f.i * p.pos_ss)
                     : "memory");
      else *at_pos = f.i;
    }
  };

  Walk f, v;
  f.begin(p);
  v = f;
  bool f_fresh = true;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (f.left > 0) {
      issue(f, f_fresh, s);
      f_fresh = f.next(p);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  stage_weights<F16, LAYOUT, kLanes>(p.t[0].w, p.t[1].w, half, s_w);
  int stage = 0, n = -1;
  bool fresh = true;
  while (v.left > 0) {
    if (v.n != n) {
      if (n >= 0) flush(n);
      n = v.n;
    }
    const NormRows& r = p.t[n];
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    if (half > 0) {
      __syncwarp();  // the position came by lane 0's copy
      if (fresh) make_turns<LAYOUT>(s_pos[warp][stage], u, half, p.mscale, true, lane, s_cs[warp]);
    }
    const uint4* in = &s_in[warp][stage][0][lane];
    Pairs x = unpack_pairs<F16, LAYOUT>(in[0], in[32]), g = unpack_pairs<F16, LAYOUT>(in[64], in[96]);
    if (f.left > 0) {
      issue(f, f_fresh, (stage + kStages - 1) % kStages);
      f_fresh = f.next(p);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage = (stage + 1) % kStages;
    {
      Turns tw;
      load_turns<D, LAYOUT>(s_cs[warp], c, tw);
      rotate<D, LAYOUT>(g, tw, s_cs[warp], c, half, row);
    }
    const float inv = rsqrtf(fmaf(dot<kLanes>(x, x), 1.f / D, p.eps));
    scale_by(x, inv);  // the unit row
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dw.a[k] = fma2(g.a[k], x.a[k], dw.a[k]);
      dw.b[k] = fma2(g.b[k], x.b[k], dw.b[k]);
    }
    multiply(g, weight_of<kLanes>(s_w, n, c));
    const float2 m = both(-dot<kLanes>(g, x) * (1.f / D));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      g.a[k] = fma2(x.a[k], m, g.a[k]);
      g.b[k] = fma2(x.b[k], m, g.b[k]);
    }
    scale_by(g, inv);
    const int h = v.round * kHeads + slot;
    if (h < r.heads) {
      uint4 a, b;
      pack_pairs<F16, LAYOUT>(g, a, b);
      uint16_t* dst = r.out + v.b * r.out_sb + v.i * r.out_ss + h * r.out_sh;
      *reinterpret_cast<uint4*>(dst + at.xa) = a;
      *reinterpret_cast<uint4*>(dst + at.xb) = b;
    }
    fresh = v.next(p);
  }
  if (!p.part) return;
  if (n >= 0) flush(n);
  __syncthreads();
  for (int k = threadIdx.x; k < 2 * D; k += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_sum[k / D][w][k % D];
    p.part[(int64_t)blockIdx.x * 2 * D + k] = sum;
  }
}

// dw: eight columns of q's or k's per CTA, a part for every eight threads at a time.
template <int D>
__global__ void __launch_bounds__(kDwThreads) norm_dw_kernel(const __grid_constant__ NormParams p) {
  constexpr int kDwWarps = kDwThreads / 32;
  __shared__ float2 s[kDwWarps][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x / (D / 8), col = blockIdx.x % (D / 8) * 8 + lane % 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!p.t[n].dw) return;
  // (in two fp32 words, the second the first's rounding errors: fp64 would take 16 us)
  float v = 0.f, rest = 0.f;
  auto add = [&](float x) {
    const float sum = v + x, t = sum - v;
    rest += (v - (sum - t)) + (x - t);
    v = sum;
  };
#pragma unroll 8
  for (int k = threadIdx.x / 8; k < p.n_parts; k += kDwThreads / 8) add(p.part[((int64_t)k * 2 + n) * D + col]);
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v, o), y = __shfl_xor_sync(0xffffffffu, rest, o);
    add(x);
    rest += y;
  }
  if (lane < 8) s[warp][lane] = make_float2(v, rest);
  __syncthreads();
  if (warp > 0) return;
  v = rest = 0.f;
#pragma unroll
  for (int k = 0; k < kDwWarps; k += 4) {
    const float2 x = s[k + lane / 8][lane % 8];
    add(x.x);
    rest += x.y;
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v, o), y = __shfl_xor_sync(0xffffffffu, rest, o);
    add(x);
    rest += y;
  }
  // (an infinite or NaN sum has a NaN rest)
  if (lane < 8) p.t[n].dw[col] = isfinite(v) ? v + rest : v;
}

template <int D, bool F16>
void launch_fwd(const NormParams& p, int layout, unsigned grid, cudaStream_t st) {
  if (layout == kInterleaved) norm_kernel<D, F16, kInterleaved><<<grid, kThreads, 0, st>>>(p);
  else if (layout == kHalf) norm_kernel<D, F16, kHalf><<<grid, kThreads, 0, st>>>(p);
  else norm_kernel<D, F16, kHalfOdd><<<grid, kThreads, 0, st>>>(p);
}
template <int D, bool F16>
void launch_bwd(const NormParams& p, int layout, int grid, cudaStream_t st) {
  if (layout == kInterleaved) norm_bwd_kernel<D, F16, kInterleaved><<<grid, kThreads, 0, st>>>(p);
  else if (layout == kHalf) norm_bwd_kernel<D, F16, kHalf><<<grid, kThreads, 0, st>>>(p);
  else norm_bwd_kernel<D, F16, kHalfOdd><<<grid, kThreads, 0, st>>>(p);
}
template <int D>
cudaError_t launch_dw(const NormParams& p, bool overlap, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(2 * D / 8);
  c.blockDim = dim3(kDwThreads);
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&c, norm_dw_kernel<D>, p);
}

int check_dw(const fa_tensor* w, const fa_tensor* x, NormRows& r) {
  if (!w) return FA_OK;
  if (!w->data || w->dtype != FA_DTYPE_F32 || w->ndim != 1 || w->shape[0] != x->shape[x->ndim - 1] || w->stride[0] != 1 ||
      (reinterpret_cast<uintptr_t>(w->data) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  r.dw = static_cast<float*>(w->data);
  return FA_OK;
}

// What both passes share: x (q or k) and its written counterpart, weights,
// positions, frequencies.
int check_norm(const fa_tensor* const (&x)[2], const fa_tensor* const (&out)[2], const fa_tensor* const (&w)[2],
               const fa_tensor* positions, const fa_tensor* inv_freq, float eps, float mscale, NormParams& p) {
  const fa_tensor* q = x[0];
  memset(&p, 0, sizeof(p));
  int rc;
  if (!q || !out[0] || (x[1] == nullptr) != (out[1] == nullptr) || (!x[1] && w[1])) return FA_ERR_INVALID_ARG;
  if (q->ndim != 3 && q->ndim != 4) return FA_ERR_INVALID_ARG;
  const int64_t d = q->shape[q->ndim - 1];
  if (d != 64 && d != 128) return FA_ERR_INVALID_ARG;
  int64_t heads = 0;
  for (int n = 0; n < 2; ++n) {
    if (!x[n]) continue;
    if ((rc = check_pair(x[n], out[n], q)) || (rc = check_weight(w[n], x[n], p.t[n].w))) return rc;
    NormRows& r = p.t[n];
    const int64_t h = x[n]->shape[q->ndim - 2];
    heads += h;
    if (heads > INT32_MAX / 1024) return FA_ERR_INVALID_ARG;
    r.heads = (int32_t)h;
    const int64_t at_once = 32 / (d / 16);
    r.rounds = (int32_t)((h + at_once - 1) / at_once);
    r.x = static_cast<const uint16_t*>(x[n]->data);
    r.out = static_cast<uint16_t*>(out[n]->data);
    strides_of(x[n], r.x_sb, r.x_ss, r.x_sh);
    strides_of(out[n], r.out_sb, r.out_ss, r.out_sh);
  }
  if ((rc = check_rows(q, p))) return rc;
  if (inv_freq) {
    if ((rc = check_freq(inv_freq, d, &p.half))) return rc;
    p.inv_freq = static_cast<const double*>(inv_freq->data);
    if (!std::isfinite(mscale)) return FA_ERR_INVALID_ARG;
    p.mscale = mscale;
    if (!positions && q->ndim == 3) return FA_ERR_INVALID_ARG;
  }
  if (positions && (rc = check_positions(positions, q, p))) return rc;
  if (!(eps > 0.f) || !std::isfinite(eps)) return FA_ERR_INVALID_ARG;
  p.eps = eps;
  return FA_OK;
}

cudaError_t record(void* ev, cudaStream_t st) {
  return ev ? cudaEventRecord(static_cast<cudaEvent_t>(ev), st) : cudaSuccess;
}

}  // namespace

extern "C" {

int fa_qk_norm_rope(const fa_tensor* q, const fa_tensor* k, const fa_tensor* q_weight, const fa_tensor* k_weight,
                    const fa_tensor* q_out, const fa_tensor* k_out, const fa_tensor* positions,
                    const fa_tensor* inv_freq, float eps, float mscale, int32_t interleaved, const fa_opts* opts) {
  if (!opts) return FA_ERR_INVALID_ARG;
  NormParams p;
  int rc;
  if ((rc = check_norm({q, k}, {q_out, k_out}, {q_weight, k_weight}, positions, inv_freq, eps, mscale, p))) return rc;
  if ((rc = check_device()) != FA_OK) return rc;
  TraceRange tr("mfa.qk_norm_rope");
  cudaStream_t st = static_cast<cudaStream_t>(opts->stream);
  cudaError_t e = record(opts->event_begin, st);
  const int d = (int)q->shape[q->ndim - 1], layout = layout_of(interleaved != 0, p.half);
  const bool f16 = q->dtype == FA_DTYPE_F16;
  // A warp takes a whole token where that makes two waves of warps, otherwise the
  // token's rounds are dealt to as many warps as do.
  const int64_t rounds = p.t[0].rounds + p.t[1].rounds, groups = (p.rows + kWarps - 1) / kWarps;
  const int64_t ctas = 2 * (int64_t)sm_count() * kFwdBlocks, units = std::min(rounds, (ctas + groups - 1) / std::max<int64_t>(1, groups));
  p.span = (int32_t)((rounds + units - 1) / units);
  p.units = (int32_t)((rounds + p.span - 1) / p.span);
  const int64_t grid = groups * p.units;
  if (grid > INT32_MAX) return FA_ERR_INVALID_ARG;
  if (e == cudaSuccess && p.rows > 0) {
    if (d == 64) f16 ? launch_fwd<64, true>(p, layout, (unsigned)grid, st) : launch_fwd<64, false>(p, layout, (unsigned)grid, st);
    else f16 ? launch_fwd<128, true>(p, layout, (unsigned)grid, st) : launch_fwd<128, false>(p, layout, (unsigned)grid, st);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = record(opts->event_end, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

int fa_qk_norm_rope_bwd(const fa_tensor* dq_out, const fa_tensor* dk_out, const fa_tensor* q, const fa_tensor* k,
                        const fa_tensor* q_weight, const fa_tensor* k_weight, const fa_tensor* dq, const fa_tensor* dk,
                        const fa_tensor* dq_weight, const fa_tensor* dk_weight, const fa_tensor* positions,
                        const fa_tensor* inv_freq, float eps, float mscale, int32_t interleaved, const fa_opts* opts) {
  if (!opts || !dq_out || (k == nullptr) != (dk_out == nullptr) || (!k && dk_weight)) return FA_ERR_INVALID_ARG;
  NormParams p;
  int rc;
  if ((rc = check_norm({q, k}, {dq, dk}, {q_weight, k_weight}, positions, inv_freq, eps, mscale, p))) return rc;
  const fa_tensor* x[2] = {q, k};
  const fa_tensor* dy[2] = {dq_out, dk_out};
  const fa_tensor* dw[2] = {dq_weight, dk_weight};
  for (int n = 0; n < 2; ++n) {
    if (!x[n]) continue;
    if ((rc = check_bf16(dy[n], x[n]->ndim))) return rc;
    if (dy[n]->dtype != x[n]->dtype || !same_shape(dy[n], x[n])) return FA_ERR_INVALID_ARG;
    p.t[n].dy = static_cast<const uint16_t*>(dy[n]->data);
    strides_of(dy[n], p.t[n].dy_sb, p.t[n].dy_ss, p.t[n].dy_sh);
    if ((rc = check_dw(dw[n], x[n], p.t[n]))) return rc;
  }
  const bool sums = p.t[0].dw || p.t[1].dw;
  if (sums) {
    if (!opts->workspace || (reinterpret_cast<uintptr_t>(opts->workspace) % kAlign) != 0 ||
        opts->workspace_bytes < FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES)
      return FA_ERR_WORKSPACE;
    p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(opts->workspace) + kWsHeadBytes);
  }
  if ((rc = check_device()) != FA_OK) return rc;
  TraceRange tr("mfa.qk_norm_rope_bwd");
  cudaStream_t st = static_cast<cudaStream_t>(opts->stream);
  cudaError_t e = record(opts->event_begin, st);
  const int d = (int)q->shape[q->ndim - 1], layout = layout_of(interleaved != 0, p.half);
  const bool f16 = q->dtype == FA_DTYPE_F16;
  const int most = std::min(sm_count() * kBwdBlocks, kMaxParts);
  const int64_t rounds = p.rows * (p.t[0].rounds + p.t[1].rounds);
  p.n_parts = (int32_t)std::min<int64_t>(most, (rounds + kWarps - 1) / kWarps);
  for (NormRows& r : p.t) {
    const int64_t warps = std::max<int64_t>(1, (int64_t)p.n_parts * kWarps);
    r.share = p.rows * r.rounds / warps;
    r.more = p.rows * r.rounds % warps;
  }
  if (e == cudaSuccess && p.rows > 0) {
    if (d == 64) f16 ? launch_bwd<64, true>(p, layout, p.n_parts, st) : launch_bwd<64, false>(p, layout, p.n_parts, st);
    else f16 ? launch_bwd<128, true>(p, layout, p.n_parts, st) : launch_bwd<128, false>(p, layout, p.n_parts, st);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && sums) e = d == 64 ? launch_dw<64>(p, p.rows > 0, st) : launch_dw<128>(p, p.rows > 0, st);
  if (e == cudaSuccess) e = record(opts->event_end, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // extern "C"
