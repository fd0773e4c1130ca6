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
// at the store.  A CTA makes the (cos, sin) of up to eight tokens once, in shared
// memory, for all heads; a thread keeps its columns' weights in registers.  The
// backward pass runs a grid of one wave whose threads keep their columns' dw in
// registers over all their rows; a CTA's sum goes to the workspace and a second
// kernel adds the CTAs' in their order, in fp64: no atomics, and the result
// does not depend on scheduling.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "rope_common.cuh"

using namespace mfa;

namespace {

constexpr int kThreads = 256;
constexpr int kFwdBlocks = 3;  // CTAs per SM
constexpr int kBwdBlocks = 2;
constexpr int kMaxTokens = 8;  // tokens per CTA and step
constexpr int kMaxParts = 1024;  // CTAs of the backward pass
static_assert(FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES >= kWsHeadBytes + (size_t)kMaxParts * 2 * 128 * 4, "partials of dw");

enum { kNoWeight = 0, kWeightF32 = 1, kWeight16 = 2 };

// q or k.
struct NormRows {
  const uint16_t* x;
  const uint16_t* dy;  // backward
  uint16_t* out;       // y, or dx
  int64_t x_sb, x_ss, x_sh, dy_sb, dy_ss, dy_sh, out_sb, out_ss, out_sh;
  const void* w;
  float* dw;  // nullable
  int32_t w_kind, heads;
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
  int32_t tb;  // tokens per CTA and step, a power of two
  int64_t steps;  // of tb tokens
  float* part;  // backward: [CTAs][2][D], null without weight gradients
  int32_t n_parts;
};

// Sum over the lanes of a head, in every one of them.
template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool F16>
__device__ __forceinline__ void load_weight(const NormRows& r, Columns at, float (&w)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int col = e < 8 ? at.xa + e : at.xb + e - 8;
    w[e] = r.w_kind == kWeightF32 ? __ldg(static_cast<const float*>(r.w) + col)
         : r.w_kind == kWeight16  ? to_float<F16>(__ldg(static_cast<const uint16_t*>(r.w) + col))
                                  : 1.f;
  }
}

// Tokens row0 .. row0 + tb - 1: their sequences (-1: no such token), rows and turns.
template <int D>
__device__ __forceinline__ void load_tokens(const NormParams& p, int64_t row0, bool inverse, float2* cs, int* s_b, int* s_i,
                                            int* s_pos) {
  const int tid = threadIdx.x;
  if (tid < p.tb) {
    const int64_t row = row0 + tid;
    int b = -1, i = 0, pos = 0;
    if (row < p.rows) {
      b = (int)(row / p.S);
      i = (int)(row - (int64_t)b * p.S);
      pos = p.positions ? __ldg(p.positions + b * p.pos_sb + i * p.pos_ss) : i;
    }
    s_b[tid] = b;
    s_i[tid] = i;
    s_pos[tid] = pos;
  }
  __syncthreads();
  if (p.half > 0) {
    const int groups = kThreads / p.half;  // half <= 64
    if (tid < groups * p.half) {
      const int i = tid % p.half;
      const uint64_t u = turn_step(__ldg(p.inv_freq + i));
      for (int t = tid / p.half; t < p.tb; t += groups) cs[t * (D / 2) + i] = position_turn(s_pos[t], u, p.mscale, inverse);
    }
    __syncthreads();
  }
}

template <int D, bool F16, int LAYOUT>
__global__ void __launch_bounds__(kThreads, kFwdBlocks) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 16, kSlots = kThreads / kLanes;  // threads per head; heads at a time
  __shared__ float2 cs[kMaxTokens * D / 2];
  __shared__ int s_b[kMaxTokens], s_i[kMaxTokens], s_pos[kMaxTokens];
  __shared__ float s_row[LAYOUT == kHalfOdd ? kSlots * D : 1];
  const int c = threadIdx.x % kLanes, slot = threadIdx.x / kLanes, half = p.half;
  load_tokens<D>(p, (int64_t)blockIdx.x * p.tb, false, cs, s_b, s_i, s_pos);
  const int per = kSlots / p.tb;  // slots per token
  const int t = slot / per, b = s_b[t], i = s_i[t];
  const Columns at = columns_of<LAYOUT>(c, half);
  float* row = s_row + (LAYOUT == kHalfOdd ? slot * D : 0);
  const int step = per * gridDim.y;
  // (the lanes of a warp stay together through the shuffles: a slot without a
  // token or head computes on zeros and stores nothing)
#pragma unroll 1
  for (int n = 0; n < 2; ++n) {
    const NormRows& r = p.t[n];
    if (r.heads == 0) continue;
    float w[16];
    load_weight<F16>(r, at, w);
    const uint16_t* src = r.x + b * r.x_sb + i * r.x_ss;
    uint16_t* dst = r.out + b * r.out_sb + i * r.out_ss;
    // as many rounds for every slot
    for (int h0 = blockIdx.y * per; h0 < r.heads; h0 += 2 * step) {
      uint4 va[2], vb[2];
      int h[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        h[k] = h0 + k * step + slot % per;
        if (b < 0 || h[k] >= r.heads) h[k] = -1;
        va[k] = vb[k] = make_uint4(0, 0, 0, 0);
        if (h[k] >= 0) {
          va[k] = *reinterpret_cast<const uint4*>(src + h[k] * r.x_sh + at.xa);
          vb[k] = *reinterpret_cast<const uint4*>(src + h[k] * r.x_sh + at.xb);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[16];
        unpack16<F16>(va[k], vb[k], x);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float inv = rsqrtf(fmaf(head_sum<kLanes>(ss), 1.f / D, p.eps));
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * w[e];
        rotate16<LAYOUT>(x, cs + t * (D / 2), c, half, row);
        if (h[k] >= 0) {
          pack16<F16>(x, va[k], vb[k]);
          *reinterpret_cast<uint4*>(dst + h[k] * r.out_sh + at.xa) = va[k];
          *reinterpret_cast<uint4*>(dst + h[k] * r.out_sh + at.xb) = vb[k];
        }
      }
    }
  }
}

template <int D, bool F16, int LAYOUT>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 16, kSlots = kThreads / kLanes;
  // the turns of a step; after the last step the slots' sums of dw
  __shared__ union {
    float2 cs[kMaxTokens * D / 2];
    float sum[kThreads / 32][D];
  } u;
  __shared__ int s_b[kMaxTokens], s_i[kMaxTokens], s_pos[kMaxTokens];
  __shared__ float s_row[LAYOUT == kHalfOdd ? kSlots * D : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = threadIdx.x % kLanes, slot = threadIdx.x / kLanes, half = p.half, lane = threadIdx.x & 31;
  const int per = kSlots / p.tb, t = slot / per;
  const Columns at = columns_of<LAYOUT>(c, half);
  float* row = s_row + (LAYOUT == kHalfOdd ? slot * D : 0);
  float dw[2][16];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[n][e] = 0.f;

  for (int64_t s = blockIdx.x; s < p.steps; s += gridDim.x) {
    load_tokens<D>(p, s * p.tb, true, u.cs, s_b, s_i, s_pos);
    const int b = s_b[t], i = s_i[t];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const NormRows& r = p.t[n];
      if (r.heads == 0) continue;
      float w[16];
      load_weight<F16>(r, at, w);
      const uint16_t* src = r.x + b * r.x_sb + i * r.x_ss;
      const uint16_t* grad = r.dy + b * r.dy_sb + i * r.dy_ss;
      uint16_t* dst = r.out + b * r.out_sb + i * r.out_ss;
      for (int h0 = 0; h0 < r.heads; h0 += per) {
        int h = h0 + slot % per;
        if (b < 0 || h >= r.heads) h = -1;
        uint4 xa = make_uint4(0, 0, 0, 0), xb = xa, ga = xa, gb = xa;
        if (h >= 0) {
          xa = *reinterpret_cast<const uint4*>(src + h * r.x_sh + at.xa);
          xb = *reinterpret_cast<const uint4*>(src + h * r.x_sh + at.xb);
          ga = *reinterpret_cast<const uint4*>(grad + h * r.dy_sh + at.xa);
          gb = *reinterpret_cast<const uint4*>(grad + h * r.dy_sh + at.xb);
        }
        float x[16], g[16];
        unpack16<F16>(xa, xb, x);
        unpack16<F16>(ga, gb, g);
        rotate16<LAYOUT>(g, u.cs + t * (D / 2), c, half, row);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float inv = rsqrtf(fmaf(head_sum<kLanes>(ss), 1.f / D, p.eps));
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] *= inv;  // the unit row
          dw[n][e] = fmaf(g[e], x[e], dw[n][e]);
          g[e] *= w[e];
          dot = fmaf(g[e], x[e], dot);
        }
        dot = head_sum<kLanes>(dot) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = inv * fmaf(-x[e], dot, g[e]);
        if (h >= 0) {
          pack16<F16>(g, xa, xb);
          *reinterpret_cast<uint4*>(dst + h * r.out_sh + at.xa) = xa;
          *reinterpret_cast<uint4*>(dst + h * r.out_sh + at.xb) = xb;
        }
      }
    }
    __syncthreads();  // the turns are read
  }
  if (!p.part) return;
  // the CTA's sums: over the heads of a warp by shuffles, over its warps in order
#pragma unroll
  for (int n = 0; n < 2; ++n) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = dw[n][e];
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < kLanes) u.sum[threadIdx.x / 32][e < 8 ? at.xa + e : at.xb + e - 8] = v;
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) v += u.sum[k][threadIdx.x];
      p.part[((int64_t)blockIdx.x * 2 + n) * D + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// dw: 32 columns of q's or k's per CTA, the parts dealt to its warps.
template <int D>
__global__ void __launch_bounds__(kThreads) norm_dw_kernel(const __grid_constant__ NormParams p) {
  __shared__ double s[kThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x / (D / 32), col = blockIdx.x % (D / 32) * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!p.t[n].dw) return;
  double v = 0.0;
#pragma unroll 4
  for (int k = warp; k < p.n_parts; k += kThreads / 32) v += p.part[((int64_t)k * 2 + n) * D + col];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int k = 1; k < kThreads / 32; ++k) v += s[k][lane];
    p.t[n].dw[col] = (float)v;
  }
}

template <int D, bool F16>
void launch_fwd(const NormParams& p, int layout, dim3 grid, cudaStream_t st) {
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
  c.gridDim = dim3(2 * D / 32);
  c.blockDim = dim3(kThreads);
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&c, norm_dw_kernel<D>, p);
}

int check_weight(const fa_tensor* w, const fa_tensor* x, NormRows& r) {
  if (!w) return FA_OK;
  const int64_t d = x->shape[x->ndim - 1];
  const bool f32 = w->dtype == FA_DTYPE_F32;
  if (!w->data || (!f32 && w->dtype != x->dtype) || w->ndim != 1 || w->shape[0] != d || w->stride[0] != 1 ||
      (reinterpret_cast<uintptr_t>(w->data) & (f32 ? 3u : 1u)) != 0)
    return FA_ERR_INVALID_ARG;
  r.w = w->data;
  r.w_kind = f32 ? kWeightF32 : kWeight16;
  return FA_OK;
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
    if ((rc = check_pair(x[n], out[n], q)) || (rc = check_weight(w[n], x[n], p.t[n]))) return rc;
    NormRows& r = p.t[n];
    const int64_t h = x[n]->shape[q->ndim - 2];
    heads += h;
    if (heads > INT32_MAX / 1024) return FA_ERR_INVALID_ARG;
    r.heads = (int32_t)h;
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
  // Tokens per CTA: the fewest that one wave of CTAs takes, at most eight; with
  // one, its heads go over the grid's second dimension too.
  const int slots = kThreads / (d / 16), sms = sm_count();
  p.tb = 1;
  while (p.tb < kMaxTokens && p.rows > (int64_t)sms * kFwdBlocks * p.tb) p.tb *= 2;
  p.steps = (p.rows + p.tb - 1) / p.tb;
  int ysplit = 1;
  if (p.tb == 1) {
    const int most = (std::max(p.t[0].heads, p.t[1].heads) + slots - 1) / slots;
    ysplit = p.steps * most <= 8 * sms ? most : 1;
  }
  if (e == cudaSuccess && p.rows > 0) {
    const dim3 grid((unsigned)p.steps, (unsigned)ysplit);
    if (d == 64) f16 ? launch_fwd<64, true>(p, layout, grid, st) : launch_fwd<64, false>(p, layout, grid, st);
    else f16 ? launch_fwd<128, true>(p, layout, grid, st) : launch_fwd<128, false>(p, layout, grid, st);
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
  p.tb = 1;
  while (p.tb < kMaxTokens && p.rows > (int64_t)most * p.tb) p.tb *= 2;
  p.steps = (p.rows + p.tb - 1) / p.tb;
  p.n_parts = (int32_t)std::min<int64_t>(most, p.steps);
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
