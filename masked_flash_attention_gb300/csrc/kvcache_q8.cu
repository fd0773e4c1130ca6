// kvcache_q8.cu -- the KV cache held in 8 bits (q8_device.cuh): fa_kvcache_append_q8
// quantises the step's keys (normalised and rotated on the way) and values into
// it, with q beside them, and fa_kvcache_read_q8 reads sequences' keys back.
//
// A block's scale is 2^E with the smallest E whose 448 * 2^E holds every finite
// value of the block.  A block that earlier tokens have begun keeps its scale
// unless the new ones need a larger one; then the tokens before them are
// rounded again to the new scale, so that a block has one scale whenever its tokens
// came.  Values are quantised from fp32 (rotated keys are not rounded to the
// input type first).
//
// Append: HBM (prompts) or latency (single tokens) is the bound; 2 bytes read and
// 1 written per element of k and v, 2 and 2 per element of q.  The CTA of a run of
// packed rows takes the cache blocks whose first new row lies in the run.  A
// team of warps holds one head's block in registers, 16 columns of up to four
// tokens a thread, so that the maximum and the rounding need one read; old
// tokens of the block stand beside the new ones as their values.  Other CTAs
// (the grid's second dimension) rotate the same rows of q.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "q8_device.cuh"
#include "rope_common.cuh"

using namespace mfa;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPasses = 4;  // tokens of a block per thread at most

struct Q8Params {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_sb, q_ss, q_sh, qo_sb, qo_ss, qo_sh, k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;
  uint8_t* code[2];  // K, V
  float* scale[2];
  int64_t c_sb[2], c_ss[2], c_sh[2], s_sb[2], s_ss[2], s_sh[2];
  int32_t hq, hk;
  FastDiv div_hq;
  int64_t rows;
  int32_t S;
  const int32_t* cu_q;
  const int32_t* cache_len;
  int32_t* len_out;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t n_seq, page_size, num_pages;
  int64_t cap;
  const int32_t* positions;
  int64_t pos_sb, pos_ss;
  const double* inv_freq;
  int32_t half;
  float mscale, eps;  // eps 0: no norm
  const void* w[2];   // weights of q, k
  int32_t w_f32[2];
  int32_t block, team;  // tokens of a block, warps that hold one
  int32_t span;         // packed rows per CTA
  int32_t kv_y, q_y;    // CTAs per run for k and v, for q
  WsHeader* ws;
};

// n / f.d for 0 <= n < 2^31.
__device__ __forceinline__ int divide(int n, const FastDiv& f) {
  return f.d == 1 ? n : (int)(__umulhi((uint32_t)n, f.mul) >> f.shr);
}

__device__ __forceinline__ void q8_error(WsHeader* ws, uint32_t info) {
  if (atomicCAS(&ws->error, 0u, (uint32_t)FA_ERR_DEVICE_BOUNDS) == 0u) atomicExch(&ws->error_info, info);
}

// The sequence of a packed row at or after those of sequence s0 (-1: none), by one thread.
__device__ __forceinline__ int seq_from(const int32_t* cu, int n_seq, int s0, int64_t row) {
  if (row < __ldg(cu + s0 + 1)) return row >= __ldg(cu + s0) ? s0 : -1;
  int lo = s0, hi = n_seq;  // the last sequence that starts at or before row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= row) lo = mid;
    else hi = mid;
  }
  return (__ldg(cu + lo) <= row && row < __ldg(cu + lo + 1)) ? lo : -1;
}

__device__ __forceinline__ bool seq_bad(const Q8Params& p, int64_t L, int64_t c0, int64_t n) {
  return L < 0 || n < 0 || c0 < 0 || c0 + n > p.rows || L + n > p.cap;
}

template <bool F16>
__device__ __forceinline__ void load_weight(const void* w, bool f32, Columns at, float (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int col = e < 8 ? at.xa + e : at.xb + e - 8;
    x[e] = !w ? 1.f : f32 ? __ldg(static_cast<const float*>(w) + col) : to_float<F16>(__ldg(static_cast<const uint16_t*>(w) + col));
  }
}

// The row's columns x divided by its root mean square, times w.
template <int kLanes>
__device__ __forceinline__ void norm16(float (&x)[16], const float (&w)[16], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = rsqrtf(fmaf(ss, 1.f / (16 * kLanes), eps));
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * w[e];
}

// One head's block of a cache (n_new new tokens after n_old old ones), by a team of warps.
// src: the first new token's row of the head, or null (a team without a head).
template <int D, bool F16, int LAYOUT, bool IS_K>
__device__ __forceinline__ void enter_block(const Q8Params& p, const uint16_t* src, int64_t src_ss, uint8_t* code,
                                            int64_t code_ss, float* scale, int n_old, int n_new, const float2* cs,
                                            const float (&w)[16], float* row_mem, float* s_top) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;  // tokens of a warp's pass
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % kLanes;
  const int member = warp % p.team;
  const Columns at = columns_of<IS_K ? LAYOUT : kInterleaved>(c, p.half);
  float x[kPasses][16];
  float before = 0.f;
  if (src && n_old > 0) before = *scale;
  const float held = pow2f(scale_exponent(before));
  int tok[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) tok[k] = (member * kPasses + k) * kRows + lane / kLanes;
  uint4 va[kPasses], vb[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    va[k] = vb[k] = make_uint4(0, 0, 0, 0);
    if (!src || tok[k] >= n_old + n_new) continue;
    if (tok[k] < n_old) {
      const uint2 a = *reinterpret_cast<const uint2*>(code + tok[k] * code_ss + at.xa);
      const uint2 b = *reinterpret_cast<const uint2*>(code + tok[k] * code_ss + at.xb);
      va[k].x = a.x; va[k].y = a.y; vb[k].x = b.x; vb[k].y = b.y;
    } else {
      const uint16_t* s = src + (tok[k] - n_old) * src_ss;
      va[k] = *reinterpret_cast<const uint4*>(s + at.xa);
      vb[k] = *reinterpret_cast<const uint4*>(s + at.xb);
    }
  }
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const bool old = tok[k] < n_old;
    unpack16<F16>(va[k], vb[k], x[k]);
    if constexpr (IS_K) {
      if (p.eps > 0.f) norm16<kLanes>(x[k], w, p.eps);
      if (p.half > 0) rotate16<LAYOUT>(x[k], cs + min(max(tok[k] - n_old, 0), max(n_new - 1, 0)) * (D / 2), c, p.half, row_mem);
    }
    if (old) {
      const uint32_t u[4] = {va[k].x, va[k].y, vb[k].x, vb[k].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = e4m3x2_to_float2((uint16_t)u[e]), b = e4m3x2_to_float2((uint16_t)(u[e] >> 16));
        x[k][4 * e] = a.x * held; x[k][4 * e + 1] = a.y * held;
        x[k][4 * e + 2] = b.x * held; x[k][4 * e + 3] = b.y * held;
      }
    } else if (tok[k] < n_old + n_new) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[k][e] = fmaf(x[k][e], 0.f, x[k][e]);  // an infinity becomes a NaN, which the maximum leaves out
        top = fmaxf(top, fabsf(x[k][e]));
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (p.team > 1) {
    // (a barrier of the team's own: its neighbours may be at K while it is at V)
    const int w0 = warp - member;
    auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / p.team), "r"(32 * p.team) : "memory"); };
    if (lane == 0) s_top[warp] = top;
    meet();
    for (int m = 0; m < p.team; ++m) top = fmaxf(top, s_top[w0 + m]);
    meet();
  }
  if (!src) return;
  const int e_old = scale_exponent(before), e_new = block_exponent(top);
  const bool grows = n_old == 0 || e_new > e_old;
  const int e = grows ? e_new : e_old;
  if (grows && member == 0 && lane == 0) *scale = pow2f(e);
  const float down = pow2f(-e);
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    if (tok[k] >= n_old + n_new || (tok[k] < n_old && !grows)) continue;
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = to_e4m3x4(x[k][4 * i] * down, x[k][4 * i + 1] * down, x[k][4 * i + 2] * down, x[k][4 * i + 3] * down);
    *reinterpret_cast<uint2*>(code + tok[k] * code_ss + at.xa) = make_uint2(u[0], u[1]);
    *reinterpret_cast<uint2*>(code + tok[k] * code_ss + at.xb) = make_uint2(u[2], u[3]);
  }
}

template <int D, bool F16, int LAYOUT>
__global__ void __launch_bounds__(kThreads, 2) append_q8_kernel(const __grid_constant__ Q8Params p) {
  constexpr int kLanes = D / 16, kSlots = kThreads / kLanes;
  extern __shared__ float2 cs[];  // [block][D / 2]
  __shared__ float s_row[LAYOUT == kHalfOdd ? kSlots * D : 1];
  __shared__ float s_top[kWarps];
  __shared__ int s_seq[kQ8MaxBlock], s_i[kQ8MaxBlock], s_pos[kQ8MaxBlock];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * p.span;
  const int slot = tid / kLanes, c = tid % kLanes;
  float* row_mem = s_row + (LAYOUT == kHalfOdd ? slot * D : 0);

  // ---- the run's rows: sequence (-1: none, or one whose lengths do not fit) and place in it
  int s0 = -1;
  if (p.cu_q && p.n_seq > 0) {
    // (the last sequence that starts at or before the first row, by every warp)
    int lo = 0, hi = p.n_seq;
    while (hi - lo > 32) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const int n = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(p.cu_q + at) <= row0));
      lo += max(n - 1, 0) * step;
      hi = min(hi, lo + step);
    }
    const int n = __popc(__ballot_sync(0xffffffffu, lo + lane < hi && __ldg(p.cu_q + lo + lane) <= row0));
    s0 = lo + max(n - 1, 0);
  }
  if (tid < p.span) {
    const int64_t row = row0 + tid;
    int s = -1, i = 0, pos = 0;
    if (row < p.rows) s = p.cu_q ? (s0 >= 0 ? seq_from(p.cu_q, p.n_seq, s0, row) : -1) : (int)(row / p.S);
    if (s >= 0) {
      const int64_t c0 = p.cu_q ? __ldg(p.cu_q + s) : (int64_t)s * p.S;
      const int64_t n = p.cu_q ? (int64_t)__ldg(p.cu_q + s + 1) - c0 : p.S;
      const int64_t L = __ldg(p.cache_len + s);
      i = (int)(row - c0);
      if (seq_bad(p, L, c0, n)) s = -1;  // recorded below, once per sequence
      else pos = p.positions ? __ldg(p.positions + (p.cu_q ? row * p.pos_ss : s * p.pos_sb + i * p.pos_ss)) : (int)(L + i);
    }
    s_seq[tid] = s;
    s_i[tid] = i;
    s_pos[tid] = pos;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int s = tid; s < p.n_seq; s += kThreads) {
      const int64_t L = __ldg(p.cache_len + s), c0 = p.cu_q ? __ldg(p.cu_q + s) : (int64_t)s * p.S;
      const int64_t n = p.cu_q ? (int64_t)__ldg(p.cu_q + s + 1) - c0 : p.S;
      const bool bad = seq_bad(p, L, c0, n);
      if (bad) q8_error(p.ws, (uint32_t)s);
      if (p.len_out) p.len_out[s] = (int32_t)(bad ? L : L + n);
    }
  }
  __syncthreads();

  // this thread's pair and its step, for the turns it makes
  const int groups = p.half > 0 ? kThreads / p.half : 0, pair = p.half > 0 ? tid % p.half : 0;
  const uint64_t step = p.half > 0 ? turn_step(__ldg(p.inv_freq + pair)) : 0;

  if ((int)blockIdx.y >= p.kv_y) {
    // ---------------------------------------------------------------- q
    for (int t = p.half > 0 ? tid / p.half : p.span; t < p.span && tid < groups * p.half; t += groups)
      cs[t * (D / 2) + pair] = position_turn(s_pos[t], step, p.mscale, false);
    __syncthreads();
    const Columns at = columns_of<LAYOUT>(c, p.half);
    float w[16];
    load_weight<F16>(p.w[0], p.w_f32[0], at, w);
    const int n = p.span * p.hq;
    for (int e0 = (blockIdx.y - p.kv_y) * kSlots; e0 < n; e0 += 2 * kSlots * p.q_y) {
      uint4 va[2], vb[2];
      uint16_t* dst[2];
      int t[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = e0 + k * kSlots * p.q_y + slot;
        t[k] = 0;
        dst[k] = nullptr;
        va[k] = vb[k] = make_uint4(0, 0, 0, 0);
        if (e < n) {
          t[k] = divide(e, p.div_hq);
          const int h = e - t[k] * p.hq, s = s_seq[t[k]];
          if (s >= 0) {
            const int64_t b = p.cu_q ? 0 : s, i = p.cu_q ? row0 + t[k] : s_i[t[k]];
            const uint16_t* src = p.q + b * p.q_sb + i * p.q_ss + h * p.q_sh;
            dst[k] = p.q_out + b * p.qo_sb + i * p.qo_ss + h * p.qo_sh;
            va[k] = *reinterpret_cast<const uint4*>(src + at.xa);
            vb[k] = *reinterpret_cast<const uint4*>(src + at.xb);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (p.eps > 0.f || p.half > 0) {  // (else the bits are copied)
          float x[16];
          unpack16<F16>(va[k], vb[k], x);
          if (p.eps > 0.f) norm16<kLanes>(x, w, p.eps);
          if (p.half > 0) rotate16<LAYOUT>(x, cs + t[k] * (D / 2), c, p.half, row_mem);
          pack16<F16>(x, va[k], vb[k]);
        }
        if (dst[k]) {
          *reinterpret_cast<uint4*>(dst[k] + at.xa) = va[k];
          *reinterpret_cast<uint4*>(dst[k] + at.xb) = vb[k];
        }
      }
    }
    return;
  }

  // ------------------------------------------------------------------ k and v
  const int teams = kWarps / p.team, team = warp / p.team;
  float w[16];
  load_weight<F16>(p.w[1], p.w_f32[1], columns_of<LAYOUT>(c, p.half), w);
  for (int t = 0; t < p.span; ++t) {
    const int s = s_seq[t], i = s_i[t];
    if (s < 0) continue;
    const int64_t L = __ldg(p.cache_len + s), j = L + i;
    if (i > 0 && j % p.block != 0) continue;  // not the block's first new row
    const int64_t c0 = p.cu_q ? __ldg(p.cu_q + s) : (int64_t)s * p.S;
    const int n_left = (int)((p.cu_q ? (int64_t)__ldg(p.cu_q + s + 1) - c0 : p.S) - i);
    const int n_old = (int)(j % p.block), n_new = min(p.block - n_old, n_left);
    const int64_t j0 = j - n_old;
    int64_t page = s, r = j0;
    if (p.block_table) {
      page = __ldg(p.block_table + s * p.bt_stride + j0 / p.page_size);
      r = j0 % p.page_size;
      if (page < 0 || page >= p.num_pages) {
        if (blockIdx.y == 0 && tid == 0) q8_error(p.ws, (uint32_t)page);
        continue;
      }
    }
    if (p.half > 0 && tid < groups * p.half) {
      const int64_t row = row0 + t;
      for (int m = tid / p.half; m < n_new; m += groups) {
        const int pos = p.positions ? __ldg(p.positions + (p.cu_q ? (row + m) * p.pos_ss : s * p.pos_sb + (i + m) * p.pos_ss)) : (int)(j + m);
        cs[m * (D / 2) + pair] = position_turn(pos, step, p.mscale, false);
      }
    }
    __syncthreads();
    const int64_t sb = p.cu_q ? 0 : s, si = p.cu_q ? row0 + t : i;
    for (int e0 = blockIdx.y * teams; e0 < 2 * p.hk; e0 += teams * p.kv_y) {
      // (a team's head is K or V by itself; a round may hold both)
      const int e = e0 + team, h = e < p.hk ? e : e - p.hk;
      const bool any = e < 2 * p.hk;
      const int which = e < p.hk ? 0 : 1;
      uint8_t* code = p.code[which] + page * p.c_sb[which] + r * p.c_ss[which] + h * p.c_sh[which];
      float* scale = p.scale[which] + page * p.s_sb[which] + (r / p.block) * p.s_ss[which] + h * p.s_sh[which];
      if (which == 0)
        enter_block<D, F16, LAYOUT, true>(p, p.k + sb * p.k_sb + si * p.k_ss + h * p.k_sh, p.k_ss, code, p.c_ss[0], scale, n_old,
                                          n_new, cs, w, row_mem, s_top);
      else
        enter_block<D, F16, LAYOUT, false>(p, any ? p.v + sb * p.v_sb + si * p.v_ss + h * p.v_sh : nullptr, p.v_ss, code, p.c_ss[1],
                                           scale, n_old, n_new, cs, w, row_mem, s_top);
    }
    __syncthreads();  // the turns are read
  }
}

// ---- reading back

constexpr int kReadRows = 32;  // tokens per CTA

struct ReadParams {
  const uint8_t* code[2];
  const float* scale[2];
  uint16_t* out[2];
  int64_t c_sb[2], c_ss[2], c_sh[2], s_sb[2], s_ss[2], s_sh[2], o_sb[2], o_ss[2], o_sh[2];
  int64_t rows, most;  // most: rows per sequence (packed: all)
  int32_t S, hk;
  FastDiv div_hk;
  const int32_t* cu_k;
  const int32_t* lens;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t n_seq, page_size, num_pages, block;
  int64_t cap;
  WsHeader* ws;
};

// Bound: HBM, 1 byte read and 2 written per element.  A thread turns 16 codes
// (one load) into 16 values (two stores), four of them in flight.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) read_q8_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kChunks = D / 16, kAhead = 4;
  __shared__ int64_t s_page[kReadRows], s_at[kReadRows], s_b[kReadRows], s_i[kReadRows];  // page (-1: none), row in it; output row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * kReadRows;
  if (blockIdx.x == 0) {
    for (int s = tid; s < p.n_seq; s += kThreads) {
      const int64_t c0 = p.cu_k ? __ldg(p.cu_k + s) : 0, c1 = p.cu_k ? __ldg(p.cu_k + s + 1) : __ldg(p.lens + s);
      if (c0 < 0 || c1 < c0 || c1 > p.most || c1 - c0 > p.cap) q8_error(p.ws, (uint32_t)s);
    }
  }
  for (int t = warp; t < kReadRows; t += kWarps) {
    const int64_t row = row0 + t;
    int s = -1;
    if (row < p.rows) s = p.cu_k ? find_seq(p.cu_k, p.n_seq, row, lane) : (int)(row / p.S);
    if (lane == 0) {
      int64_t page = -1, at = 0, b = 0, i = row;
      if (s >= 0) {
        int64_t j, n;
        if (p.cu_k) {
          const int64_t c0 = __ldg(p.cu_k + s);
          n = (int64_t)__ldg(p.cu_k + s + 1) - c0;
          j = row - c0;
          if (c0 < 0 || c0 + n > p.rows) n = -1;
        } else {
          n = __ldg(p.lens + s);
          b = s;
          i = j = row - (int64_t)s * p.S;
          if (n > p.most) n = -1;
        }
        if (n >= 0 && n <= p.cap && j < n) {  // (lengths that do not fit are recorded below)
          page = s;
          at = j;
          if (p.block_table) {
            page = __ldg(p.block_table + s * p.bt_stride + j / p.page_size);
            at = j % p.page_size;
            if (page < 0 || page >= p.num_pages) {
              q8_error(p.ws, (uint32_t)page);
              page = -1;
            }
          }
        }
      }
      s_page[t] = page;
      s_at[t] = at;
      s_b[t] = b;
      s_i[t] = i;
    }
  }
  __syncthreads();
  const int n = kReadRows * p.hk * kChunks;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    for (int e0 = tid; e0 < n; e0 += kAhead * kThreads) {
      uint4 u[kAhead];
      float f[kAhead];
      uint16_t* dst[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int e = e0 + k * kThreads;
        dst[k] = nullptr;
        if (e >= n) continue;
        const int c = e % kChunks, th = e / kChunks, t = divide(th, p.div_hk), h = th - t * p.hk;
        const int64_t page = s_page[t], at = s_at[t];
        if (page < 0) continue;
        u[k] = *reinterpret_cast<const uint4*>(p.code[which] + page * p.c_sb[which] + at * p.c_ss[which] + h * p.c_sh[which] + 16 * c);
        f[k] = __ldg(p.scale[which] + page * p.s_sb[which] + (at / p.block) * p.s_ss[which] + h * p.s_sh[which]);
        dst[k] = p.out[which] + s_b[t] * p.o_sb[which] + s_i[t] * p.o_ss[which] + h * p.o_sh[which] + 16 * c;
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (!dst[k]) continue;
        const float s = pow2f(scale_exponent(f[k]));
        const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = e4m3x2_to_float2((uint16_t)w[i]), b = e4m3x2_to_float2((uint16_t)(w[i] >> 16));
          o[2 * i] = pack2<F16>(a.x * s, a.y * s);
          o[2 * i + 1] = pack2<F16>(b.x * s, b.y * s);
        }
        *reinterpret_cast<uint4*>(dst[k]) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst[k] + 8) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

// ---- host

// The 8-bit caches and their scales; heads and head dim as given; block_table and sequences.
template <typename P>
int check_caches(const fa_tensor* const (&code)[2], const fa_tensor* const (&scale)[2], int64_t n_seq, int64_t* block,
                 const fa_tensor* block_table, P& p) {
  int rc;
  int64_t b2 = 0;
  if ((rc = check_q8(code[0], scale[0], block)) || (rc = check_q8(code[1], scale[1], &b2))) return rc;
  if (!same_shape(code[0], code[1]) || *block != b2) return FA_ERR_INVALID_ARG;
  const int64_t d = code[0]->shape[3], hk = code[0]->shape[2];
  if ((d != 64 && d != 128) || hk < 1 || hk > INT32_MAX / 4096) return FA_ERR_INVALID_ARG;
  if (block_table) {
    const int64_t page = code[0]->shape[1];
    if (!block_table->data || block_table->dtype != FA_DTYPE_I32 || block_table->ndim != 2 || block_table->shape[0] != n_seq ||
        block_table->stride[1] != 1 || block_table->stride[0] < 0 || block_table->shape[1] < 1 || page > INT32_MAX ||
        code[0]->shape[0] > INT32_MAX)
      return FA_ERR_INVALID_ARG;
    p.block_table = static_cast<const int32_t*>(block_table->data);
    p.bt_stride = block_table->stride[0];
    p.page_size = (int32_t)page;
    p.num_pages = (int32_t)code[0]->shape[0];
    p.cap = block_table->shape[1] * page;
  } else {
    if (code[0]->shape[0] != n_seq) return FA_ERR_INVALID_ARG;
    p.cap = code[0]->shape[1];
  }
  p.cap = std::min<int64_t>(p.cap, INT32_MAX);
  p.hk = (int32_t)hk;
  p.block = (int32_t)*block;
  for (int n = 0; n < 2; ++n) {
    p.code[n] = static_cast<uint8_t*>(code[n]->data);
    p.scale[n] = static_cast<float*>(scale[n]->data);
    p.c_sb[n] = code[n]->stride[0]; p.c_ss[n] = code[n]->stride[1]; p.c_sh[n] = code[n]->stride[2];
    p.s_sb[n] = scale[n]->stride[0]; p.s_ss[n] = scale[n]->stride[1]; p.s_sh[n] = scale[n]->stride[2];
  }
  return FA_OK;
}

int check_error_word(const fa_opts* opts) {
  return (!opts->workspace || (reinterpret_cast<uintptr_t>(opts->workspace) % kAlign) != 0 ||
          opts->workspace_bytes < FA_KVCACHE_APPEND_WORKSPACE_BYTES)
             ? FA_ERR_WORKSPACE
             : FA_OK;
}

template <int D, bool F16, int LAYOUT>
cudaError_t launch_append(const Q8Params& p, dim3 grid, cudaStream_t st) {
  const int smem = p.block * (D / 2) * (int)sizeof(float2);
  static std::atomic<uint64_t> done{0};  // devices where the kernel may have all the shared memory it can want
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0;
  if (e == cudaSuccess && !(bit && (done.load(std::memory_order_acquire) & bit))) {
    e = cudaFuncSetAttribute(append_q8_kernel<D, F16, LAYOUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kQ8MaxBlock * (D / 2) * (int)sizeof(float2));
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  }
  if (e != cudaSuccess) return e;
  append_q8_kernel<D, F16, LAYOUT><<<grid, kThreads, p.half > 0 ? smem : 0, st>>>(p);
  return cudaGetLastError();
}
template <int D, bool F16>
cudaError_t launch_append(const Q8Params& p, int layout, dim3 grid, cudaStream_t st) {
  if (layout == kInterleaved) return launch_append<D, F16, kInterleaved>(p, grid, st);
  return layout == kHalf ? launch_append<D, F16, kHalf>(p, grid, st) : launch_append<D, F16, kHalfOdd>(p, grid, st);
}

cudaError_t record(void* ev, cudaStream_t st) {
  return ev ? cudaEventRecord(static_cast<cudaEvent_t>(ev), st) : cudaSuccess;
}

int check_weight(const fa_tensor* w, const fa_tensor* x, const void** at, int32_t* is_f32) {
  if (!w) return FA_OK;
  const bool f32 = w->dtype == FA_DTYPE_F32;
  if (!w->data || (!f32 && w->dtype != x->dtype) || w->ndim != 1 || w->shape[0] != x->shape[x->ndim - 1] || w->stride[0] != 1 ||
      (reinterpret_cast<uintptr_t>(w->data) & (f32 ? 3u : 1u)) != 0)
    return FA_ERR_INVALID_ARG;
  *at = w->data;
  *is_f32 = f32;
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_kvcache_append_q8(const fa_tensor* q, const fa_tensor* q_out, const fa_tensor* k_new, const fa_tensor* v_new,
                         const fa_tensor* k_cache, const fa_tensor* v_cache, const fa_tensor* k_scale,
                         const fa_tensor* v_scale, const fa_tensor* cu_seqlens_q, const fa_tensor* cache_seqlens,
                         const fa_tensor* block_table, const fa_tensor* positions, const fa_tensor* inv_freq,
                         float mscale, int32_t interleaved, const fa_tensor* q_weight, const fa_tensor* k_weight,
                         float eps, const fa_tensor* seqlens_out, const fa_opts* opts) {
  if (!k_new || !v_new || !cache_seqlens || !opts || (q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
  Q8Params p;
  memset(&p, 0, sizeof(p));
  int rc;
  const int nd = cu_seqlens_q ? 3 : 4;
  if ((rc = check_bf16(k_new, nd)) || (rc = check_bf16(v_new, nd))) return rc;
  if (!same_shape(k_new, v_new) || v_new->dtype != k_new->dtype) return FA_ERR_INVALID_ARG;
  const int64_t hk = k_new->shape[nd - 2], d = k_new->shape[nd - 1];
  if ((rc = check_rows(k_new, p))) return rc;
  int64_t n_seq;
  if (cu_seqlens_q) {
    if (cu_seqlens_q->ndim != 1 || cu_seqlens_q->shape[0] < 1) return FA_ERR_INVALID_ARG;
    n_seq = cu_seqlens_q->shape[0] - 1;
    if ((rc = check_i32_vec(cu_seqlens_q, n_seq + 1))) return rc;
    p.cu_q = static_cast<const int32_t*>(cu_seqlens_q->data);
  } else {
    n_seq = k_new->shape[0];
    p.S = (int32_t)k_new->shape[1];
  }
  if (n_seq > INT32_MAX / 64) return FA_ERR_INVALID_ARG;
  p.n_seq = (int32_t)n_seq;
  if ((rc = check_i32_vec(cache_seqlens, n_seq))) return rc;
  p.cache_len = static_cast<const int32_t*>(cache_seqlens->data);
  int64_t block = 0;
  if ((rc = check_caches({k_cache, v_cache}, {k_scale, v_scale}, n_seq, &block, block_table, p))) return rc;
  if (k_cache->shape[2] != hk || k_cache->shape[3] != d || !writable(k_cache) || !writable(v_cache) || !writable(k_scale) ||
      !writable(v_scale))
    return FA_ERR_INVALID_ARG;
  // ---- q, norm, rotation
  int64_t hq = 0;
  if (q) {
    if ((rc = check_pair(q, q_out, k_new))) return rc;
    hq = q->shape[nd - 2];
    p.q = static_cast<const uint16_t*>(q->data);
    p.q_out = static_cast<uint16_t*>(q_out->data);
    strides_of(q, p.q_sb, p.q_ss, p.q_sh);
    strides_of(q_out, p.qo_sb, p.qo_ss, p.qo_sh);
  }
  if (hq > INT32_MAX / 1024) return FA_ERR_INVALID_ARG;
  p.hq = (int32_t)hq;
  p.div_hq = make_fastdiv((uint32_t)std::max<int64_t>(hq, 1));
  p.k = static_cast<const uint16_t*>(k_new->data);
  p.v = static_cast<const uint16_t*>(v_new->data);
  strides_of(k_new, p.k_sb, p.k_ss, p.k_sh);
  strides_of(v_new, p.v_sb, p.v_ss, p.v_sh);
  if (!(eps >= 0.f) || !std::isfinite(eps) || (eps == 0.f && (q_weight || k_weight)) || (!q && q_weight)) return FA_ERR_INVALID_ARG;
  p.eps = eps;
  if ((rc = check_weight(q_weight, k_new, &p.w[0], &p.w_f32[0])) || (rc = check_weight(k_weight, k_new, &p.w[1], &p.w_f32[1])))
    return rc;
  if (positions && (rc = check_positions(positions, k_new, p))) return rc;
  if (inv_freq) {
    if ((rc = check_freq(inv_freq, d, &p.half))) return rc;
    if (!std::isfinite(mscale)) return FA_ERR_INVALID_ARG;
    p.inv_freq = static_cast<const double*>(inv_freq->data);
    p.mscale = mscale;
  }
  if (seqlens_out) {
    if ((rc = check_i32_vec(seqlens_out, n_seq))) return rc;
    const int32_t* o = static_cast<const int32_t*>(seqlens_out->data);
    if (n_seq > 0 && o < p.cache_len + n_seq && p.cache_len < o + n_seq) return FA_ERR_INVALID_ARG;
    p.len_out = static_cast<int32_t*>(seqlens_out->data);
  }
  if ((rc = check_error_word(opts)) || (rc = check_device())) return rc;
  p.ws = static_cast<WsHeader*>(opts->workspace);

  TraceRange tr("mfa.kvcache_append_q8");
  cudaStream_t st = static_cast<cudaStream_t>(opts->stream);
  cudaError_t e = record(opts->event_begin, st);
  const int sms = sm_count(), rows_per_warp = kPasses * 512 / (int)d;
  p.team = std::max(1, p.block / rows_per_warp);
  // Rows per CTA: a block's, fewer where that would leave SMs without any; the
  // heads then go over more CTAs too.
  p.span = p.block;
  while (p.span > 1 && p.rows < (int64_t)p.span * sms) p.span /= 2;
  const int64_t runs = (p.rows + p.span - 1) / p.span;
  const int teams = kWarps / p.team, slots = kThreads / ((int)d / 16);
  const int kv_most = (2 * p.hk + teams - 1) / teams, q_most = (int)std::min<int64_t>(1024, ((int64_t)p.span * hq + slots - 1) / slots);
  const int room = (int)std::max<int64_t>(1, 4 * sms / std::max<int64_t>(runs, 1));  // CTAs per run, about
  p.kv_y = std::min(kv_most, room);
  p.q_y = hq ? std::min(q_most, std::max(room, (int)((hq + 2 * hk - 1) / (2 * hk)))) : 0;
  if (e == cudaSuccess && (runs > 0 || n_seq > 0)) {
    const dim3 grid((unsigned)std::max<int64_t>(runs, 1), (unsigned)(p.kv_y + p.q_y));
    const int layout = layout_of(interleaved != 0, p.half);
    const bool f16 = k_new->dtype == FA_DTYPE_F16;
    if (d == 64) e = f16 ? launch_append<64, true>(p, layout, grid, st) : launch_append<64, false>(p, layout, grid, st);
    else e = f16 ? launch_append<128, true>(p, layout, grid, st) : launch_append<128, false>(p, layout, grid, st);
  }
  if (e == cudaSuccess) e = record(opts->event_end, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

int fa_kvcache_read_q8(const fa_tensor* k_cache, const fa_tensor* v_cache, const fa_tensor* k_scale,
                       const fa_tensor* v_scale, const fa_tensor* cu_seqlens_k, const fa_tensor* seqlens_k,
                       const fa_tensor* block_table, const fa_tensor* k_out, const fa_tensor* v_out,
                       const fa_opts* opts) {
  if (!k_out || !v_out || !opts || (cu_seqlens_k == nullptr) == (seqlens_k == nullptr)) return FA_ERR_INVALID_ARG;
  ReadParams p;
  memset(&p, 0, sizeof(p));
  int rc;
  const int nd = cu_seqlens_k ? 3 : 4;
  if ((rc = check_bf16(k_out, nd)) || (rc = check_bf16(v_out, nd))) return rc;
  if (!same_shape(k_out, v_out) || k_out->dtype != v_out->dtype || !writable(k_out) || !writable(v_out)) return FA_ERR_INVALID_ARG;
  if ((rc = check_rows(k_out, p))) return rc;
  p.most = cu_seqlens_k ? p.rows : k_out->shape[1];
  int64_t n_seq;
  if (cu_seqlens_k) {
    if (cu_seqlens_k->ndim != 1 || cu_seqlens_k->shape[0] < 1) return FA_ERR_INVALID_ARG;
    n_seq = cu_seqlens_k->shape[0] - 1;
    if ((rc = check_i32_vec(cu_seqlens_k, n_seq + 1))) return rc;
    p.cu_k = static_cast<const int32_t*>(cu_seqlens_k->data);
  } else {
    n_seq = k_out->shape[0];
    if ((rc = check_i32_vec(seqlens_k, n_seq))) return rc;
    p.lens = static_cast<const int32_t*>(seqlens_k->data);
  }
  if (n_seq > INT32_MAX / 64) return FA_ERR_INVALID_ARG;
  p.n_seq = (int32_t)n_seq;
  int64_t block = 0;
  if ((rc = check_caches({k_cache, v_cache}, {k_scale, v_scale}, n_seq, &block, block_table, p))) return rc;
  const int64_t d = k_cache->shape[3];
  if (k_out->shape[nd - 2] != p.hk || k_out->shape[nd - 1] != d) return FA_ERR_INVALID_ARG;
  p.div_hk = make_fastdiv((uint32_t)p.hk);
  const fa_tensor* out[2] = {k_out, v_out};
  for (int n = 0; n < 2; ++n) {
    p.out[n] = static_cast<uint16_t*>(out[n]->data);
    strides_of(out[n], p.o_sb[n], p.o_ss[n], p.o_sh[n]);
  }
  if ((rc = check_error_word(opts)) || (rc = check_device())) return rc;
  p.ws = static_cast<WsHeader*>(opts->workspace);
  TraceRange tr("mfa.kvcache_read_q8");
  cudaStream_t st = static_cast<cudaStream_t>(opts->stream);
  cudaError_t e = record(opts->event_begin, st);
  if (e == cudaSuccess && (p.rows > 0 || n_seq > 0)) {
    const unsigned grid = (unsigned)std::max<int64_t>(1, (p.rows + kReadRows - 1) / kReadRows);
    const bool f16 = k_out->dtype == FA_DTYPE_F16;
    if (d == 64) f16 ? read_q8_kernel<64, true><<<grid, kThreads, 0, st>>>(p) : read_q8_kernel<64, false><<<grid, kThreads, 0, st>>>(p);
    else f16 ? read_q8_kernel<128, true><<<grid, kThreads, 0, st>>>(p) : read_q8_kernel<128, false><<<grid, kThreads, 0, st>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = record(opts->event_end, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // extern "C"
