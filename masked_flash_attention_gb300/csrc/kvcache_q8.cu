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
// tokens of the block stand beside the new ones as their values.  Other CTAs work
// on q, a warp to a token as in qknorm.cu.
// Measured (4 prompts of 4096 tokens, 32 + 8 heads, d 128, bf16, norms and rotation, pages
// of 64 keys): 92 us (4.0 TB/s), 45 of it k and v and 43 q, both by their instructions;
// 64 single tokens 8 us.  Three CTAs per SM, their values made twice, took 112 us, q's CTAs
// between those of k and v 94.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "norm_rows.cuh"
#include "q8_device.cuh"

using namespace mfa;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPasses = 4;  // tokens of a block per thread at most
constexpr int kAppendBlocks = 2;  // CTAs per SM
constexpr int kAhead = 4;   // rounds of q under way

struct Q8Params {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_sb, q_ss, q_sh, qo_sb, qo_ss, qo_sh, k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;
  uint8_t* code[2];  // K, V
  float* scale[2];
  int64_t c_sb[2], c_ss[2], c_sh[2], s_sb[2], s_ss[2], s_sh[2];
  int32_t hq, hk;
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
  HeadWeight w[2];    // of q, k
  int32_t block, block_shift, team;  // tokens of a block (and its log2), warps that hold one
  FastDiv div_page;
  int32_t span;         // packed rows per CTA
  int32_t kv_y, kv_ctas;  // CTAs per run for k and v, and all of them; the others are q's
  int32_t q_units, q_span, q_rounds;  // q: warps of a token, rounds of heads of a warp and of a token
  WsHeader* ws;
};

// n / f.d for 0 <= n < 2^31.
__device__ __forceinline__ int divide(int n, const FastDiv& f) {
  return f.d == 1 ? n : (int)(__umulhi((uint32_t)n, f.mul) >> f.shr);
}

__device__ __forceinline__ void q8_error(WsHeader* ws, uint32_t info) {
  if (atomicCAS(&ws->error, 0u, (uint32_t)FA_ERR_DEVICE_BOUNDS) == 0u) atomicExch(&ws->error_info, info);
}

// The last sequence that starts at or before a packed row (the first if none does; -1: there
// are none), by a warp.
__device__ __forceinline__ int start_before(const int32_t* cu, int n_seq, int64_t row, int lane) {
  if (n_seq == 0) return -1;
  int lo = 0, hi = n_seq;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(cu + at) <= row));
    lo += max(n - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  const int n = __popc(__ballot_sync(0xffffffffu, lo + lane < hi && __ldg(cu + lo + lane) <= row));
  return lo + max(n - 1, 0);
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

// Where sequence s of the step has its rows; bad: its lengths do not fit.
struct Step {
  int64_t c0, n, L;
  bool bad;
};
__device__ __forceinline__ Step step_of(const Q8Params& p, int s) {
  Step t;
  t.c0 = p.cu_q ? __ldg(p.cu_q + s) : (int64_t)s * p.S;
  t.n = p.cu_q ? (int64_t)__ldg(p.cu_q + s + 1) - t.c0 : p.S;
  t.L = __ldg(p.cache_len + s);
  t.bad = seq_bad(p, t.L, t.c0, t.n);
  return t;
}
__device__ __forceinline__ int position_of(const Q8Params& p, int s, int64_t row, int64_t i, int64_t L) {
  return p.positions ? __ldg(p.positions + (p.cu_q ? row * p.pos_ss : s * p.pos_sb + i * p.pos_ss)) : (int)(L + i);
}

// One head's block of a cache (n_new new tokens after n_old old ones), by a team of warps.
// va, vb: this lane's columns of tokens tok (new rows, or old codes in x and y).
template <int D, bool F16, int LAYOUT, bool IS_K>
__device__ __forceinline__ void enter_block(const Q8Params& p, const uint4 (&va)[kPasses], const uint4 (&vb)[kPasses],
                                            const int (&tok)[kPasses], bool any, uint8_t* code, int64_t code_ss, float* scale,
                                            float before, int n_old, int n_new, const float2* cs, const Weights<D / 16>& s_w,
                                            float* row_mem, float* s_top) {
  constexpr int kLanes = D / 16, kLayout = IS_K ? LAYOUT : kInterleaved;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % kLanes;
  const int member = warp % p.team;
  const Columns at = lane_columns<D, kLayout>(c, p.half);
  const float held = pow2f(scale_exponent(before));
  Pairs y[kPasses];
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    y[k] = unpack_pairs<F16, kLayout>(va[k], vb[k]);
    if constexpr (IS_K) {
      if (p.eps > 0.f) {
        scale_by(y[k], rsqrtf(fmaf(dot<kLanes>(y[k], y[k]), 1.f / D, p.eps)));
        multiply(y[k], weight_of<kLanes>(s_w, 1, c));
      }
      if (p.half > 0) {
        const float2* of = cs + min(max(tok[k] - n_old, 0), max(n_new - 1, 0)) * (D / 2);
        Turns tw;
        load_turns<D, LAYOUT>(of, c, tw);
        rotate<D, LAYOUT>(y[k], tw, of, c, p.half, row_mem);
      }
    }
    if (tok[k] < n_old) {
      const uint32_t u[4] = {va[k].x, va[k].y, vb[k].x, vb[k].y};
      float x[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = e4m3x2_to_float2((uint16_t)u[e]), b = e4m3x2_to_float2((uint16_t)(u[e] >> 16));
        x[4 * e] = a.x * held; x[4 * e + 1] = a.y * held;
        x[4 * e + 2] = b.x * held; x[4 * e + 3] = b.y * held;
      }
      y[k] = pairs_of<kLayout>(x);
    } else if (tok[k] < n_old + n_new) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // an infinity becomes a NaN, which the maximum leaves out
        y[k].a[i] = fma2(y[k].a[i], both(0.f), y[k].a[i]);
        y[k].b[i] = fma2(y[k].b[i], both(0.f), y[k].b[i]);
        top = fmaxf(top, fmaxf(fabsf(y[k].a[i].x), fabsf(y[k].a[i].y)));
        top = fmaxf(top, fmaxf(fabsf(y[k].b[i].x), fabsf(y[k].b[i].y)));
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
  const int e_old = scale_exponent(before), e_new = block_exponent(top);
  const bool grows = n_old == 0 || e_new > e_old;
  const int e = grows ? e_new : e_old;
  if (any && grows && member == 0 && lane == 0) *scale = pow2f(e);
  const float down = pow2f(-e);
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    if (!any || tok[k] >= n_old + n_new || (tok[k] < n_old && !grows)) continue;
    scale_by(y[k], down);
    float x[16];
    columns_from<kLayout>(y[k], x);
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = to_e4m3x4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    *reinterpret_cast<uint2*>(code + tok[k] * code_ss + at.xa) = make_uint2(u[0], u[1]);
    *reinterpret_cast<uint2*>(code + tok[k] * code_ss + at.xb) = make_uint2(u[2], u[3]);
  }
}

// q's token of this warp: its rounds r0 .. of heads.
template <int D, bool F16, int LAYOUT>
__device__ __forceinline__ void q_rows(const Q8Params& p, int64_t row, int r0, float2* cs, const Weights<D / 16>& s_w, float* row_mem) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
  const int lane = threadIdx.x & 31, c = lane % kLanes, slot = lane / kLanes, r1 = min(r0 + p.q_span, p.q_rounds);
  const Columns at = lane_columns<D, LAYOUT>(c, p.half);
  const int b = p.cu_q ? 0 : (int)row / p.S;
  const int64_t i = p.cu_q ? row : row - (int64_t)b * p.S;
  const uint16_t* src = p.q + b * p.q_sb + i * p.q_ss;
  uint4 va[kAhead], vb[kAhead];
  auto load = [&](int r, uint4& x, uint4& y) {
    const int h = r * kHeads + slot;
    x = y = make_uint4(0, 0, 0, 0);
    if (r < r1 && h < p.hq) {
      x = *reinterpret_cast<const uint4*>(src + h * p.q_sh + at.xa);
      y = *reinterpret_cast<const uint4*>(src + h * p.q_sh + at.xb);
    }
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(r0 + k, va[k], vb[k]);
  const int s = p.cu_q ? find_seq(p.cu_q, p.n_seq, row, lane) : b;
  if (s < 0) return;
  const Step st = step_of(p, s);
  if (st.bad) return;
  Turns tw;
  if (p.half > 0) {
    const int pos = position_of(p, s, row, p.cu_q ? row - st.c0 : i, st.L);
    uint64_t u[2];
    turn_steps(p.inv_freq, p.half, lane, u);
    make_turns<LAYOUT>(pos, u, p.half, p.mscale, false, lane, cs);
    load_turns<D, LAYOUT>(cs, c, tw);
  }
  uint16_t* dst = p.q_out + b * p.qo_sb + i * p.qo_ss;
#pragma unroll 1
  for (int r = r0; r < r1; r += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (r + k >= r1) break;
      uint4 ya = va[k], yb = vb[k];
      load(r + k + kAhead, va[k], vb[k]);
      if (p.eps > 0.f || p.half > 0) {  // (else the bits are copied)
        Pairs x = unpack_pairs<F16, LAYOUT>(ya, yb);
        if (p.eps > 0.f) {
          scale_by(x, rsqrtf(fmaf(dot<kLanes>(x, x), 1.f / D, p.eps)));
          multiply(x, weight_of<kLanes>(s_w, 0, c));
        }
        if (p.half > 0) rotate<D, LAYOUT>(x, tw, cs, c, p.half, row_mem);
        pack_pairs<F16, LAYOUT>(x, ya, yb);
      }
      const int h = (r + k) * kHeads + slot;
      if (h < p.hq) {
        *reinterpret_cast<uint4*>(dst + h * p.qo_sh + at.xa) = ya;
        *reinterpret_cast<uint4*>(dst + h * p.qo_sh + at.xb) = yb;
      }
    }
  }
}

template <int D, bool F16, int LAYOUT>
__global__ void __launch_bounds__(kThreads, kAppendBlocks) append_q8_kernel(const __grid_constant__ Q8Params p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kSlots = kThreads / kLanes;
  extern __shared__ __align__(16) float2 cs[];  // [block, at least the warps][D / 2]
  __shared__ Weights<kLanes> s_w;
  __shared__ float s_row[LAYOUT == kHalfOdd ? kSlots * D : 1];
  __shared__ float s_top[kWarps];
  __shared__ int s_seq[kQ8MaxBlock], s_i[kQ8MaxBlock];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = tid % kLanes;
  float* row_mem = s_row + (LAYOUT == kHalfOdd ? tid / kLanes * D : 0);

  if ((int)blockIdx.x >= p.kv_ctas) {
    const uint32_t x = blockIdx.x - p.kv_ctas, group = x / (uint32_t)p.q_units;
    const int64_t row = (int64_t)group * kWarps + warp;
    if (p.eps > 0.f) stage_weights<F16, LAYOUT, kLanes>(p.w[0], p.w[1], p.half, s_w);
    if (row < p.rows) q_rows<D, F16, LAYOUT>(p, row, (int)(x - group * p.q_units) * p.q_span, cs + warp * (D / 2), s_w, row_mem);
    return;
  }

  // ------------------------------------------------------------------ k and v
  const uint32_t run = blockIdx.x / (uint32_t)p.kv_y;
  const int y = (int)(blockIdx.x - run * p.kv_y);
  const int64_t row0 = (int64_t)run * p.span;
  // ---- the run's rows: sequence (-1: none, or one whose lengths do not fit) and place in it
  const int s0 = p.cu_q ? start_before(p.cu_q, p.n_seq, row0, lane) : -1;
  if (tid < p.span) {
    const int64_t row = row0 + tid;
    int s = -1, i = 0;
    if (row < p.rows) s = p.cu_q ? (s0 >= 0 ? seq_from(p.cu_q, p.n_seq, s0, row) : -1) : (int)((uint32_t)row / (uint32_t)p.S);
    if (s >= 0) {
      const Step st = step_of(p, s);
      i = (int)(row - st.c0);
      if (st.bad) s = -1;  // recorded below, once per sequence
      else if (i > 0 && ((int)st.L + i & p.block - 1) != 0) s = -1;  // not the block's first new row
    }
    s_seq[tid] = s;
    s_i[tid] = i;
  }
  if (blockIdx.x == 0) {
    for (int s = tid; s < p.n_seq; s += kThreads) {
      const Step st = step_of(p, s);
      if (st.bad) q8_error(p.ws, (uint32_t)s);
      if (p.len_out) p.len_out[s] = (int32_t)(st.bad ? st.L : st.L + st.n);
    }
  }
  // this thread's pair and its step, for the turns it makes
  const int groups = p.half > 0 ? kThreads / p.half : 0, pair = p.half > 0 ? tid % p.half : 0;
  const uint64_t step = p.half > 0 ? turn_step(__ldg(p.inv_freq + pair)) : 0;
  stage_weights<F16, LAYOUT, kLanes>(p.w[0], p.w[1], p.half, s_w);  // (and the rows are there)

  const int teams = kWarps / p.team, team = warp / p.team, member = warp % p.team;
  uint32_t starts = 0;  // of these 32 rows, those that begin a block, from t on
  for (int t = 0; t < p.span; ++t) {
    if (t % 32 == 0) starts = __ballot_sync(0xffffffffu, t + lane < p.span && s_seq[t + lane] >= 0);
    if (starts == 0) {
      t |= 31;
      continue;
    }
    t = t & ~31 | __ffs(starts) - 1;
    starts &= starts - 1;
    const int s = s_seq[t], i = s_i[t];
    const Step st = step_of(p, s);
    const int j = (int)st.L + i, n_old = j & p.block - 1, n_new = min(p.block - n_old, (int)st.n - i), j0 = j - n_old;
    int64_t page = s, r = j0;
    if (p.block_table) {
      const int column = divide(j0, p.div_page);
      page = __ldg(p.block_table + s * p.bt_stride + column);
      r = j0 - (int64_t)column * p.page_size;
      if (page < 0 || page >= p.num_pages) {
        if (y == 0 && tid == 0) q8_error(p.ws, (uint32_t)page);
        continue;
      }
    }
    const int64_t sb = p.cu_q ? 0 : s, si = p.cu_q ? row0 + t : i;
    for (int e0 = y * teams; e0 < 2 * p.hk; e0 += teams * p.kv_y) {
      // (a team's head is K or V by itself; a round may hold both)
      const int e = min(e0 + team, 2 * p.hk - 1), which = e < p.hk ? 0 : 1, h = e - which * p.hk;
      const bool any = e0 + team < 2 * p.hk;
      const uint16_t* src = which == 0 ? p.k + sb * p.k_sb + si * p.k_ss + h * p.k_sh : p.v + sb * p.v_sb + si * p.v_ss + h * p.v_sh;
      const int64_t src_ss = which == 0 ? p.k_ss : p.v_ss, code_ss = p.c_ss[which];
      uint8_t* code = p.code[which] + page * p.c_sb[which] + r * p.c_ss[which] + h * p.c_sh[which];
      float* scale = p.scale[which] + page * p.s_sb[which] + (r >> p.block_shift) * p.s_ss[which] + h * p.s_sh[which];
      const Columns at = which == 0 ? lane_columns<D, LAYOUT>(c, p.half) : lane_columns<D, kInterleaved>(c, p.half);
      int tok[kPasses];
      uint4 va[kPasses], vb[kPasses];
      const float before = any && n_old > 0 ? *scale : 0.f;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        tok[k] = (member * kPasses + k) * kRows + lane / kLanes;
        va[k] = vb[k] = make_uint4(0, 0, 0, 0);
        if (!any || tok[k] >= n_old + n_new) continue;
        if (tok[k] < n_old) {
          const uint2 a = *reinterpret_cast<const uint2*>(code + tok[k] * code_ss + at.xa);
          const uint2 b = *reinterpret_cast<const uint2*>(code + tok[k] * code_ss + at.xb);
          va[k].x = a.x; va[k].y = a.y; vb[k].x = b.x; vb[k].y = b.y;
        } else {
          const uint16_t* from = src + (tok[k] - n_old) * src_ss;
          va[k] = *reinterpret_cast<const uint4*>(from + at.xa);
          vb[k] = *reinterpret_cast<const uint4*>(from + at.xb);
        }
      }
      if (e0 == y * teams && e0 < p.hk && p.half > 0) {
        // the block's turns, while the rows come
        if (tid < groups * p.half) {
          for (int m = tid / p.half; m < n_new; m += groups)
            cs[m * (D / 2) + turn_place<LAYOUT>(pair)] = position_turn(position_of(p, s, row0 + t + m, i + m, st.L), step, p.mscale, false);
        }
        __syncthreads();
      }
      if (which == 0) enter_block<D, F16, LAYOUT, true>(p, va, vb, tok, any, code, code_ss, scale, before, n_old, n_new, cs, s_w, row_mem, s_top);
      else enter_block<D, F16, LAYOUT, false>(p, va, vb, tok, any, code, code_ss, scale, before, n_old, n_new, cs, s_w, row_mem, s_top);
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
  int32_t n_seq, page_size, num_pages, block, block_shift;
  FastDiv div_page;
  int64_t cap;
  WsHeader* ws;
};

// Bound: HBM, 1 byte read and 2 written per element.  A thread turns 16 codes
// (one load) into 16 values (two stores), four of them in flight.  Measured (64 sequences of
// 128 .. 8192 tokens, 8 heads, d 128, pages of 16): 310 us (6.0 TB/s); 334 us with a
// warp to look up each token, instead of a lane.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) read_q8_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kChunks = D / 16;
  // a token's codes, scales and output, from their tensors' starts; codes -1: no token
  __shared__ int64_t s_code[2][kReadRows], s_scale[2][kReadRows], s_out[2][kReadRows];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t row0 = (int64_t)blockIdx.x * kReadRows;
  if (blockIdx.x == 0) {
    for (int s = tid; s < p.n_seq; s += kThreads) {
      const int64_t c0 = p.cu_k ? __ldg(p.cu_k + s) : 0, c1 = p.cu_k ? __ldg(p.cu_k + s + 1) : __ldg(p.lens + s);
      if (c0 < 0 || c1 < c0 || c1 > p.most || c1 - c0 > p.cap) q8_error(p.ws, (uint32_t)s);
    }
  }
  if (tid < kReadRows) {  // (one warp)
    const int64_t row = row0 + lane;
    const int s0 = p.cu_k ? start_before(p.cu_k, p.n_seq, row0, lane) : 0;
    int s = -1;
    if (row < p.rows) s = p.cu_k ? (s0 >= 0 ? seq_from(p.cu_k, p.n_seq, s0, row) : -1) : (int)((uint32_t)row / (uint32_t)p.S);
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
      if (n >= 0 && n <= p.cap && j < n) {  // (lengths that do not fit are recorded above)
        page = s;
        at = j;
        if (p.block_table) {
          const int column = divide((int)j, p.div_page);
          page = __ldg(p.block_table + s * p.bt_stride + column);
          at = j - (int64_t)column * p.page_size;
          if (page < 0 || page >= p.num_pages) {
            q8_error(p.ws, (uint32_t)page);
            page = -1;
          }
        }
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      s_code[which][lane] = page < 0 ? -1 : page * p.c_sb[which] + at * p.c_ss[which];
      s_scale[which][lane] = page * p.s_sb[which] + (at >> p.block_shift) * p.s_ss[which];
      s_out[which][lane] = b * p.o_sb[which] + i * p.o_ss[which];
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
        const int64_t code = s_code[which][t];
        if (code < 0) continue;
        u[k] = *reinterpret_cast<const uint4*>(p.code[which] + code + h * p.c_sh[which] + 16 * c);
        f[k] = __ldg(p.scale[which] + s_scale[which][t] + h * p.s_sh[which]);
        dst[k] = p.out[which] + s_out[which][t] + h * p.o_sh[which] + 16 * c;
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
  const int smem = std::max(p.block, kWarps) * (D / 2) * (int)sizeof(float2);
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
  p.k = static_cast<const uint16_t*>(k_new->data);
  p.v = static_cast<const uint16_t*>(v_new->data);
  strides_of(k_new, p.k_sb, p.k_ss, p.k_sh);
  strides_of(v_new, p.v_sb, p.v_ss, p.v_sh);
  if (!(eps >= 0.f) || !std::isfinite(eps) || (eps == 0.f && (q_weight || k_weight)) || (!q && q_weight)) return FA_ERR_INVALID_ARG;
  p.eps = eps;
  if ((rc = check_weight(q_weight, k_new, p.w[0])) || (rc = check_weight(k_weight, k_new, p.w[1]))) return rc;
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
  p.div_page = make_fastdiv((uint32_t)std::max(p.page_size, 1));
  while ((1 << p.block_shift) < p.block) ++p.block_shift;

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
  // Their heads go over more CTAs where the runs do not make four waves.
  const int64_t wave = (int64_t)sms * kAppendBlocks;
  const int teams = kWarps / p.team, kv_most = (2 * p.hk + teams - 1) / teams;
  const int64_t kv_want = std::min<int64_t>(kv_most, (4 * wave + runs - 1) / std::max<int64_t>(runs, 1));
  const int64_t kv_each = (kv_most + kv_want - 1) / kv_want;  // (as many rounds to each)
  p.kv_y = (int32_t)((kv_most + kv_each - 1) / kv_each);
  const int64_t kv_ctas = std::max<int64_t>(runs, 1) * p.kv_y;
  // q: a warp takes a whole token where that makes two waves, else fewer of its heads.
  int64_t q_ctas = 0;
  p.q_units = 1;
  if (hq && p.rows > 0) {
    const int at_once = 512 / (int)d;
    const int64_t groups = (p.rows + kWarps - 1) / kWarps;
    p.q_rounds = (p.hq + at_once - 1) / at_once;
    const int64_t units = std::min<int64_t>(p.q_rounds, (2 * wave + groups - 1) / groups);
    p.q_span = (int32_t)((p.q_rounds + units - 1) / units);
    p.q_units = (p.q_rounds + p.q_span - 1) / p.q_span;
    q_ctas = groups * p.q_units;
  }
  if (kv_ctas + q_ctas > INT32_MAX) return FA_ERR_INVALID_ARG;
  p.kv_ctas = (int32_t)kv_ctas;
  if (e == cudaSuccess && (runs > 0 || n_seq > 0)) {
    const dim3 grid((unsigned)(kv_ctas + q_ctas));
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
  p.div_page = make_fastdiv((uint32_t)std::max(p.page_size, 1));
  while ((1 << p.block_shift) < p.block) ++p.block_shift;
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
