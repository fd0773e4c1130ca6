// rope.cu -- rotary positions: fa_rope (forward and inverse), the frequencies
// of scaled embeddings, and fa_kvcache_append, which rotates the new keys on
// their way into a paged or padded KV cache and q beside them.
//
// Pair i of a row at position p turns by the angle p * f_i.  In turns that is
// p * f_i / (2 pi), of which only the fraction matters: f_i / (2 pi) is held as
// a 64-bit binary fraction (units of 2^-64 turn), so the product with an
// integer position, wrapped to 64 bits, is the fraction of the angle, exact to
// |p| * 2^-64 turn at any distance (the fp64 frequency's own rounding is
// larger).  The top 32 bits of it go to sincospif.
//
// Bound: HBM.  Every element is read once and written once (4 bytes per
// element), 3 flop each; the angles are made once per (token, pair) in shared
// memory and serve all heads of the token.  A thread takes 16 elements of one
// head (two 16-byte loads) of one token, keeps the 8 (cos, sin) of its columns
// in registers and walks the token's heads, two of them in flight; four CTAs per
// SM hide each other's starts (three with four heads in flight were 4 % slower,
// six spill).  Measured (copy rate 6792 GB/s): q and k of 8192 tokens, 32 / 8
// heads, d = 128, in a graph 29.5 us, 0.84 of the copy rate; of 65536 tokens 196
// us, 1.01 (201, 0.98, after an L2 flush); 16384 tokens appended with q 67.2 us,
// 0.88; one token 3.2 us.  Pairs whose
// columns no 16-byte load holds (kHalfOdd) run at 0.46.
#include <climits>
#include <cmath>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "fa_internal.h"

using namespace mfa;

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBlocks = 4;  // CTAs per SM
constexpr int kMaxTokens = 8;   // tokens per CTA

// One of q, k, v: rows of `heads` heads, read at in + b * in_sb + i * in_ss,
// written at out + b * out_sb + i * out_ss (the cache's page and row strides
// for the appended k and v).
struct RopeRows {
  const uint16_t* in;
  uint16_t* out;
  int64_t in_sb, in_ss, in_sh, out_sb, out_ss, out_sh;
};

struct RopeParams {
  RopeRows t[3];  // q, k, v (v in the append only)
  int32_t hq, hk, heads;  // heads = hq + hk (+ hk of v in the append)
  int64_t rows;
  int32_t S;  // rows per sequence of the fixed-length form; packed: rows
  const int32_t* positions;
  int64_t pos_sb, pos_ss;
  const double* inv_freq;
  int32_t half;  // pairs
  float mscale;
  int32_t inverse;
  int32_t tb;  // tokens per CTA, a power of two
  // append
  const int32_t* cu_q;
  const int32_t* cache_len;
  int32_t* len_out;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t n_seq, page_size, num_pages;
  int64_t cap;
  WsHeader* ws;
};

// f / (2 pi) modulo 1 in units of 2^-64: f = m * 2^(e - 63) with the 64-bit
// mantissa m, and m * round(2^66 / (2 pi)) / 2^64 = m * 4 / (2 pi), so the
// fraction is that product times 2^(e - 1).
__device__ __forceinline__ uint64_t turn_step(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int ex = (int)((bits >> 52) & 0x7ff);
  if (ex == 0 || ex == 0x7ff) return 0;  // zero (and what is too small to turn); not finite: not accepted
  const uint64_t m = (bits << 11) | (1ull << 63);
  const uint64_t hi = __umul64hi(m, 0xa2f9836e4e44152aull);
  const int sh = ex - 1023 - 1;
  uint64_t u = 0;
  if (sh >= 0) u = sh < 64 ? hi << sh : 0;
  else u = -sh < 64 ? hi >> -sh : 0;
  return (bits >> 63) ? 0 - u : u;
}

// The sequence whose rows [cu[s], cu[s + 1]) hold `row`, found by a warp: 32
// probes a step instead of one.  -1 when there is none.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n_seq, int64_t row, int lane) {
  int lo = 0, hi = n_seq;  // the number of sequences that start at or before row is in (lo, hi]
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int c = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(cu + at) <= row));
    if (c == 0) return -1;
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
  }
  const int at = lo + lane;
  const int c = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(cu + at) <= row));
  if (c == 0) return -1;
  const int s = lo + c - 1;
  return (__ldg(cu + s) <= row && row < __ldg(cu + s + 1)) ? s : -1;
}

// Append: a sequence whose rows [c0, c0 + n) or L cached keys do not fit.
__device__ __forceinline__ bool seq_bad(const RopeParams& p, int64_t L, int64_t c0, int64_t n) {
  return L < 0 || n < 0 || c0 < 0 || c0 + n > p.rows || L + n > p.cap;
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  else return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}
template <bool F16>
__device__ __forceinline__ float to_float(uint16_t u) {
  if constexpr (F16) return __half2float(__ushort_as_half(u));
  else return __uint_as_float((uint32_t)u << 16);
}

// Layouts of the pairs.  kHalf: columns i and i + half, half a multiple of 8,
// so a thread's two 16-byte pieces are the two sides of 8 pairs.
// kInterleaved: columns 2i and 2i + 1 of 16 consecutive columns.  kHalfOdd: as
// kHalf with any half; a thread reads its columns' partners one by one (they
// come from L1) and the head's threads, all of one warp, meet between reads and
// writes, so that in-place calls hold.
enum { kHalf = 0, kInterleaved = 1, kHalfOdd = 2 };

template <int D, bool F16, int LAYOUT, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 16;  // threads per head
  __shared__ float2 cs[kMaxTokens * D / 2];
  __shared__ int s_pos[kMaxTokens], s_b[kMaxTokens], s_i[kMaxTokens];
  __shared__ int64_t s_ko[kMaxTokens], s_vo[kMaxTokens];  // append: cache row offsets, -1 = not written
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * p.tb;

  // ---- where each token goes: sequence (-1: none), row in it, position
  if constexpr (APPEND) {
    for (int t = warp; t < p.tb; t += kRopeThreads / 32) {
      const int64_t row = row0 + t;
      int s = -1;
      if (row < p.rows) s = p.cu_q ? find_seq(p.cu_q, p.n_seq, row, lane) : (int)(row / p.S);
      if (lane == 0) {
        int pos = 0, i = 0;
        int64_t ko = -1, vo = -1;
        if (s >= 0) {
          const int64_t c0 = p.cu_q ? __ldg(p.cu_q + s) : (int64_t)s * p.S;
          const int64_t n = p.cu_q ? (int64_t)__ldg(p.cu_q + s + 1) - c0 : p.S;
          const int64_t L = __ldg(p.cache_len + s);
          i = (int)(row - c0);
          if (seq_bad(p, L, c0, n)) {
            s = -1;  // recorded below, once per sequence
          } else {
            const int64_t j = L + i;
            pos = p.positions ? __ldg(p.positions + (p.cu_q ? row * p.pos_ss : s * p.pos_sb + i * p.pos_ss)) : (int)j;
            int64_t page = s, r = j;
            bool ok = true;
            if (p.block_table) {
              r = j % p.page_size;
              page = __ldg(p.block_table + s * p.bt_stride + j / p.page_size);
              ok = page >= 0 && page < p.num_pages;
              if (!ok && blockIdx.y == 0 && atomicCAS(&p.ws->error, 0u, (uint32_t)FA_ERR_DEVICE_BOUNDS) == 0u)
                atomicExch(&p.ws->error_info, (uint32_t)page);
            }
            if (ok) {
              ko = page * p.t[1].out_sb + r * p.t[1].out_ss;
              vo = page * p.t[2].out_sb + r * p.t[2].out_ss;
            }
          }
        }
        s_b[t] = s;
        s_i[t] = i;
        s_pos[t] = pos;
        s_ko[t] = ko;
        s_vo[t] = vo;
      }
    }
    // the new lengths, and the sequences whose lengths do not fit
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      for (int s = tid; s < p.n_seq; s += kRopeThreads) {
        const int64_t L = __ldg(p.cache_len + s), c0 = p.cu_q ? __ldg(p.cu_q + s) : (int64_t)s * p.S;
        const int64_t n = p.cu_q ? (int64_t)__ldg(p.cu_q + s + 1) - c0 : p.S;
        const bool bad = seq_bad(p, L, c0, n);
        if (bad && atomicCAS(&p.ws->error, 0u, (uint32_t)FA_ERR_DEVICE_BOUNDS) == 0u)
          atomicExch(&p.ws->error_info, (uint32_t)s);
        if (p.len_out) p.len_out[s] = (int32_t)(bad ? L : L + n);
      }
    }
  } else if (tid < p.tb) {
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

  // ---- the angles of the CTA's tokens
  if (p.half > 0) {
    const int groups = kRopeThreads / p.half;  // half <= 64
    if (tid < groups * p.half) {
      const int i = tid % p.half;
      const uint64_t u = turn_step(__ldg(p.inv_freq + i));
      for (int t = tid / p.half; t < p.tb; t += groups) {
        const uint64_t a = (uint64_t)(int64_t)s_pos[t] * u;
        // [-1, 1) half turns
        const float x = (float)(int32_t)(uint32_t)(a >> 32) * 4.656612873077393e-10f;  // 2^-31
        float sn, co;
        sincospif(x, &sn, &co);
        cs[t * (D / 2) + i] = make_float2(co * p.mscale, (p.inverse ? -sn : sn) * p.mscale);
      }
    }
    __syncthreads();
  }

  // ---- the rows
  constexpr int kSlots = kRopeThreads / kLanes;
  const int c = tid % kLanes, slot = tid / kLanes;
  const int per = kSlots / p.tb;  // slots per token
  const int t = slot / per;
  const int b = s_b[t], i = s_i[t];
  if (b < 0) return;
  const int half = p.half;
  // packed rows: the fixed-length form's b is 0 or the sequence's own (append)
  const int64_t ib = (APPEND && p.cu_q) ? 0 : b, ii = (APPEND && p.cu_q) ? row0 + t : i;
  int64_t ko = 0, vo = 0;
  if constexpr (APPEND) {
    ko = s_ko[t];
    vo = s_vo[t];
  }
  // this thread's columns: two runs of 8 from xa and xb, and their angles
  int xa = 16 * c, xb = 16 * c + 8;
  bool turned = false;
  float2 w[8];
  if (LAYOUT == kHalf && 8 * c < half) {
    xa = 8 * c;
    xb = half + 8 * c;
  }
  if (LAYOUT != kHalfOdd && 8 * c < half) {
    turned = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 8 * c + e < half ? cs[t * (D / 2) + 8 * c + e] : make_float2(1.f, 0.f);
  }
  if (LAYOUT == kHalfOdd) turned = 16 * c < 2 * half;
  const unsigned group = ((1u << kLanes) - 1u) << (lane & ~(kLanes - 1));

  const int step = per * gridDim.y;
  constexpr int U = LAYOUT == kHalfOdd ? 1 : 2;  // heads in flight
  for (int h0 = blockIdx.y * per + slot % per; h0 < p.heads; h0 += U * step) {
    uint4 va[U], vb[U];
    uint16_t* dst[U];
    bool rot[U];
    uint32_t mate[8];  // kHalfOdd: the 16 partners
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = h0 + k * step;
      dst[k] = nullptr;
      rot[k] = false;
      if (h < p.heads) {
        const int n = h < p.hq ? 0 : (h < p.hq + p.hk ? 1 : 2);
        const RopeRows& r = p.t[n];
        const int hh = h - (n == 0 ? 0 : (n == 1 ? p.hq : p.hq + p.hk));
        const uint16_t* src = r.in + ib * r.in_sb + ii * r.in_ss + hh * r.in_sh;
        const int64_t at = (APPEND && n > 0) ? (n == 1 ? ko : vo) : ib * r.out_sb + ii * r.out_ss;
        if (at >= 0) {
          dst[k] = r.out + at + hh * r.out_sh;
          rot[k] = turned && n < 2;
          va[k] = *reinterpret_cast<const uint4*>(src + xa);
          vb[k] = *reinterpret_cast<const uint4*>(src + xb);
          if constexpr (LAYOUT == kHalfOdd) {
            if (rot[k]) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int x0 = 16 * c + 2 * e, x1 = x0 + 1;
                const int y0 = x0 < half ? x0 + half : (x0 < 2 * half ? x0 - half : x0);
                const int y1 = x1 < half ? x1 + half : (x1 < 2 * half ? x1 - half : x1);
                mate[e] = (uint32_t)src[y0] | ((uint32_t)src[y1] << 16);
              }
            }
          }
        }
      }
    }
    if (LAYOUT == kHalfOdd) __syncwarp(group);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (!dst[k]) continue;
      if (rot[k]) {
        uint32_t* a = reinterpret_cast<uint32_t*>(&va[k]);
        uint32_t* bq = reinterpret_cast<uint32_t*>(&vb[k]);
        if constexpr (LAYOUT == kHalf) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack2<F16>(a[e]), y = unpack2<F16>(bq[e]);
            const float2 w0 = w[2 * e], w1 = w[2 * e + 1];
            a[e] = pack2<F16>(x.x * w0.x - y.x * w0.y, x.y * w1.x - y.y * w1.y);
            bq[e] = pack2<F16>(x.x * w0.y + y.x * w0.x, x.y * w1.y + y.y * w1.x);
          }
        } else if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t& u = e < 4 ? a[e & 3] : bq[e & 3];
            const float2 x = unpack2<F16>(u);
            if (8 * c + e < half) u = pack2<F16>(x.x * w[e].x - x.y * w[e].y, x.x * w[e].y + x.y * w[e].x);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t& u = e < 4 ? a[e & 3] : bq[e & 3];
            uint32_t o = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int x = 16 * c + 2 * e + q;
              const uint16_t own = (uint16_t)(u >> (16 * q));
              uint16_t res = own;
              if (x < 2 * half) {
                const float2 ww = cs[t * (D / 2) + (x < half ? x : x - half)];
                const float v = to_float<F16>(own), m = to_float<F16>((uint16_t)(mate[e] >> (16 * q)));
                res = (uint16_t)pack2<F16>(x < half ? v * ww.x - m * ww.y : m * ww.y + v * ww.x, 0.f);
              }
              o |= (uint32_t)res << (16 * q);
            }
            u = o;
          }
        }
      }
      *reinterpret_cast<uint4*>(dst[k] + xa) = va[k];
      *reinterpret_cast<uint4*>(dst[k] + xb) = vb[k];
    }
  }
}

template <int D, bool F16, bool APPEND>
void launch_layout(const RopeParams& p, bool interleaved, dim3 grid, cudaStream_t st) {
  if (interleaved || p.half == 0)
    rope_kernel<D, F16, kInterleaved, APPEND><<<grid, kRopeThreads, 0, st>>>(p);
  else if (p.half % 8 == 0)
    rope_kernel<D, F16, kHalf, APPEND><<<grid, kRopeThreads, 0, st>>>(p);
  else
    rope_kernel<D, F16, kHalfOdd, APPEND><<<grid, kRopeThreads, 0, st>>>(p);
}

template <bool APPEND>
int launch_rope(RopeParams& p, int d, bool f16, bool interleaved, const fa_opts* opts, const char* range) {
  TraceRange tr(range);
  cudaStream_t st = static_cast<cudaStream_t>(opts->stream);
  cudaError_t e = cudaSuccess;
  if (opts->event_begin) e = cudaEventRecord(static_cast<cudaEvent_t>(opts->event_begin), st);
  // Tokens per CTA: the fewest that one wave of CTAs takes, at most eight.  With
  // one, the heads go over the grid's second dimension too, so that a thread has
  // one head (1050 tokens in two waves of one each took 9.1 us, in one of four 4.7).
  const int slots = kRopeThreads / (d / 16), sms = sm_count();
  p.tb = 1;
  while (p.tb < kMaxTokens && p.rows > (int64_t)sms * kRopeBlocks * p.tb) p.tb *= 2;
  const int64_t blocks = (p.rows + p.tb - 1) / p.tb;
  int ysplit = 1;
  if (p.tb == 1) {
    const int most = (p.heads + slots - 1) / slots;
    ysplit = blocks * most <= 8 * sms ? most : 1;
  }
  if (e == cudaSuccess && (blocks > 0 || p.n_seq > 0)) {
    const dim3 grid((unsigned)(blocks > 0 ? blocks : 1), (unsigned)ysplit);
    if (d == 64) {
      if (f16) launch_layout<64, true, APPEND>(p, interleaved, grid, st);
      else launch_layout<64, false, APPEND>(p, interleaved, grid, st);
    } else {
      if (f16) launch_layout<128, true, APPEND>(p, interleaved, grid, st);
      else launch_layout<128, false, APPEND>(p, interleaved, grid, st);
    }
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && opts->event_end) e = cudaEventRecord(static_cast<cudaEvent_t>(opts->event_end), st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

// Strides of a [B, S, H, d] or [total, H, d] tensor.
void strides_of(const fa_tensor* t, int64_t& sb, int64_t& ss, int64_t& sh) {
  if (t->ndim == 3) { sb = 0; ss = t->stride[0]; sh = t->stride[1]; }
  else { sb = t->stride[0]; ss = t->stride[1]; sh = t->stride[2]; }
}

bool same_shape(const fa_tensor* a, const fa_tensor* b) {
  if (a->ndim != b->ndim) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i]) return false;
  return true;
}

// A written tensor holds every element once: no stride of 0 along more than
// one element.
bool writable(const fa_tensor* t) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] == 0) return false;
  return true;
}

// x and its output: one shape and type, like `like` but for the heads.
int check_pair(const fa_tensor* x, const fa_tensor* y, const fa_tensor* like) {
  int rc;
  if ((rc = check_bf16(x, like->ndim)) || (rc = check_bf16(y, like->ndim))) return rc;
  if (x->dtype != like->dtype || y->dtype != like->dtype || !same_shape(x, y) || !writable(y))
    return FA_ERR_INVALID_ARG;
  for (int i = 0; i < like->ndim; ++i)
    if (i != like->ndim - 2 && x->shape[i] != like->shape[i]) return FA_ERR_INVALID_ARG;
  return x->shape[like->ndim - 2] < 1 ? FA_ERR_INVALID_ARG : FA_OK;
}

int check_freq(const fa_tensor* f, int64_t d, int32_t* half) {
  if (!f->data || f->dtype != FA_DTYPE_F64 || f->ndim != 1 || f->stride[0] != 1 ||
      (reinterpret_cast<uintptr_t>(f->data) & 7u) != 0 || f->shape[0] < 1 || 2 * f->shape[0] > d)
    return FA_ERR_INVALID_ARG;
  *half = (int32_t)f->shape[0];
  return FA_OK;
}

int check_positions(const fa_tensor* t, const fa_tensor* x, RopeParams& p) {
  const int nd = x->ndim - 2;  // [B, S] or [total]
  if (!t->data || t->dtype != FA_DTYPE_I32 || t->ndim != nd || (reinterpret_cast<uintptr_t>(t->data) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  for (int i = 0; i < nd; ++i)
    if (t->shape[i] != x->shape[i] || t->stride[i] < 0) return FA_ERR_INVALID_ARG;
  p.positions = static_cast<const int32_t*>(t->data);
  p.pos_sb = nd == 2 ? t->stride[0] : 0;
  p.pos_ss = t->stride[nd - 1];
  return FA_OK;
}

void set_rows(RopeRows& r, const fa_tensor* x, const fa_tensor* y) {
  r.in = static_cast<const uint16_t*>(x->data);
  r.out = static_cast<uint16_t*>(y->data);
  strides_of(x, r.in_sb, r.in_ss, r.in_sh);
  strides_of(y, r.out_sb, r.out_ss, r.out_sh);
}

// Rows of q-like tensor x: total, and rows per sequence of its layout.
int check_rows(const fa_tensor* x, RopeParams& p) {
  const int64_t B = x->ndim == 4 ? x->shape[0] : 1, S = x->shape[x->ndim - 3];
  if (B > INT32_MAX / 64 || S > INT32_MAX / 64 || (S > 0 && B > INT32_MAX / S)) return FA_ERR_INVALID_ARG;
  p.rows = B * S;
  p.S = (int32_t)(S > 0 ? S : 1);
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_rope(const fa_tensor* q, const fa_tensor* k, const fa_tensor* q_out, const fa_tensor* k_out,
            const fa_tensor* positions, const fa_tensor* inv_freq, float mscale, int32_t interleaved,
            int32_t inverse, const fa_opts* opts) {
  if (!q || !q_out || !inv_freq || !opts || (k == nullptr) != (k_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (q->ndim != 3 && q->ndim != 4) return FA_ERR_INVALID_ARG;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  int rc;
  if ((rc = check_pair(q, q_out, q))) return rc;
  const int64_t d = q->shape[q->ndim - 1];
  if (d != 64 && d != 128) return FA_ERR_INVALID_ARG;
  if (k && (rc = check_pair(k, k_out, q))) return rc;
  if ((rc = check_rows(q, p)) || (rc = check_freq(inv_freq, d, &p.half))) return rc;
  if (positions) {
    if ((rc = check_positions(positions, q, p))) return rc;
  } else if (q->ndim == 3) {
    return FA_ERR_INVALID_ARG;
  }
  if (!std::isfinite(mscale)) return FA_ERR_INVALID_ARG;
  const int64_t hq = q->shape[q->ndim - 2], hk = k ? k->shape[q->ndim - 2] : 0;
  if (hq + hk > INT32_MAX / 1024) return FA_ERR_INVALID_ARG;
  p.hq = (int32_t)hq;
  p.hk = (int32_t)hk;
  p.heads = p.hq + p.hk;
  set_rows(p.t[0], q, q_out);
  if (k) set_rows(p.t[1], k, k_out);
  p.inv_freq = static_cast<const double*>(inv_freq->data);
  p.mscale = mscale;
  p.inverse = inverse ? 1 : 0;
  if ((rc = check_device()) != FA_OK) return rc;
  return launch_rope<false>(p, (int)d, q->dtype == FA_DTYPE_F16, interleaved != 0, opts, "mfa.rope");
}

int fa_rope_inv_freq(int32_t rot, double base, const fa_rope_scaling* scaling, double* inv_freq, float* mscale) {
  if (!inv_freq || !mscale || rot < 2 || rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
    return FA_ERR_INVALID_ARG;
  const int kind = scaling ? scaling->kind : FA_ROPE_PLAIN;
  const int half = rot / 2;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (kind < FA_ROPE_PLAIN || kind > FA_ROPE_YARN) return FA_ERR_INVALID_ARG;
  if (kind != FA_ROPE_PLAIN && (!(scaling->factor >= 1.0) || !std::isfinite(scaling->factor))) return FA_ERR_INVALID_ARG;
  if (kind == FA_ROPE_NTK && rot == 2) return FA_ERR_INVALID_ARG;
  const bool turns = kind == FA_ROPE_BLEND || kind == FA_ROPE_YARN;
  if (turns && (scaling->original_len < 1 || !(scaling->low > 0.0) || !(scaling->high > scaling->low) ||
                !std::isfinite(scaling->high)))
    return FA_ERR_INVALID_ARG;
  if (kind == FA_ROPE_NTK) base *= std::pow(scaling->factor, (double)rot / (rot - 2));
  if (!std::isfinite(base)) return FA_ERR_INVALID_ARG;
  *mscale = 1.0f;
  // YaRN: pair index (real) whose frequency makes n turns in original_len
  // positions, original_len * base^(-2i/rot) = 2 pi n
  double lo = 0.0, hi = 0.0;
  if (kind == FA_ROPE_YARN) {
    auto index = [&](double n) { return rot * std::log(scaling->original_len / (kTwoPi * n)) / (2.0 * std::log(base)); };
    lo = std::fmax(0.0, std::floor(index(scaling->high)));
    hi = std::fmin((double)rot - 1.0, std::ceil(index(scaling->low)));
    if (!(hi > lo)) hi = lo + 1e-3;
    *mscale = (float)(0.1 * std::log(scaling->factor) + 1.0);
  }
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    double kept = 1.0;  // share of the unscaled frequency
    if (kind == FA_ROPE_LINEAR) kept = 0.0;
    if (kind == FA_ROPE_BLEND) kept = (scaling->original_len * f / kTwoPi - scaling->low) / (scaling->high - scaling->low);
    if (kind == FA_ROPE_YARN) kept = 1.0 - (i - lo) / (hi - lo);
    kept = std::fmin(1.0, std::fmax(0.0, kept));
    inv_freq[i] = kept >= 1.0 ? f : kept * f + (1.0 - kept) * (f / scaling->factor);
  }
  return FA_OK;
}

int fa_kvcache_append(const fa_tensor* q, const fa_tensor* q_out, const fa_tensor* k_new, const fa_tensor* v_new,
                      const fa_tensor* k_cache, const fa_tensor* v_cache, const fa_tensor* cu_seqlens_q,
                      const fa_tensor* cache_seqlens, const fa_tensor* block_table, const fa_tensor* positions,
                      const fa_tensor* inv_freq, float mscale, int32_t interleaved, const fa_tensor* seqlens_out,
                      const fa_opts* opts) {
  if (!k_new || !v_new || !k_cache || !v_cache || !cache_seqlens || !opts || (q == nullptr) != (q_out == nullptr))
    return FA_ERR_INVALID_ARG;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  int rc;
  const int nd = cu_seqlens_q ? 3 : 4;
  if ((rc = check_bf16(k_new, nd)) || (rc = check_bf16(v_new, nd))) return rc;
  if (!same_shape(k_new, v_new) || v_new->dtype != k_new->dtype) return FA_ERR_INVALID_ARG;
  const int64_t hk = k_new->shape[nd - 2], d = k_new->shape[nd - 1];
  if ((d != 64 && d != 128) || hk < 1) return FA_ERR_INVALID_ARG;
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
  // ---- cache
  if ((rc = check_bf16(k_cache, 4)) || (rc = check_bf16(v_cache, 4))) return rc;
  if (k_cache->dtype != k_new->dtype || v_cache->dtype != k_new->dtype || !same_shape(k_cache, v_cache) ||
      !writable(k_cache) || !writable(v_cache) || k_cache->shape[2] != hk || k_cache->shape[3] != d)
    return FA_ERR_INVALID_ARG;
  if (block_table) {
    const int64_t page = k_cache->shape[1];
    if (!block_table->data || block_table->dtype != FA_DTYPE_I32 || block_table->ndim != 2 ||
        block_table->shape[0] != n_seq || block_table->stride[1] != 1 || block_table->stride[0] < 0 ||
        block_table->shape[1] < 1 || page < 1 || page > INT32_MAX || k_cache->shape[0] > INT32_MAX)
      return FA_ERR_INVALID_ARG;
    p.block_table = static_cast<const int32_t*>(block_table->data);
    p.bt_stride = block_table->stride[0];
    p.page_size = (int32_t)page;
    p.num_pages = (int32_t)k_cache->shape[0];
    p.cap = block_table->shape[1] * page;
  } else {
    if (k_cache->shape[0] != n_seq) return FA_ERR_INVALID_ARG;
    p.cap = k_cache->shape[1];
  }
  if (p.cap > INT32_MAX) p.cap = INT32_MAX;  // lengths and positions are int32
  // ---- q, rotation
  int64_t hq = 0;
  if (q) {
    if ((rc = check_pair(q, q_out, k_new))) return rc;
    hq = q->shape[nd - 2];
    set_rows(p.t[0], q, q_out);
  }
  if (hq + 2 * hk > INT32_MAX / 1024) return FA_ERR_INVALID_ARG;
  set_rows(p.t[1], k_new, k_cache);
  set_rows(p.t[2], v_new, v_cache);
  p.t[1].out_sb = k_cache->stride[0]; p.t[1].out_ss = k_cache->stride[1]; p.t[1].out_sh = k_cache->stride[2];
  p.t[2].out_sb = v_cache->stride[0]; p.t[2].out_ss = v_cache->stride[1]; p.t[2].out_sh = v_cache->stride[2];
  p.hq = (int32_t)hq;
  p.hk = (int32_t)hk;
  p.heads = p.hq + 2 * p.hk;
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
  if (!opts->workspace || (reinterpret_cast<uintptr_t>(opts->workspace) % kAlign) != 0 ||
      opts->workspace_bytes < FA_KVCACHE_APPEND_WORKSPACE_BYTES)
    return FA_ERR_WORKSPACE;
  if ((rc = check_device()) != FA_OK) return rc;
  p.ws = static_cast<WsHeader*>(opts->workspace);
  return launch_rope<true>(p, (int)d, k_new->dtype == FA_DTYPE_F16, interleaved != 0, opts, "mfa.kvcache_append");
}

}  // extern "C"
