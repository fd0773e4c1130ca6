// rope_common.cuh -- shared by the kernels around rotary positions: the angle of
// a position in turns, the sequence of a packed row, 16-bit conversions, and the
// argument checks of their entry points.
#pragma once

#include <climits>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "fa_internal.h"

namespace mfa {

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

// The (cosine, sine) of position pos for the pair whose step is u (turn_step), times mscale.
__device__ __forceinline__ float2 position_turn(int pos, uint64_t u, float mscale, bool inverse) {
  const uint64_t a = (uint64_t)(int64_t)pos * u;
  const float x = (float)(int32_t)(uint32_t)(a >> 32) * 4.656612873077393e-10f;  // [-1, 1) half turns, 2^-31 a step
  float sn, co;
  sincospif(x, &sn, &co);
  return make_float2(co * mscale, (inverse ? -sn : sn) * mscale);
}

enum { kHalf = 0, kInterleaved = 1, kHalfOdd = 2 };
inline int layout_of(bool interleaved, int half) {
  return interleaved || half == 0 ? kInterleaved : (half % 8 == 0 ? kHalf : kHalfOdd);
}

// Sixteen columns of a head in fp32, columns xa .. xa + 7 and xb .. xb + 7 of
// lane c's share (kHalf: the two sides of 8 pairs where those are rotated).
struct Columns {
  int xa, xb;
};
template <int LAYOUT>
__device__ __forceinline__ Columns columns_of(int c, int half) {
  if (LAYOUT == kHalf && 8 * c < half) return {8 * c, half + 8 * c};
  return {16 * c, 16 * c + 8};
}
template <bool F16>
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&x)[16]) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(&a);
  const uint32_t* v = reinterpret_cast<const uint32_t*>(&b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = unpack2<F16>(u[e]), q = unpack2<F16>(v[e]);
    x[2 * e] = p.x; x[2 * e + 1] = p.y;
    x[8 + 2 * e] = q.x; x[9 + 2 * e] = q.y;
  }
}
template <bool F16>
__device__ __forceinline__ void pack16(const float (&x)[16], uint4& a, uint4& b) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&a);
  uint32_t* v = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    u[e] = pack2<F16>(x[2 * e], x[2 * e + 1]);
    v[e] = pack2<F16>(x[8 + 2 * e], x[9 + 2 * e]);
  }
}
// Rotates lane c's columns x of one row by that row's turns cs[0 .. half).
// kHalfOdd: through `row`, shared memory of the row's lanes (all in one warp,
// all here).
template <int LAYOUT>
__device__ __forceinline__ void rotate16(float (&x)[16], const float2* cs, int c, int half, float* row) {
  if constexpr (LAYOUT == kHalf) {
    if (8 * c < half) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = cs[8 * c + e];
        const float a = x[e], b = x[8 + e];
        x[e] = a * w.x - b * w.y;
        x[8 + e] = a * w.y + b * w.x;
      }
    }
  } else if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (8 * c + e < half) {
        const float2 w = cs[8 * c + e];
        const float a = x[2 * e], b = x[2 * e + 1];
        x[2 * e] = a * w.x - b * w.y;
        x[2 * e + 1] = a * w.y + b * w.x;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) row[16 * c + e] = x[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int col = 16 * c + e;
      if (col < 2 * half) {
        const float2 w = cs[col < half ? col : col - half];
        const float m = row[col < half ? col + half : col - half];
        x[e] = col < half ? x[e] * w.x - m * w.y : m * w.y + x[e] * w.x;
      }
    }
    __syncwarp();
  }
}

// Strides of a [B, S, H, d] or [total, H, d] tensor.
inline void strides_of(const fa_tensor* t, int64_t& sb, int64_t& ss, int64_t& sh) {
  if (t->ndim == 3) { sb = 0; ss = t->stride[0]; sh = t->stride[1]; }
  else { sb = t->stride[0]; ss = t->stride[1]; sh = t->stride[2]; }
}

inline bool same_shape(const fa_tensor* a, const fa_tensor* b) {
  if (a->ndim != b->ndim) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i]) return false;
  return true;
}

// A written tensor holds every element once: no stride of 0 along more than
// one element.
inline bool writable(const fa_tensor* t) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] == 0) return false;
  return true;
}

inline int check_freq(const fa_tensor* f, int64_t d, int32_t* half) {
  if (!f->data || f->dtype != FA_DTYPE_F64 || f->ndim != 1 || f->stride[0] != 1 ||
      (reinterpret_cast<uintptr_t>(f->data) & 7u) != 0 || f->shape[0] < 1 || 2 * f->shape[0] > d)
    return FA_ERR_INVALID_ARG;
  *half = (int32_t)f->shape[0];
  return FA_OK;
}

// x and its output: one shape and type, like `like` but for the heads.
inline int check_pair(const fa_tensor* x, const fa_tensor* y, const fa_tensor* like) {
  int rc;
  if ((rc = check_bf16(x, like->ndim)) || (rc = check_bf16(y, like->ndim))) return rc;
  if (x->dtype != like->dtype || y->dtype != like->dtype || !same_shape(x, y) || !writable(y))
    return FA_ERR_INVALID_ARG;
  for (int i = 0; i < like->ndim; ++i)
    if (i != like->ndim - 2 && x->shape[i] != like->shape[i]) return FA_ERR_INVALID_ARG;
  return x->shape[like->ndim - 2] < 1 ? FA_ERR_INVALID_ARG : FA_OK;
}

// Positions of x's rows, int32 [B, S] or [total]; sets positions, pos_sb and pos_ss of p.
template <typename P>
inline int check_positions(const fa_tensor* t, const fa_tensor* x, P& p) {
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

// Rows of q-like tensor x: total, and rows per sequence of its layout.
template <typename P>
inline int check_rows(const fa_tensor* x, P& p) {
  const int64_t B = x->ndim == 4 ? x->shape[0] : 1, S = x->shape[x->ndim - 3];
  if (B > INT32_MAX / 64 || S > INT32_MAX / 64 || (S > 0 && B > INT32_MAX / S)) return FA_ERR_INVALID_ARG;
  p.rows = B * S;
  p.S = (int32_t)(S > 0 ? S : 1);
  return FA_OK;
}

}  // namespace mfa
