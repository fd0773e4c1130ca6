// q8_device.cuh -- the 8-bit KV cache: e4m3 values, and per block of tokens of a
// page and per head one scale, a power of two (fp32), for K and V each.
//
// A power of two costs nothing here: a value keeps e4m3's four significant bits
// whatever the scale (only its smallest values differ), reading back is exact in
// 16 bits, and a block whose scale has to grow is rounded again only where its
// values become subnormal.  Scales lie within 2^-40 .. 2^40, so that the
// attention's ratios of them stay well inside fp32.
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "host_util.h"

namespace mfa {

constexpr int kQ8Low = -40, kQ8High = 40;  // exponents of the scales
constexpr int kQ8MinBlock = 16, kQ8MaxBlock = 128;

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The exponent of a scale (what its other bits say is not looked at).
__device__ __forceinline__ int scale_exponent(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 0xff) - 127;
  return min(max(e, kQ8Low), kQ8High);
}

// The smallest exponent with top <= 448 * 2^e in range; top is finite, >= 0.
__device__ __forceinline__ int block_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  return min(max(e, kQ8Low), kQ8High);
}

// The power of two that a row of Q is divided by on its way to fp16: its largest
// finite element comes to 2^7 .. 2^8.
__device__ __forceinline__ int q_exponent(float top) {
  return top > 0.f ? min(max((int)(__float_as_uint(top) >> 23) - 127 - 7, -100), 120) : 0;
}

// Four fp32 values as e4m3 bytes, rounded to nearest even, saturated (NaN stays NaN).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// 0xff in the bytes that are NaN codes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t codes) {
  const uint32_t m = ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return m | (m - (m >> 7));
}

// Two e4m3 bytes (the low half of u) as two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t u) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(u));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t u) {
  const uint32_t h = e4m3x2_to_f16x2(u);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// An 8-bit cache and its scales: [num_pages, page_size, Hkv, d] or [n_seq, cap,
// Hkv, d], and fp32 [num_pages, page_size / block, Hkv] or [n_seq, cap / block,
// Hkv]; the codes' strides are multiples of 16 bytes.  Sets the tokens of a block.
inline int check_q8(const fa_tensor* c, const fa_tensor* s, int64_t* block) {
  if (!c || !s || !c->data || !s->data || c->dtype != FA_DTYPE_E4M3 || c->ndim != 4 || s->dtype != FA_DTYPE_F32 || s->ndim != 3)
    return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (c->shape[i] < 0 || c->stride[i] < 0 || (i < 3 && c->stride[i] % 16 != 0)) return FA_ERR_INVALID_ARG;
  if (c->stride[3] != 1 || !aligned16(c->data) || (reinterpret_cast<uintptr_t>(s->data) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (s->shape[0] != c->shape[0] || s->shape[2] != c->shape[2]) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (s->stride[i] < 0) return FA_ERR_INVALID_ARG;
  const int64_t rows = c->shape[1], n = s->shape[1];
  if (rows == 0 || n < 1 || rows % n != 0) return FA_ERR_INVALID_ARG;
  const int64_t b = rows / n;
  if (b < kQ8MinBlock || b > kQ8MaxBlock || (b & (b - 1)) != 0) return FA_ERR_INVALID_ARG;
  *block = b;
  return FA_OK;
}

// Tensor map of a cache's codes {d, heads, rows, outer} (strides in bytes), box_rows
// rows of a head per copy.  False when the driver rejects it or has no encoder.
inline bool encode_codes(CUtensorMap* m, const uint8_t* base, int d, int heads, int64_t rows, int64_t outer, int64_t s_h,
                         int64_t s_row, int64_t s_outer, int box_rows, CUtensorMapSwizzle swz) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  outer = std::max<int64_t>(outer, 1);
  if (heads == 1) s_h = d;
  if (outer == 1) s_outer = s_row;  // (an extent of 1 gets a harmless stride)
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[3] = {(cuuint64_t)s_h, (cuuint64_t)s_row, (cuuint64_t)s_outer};
  cuuint32_t box[4] = {(cuuint32_t)d, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mfa
