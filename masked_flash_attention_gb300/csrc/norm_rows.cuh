// norm_rows.cuh -- rows of heads normalised by their root mean square, weighted and
// rotated, 16 columns of a head to a lane as pairs of fp32 in register pairs.
#pragma once

#include <cuda_runtime.h>

#include "f32x2.cuh"
#include "rope_common.cuh"

namespace mfa {

enum { kNoWeight = 0, kWeightF32 = 1, kWeight16 = 2 };
// A weight per column of a head.
struct HeadWeight {
  const void* data;
  int32_t kind, wide;  // wide: 16-byte loads of it
};

// Sum over the lanes of a head, in every one of them.
template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Lane c's columns; of kInterleaved's pairs both halves' 4 c .. 4 c + 3 (a warp's
// 16 bytes are then whole sectors).
template <int D, int LAYOUT>
__device__ __forceinline__ Columns lane_columns(int c, int half) {
  if (LAYOUT == kInterleaved) return {8 * c, D / 2 + 8 * c};
  return columns_of<LAYOUT>(c, half);
}

template <bool F16>
__device__ __forceinline__ void load_weight(const HeadWeight& r, Columns at, float (&w)[16]) {
  if (r.wide && r.kind == kWeight16) {
    const uint16_t* src = static_cast<const uint16_t*>(r.data);
    unpack16<F16>(__ldg(reinterpret_cast<const uint4*>(src + at.xa)), __ldg(reinterpret_cast<const uint4*>(src + at.xb)), w);
    return;
  }
  if (r.wide && r.kind == kWeightF32) {
    const float* src = static_cast<const float*>(r.data);
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src + (e < 8 ? at.xa + e : at.xb + e - 8)));
      w[e] = v.x; w[e + 1] = v.y; w[e + 2] = v.z; w[e + 3] = v.w;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int col = e < 8 ? at.xa + e : at.xb + e - 8;
    w[e] = r.kind == kWeightF32 ? __ldg(static_cast<const float*>(r.data) + col)
         : r.kind == kWeight16  ? to_float<F16>(__ldg(static_cast<const uint16_t*>(r.data) + col))
                                  : 1.f;
  }
}

// A lane's part of its warp's turns: pairs lane and lane + 32.
__device__ __forceinline__ void turn_steps(const double* inv_freq, int half, int lane, uint64_t (&u)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) u[k] = lane + 32 * k < half ? turn_step(__ldg(inv_freq + lane + 32 * k)) : 0;
}
// A lane's 16 columns as 8 rotated pairs (a, b), two of each to a register pair:
// column e and the one a half behind, or columns 2 e and 2 e + 1.
struct Pairs {
  float2 a[4], b[4];
};
template <int LAYOUT>
__device__ __forceinline__ Pairs pairs_of(const float (&x)[16]) {
  Pairs y;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    y.a[k] = LAYOUT == kInterleaved ? make_float2(x[4 * k], x[4 * k + 2]) : make_float2(x[2 * k], x[2 * k + 1]);
    y.b[k] = LAYOUT == kInterleaved ? make_float2(x[4 * k + 1], x[4 * k + 3]) : make_float2(x[8 + 2 * k], x[9 + 2 * k]);
  }
  return y;
}
template <int LAYOUT>
__device__ __forceinline__ void columns_from(const Pairs& y, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[LAYOUT == kInterleaved ? 4 * k : 2 * k] = y.a[k].x;
    x[LAYOUT == kInterleaved ? 4 * k + 2 : 2 * k + 1] = y.a[k].y;
    x[LAYOUT == kInterleaved ? 4 * k + 1 : 8 + 2 * k] = y.b[k].x;
    x[LAYOUT == kInterleaved ? 4 * k + 3 : 9 + 2 * k] = y.b[k].y;
  }
}
template <bool F16, int LAYOUT>
__device__ __forceinline__ Pairs unpack_pairs(const uint4& a, const uint4& b) {
  float x[16];
  unpack16<F16>(a, b, x);
  return pairs_of<LAYOUT>(x);
}
template <bool F16, int LAYOUT>
__device__ __forceinline__ void pack_pairs(const Pairs& y, uint4& a, uint4& b) {
  float x[16];
  columns_from<LAYOUT>(y, x);
  pack16<F16>(x, a, b);
}
// Sum of the products of two rows, over the lanes of their head.
template <int kLanes>
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) {
  float2 s = mul2(x.a[0], y.a[0]), t = mul2(x.b[0], y.b[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    s = fma2(x.a[k], y.a[k], s);
    t = fma2(x.b[k], y.b[k], t);
  }
  s = add2(s, t);
  return head_sum<kLanes>(s.x + s.y);
}
__device__ __forceinline__ void scale_by(Pairs& x, float f) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x.a[k] = mul2(x.a[k], both(f));
    x.b[k] = mul2(x.b[k], both(f));
  }
}
__device__ __forceinline__ void multiply(Pairs& x, const Pairs& y) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x.a[k] = mul2(x.a[k], y.a[k]);
    x.b[k] = mul2(x.b[k], y.b[k]);
  }
}

// q's and k's weights, lane c's pairs at [n][0 .. 3][c].
template <int kLanes>
using Weights = float4[2][4][kLanes];
template <bool F16, int LAYOUT, int kLanes>
__device__ __forceinline__ void stage_weights(const HeadWeight& q, const HeadWeight& k, int half, Weights<kLanes>& s_w) {
  const int n = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  if (n < 2) {
    float w[16];
    load_weight<F16>(n ? k : q, lane_columns<16 * kLanes, LAYOUT>(c, half), w);
    const Pairs y = pairs_of<LAYOUT>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) s_w[n][i][c] = make_float4(y.a[i].x, y.a[i].y, y.b[i].x, y.b[i].y);
  }
  __syncthreads();
}
template <int kLanes>
__device__ __forceinline__ Pairs weight_of(const Weights<kLanes>& s_w, int n, int c) {
  Pairs w;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 v = s_w[n][k][c];
    w.a[k] = make_float2(v.x, v.y);
    w.b[k] = make_float2(v.z, v.w);
  }
  return w;
}

// The turns of a lane's pairs.
struct Turns {
  float2 co[4], sn[4];
};
// The first pair of lane c's register pairs k.
template <int D, int LAYOUT>
__device__ __forceinline__ int first_pair(int c, int k) {
  return LAYOUT == kInterleaved ? (k / 2) * (D / 4) + 4 * c + 2 * (k % 2) : 8 * c + 2 * k;
}
// The place of pair i's turn: such that the lanes of a head read different banks, 16 bytes each.
template <int LAYOUT>
__device__ __forceinline__ int turn_place(int i) {
  return LAYOUT == kInterleaved ? i ^ (i >> 4 & 1) << 1 : LAYOUT == kHalf ? i ^ (i >> 4 & 3) << 1 : i;
}
// The turns of position pos, to cs.  (By all the lanes of a warp.)
template <int LAYOUT>
__device__ __forceinline__ void make_turns(int pos, const uint64_t (&u)[2], int half, float mscale, bool inverse, int lane, float2* cs) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane + 32 * k < half) cs[turn_place<LAYOUT>(lane + 32 * k)] = position_turn(pos, u[k], mscale, inverse);
  __syncwarp();
}
// Those of lane c's pairs (of its pairs that are not rotated: anything).
template <int D, int LAYOUT>
__device__ __forceinline__ void load_turns(const float2* cs, int c, Turns& tw) {
  if constexpr (LAYOUT != kHalfOdd) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(cs + turn_place<LAYOUT>(first_pair<D, LAYOUT>(c, k)));
      tw.co[k] = make_float2(v.x, v.z);
      tw.sn[k] = make_float2(v.y, v.w);
    }
  }
}

// rotate16, of pairs and with the turns in registers where lanes do not exchange columns.
template <int D, int LAYOUT>
__device__ __forceinline__ void rotate(Pairs& x, const Turns& tw, const float2* cs, int c, int half, float* row) {
  if constexpr (LAYOUT == kHalfOdd) {
    float y[16];
    columns_from<LAYOUT>(x, y);
    rotate16<LAYOUT>(y, cs, c, half, row);
    x = pairs_of<LAYOUT>(y);
  } else {
    // (kHalf: all eight pairs or none; kInterleaved: so for each four but where half % 4 is not 0)
    constexpr int kSame = LAYOUT == kInterleaved ? 2 : 4;
#pragma unroll
    for (int k0 = 0; k0 < 4; k0 += kSame) {
      const int left = half - first_pair<D, LAYOUT>(c, k0);  // pairs from here on that are rotated
      if (left <= 0) continue;
      Pairs was = x;
#pragma unroll
      for (int k = k0; k < k0 + kSame; ++k) {
        const float2 t = mul2(x.b[k], tw.sn[k]), a = x.a[k];
        x.a[k] = fma2(a, tw.co[k], make_float2(-t.x, -t.y));
        x.b[k] = fma2(a, tw.sn[k], mul2(x.b[k], tw.co[k]));
      }
      if (LAYOUT == kInterleaved && left < 4) {
#pragma unroll
        for (int k = k0; k < k0 + kSame; ++k) {
          if (left <= 2 * (k - k0)) x.a[k].x = was.a[k].x, x.b[k].x = was.b[k].x;
          if (left <= 2 * (k - k0) + 1) x.a[k].y = was.a[k].y, x.b[k].y = was.b[k].y;
        }
      }
    }
  }
}

// A weight's checks: [d], fp32 or of x's type; null is none.
inline int check_weight(const fa_tensor* w, const fa_tensor* x, HeadWeight& r) {
  if (!w) return FA_OK;
  const int64_t d = x->shape[x->ndim - 1];
  const bool f32 = w->dtype == FA_DTYPE_F32;
  if (!w->data || (!f32 && w->dtype != x->dtype) || w->ndim != 1 || w->shape[0] != d || w->stride[0] != 1 ||
      (reinterpret_cast<uintptr_t>(w->data) & (f32 ? 3u : 1u)) != 0)
    return FA_ERR_INVALID_ARG;
  r.data = w->data;
  r.kind = f32 ? kWeightF32 : kWeight16;
  r.wide = (reinterpret_cast<uintptr_t>(w->data) & 15u) == 0;
  return FA_OK;
}

}  // namespace mfa
