// chunk_logit.cuh -- the soft-cap of the chunk attention kernels' logits.
#pragma once

#include "chunk.h"
#include "fa_device.cuh"

namespace mfa {

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Soft-caps above this one are far from most logits, and what 1 + e^(2 y) rounds
// off near y = 0 would grow with them: there the logit is scale x (tanh y) / y by
// the power series (cut after y^8: 2e-8 at |y| = 1/4).
constexpr float kPlainSoftcap = 128.f;
__device__ __forceinline__ float wide_softcap(float x, float k, float c1, const ChunkParams& p) {
  const float y = x * p.scale * p.inv_softcap, y2 = y * y;
  const float series = fmaf(y2, fmaf(y2, fmaf(y2, fmaf(y2, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
  const float far = fmaf(-2.f * c1, fast_rcp(1.f + fast_exp2(x * k)), c1);
  return fabsf(y) > 0.25f ? far : x * p.scale_log2 * series;
}

}  // namespace mfa
