// chunk_device.cuh -- device helpers that the chunk attention kernels share: the soft-cap
// of the logits, packed arithmetic, TMEM loads, time-outs.
#pragma once

#include "chunk.h"
#include "f32x2.cuh"
#include "fa_device.cuh"
#include "tc_sm103.cuh"

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

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Waits for this thread's TMEM loads; the registers pass through, so that no use
// of theirs moves before the wait.
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void fail(const ChunkParams& p, volatile int* abort_flag, uint32_t where) {
  if (!*abort_flag) {
    *abort_flag = 1;
    chunk_error(p, FA_ERR_DEVICE_TIMEOUT, where);
  }
}

// Adds to the bytes a barrier's current phase waits for, without an arrival.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(bytes)
               : "memory");
}

// The dynamic shared memory, from its first 1024-byte boundary.
__device__ __forceinline__ unsigned char* smem_base() {
  extern __shared__ unsigned char smem_raw[];
  return reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}

// No planner: the piece of CTA i (count -1: the sequence has no such tile), and the check of its lengths.
__device__ __forceinline__ ChunkPiece q8_own_piece(const ChunkParams& p, int i) {
  const int n_rt = (p.Sq + p.rt_tokens - 1) / p.rt_tokens;
  ChunkPiece w;
  w.hg = i % p.n_hg;
  w.rt = i / p.n_hg % n_rt;
  w.b = i / p.n_hg / n_rt;
  w.kt0 = 0;
  w.count = -1;
  w.slot = -1;
  w.pad[0] = w.pad[1] = 0;
  int4 q = make_int4(0, 0, 0, 0);
  if (!chunk_seq(p, w.b, q)) {
    if (w.rt == 0 && w.hg == 0) chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)w.b);
  } else if (w.rt * p.rt_tokens < q.y) {
    const SinkTiles t = row_tile_sinks(p, q, w.rt);
    w.kt0 = t.kt0;
    w.count = t.count;
  }
  return w;
}

}  // namespace mfa
