// chunk_sm103.cu -- the attention kernel of fa_fwd_chunk on the 5th-generation
// tensor cores of sm_103a (tcgen05 + TMEM + TMA), over a paged KV cache.
//
// Tiled online-softmax attention: per 128-row query tile and 128-key tile,
// S = Q K^T into TMEM, P = 2^(x - ref) packed to the input type back into TMEM,
// O += P V; `ref` follows the row maximum (raised only when it is outgrown by
// more than 2^8, so O is rarely rescaled), the row sums are fp32, and a row that
// keeps no key ends with sum 0: O = 0, LSE = -inf.
//
// Against the contiguous prefill kernel three things differ:
//  - a tile's rows are (token, q-head) pairs of one K/V head (chunk.h), fetched
//    as one TMA box {64 columns, gp heads, tokens}: a single token still fills
//    gp rows, and a K/V tile is read once for the whole group;
//  - K and V tiles are gathered from pages: a box of box_rows rows (the largest
//    power of two that divides the page size, at most 128) per copy, the copies
//    of a tile issued by the lanes of one warp, which look up their own pages.
//    Rows past the sequence's end are not copied where they fill a box; the
//    ones of V that the last 16-key MMA step still reads are zeroed (a page's
//    unused rows may hold anything, and 0 times NaN is NaN), and the steps past
//    them are not issued;
//  - work comes as pieces from the planner's list (chunk.cu), taken in rounds of
//    one per CTA, longest first; a piece of a split unit leaves its normalised
//    rows and log-sum-exp in fp32 for the join.
//
// Warp roles (12 warps; 8 at d = 64, two CTAs per SM): 0 K producer, 1 QK
// issuer and Q producer, 2 V producer, 3 PV issuer, 4.. one or two softmax
// warpgroups, which at d = 128 take alternate key tiles of a piece and hand the
// row references from tile to tile through shared memory.  A warp none of whose
// rows exists keeps step on the barriers and computes nothing.
//
// Every mbarrier wait is bounded (1 s); on a time-out the kernel records
// FA_ERR_DEVICE_TIMEOUT, every role stops, issued copies and MMAs are drained and
// TMEM is released before the CTA exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "chunk.h"
#include "fa_device.cuh"
#include "host_util.h"
#include "tc_sm103.cuh"

namespace mfa {

namespace {

// Register split: d = 128 launches 384 threads at 168 registers, of which the
// producers and issuers keep 72 and the softmax warpgroups take 216; d = 64
// 256 threads at 128, split 40 / 216.
template <int D>
struct CCfg {
  static constexpr int NW = D == 64 ? 1 : 2;  // softmax warpgroups
  static constexpr int kThreads = 128 + 128 * NW;
  static constexpr int kCtas = D == 64 ? 2 : 1;  // per SM
  static constexpr int kLaunchRegs = D == 64 ? 128 : 168;
  static constexpr int kIssueRegs = D == 64 ? 40 : 72;
  static constexpr int kSoftmaxRegs = 216;
  static_assert(128 * kIssueRegs + 128 * NW * kSoftmaxRegs <= kThreads * kLaunchRegs,
                "the register split must fit the block's launch allocation");
  static constexpr uint32_t kCols = NW == 2 ? 512 : 256;  // TMEM: S and P buffers, O
  static constexpr uint32_t kSCol = 0;
  static constexpr uint32_t kPCol = 128 * NW;
  static constexpr uint32_t kOCol = kPCol + 64 * NW;
  static constexpr int NQ = D == 128 ? 1 : 2;
  static constexpr int NSK = D == 128 ? 3 : 2;
  static constexpr int NSV = 2;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = NQ * kTileBytes;
  static constexpr int kVOff = kKOff + NSK * kTileBytes;
  static constexpr int kAuxOff = kVOff + NSV * kTileBytes;  // barriers and flags
  static constexpr int kRefOff = kAuxOff + 512;             // row references [2][128]
  static constexpr int kSumOff = kRefOff + 2 * 128 * 4;     // row sums [2][128]
  static constexpr int kStageOff = kSumOff + 2 * 128 * 4;   // output staging, 2 KB per softmax warp
  static constexpr int kSmem = kStageOff + 4 * NW * 2048 + 1024;
  static_assert(kSmem <= (kCtas == 1 ? 227 * 1024 : 113 * 1024), "shared memory budget");
  static_assert(kOCol + D <= kCols, "TMEM budget");
};

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

// Packed fp32 pair arithmetic.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float row_max(const float2 (&x)[64]) {
  float m[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) m[k] = fmaxf(x[k].x, x[k].y);
#pragma unroll
  for (int i = 8; i < 64; ++i) m[i & 7] = max3f(m[i & 7], x[i].x, x[i].y);
  return fmaxf(max3f(m[0], m[1], m[2]), max3f(m[3], m[4], max3f(m[5], m[6], m[7])));
}

__device__ __forceinline__ void chunk_error(const ChunkParams& p, uint32_t code, uint32_t info) {
  if (atomicCAS(&p.ws->error, 0u, code) == 0u) atomicExch(&p.ws->error_info, info);
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

// The piece this CTA takes in round r: rounds of one piece per CTA, every other
// one in reverse CTA order, so that the CTA with a round's longest piece gets
// the next one's shortest.  At or past n: none, nor in any later round.
__device__ __forceinline__ int round_piece(int r) {
  const int c = (r & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
  return r * (int)gridDim.x + c;
}
__device__ __forceinline__ ChunkPiece piece_at(const ChunkParams& p, int i) {
  const int4* src = reinterpret_cast<const int4*>(p.pieces + i);
  const int4 a = src[0], b = src[1];
  ChunkPiece w;
  w.b = a.x; w.rt = a.y; w.hg = a.z; w.kt0 = a.w;
  w.count = b.x; w.slot = b.y; w.fl = b.z; w.fh = b.w;
  return w;
}
// Next round at or after r whose piece has key tiles, or -1.
__device__ __forceinline__ int next_busy(const ChunkParams& p, int n, int r, ChunkPiece& w) {
  for (;; ++r) {
    const int i = round_piece(r);
    if (i >= n) return -1;
    w = piece_at(p, i);
    if (w.count > 0) return r;
  }
}

// GEN: soft-cap and / or ALiBi (the plain logits fold the scale into the exponent).
template <int D, bool GEN, bool F16>
__global__ void __launch_bounds__(CCfg<D>::kThreads, CCfg<D>::kCtas)
    chunk_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tmq,
                 const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using C = CCfg<D>;
  constexpr int NSK = C::NSK, NSV = C::NSV, NQ = C::NQ, NW = C::NW;
  constexpr uint32_t kSCol = C::kSCol, kPCol = C::kPCol, kOCol = C::kOCol;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kAuxOff);
  uint64_t* q_full = bars;           // [2] Q buffer loaded
  uint64_t* q_empty = q_full + 2;    // [2] QKs reading a Q buffer done
  uint64_t* k_full = q_empty + 2;    // [NSK]
  uint64_t* k_empty = k_full + NSK;  // [NSK]
  uint64_t* v_full = k_empty + NSK;  // [NSV]
  uint64_t* v_empty = v_full + NSV;  // [NSV]
  uint64_t* v_tail = v_empty + NSV;  // [1] copies of a V tile whose end is zeroed
  uint64_t* s_full = v_tail + 1;     // [2] S buffer written by QK
  uint64_t* s_free = s_full + 2;     // [2] S buffer read by the softmax (128 arrivals)
  uint64_t* p_full = s_free + 2;     // [2] P buffer written, O rescaled (128 arrivals)
  uint64_t* p_free = p_full + 2;     // [2] PV reading a P buffer done
  uint64_t* o_full = p_free + 2;     // [1] last PV of a piece done
  uint64_t* drained = o_full + 1;    // [2] all MMAs of an issuer done (teardown)
  uint64_t* sumx = drained + 2;      // [1] row sums of both warpgroups posted (256 arrivals)
  uint64_t* refb = sumx + 1;         // [2 tile parity] row references posted (128 arrivals)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(refb + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      tc::mbar_init(q_full + k, 1);
      tc::mbar_init(q_empty + k, 1);
      tc::mbar_init(s_full + k, 1);
      tc::mbar_init(s_free + k, 128);
      tc::mbar_init(p_full + k, 128);
      tc::mbar_init(p_free + k, 1);
      tc::mbar_init(drained + k, 1);
      tc::mbar_init(refb + k, 128);
    }
    for (int s = 0; s < NSK; ++s) {
      tc::mbar_init(k_full + s, 1);
      tc::mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < NSV; ++s) {
      tc::mbar_init(v_full + s, 1);
      tc::mbar_init(v_empty + s, 1);
    }
    tc::mbar_init(v_tail, 1);
    tc::mbar_init(sumx, 256);
    tc::mbar_init(o_full, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const int n_pieces = p.counts->n_pieces;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers
    // K (warp 0) and V (warp 2) tiles of every piece, in order, through their
    // rings.  Box r of a tile (its rows r * box_rows ..) is sent by lane r % 32.
    const bool is_k = (warp == 0);
    const CUtensorMap* map = is_k ? &tmk : &tmv;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    unsigned char* ring = smem + (is_k ? C::kKOff : C::kVOff);
    const int NS = is_k ? NSK : NSV;
    const int br = p.box_rows;
    const uint32_t box_bytes = (uint32_t)br * D * 2;
    // test only: the first key tile is never sent (FA_DEBUG_WITHHOLD)
    const bool withhold = is_k && (p.debug_flags & FA_DEBUG_WITHHOLD);
    if (lane == 0) tc::tma_prefetch_desc(map);
    int j = 0, tails = 0;
    bool ok = true;
    ChunkPiece w;
    for (int r = next_busy(p, n_pieces, 0, w); ok && r >= 0; r = next_busy(p, n_pieces, r + 1, w)) {
      const int kv = p.kv_len[w.b];
      const int head = w.hg * p.gp / p.G;
      const int32_t* table = p.block_table ? p.block_table + (int64_t)w.b * p.bt_stride : nullptr;
      for (int i = 0; i < w.count; ++i, ++j) {
        if (withhold && j == 0) continue;
        const int j0 = (w.kt0 + i) * kKeysPerTile;
        const int rows = min(kKeysPerTile, kv - j0);
        const int nb = (rows + br - 1) / br;
        const int s = j % NS;
        // this lane's page, read before the wait
        auto page_of = [&](int box, int& row) {
          const int key = j0 + box * br, pi = fast_div(key, p.div_page);
          row = key - pi * p.page_size;
          return table ? table[pi] : w.b;
        };
        int row = 0, page = -1;
        if (lane < nb) page = page_of(lane, row);
        bool go = true;
        if (lane == 0 && j >= NS) go = tc::mbar_wait(empty + s, ((j / NS) - 1) & 1, abort_flag);
        go = __shfl_sync(0xffffffffu, go, 0);
        if (!go) {
          if (lane == 0) fail(p, abort_flag, is_k ? 1 : 7);
          ok = false;
          break;
        }
        const bool tail = !is_k && rows < kKeysPerTile;
        uint64_t* bar = tail ? v_tail : full + s;
        for (int b0 = 0; b0 < nb; b0 += 32) {
          if (b0 && b0 + lane < nb) page = page_of(b0 + lane, row);
          const bool mine = b0 + lane < nb;
          const bool good = mine && page >= 0 && page < p.num_pages;
          if (mine && !good) chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)page);
          const int n = __popc(__ballot_sync(0xffffffffu, good));
          if (lane == 0) {
            // the barrier's one arrival comes with the last group of boxes
            if (b0 + 32 < nb) mbar_expect_tx(bar, n * box_bytes);
            else tc::mbar_arrive_expect_tx(bar, n * box_bytes);
          }
          __syncwarp();
          if (good) {
            unsigned char* dst = ring + s * C::kTileBytes + (b0 + lane) * br * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tc::tma_load_4d(dst + c * 16384, map, bar, c * 64, head, row, page);
          }
          __syncwarp();
        }
        if (tail) {
          // rows past the last key in its 16-key step: zero once the copies have landed
          if (!tc::mbar_wait_drain(v_tail, tails & 1, 1000000000ull)) {
            if (lane == 0) fail(p, abort_flag, 8);
            ok = false;
            break;
          }
          ++tails;
          const int end = (rows + 15) & ~15;
          for (int e = lane; e < (end - rows) * (D / 8); e += 32) {
            const int rr = rows + e / (D / 8), ch = e % (D / 8);
            *reinterpret_cast<uint4*>(ring + s * C::kTileBytes + (ch >> 3) * 16384 + rr * 128 + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(full + s);
        }
      }
    }
    if (lane == 0 && *abort_flag) {
      // let the copies already issued land before the CTA can exit
      const int first = j > NS ? j - NS : 0;
      for (int jj = first; jj < j; ++jj)
        if (!(withhold && jj == 0)) tc::mbar_wait_drain(full + jj % NS, (jj / NS) & 1, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK issuer
    // S[g % NW] = Q K_g^T for the g-th tile of this CTA, as soon as the softmax
    // has read that S buffer NW tiles back; and Q: with two buffers the next
    // piece's while the current one runs, with one once its QKs are done.
    if (lane == 0) {
      constexpr uint32_t idS = tc::idesc_bf16_f32(128, 128, false, false, F16);
      const uint32_t sQ = tc::smem_u32(smem + C::kQOff);
      const uint32_t sK = tc::smem_u32(smem + C::kKOff);
      const uint32_t q_bytes = (uint32_t)(p.rt_tokens * p.gp) * D * 2;
      tc::tma_prefetch_desc(&tmq);
      int nq = 0;  // Q copies issued; copy l goes to buffer l % NQ
      auto load_q = [&](const ChunkPiece& w, int qb) {
        ++nq;
        const int q_row0 = p.cu_q ? p.cu_q[w.b] : 0;
        const int q_b = p.cu_q ? 0 : w.b;
        unsigned char* dst = smem + C::kQOff + qb * C::kTileBytes;
        tc::mbar_arrive_expect_tx(q_full + qb, q_bytes);
        for (int c = 0; c < D / 64; ++c)
          tc::tma_load_4d(dst + c * 16384, &tmq, q_full + qb, c * 64, w.hg * p.gp, q_row0 + w.rt * p.rt_tokens, q_b);
      };
      bool ok = true;
      int g = 0, kk = 0;  // tiles and busy pieces so far
      ChunkPiece w, wn;
      int u = next_busy(p, n_pieces, 0, w);
      if (u >= 0) load_q(w, 0);
      for (; ok && u >= 0; ++kk) {
        const int qb = kk % NQ;
        const int un = next_busy(p, n_pieces, u + 1, wn);
        if (!tc::mbar_wait(q_full + qb, (kk / NQ) & 1, abort_flag)) { ok = false; break; }
        for (int i = 0; i < w.count; ++i, ++g) {
          const int s = g % NSK, sb = g % NW;
          if (!tc::mbar_wait(k_full + s, (g / NSK) & 1, abort_flag)) { ok = false; break; }
          if (g >= NW && !tc::mbar_wait(s_free + sb, ((g - NW) / NW) & 1, abort_flag)) { ok = false; break; }
          tc::fence_after_sync();
          const uint32_t qa = sQ + qb * C::kTileBytes, ka = sK + s * C::kTileBytes;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks >> 2) * 16384 + (ks & 3) * 32;
            tc::mma_ss(tbase + kSCol + sb * 128, tc::sdesc_sw128(qa + o, 16, 1024),
                       tc::sdesc_sw128(ka + o, 16, 1024), idS, ks > 0 ? 1u : 0u);
          }
          tc::mma_commit(s_full + sb);
          tc::mma_commit(k_empty + s);
          if (NQ == 2 && i == 0 && un >= 0) {
            // next piece's Q into the other buffer, last read by piece kk - 1
            if (kk >= 1 && !tc::mbar_wait(q_empty + (qb ^ 1), ((kk - 1) >> 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            load_q(wn, qb ^ 1);
          }
        }
        if (!ok) break;
        tc::mma_commit(q_empty + qb);
        if (NQ == 1 && un >= 0) {
          if (!tc::mbar_wait(q_empty, kk & 1, abort_flag)) {
            ok = false;
            break;
          }
          load_q(wn, 0);
        }
        u = un;
        w = wn;
      }
      if (!ok) fail(p, abort_flag, 2);
      tc::mma_commit(drained);
      tc::mbar_wait_drain(drained, 0, 200000000ull);
      if (*abort_flag) {
        for (int l = nq > NQ ? nq - NQ : 0; l < nq; ++l)
          tc::mbar_wait_drain(q_full + (l % NQ), (l / NQ) & 1, 100000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ PV issuer
    // O (+)= P[g % NW] V_g once the softmax of tile g has written P (and
    // rescaled O), over the 16-key steps that hold keys.
    if (lane == 0) {
      constexpr uint32_t idO = tc::idesc_bf16_f32(128, D, false, true, F16);
      const uint32_t sV = tc::smem_u32(smem + C::kVOff);
      bool ok = true;
      int g = 0;
      ChunkPiece w;
      for (int r = next_busy(p, n_pieces, 0, w); ok && r >= 0; r = next_busy(p, n_pieces, r + 1, w)) {
        const int kv = p.kv_len[w.b];
        for (int i = 0; i < w.count; ++i, ++g) {
          const int s = g % NSV, pb = g % NW;
          const int steps = min(8, (kv - (w.kt0 + i) * kKeysPerTile + 15) / 16);
          if (!tc::mbar_wait(p_full + pb, (g / NW) & 1, abort_flag) ||
              !tc::mbar_wait(v_full + s, (g / NSV) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t va = sV + s * C::kTileBytes;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            if (ks < steps)
              tc::mma_ts(tbase + kOCol, tbase + kPCol + pb * 64 + ks * 8,
                         tc::sdesc_sw128(va + ks * 2048, 16384, 1024), idO, (i > 0 || ks > 0) ? 1u : 0u);
          tc::mma_commit(p_free + pb);
          tc::mma_commit(v_empty + s);
          if (i == w.count - 1) tc::mma_commit(o_full);
        }
      }
      if (!ok) fail(p, abort_flag, 3);
      tc::mma_commit(drained + 1);
      tc::mbar_wait_drain(drained + 1, 0, 200000000ull);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int w = NW == 2 ? (warp - 4) >> 2 : 0;
    const int wq = warp & 3;  // TMEM lane quarter this warp may access
    const int row = 32 * wq + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(32 * wq) << 16);
    float* refv = reinterpret_cast<float*>(smem + C::kRefOff);  // [2 tile parity][128]
    float* rsum = reinterpret_cast<float*>(smem + C::kSumOff);  // [2 warpgroups][128]
    constexpr int kHalfD = D / NW;  // O columns each warpgroup stores
    const int tok = fast_div(row, p.div_gp), hd = row - tok * p.gp;  // this row's token and head in the tile
    const bool in_tile = tok < p.rt_tokens;
    bool ok = true;
    int g = 0, kk = 0;  // tiles and busy pieces so far
    for (int r = 0; ok; ++r) {
      const int pi = round_piece(r);
      if (pi >= n_pieces) break;
      const ChunkPiece un = piece_at(p, pi);
      const int b = un.b;
      const int q_len = chunk_qlen(p, b), kv_len = p.kv_len[b];
      const int off = kv_len - q_len;
      const int i = un.rt * p.rt_tokens + tok;
      const bool exists = in_tile && i < q_len;
      const int64_t qbase = p.cu_q ? (int64_t)p.cu_q[b] : 0, ob = p.cu_q ? 0 : b;
      uint16_t* obase = p.o + ob * p.o_sb + (int64_t)un.hg * p.gp * p.o_sh;
      float* lptr = p.lse + ob * p.lse_sb + (int64_t)(un.hg * p.gp + hd) * p.lse_sh + (qbase + i) * p.lse_ss;
      if (un.count == 0) {
        if (w == 0 && exists) {
          uint16_t* optr = obase + (qbase + i) * p.o_ss + (int64_t)hd * p.o_sh;
#pragma unroll
          for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(optr + c) = make_uint4(0, 0, 0, 0);
          *lptr = -INFINITY;
        }
        continue;
      }
      int jlo_r, jhi_r;
      chunk_row_keys(p, i, off, kv_len, p.prefix ? p.prefix[b] : 0, jlo_r, jhi_r);
      if (!exists) { jlo_r = 1; jhi_r = 0; }
      const bool active = __any_sync(0xffffffffu, exists);
      const float alibi_l2 = (GEN && p.alibi && exists) ? __ldg(p.alibi + un.hg * p.gp + hd) * kLog2e : 0.f;
      float m_ref = -INFINITY;  // reference after the last tile seen
      float r_own = -INFINITY;  // reference this warpgroup's row sum is against
      float l = 0.f;
      const int it0 = (NW == 1 || (g & 1) == w) ? 0 : 1;
      for (int it = it0; it < un.count; it += NW) {
        const int gt = g + it;
        const int par = w;  // == gt % NW
        const int j0 = (un.kt0 + it) * kKeysPerTile;
        const bool part = it < un.fl || it > un.fh;
        if (!tc::mbar_wait(s_full + par, (gt / NW) & 1, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        float2 x[64];
        float mx = -INFINITY;
        if (active) {
          uint32_t t[4][32];
          const uint32_t sa = lane_base + kSCol + par * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld32(sa + c * 32, t[c]);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[c * 16 + e] = make_float2(__uint_as_float(t[c][2 * e]), __uint_as_float(t[c][2 * e + 1]));
        }
        tc::fence_before_sync();
        tc::mbar_arrive_relaxed(s_free + par);  // the QK NW tiles on may overwrite this S buffer
        if (active) {
          if constexpr (GEN) {
            // logits in log2 units: soft-cap or scale, then the distance penalty
            if (p.softcap > 0.f) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                x[e] = make_float2(softcap_log2(x[e].x * p.scale, p.softcap, p.inv_softcap),
                                   softcap_log2(x[e].y * p.scale, p.softcap, p.inv_softcap));
            } else {
#pragma unroll
              for (int e = 0; e < 64; ++e) x[e] = make_float2(x[e].x * p.scale_log2, x[e].y * p.scale_log2);
            }
            if (p.alibi) {
              const float dist = (float)(i + off - j0);  // to the tile's first key
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                x[e].x -= alibi_l2 * fabsf(dist - (float)(2 * e));
                x[e].y -= alibi_l2 * fabsf(dist - (float)(2 * e + 1));
              }
            }
          }
          if (part) {
            // the row keeps keys clo .. clo + span of the tile; a row that keeps
            // none gets a start no key reaches.  (The scale is positive, so
            // a raw -inf stays -inf through it.)
            const bool none = jhi_r < jlo_r;
            const int clo = none ? (1 << 20) : jlo_r - j0;
            const unsigned span = none ? 0u : (unsigned)(jhi_r - jlo_r);
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              x[e].x = (unsigned)(2 * e - clo) <= span ? x[e].x : -INFINITY;
              x[e].y = (unsigned)(2 * e + 1 - clo) <= span ? x[e].y : -INFINITY;
            }
          }
          mx = row_max(x);
          if constexpr (!GEN) mx *= p.scale_log2;
        }
        // the reference after tile gt - 1
        if (NW == 2 && gt >= 1 && !tc::mbar_wait(refb + (par ^ 1), ((gt - 1) >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        const float m_prev = (it == 0) ? -INFINITY : (NW == 2 ? refv[(par ^ 1) * 128 + row] : m_ref);
        const bool upd = mx > m_prev + 8.f;  // raise the reference only when outgrown by 2^8
        m_ref = upd ? mx : m_prev;
        if (NW == 2) {
          refv[par * 128 + row] = m_ref;
          tc::mbar_arrive(refb + par);
        }
        if (it != 0 && __any_sync(0xffffffffu, upd && m_prev != -INFINITY)) {
          // O holds the PV of tile gt - 1 (against m_prev) once that PV is done
          if (!tc::mbar_wait(p_free + (gt - 1) % NW, ((gt - 1) / NW) & 1, abort_flag)) { ok = false; break; }
          tc::fence_after_sync();
          const float f = (upd && m_prev != -INFINITY) ? fast_exp2(m_prev - m_ref) : 1.f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t t[32];
            const uint32_t a = lane_base + kOCol + c * 32;
            tc::tmem_ld32(a, t);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) t[e] = __float_as_uint(__uint_as_float(t[e]) * f);
            tc::tmem_st32(a, t);
          }
        }
        if (r_own != m_ref) {
          l = (r_own == -INFINITY) ? 0.f : l * fast_exp2(r_own - m_ref);
          r_own = m_ref;
        }
        uint32_t pk[4][16];
        if (active) {
          const float eref = (m_ref == -INFINITY) ? 0.f : m_ref;
          const float2 ner = make_float2(-eref, -eref);
          float2 acc[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] = make_float2(0.f, 0.f);
          const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 v = GEN ? add2(x[c * 16 + e], ner) : fma2(x[c * 16 + e], sl2, ner);
              const float2 pe = make_float2(fast_exp2(v.x), fast_exp2(v.y));
              acc[e & 3] = add2(acc[e & 3], pe);
              pk[c][e] = pack2<F16>(pe.x, pe.y);
            }
          acc[0] = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
          l += acc[0].x + acc[0].y;
        }
        // this P buffer is free once the PV NW tiles back is done
        if (gt >= NW && !tc::mbar_wait(p_free + par, ((gt - NW) / NW) & 1, abort_flag)) { ok = false; break; }
        if (active) {
          const uint32_t pa = lane_base + kPCol + par * 64;
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_st16(pa + c * 16, pk[c]);
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        tc::mbar_arrive_relaxed(p_full + par);
      }
      if (!ok) break;
      // ---- epilogue: both warpgroups' row sums against the final reference
      const int gl = g + un.count - 1;  // the piece's last tile
      g += un.count;
      if (NW == 2 && (gl & 1) != w) {
        if (!tc::mbar_wait(refb + (gl & 1), (gl >> 1) & 1, abort_flag)) { ok = false; break; }
        m_ref = refv[(gl & 1) * 128 + row];
      }
      // O is read out of TMEM before this warpgroup's row sum is posted: the
      // next piece's first PV overwrites O, and its P comes from a warpgroup
      // that has passed the row-sum barrier (with one warpgroup: from this
      // one, after the read)
      if (!tc::mbar_wait(o_full, kk & 1, abort_flag)) { ok = false; break; }
      tc::fence_after_sync();
      uint32_t ro[kHalfD / 32][32];
#pragma unroll
      for (int c = 0; c < kHalfD / 32; ++c) tc::tmem_ld32(lane_base + kOCol + w * kHalfD + c * 32, ro[c]);
      float lt;
      if constexpr (NW == 2) {
        rsum[w * 128 + row] = (r_own == m_ref || r_own == -INFINITY) ? l : l * fast_exp2(r_own - m_ref);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        tc::mbar_arrive(sumx);
        if (!tc::mbar_wait(sumx, kk & 1, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        lt = rsum[row] + rsum[128 + row];
      } else {
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        lt = l;
      }
      const bool empty = !(lt > 0.f);
      const float inv = empty ? 0.f : 1.f / lt;
      const float lse2 = empty ? -INFINITY : m_ref + __log2f(lt);
      if (un.slot >= 0) {
        if (exists) {
          float* dst = p.part_o + ((int64_t)un.slot * kChunkRows + row) * D + w * kHalfD;
#pragma unroll
          for (int c = 0; c < kHalfD / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + c * 32 + e) =
                  make_float4(__uint_as_float(ro[c][e]) * inv, __uint_as_float(ro[c][e + 1]) * inv,
                              __uint_as_float(ro[c][e + 2]) * inv, __uint_as_float(ro[c][e + 3]) * inv);
          if (w == 0) p.part_lse[(int64_t)un.slot * kChunkRows + row] = lse2;
        }
      } else if (active) {
        // through a warp-private staging tile: a thread packs its own row, then
        // each store instruction writes 64 contiguous bytes of 8 rows
        uint4* stg = reinterpret_cast<uint4*>(smem + C::kStageOff + (warp - 4) * 2048);  // [32 rows][4]
        uint16_t* orow[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = 32 * wq + 8 * k + (lane >> 2), t = fast_div(rr, p.div_gp);
          const int ti = un.rt * p.rt_tokens + t;
          orow[k] = (t < p.rt_tokens && ti < q_len)
                        ? obase + (qbase + ti) * p.o_ss + (int64_t)(rr - t * p.gp) * p.o_sh + w * kHalfD + 8 * (lane & 3)
                        : nullptr;
        }
#pragma unroll
        for (int c = 0; c < kHalfD / 32; ++c) {
          const uint32_t* t = ro[c];
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            uint4 o4;
            o4.x = pack2<F16>(__uint_as_float(t[8 * v4 + 0]) * inv, __uint_as_float(t[8 * v4 + 1]) * inv);
            o4.y = pack2<F16>(__uint_as_float(t[8 * v4 + 2]) * inv, __uint_as_float(t[8 * v4 + 3]) * inv);
            o4.z = pack2<F16>(__uint_as_float(t[8 * v4 + 4]) * inv, __uint_as_float(t[8 * v4 + 5]) * inv);
            o4.w = pack2<F16>(__uint_as_float(t[8 * v4 + 6]) * inv, __uint_as_float(t[8 * v4 + 7]) * inv);
            stg[lane * 4 + (v4 ^ ((lane >> 1) & 3))] = o4;
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = 8 * k + (lane >> 2), q = lane & 3;
            const uint4 o4 = stg[rr * 4 + (q ^ ((rr >> 1) & 3))];
            if (orow[k]) *reinterpret_cast<uint4*>(orow[k] + c * 32) = o4;
          }
          __syncwarp();
        }
        if (w == 0 && exists) *lptr = lse2 * kLn2;
      }
      ++kk;
    }
    if (!ok) fail(p, abort_flag, 4 + w);
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tbase, C::kCols);
}

// Tensor map of 2-byte elements {d, heads, rows, outer} with a box of {64,
// box_heads, box_rows, 1} and 128-byte swizzle; strides in elements.  An
// extent of 1 (or 0) gets a harmless stride.
bool encode_map(CUtensorMap* m, const void* base, int d, int heads, int64_t rows, int64_t outer, int64_t s_h,
                int64_t s_row, int64_t s_outer, int box_heads, int box_rows, bool f16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  rows = std::max<int64_t>(rows, 1);
  outer = std::max<int64_t>(outer, 1);
  if (heads == 1 || s_h == 0) s_h = d;
  if (rows == 1 || s_row == 0) s_row = s_h;
  if (outer == 1 || s_outer == 0) s_outer = s_row;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[3] = {(cuuint64_t)s_h * 2, (cuuint64_t)s_row * 2, (cuuint64_t)s_outer * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int D, bool GEN, bool F16>
cudaError_t launch_v(const ChunkParams& p, cudaStream_t st) {
  using C = CCfg<D>;
  // setmaxnreg.inc would wait forever if the block were launched with fewer
  // registers than the split assumes: launch only when the build matches.
  static std::atomic<int> launch_regs{-1};
  int regs = launch_regs.load(std::memory_order_relaxed);
  cudaError_t e;
  if (regs < 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, chunk_kernel<D, GEN, F16>)) != cudaSuccess) return e;
    regs = fa.numRegs;
    launch_regs.store(regs, std::memory_order_relaxed);
  }
  if (regs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  if ((e = ensure_smem_attr<chunk_kernel<D, GEN, F16>>(C::kSmem)) != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  const bool packed = p.cu_q != nullptr;
  const int heads_kv = p.Hq / p.G;
  if (!encode_map(&mq, p.q, D, p.Hq, packed ? p.tot_q : p.Sq, packed ? 1 : p.n_seq, p.q_sh, p.q_ss, p.q_sb, p.gp,
                  p.rt_tokens, F16) ||
      !encode_map(&mk, p.k, D, heads_kv, p.cache_rows, p.cache_outer, p.k_sh, p.k_ss, p.k_sb, 1, p.box_rows, F16) ||
      !encode_map(&mv, p.v, D, heads_kv, p.cache_rows, p.cache_outer, p.v_sh, p.v_ss, p.v_sb, 1, p.box_rows, F16))
    return cudaErrorInvalidValue;
  chunk_kernel<D, GEN, F16><<<(unsigned)p.grid, C::kThreads, C::kSmem, st>>>(p, mq, mk, mv);
  return cudaGetLastError();
}

template <bool F16>
cudaError_t launch_t(const ChunkParams& p, cudaStream_t st) {
  const bool gen = p.softcap > 0.f || p.alibi;
  if (p.d == 64) return gen ? launch_v<64, true, F16>(p, st) : launch_v<64, false, F16>(p, st);
  return gen ? launch_v<128, true, F16>(p, st) : launch_v<128, false, F16>(p, st);
}

}  // namespace

// The fp16 instantiations build in their own translation unit (chunk_f16.cu
// includes this file with MFA_CHUNK_F16_UNIT defined), in parallel.
#ifndef MFA_CHUNK_F16_UNIT
int chunk_ctas_per_sm(int d) { return d == 64 ? CCfg<64>::kCtas : CCfg<128>::kCtas; }
cudaError_t launch_chunk_attn(const ChunkParams& p, cudaStream_t st) { return launch_t<false>(p, st); }
#else
cudaError_t launch_chunk_attn_f16(const ChunkParams& p, cudaStream_t st) { return launch_t<true>(p, st); }
#endif

}  // namespace mfa
