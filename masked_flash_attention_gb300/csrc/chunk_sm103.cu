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
//  - a narrow piece, of at most 32 rows (single tokens, a few speculated ones),
//    would leave its exponentials to one warp of four: its rows stand in all
//    four quarters of the tile, warp q takes keys 32 q .. 32 q + 31 of each
//    key tile for them, and the quarters are joined by log-sum-exp at the end;
//  - work comes as pieces from the planner's list (chunk.cu), taken in rounds of
//    one per CTA, longest first; a piece of a split unit leaves its normalised
//    rows and log-sum-exp in fp32 for the join.
//
// Warp roles (12 or 16 warps; 8 at d = 64, two CTAs per SM): 0 K producer, 1 QK
// issuer and Q producer, 2 V producer, 3 PV issuer, 4.. one or two softmax
// warpgroups, which at d = 128 take alternate key tiles of a piece and hand the
// row references from tile to tile through shared memory, 12 and 13 more
// producers.  A warp none of whose rows exists keeps step on the barriers and computes nothing.
//
// Every mbarrier wait is bounded (1 s); on a time-out the kernel records
// FA_ERR_DEVICE_TIMEOUT, every role stops, issued copies and MMAs are drained and
// TMEM is released before the CTA exits.
//
// Measured, this kernel alone after an L2 flush: 2048 tokens over 32768 keys, 32 /
// 8 heads, d = 128, page 64: 677 us, 1574 TFLOP/s (0.83 of the measured matmul
// rate); 64 single tokens over up to 8192 keys, page 16, window 4096, soft-cap:
// 148 us for 805 MB, 5440 GB/s (0.80 of the measured copy rate).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "chunk.h"
#include "chunk_device.cuh"
#include "fa_device.cuh"
#include "host_util.h"
#include "tc_sm103.cuh"

namespace mfa {

namespace {

// NP producer warps per operand.  One warp issues a tile's TMA copies one after
// the other, and at d = 128 a page of 16 rows makes 32 copies per K/V tile: with
// boxes that small and many query rows, two warps of a fourth warpgroup share
// them.  Otherwise one warp is better: more warps cost the others instruction
// issue.  Measured, one and two warps, by separate runs (three: 127, 180): 4 x 512
// tokens over 4096 keys, page 16: 139 and 120 us (page 64: 111 with one); 64
// single tokens over up to 8192 keys, page 16: 164 and 175 us.
// Register split: with one producer warp per operand 384 threads launch at 168
// registers, of which the softmax warpgroups take 216 and the others keep 72;
// with two, 512 threads launch at 128, split 72 / 184; d = 64 launches 256
// threads at 128, split 40 / 216.
template <int D, int NW_, int NP_>
struct CCfg {
  static constexpr int NW = NW_;  // softmax warpgroups
  static constexpr int NP = NP_;
  static constexpr int kThreads = 128 + 128 * NW + (NP > 1 ? 128 : 0);
  static constexpr int kCtas = NW == 1 ? 2 : 1;  // per SM
  static constexpr int kLaunchRegs = (NW == 1 || NP > 1) ? 128 : 168;
  static constexpr int kIssueRegs = NW == 1 ? 40 : 72;
  static constexpr int kSoftmaxRegs = NP > 1 ? 184 : 216;
  static_assert(NP == 1 || (NP == 2 && NW == 2), "the role table has one or two warps per operand");
  static_assert((kThreads - 128 * NW) * kIssueRegs + 128 * NW * kSoftmaxRegs <= kThreads * kLaunchRegs,
                "the register split must fit the block's launch allocation");
  // TMEM.  Two warpgroups: three S buffers, each overwritten by its P, and O;
  // one: S, P and O.
  static constexpr uint32_t kCols = NW == 2 ? 512 : 256;
  static constexpr int NB = NW == 2 ? 3 : 1;            // S / P buffers, 128 columns of S each
  static constexpr uint32_t kPCol = NW == 2 ? 0 : 128;  // P of buffer b: kPCol + 128 b
  static constexpr uint32_t kOCol = NW == 2 ? 384 : 192;
  static constexpr int NQ = D == 128 ? 1 : 2;
  static constexpr int NSK = D == 128 ? 3 : 2 * NW;
  static constexpr int NSV = D == 128 ? 2 : 2 * NW;
  static constexpr int kTileBytes = 128 * D * 2;
  // K/V tiles: D / 64 halves of 128 rows by 64 columns (128 bytes)
  static constexpr int kHalfStep = 16384;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = NQ * kTileBytes;
  static constexpr int kVOff = kKOff + NSK * kTileBytes;
  static constexpr int kAuxOff = kVOff + NSV * kTileBytes;  // barriers and flags
  static constexpr int kRefOff = kAuxOff + 512;             // row references [2][128]
  static constexpr int kSumOff = kRefOff + 2 * 128 * 4;     // row sums [2][2][128]
  static constexpr int kNarOff = kSumOff + 2 * 2 * 128 * 4;  // narrow pieces: LSE of the quarters' rows [2][4][32]
  static constexpr int kOwnOff = kNarOff + 2 * 4 * 32 * 4;  // the piece of a CTA that works out its own
  static constexpr int kStageOff = kOwnOff + 32;   // output staging, 2 KB per softmax warp
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

// The index of the piece this CTA takes in round r (at or past n_pieces: none,
// nor in any later round).  From the planner's list it takes one per round of
// the grid, every other round in reverse CTA order, so that the CTA with a
// round's longest piece gets the next one's shortest; without a planner its
// one piece stands in its shared memory.
__device__ __forceinline__ int round_piece(const ChunkParams& p, int r) {
  if (p.direct) return r;
  const int c = (r & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
  return r * (int)gridDim.x + c;
}
template <class C>
__device__ __forceinline__ ChunkPiece piece_at(const ChunkParams& p, int i) {
  const int4* src = p.direct ? reinterpret_cast<const int4*>(smem_base() + C::kOwnOff) + 2 * i
                             : reinterpret_cast<const int4*>(p.pieces + i);
  const int4 a = src[0], b = src[1];
  ChunkPiece w;
  w.b = a.x; w.rt = a.y; w.hg = a.z; w.kt0 = a.w;
  w.count = b.x; w.slot = b.y;
  return w;
}
// Next round at or after r whose piece has key tiles, or -1.
template <class C>
__device__ __forceinline__ int next_busy(const ChunkParams& p, int n_pieces, int r, ChunkPiece& w) {
  for (;; ++r) {
    const int i = round_piece(p, r);
    if (i >= n_pieces) return -1;
    w = piece_at<C>(p, i);
    if (w.count > 0) return r;
  }
}

// No planner: piece i of sequence i / (tiles * heads), row tile, head group
// (count -1: the sequence has no such tile), and the check of its lengths.
__device__ __forceinline__ ChunkPiece direct_piece(const ChunkParams& p, int i) {
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
    row_tile_keys(p, q, w.rt, w.kt0, w.count);
  }
  return w;
}

// Output of a row that keeps no key of its sequence.
template <int D>
__device__ __forceinline__ void write_empty_row(const ChunkParams& p, int b, int h, int i) {
  const int64_t qrow = (p.cu_q ? p.cu_q[b] : 0) + i, ob = p.cu_q ? 0 : b;
  uint16_t* o = p.o + ob * p.o_sb + qrow * p.o_ss + (int64_t)h * p.o_sh;
#pragma unroll
  for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(o + c) = make_uint4(0, 0, 0, 0);
  p.lse[ob * p.lse_sb + (int64_t)h * p.lse_sh + qrow * p.lse_ss] = -INFINITY;
}

// One producer warp: K or V tiles of every piece, in order, through a ring of
// n_stages stages.  Box x of a tile (its rows x * box_rows ..) is sent by lane
// x / NP of the operand's warp x % NP; each warp waits for the stage itself and
// arrives on its full barrier (NP arrivals) with the bytes it sends.  Written for
// few registers, and one copy of the code for both operands: with two, the
// softmax loop beside them ran a fifth slower.
template <class C, int D, int NP>
__device__ __forceinline__ void produce(const ChunkParams& p, const bool is_k, const int n_stages,
                                        const CUtensorMap* map, int n_pieces, int part, int lane, uint64_t* full,
                                        uint64_t* empty, uint64_t* v_tail, unsigned char* ring,
                                        volatile int* abort_flag) {
  constexpr int kTileBytes = 128 * D * 2, kHalfStep = 16384;
  if (lane == 0) tc::tma_prefetch_desc(map);
  int s = 0;             // stage of the next tile
  uint32_t phase = 1;    // parity its empty barrier has to have completed (a fresh barrier passes for 1)
  uint32_t tails = 0;
  bool ok = true;
  // test only: the first key tile is never sent (FA_DEBUG_WITHHOLD)
  bool withhold = is_k && (p.debug_flags & FA_DEBUG_WITHHOLD);
  ChunkPiece w;
  for (int r = next_busy<C>(p, n_pieces, 0, w); ok && r >= 0; r = next_busy<C>(p, n_pieces, r + 1, w)) {
    const int head = w.hg * p.gp / p.G;
    const int32_t* table = p.block_table ? p.block_table + (int64_t)w.b * p.bt_stride : nullptr;
    const int seq = w.b;
    int key = w.kt0 * kKeysPerTile;             // the tile's first key
    int left = p.kv_len[w.b] - key;             // keys from there to the sequence's end
    for (int i = w.count; i > 0; --i, key += kKeysPerTile, left -= kKeysPerTile) {
      const int rows = min(kKeysPerTile, left);
      const int nb = (rows + p.box_rows - 1) >> p.box_shift;
      // this lane's first page, read before the wait
      int x = part + NP * lane, row = 0, page = -1;
      auto look_up = [&] {
        const int at = key + (x << p.box_shift), pi = fast_div(at, p.div_page);
        row = at - pi * p.page_size;
        page = table ? table[pi] : seq;
      };
      if (x < nb) look_up();
      const bool tail = !is_k && rows < kKeysPerTile;
      bool go = true;
      if (lane == 0) {
        go = tc::mbar_wait(empty + s, phase, abort_flag);
        // the last tail's barrier phase ends before an arrival for the next
        if (!is_k && go && tail && tails > 0) go = tc::mbar_wait_drain(v_tail, (tails - 1) & 1, 1000000000ull);
      }
      go = __shfl_sync(0xffffffffu, go, 0);
      if (!go) {
        if (lane == 0) fail(p, abort_flag, is_k ? 1 : 7);
        ok = false;
        break;
      }
      uint64_t* bar = tail ? v_tail : full + s;
      for (int x0 = 0; !withhold; ) {
        const bool good = x < nb && page >= 0 && page < p.num_pages;
        if (x < nb && !good) chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)page);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, good)) * p.box_rows * (uint32_t)(D * 2);
        const bool last = x0 + 32 * NP >= nb;
        if (lane == 0) {
          // the warp's one arrival comes with its last group of boxes
          if (last) tc::mbar_arrive_expect_tx(bar, bytes);
          else mbar_expect_tx(bar, bytes);
        }
        __syncwarp();
        if (good) {
          unsigned char* dst = ring + s * kTileBytes + x * p.box_rows * 128;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tc::tma_load_4d(dst + c * kHalfStep, map, bar, c * 64, head, row, page);
        }
        __syncwarp();
        if (last) break;
        x0 += 32 * NP;
        x += 32 * NP;
        if (x < nb) look_up();
      }
      withhold = false;
      if (tail) {
        if (part == 0) {
          // rows past the last key in its 16-key step: zero once the copies have landed
          if (!tc::mbar_wait_drain(v_tail, tails & 1, 1000000000ull)) {
            if (lane == 0) fail(p, abort_flag, 8);
            ok = false;
            break;
          }
          const int end = (rows + 15) & ~15;
          for (int e = lane; e < (end - rows) * (D / 8); e += 32) {
            const int rr = rows + e / (D / 8), ch = e % (D / 8);
            *reinterpret_cast<uint4*>(ring + s * kTileBytes + (ch >> 3) * kHalfStep + rr * 128 + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
        }
        ++tails;
        if (lane == 0) tc::mbar_arrive(full + s);
      }
      if (++s == n_stages) {
        s = 0;
        phase ^= 1;
      }
    }
  }
  if (lane == 0 && *abort_flag) {
    // let the copies already issued land before the CTA can exit: wait, up to a
    // limit, for each stage's next full phase (a stage without copies in flight
    // runs into the limit)
    for (int k = 0; k < n_stages; ++k) {
      // stages before s were last filled in this pass of the ring, the others in the pass before
      const uint32_t ph = k < s ? phase ^ 1 : phase;
      tc::mbar_wait_drain(full + k, ph, 100000000ull);
    }
  }
  __syncwarp();
}

// GEN: soft-cap and / or ALiBi (the plain logits fold the scale into the exponent).
template <int D, int NW, int NP, bool NARROW, bool GEN, bool F16>
__global__ void __launch_bounds__(CCfg<D, NW, NP>::kThreads, CCfg<D, NW, NP>::kCtas)
    chunk_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tmq,
                 const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using C = CCfg<D, NW, NP>;
  constexpr int NSK = C::NSK, NSV = C::NSV, NQ = C::NQ;
  constexpr uint32_t kPCol = C::kPCol, kOCol = C::kOCol;
  constexpr int NB = C::NB;
  unsigned char* smem = smem_base();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kAuxOff);
  uint64_t* q_full = bars;           // [2] Q buffer loaded
  uint64_t* q_empty = q_full + 2;    // [2] QKs reading a Q buffer done
  uint64_t* k_full = q_empty + 2;    // [NSK]
  uint64_t* k_empty = k_full + NSK;  // [NSK]
  uint64_t* v_full = k_empty + NSK;  // [NSV]
  uint64_t* v_empty = v_full + NSV;  // [NSV]
  uint64_t* v_tail = v_empty + NSV;  // [1] copies of a V tile whose end is zeroed
  uint64_t* s_full = v_tail + 1;     // [NB] S buffer written by QK
  uint64_t* p_full = s_full + NB;    // [NB] P buffer written, O rescaled (128 arrivals)
  uint64_t* p_free = p_full + NB;    // [NB] PV reading a P buffer done
  uint64_t* s_free = p_free + NB;    // [1] one warpgroup: S read by the softmax (128 arrivals)
  uint64_t* o_full = s_free + 1;     // [1] last PV of a piece done
  uint64_t* drained = o_full + 1;    // [2] all MMAs of an issuer done (teardown)
  uint64_t* sumx = drained + 2;      // [1] row sums of all warpgroups posted (128 NW arrivals)
  uint64_t* refb = sumx + 1;         // [2 tile parity] row references posted (128 arrivals)
  uint64_t* narb = refb + 2;         // [2 warpgroups] steps of a narrow piece's merge (128 arrivals)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(narb + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      tc::mbar_init(q_full + k, 1);
      tc::mbar_init(q_empty + k, 1);
      tc::mbar_init(drained + k, 1);
      tc::mbar_init(refb + k, 128);
      tc::mbar_init(narb + k, 128);
    }
    for (int s = 0; s < NSK; ++s) {
      tc::mbar_init(k_full + s, NP);
      tc::mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < NSV; ++s) {
      tc::mbar_init(v_full + s, NP);
      tc::mbar_init(v_empty + s, 1);
    }
    tc::mbar_init(v_tail, NP);
    for (int k = 0; k < NB; ++k) {
      tc::mbar_init(s_full + k, 1);
      tc::mbar_init(p_full + k, 128);
      tc::mbar_init(p_free + k, 1);
    }
    tc::mbar_init(s_free, 128);
    tc::mbar_init(sumx, 128 * NW);
    tc::mbar_init(o_full, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::kCols);
    tc::tmem_relinquish();
  }
  if (p.direct && tid == 128) *reinterpret_cast<ChunkPiece*>(smem + C::kOwnOff) = direct_piece(p, blockIdx.x);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  wait_for_previous();
  const int n_pieces = p.direct ? 1 : p.counts->n_pieces;  // of the grid, or (no planner) of this CTA

  if (warp < 4 || warp >= 4 + 4 * NW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
  if (warp == 0 || warp == 2 || (NP == 2 && (warp == 12 || warp == 13))) {
    // ------------------------------------------------------------ producers
    // K: warp 0 (and 12), V: warp 2 (and 13)
    const int part = warp < 4 ? 0 : 1;
    const bool is_k = warp == 0 || warp == 12;
    produce<C, D, NP>(p, is_k, is_k ? NSK : NSV, is_k ? &tmk : &tmv, n_pieces, part, lane, is_k ? k_full : v_full,
                   is_k ? k_empty : v_empty, v_tail, smem + (is_k ? C::kKOff : C::kVOff), abort_flag);
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK issuer
    // S[g % NB] = Q K_g^T for the g-th tile of this CTA, as soon as that buffer is
    // free: the PV of its P done (one warpgroup: S read by the softmax); and Q: with two buffers the next
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
        // narrow: the same rows in each quarter of the tile
        constexpr int kCopies = NARROW ? 4 : 1;
        tc::mbar_arrive_expect_tx(q_full + qb, kCopies * q_bytes);
        for (int e = 0; e < kCopies * (D / 64); ++e)
          tc::tma_load_4d(dst + (e / kCopies) * 16384 + (e % kCopies) * 4096, &tmq, q_full + qb, (e / kCopies) * 64,
                          w.hg * p.gp, q_row0 + w.rt * p.rt_tokens, q_b);
      };
      bool ok = true;
      int g = 0, kk = 0;  // tiles and busy pieces so far
      ChunkPiece w, wn;
      int u = next_busy<C>(p, n_pieces, 0, w);
      if (u >= 0) load_q(w, 0);
      for (; ok && u >= 0; ++kk) {
        const int qb = kk % NQ;
        const int un = next_busy<C>(p, n_pieces, u + 1, wn);
        if (!tc::mbar_wait(q_full + qb, (kk / NQ) & 1, abort_flag)) { ok = false; break; }
        for (int i = 0; i < w.count; ++i, ++g) {
          const int s = g % NSK, sb = g % NB;
          if (!tc::mbar_wait(k_full + s, (g / NSK) & 1, abort_flag)) { ok = false; break; }
          if (g >= NB && !tc::mbar_wait(NW == 2 ? p_free + sb : s_free, ((g - NB) / NB) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          // (an operand's later steps: its descriptor plus a constant, the
          // address field does not overflow)
          const uint64_t qd = tc::sdesc_sw128(sQ + qb * C::kTileBytes, 16, 1024);
          const uint64_t kd = tc::sdesc_sw128(sK + s * C::kTileBytes, 16, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = ((ks >> 2) * C::kHalfStep + (ks & 3) * 32) >> 4;
            tc::mma_ss(tbase + sb * 128, qd + o, kd + o, idS, ks > 0 ? 1u : 0u);
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
    // O (+)= P[g % NB] V_g once the softmax of tile g has written P (and
    // rescaled O), over the 16-key steps that hold keys.
    if (lane == 0) {
      constexpr uint32_t idO = tc::idesc_bf16_f32(128, D, false, true, F16);
      const uint32_t sV = tc::smem_u32(smem + C::kVOff);
      bool ok = true;
      int g = 0;
      ChunkPiece w;
      for (int r = next_busy<C>(p, n_pieces, 0, w); ok && r >= 0; r = next_busy<C>(p, n_pieces, r + 1, w)) {
        const int kv = p.kv_len[w.b];
        for (int i = 0; i < w.count; ++i, ++g) {
          const int s = g % NSV, pb = g % NB;
          const int steps = min(8, (kv - (w.kt0 + i) * kKeysPerTile + 15) / 16);
          if (!tc::mbar_wait(p_full + pb, (g / NB) & 1, abort_flag) ||
              !tc::mbar_wait(v_full + s, (g / NSV) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t vd = tc::sdesc_sw128(sV + s * C::kTileBytes, C::kHalfStep, 1024);
          // (whole tiles apart: the queue of MMAs is shallow, and whatever the
          // issuing thread does between two of them idles the tensor cores)
          if (steps == 8) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc::mma_ts(tbase + kOCol, tbase + kPCol + pb * 128 + ks * 8,
                         vd + (uint32_t)(ks * 2048 >> 4), idO, (i > 0 || ks > 0) ? 1u : 0u);
          } else {
#pragma unroll 1
            for (int ks = 0; ks < steps; ++ks)
              tc::mma_ts(tbase + kOCol, tbase + kPCol + pb * 128 + ks * 8,
                         vd + (uint32_t)(ks * 2048 >> 4), idO, (i > 0 || ks > 0) ? 1u : 0u);
          }
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
  } else if (warp < 4 + 4 * NW) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int w = NW == 2 ? (warp - 4) >> 2 : 0;
    const int wq = warp & 3;  // TMEM lane quarter this warp may access
    const int row = 32 * wq + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(32 * wq) << 16);
    float* refv = reinterpret_cast<float*>(smem + C::kRefOff);  // [2 tile parity][128]
    float* rsum = reinterpret_cast<float*>(smem + C::kSumOff);  // [2][2 warpgroups][128]
    constexpr int kHalfD = D / NW;  // O columns each warpgroup stores
    bool ok = true;
    int g = 0, kk = 0;  // tiles and busy pieces so far
    uint32_t nsteps = 0;  // steps of narrow pieces' merges so far
    // buffer of this warpgroup's next tile and the parity of its use; tiles come
    // NW apart whatever the pieces' lengths
    int sb = NW == 2 ? w : 0;
    uint32_t use = 0;
    auto advance = [&] {
      sb += NW;
      if (sb >= NB) {
        sb -= NB;
        use ^= 1;
      }
    };
    for (int r = 0; ok; ++r) {
      const int pi = round_piece(p, r);
      if (pi >= n_pieces) break;
      // what the tile loop keeps live is little: the piece's tiles, this row's
      // keys, and (GEN) its place and slope; the rest is read again after it
      int kt0, count, jlo_r, jhi_r, place = 0;
      float alibi_l2 = 0.f;
      bool active;
      {
        const ChunkPiece un = piece_at<C>(p, pi);
        kt0 = un.kt0;
        count = un.count;
        const int q_len = chunk_qlen(p, un.b), kv_len = p.kv_len[un.b];
        const int rl = NARROW ? lane : row, tok = fast_div(rl, p.div_gp), i = un.rt * p.rt_tokens + tok;
        const bool exists = tok < p.rt_tokens && i < q_len;
        if (count <= 0) {
          if (count == 0 && w == 0 && exists && (!NARROW || wq == 0)) write_empty_row<D>(p, un.b, un.hg * p.gp + rl - tok * p.gp, i);
          continue;
        }
        chunk_row_keys(p, i, kv_len - q_len, kv_len, p.prefix ? p.prefix[un.b] : 0, jlo_r, jhi_r);
        if (!exists) { jlo_r = 0; jhi_r = INT_MAX; }  // whatever it computes is not stored
        active = __any_sync(0xffffffffu, exists);
        if (GEN) {
          place = i + kv_len - q_len;
          if (p.alibi && exists) alibi_l2 = __ldg(p.alibi + un.hg * p.gp + rl - tok * p.gp) * kLog2e;
        }
      }
      float m_ref = -INFINITY;  // reference after the last tile seen
      float r_own = -INFINITY;  // reference this warpgroup's row sum is against
      float l = 0.f;
      const int it0 = (NW == 1 || (g & 1) == w) ? 0 : 1;  // the piece's first tile that is this warpgroup's
      if (!active) {
        // no row of this warp exists: keep step on the barriers
        for (int it = it0; ok && it < count; it += NW) {
          const int gt = g + it;
          ok = tc::mbar_wait(s_full + sb, use, abort_flag);
          if (NW == 1) tc::mbar_arrive_relaxed(s_free);
          if (NW == 2) {
            ok = ok && (gt < 1 || tc::mbar_wait(refb + ((gt - 1) & 1), ((gt - 1) >> 1) & 1, abort_flag));
            tc::mbar_arrive(refb + (gt & 1));
          }
          if (NW == 1) ok = ok && (gt < 1 || tc::mbar_wait(p_free, (gt - 1) & 1, abort_flag));
          tc::mbar_arrive_relaxed(p_full + sb);
          advance();
        }
      } else
      for (int it = it0; it < count; it += NW) {
        const int gt = g + it;
        const int j0 = (kt0 + it) * kKeysPerTile;
        // some row of the warp does not keep the whole tile
        const bool part = __any_sync(0xffffffffu, jlo_r > j0 || jhi_r < j0 + kKeysPerTile - 1);
        if (!tc::mbar_wait(s_full + sb, use, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        // The row is taken in four runs of 32 columns, twice: from the last to the
        // first for the maximum (with the logits' transforms, which are left in
        // TMEM), and back for the exponentials, each run loaded while the one
        // before it is worked on.  The loops are not unrolled further: four warps
        // of instruction stream share a fetch path that this code is bound by.
        const uint32_t sa = lane_base + sb * 128, pa = lane_base + kPCol + sb * 128;
        uint32_t xa[32], xb[32];
        float mx = -INFINITY;
        auto first_pass = [&](uint32_t (&x)[32], int c, bool keep) {
          if constexpr (GEN) {
            // logits in log2 units: soft-cap or scale, then the distance penalty
            if (p.softcap > 0.f) {
              // cap tanh(y) = cap - 2 cap / (1 + e^(2 y)); the rounding near 1 leaves
              // about 3e-7 cap in the logit (1e-5 at cap 30)
              const float k = 2.f * p.scale_log2 * p.inv_softcap, c1 = p.softcap * kLog2e;
              if (p.softcap <= kPlainSoftcap) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  x[e] = __float_as_uint(fmaf(-2.f * c1, fast_rcp(1.f + fast_exp2(__uint_as_float(x[e]) * k)), c1));
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(wide_softcap(__uint_as_float(x[e]), k, c1, p));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * p.scale_log2);
            }
            if (p.alibi) {
              const float dist = (float)(place - j0 - 32 * c);  // to the run's first key
#pragma unroll
              for (int e = 0; e < 32; ++e)
                x[e] = __float_as_uint(__uint_as_float(x[e]) - alibi_l2 * fabsf(dist - (float)e));
            }
          }
          if (part) {
            // the row keeps keys clo .. clo + span of the run; a row that keeps
            // none gets a start no key reaches.  (The scale is positive, so
            // a raw -inf stays -inf through it.)
            const bool none = jhi_r < jlo_r;
            const int clo = none ? (1 << 20) : jlo_r - j0 - 32 * c;
            const unsigned span = none ? 0u : (unsigned)(jhi_r - jlo_r);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = (unsigned)(e - clo) <= span ? x[e] : __float_as_uint(-INFINITY);
          }
          if ((GEN || part) && keep) tc::tmem_st32(sa + c * 32, x);
          float m[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = __uint_as_float(x[k]);
#pragma unroll
          for (int e = 4; e < 32; e += 2)
            m[(e >> 1) & 3] = max3f(m[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          mx = max3f(mx, max3f(m[0], m[1], m[2]), m[3]);
        };
        if constexpr (NARROW) {
          // the warp's quarter of the tile's keys
          tc::tmem_ld32(sa + wq * 32, xb);
          tmem_loaded(xb);
          first_pass(xb, wq, false);
        } else {
          tc::tmem_ld32(sa + 96, xa);
          tmem_loaded(xa);
#pragma unroll 1
          for (int c = 3; c > 0; c -= 2) {
            tc::tmem_ld32(sa + (c - 1) * 32, xb);
            first_pass(xa, c, true);
            tmem_loaded(xb);
            if (c > 1) tc::tmem_ld32(sa + (c - 2) * 32, xa);
            first_pass(xb, c - 1, c > 1);
            if (c > 1) tmem_loaded(xa);
          }
        }
        if constexpr (!GEN) mx *= p.scale_log2;
        if (GEN || part) tc::tmem_wait_st();
        // the reference after tile gt - 1
        if (NW == 2 && gt >= 1 && !tc::mbar_wait(refb + ((gt - 1) & 1), ((gt - 1) >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        const float m_prev = (it == 0) ? -INFINITY : (NW == 2 ? refv[((gt - 1) & 1) * 128 + row] : m_ref);
        const bool upd = mx > m_prev + 8.f;  // raise the reference only when outgrown by 2^8
        m_ref = upd ? mx : m_prev;
        if (NW == 2) {
          refv[(gt & 1) * 128 + row] = m_ref;
          tc::mbar_arrive(refb + (gt & 1));
        }
        if (it != 0 && __any_sync(0xffffffffu, upd && m_prev != -INFINITY)) {
          // O holds the PV of tile gt - 1 (against m_prev) once that PV is done
          const int pb = sb > 0 ? sb - 1 : NB - 1;
          if (!tc::mbar_wait(p_free + pb, sb > 0 ? use : use ^ 1, abort_flag)) { ok = false; break; }
          tc::fence_after_sync();
          const float f = (upd && m_prev != -INFINITY) ? fast_exp2(m_prev - m_ref) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            const uint32_t a = lane_base + kOCol + c * 32;
            tc::tmem_ld32(a, xa);
            tmem_loaded(xa);
#pragma unroll
            for (int e = 0; e < 32; ++e) xa[e] = __float_as_uint(__uint_as_float(xa[e]) * f);
            tc::tmem_st32(a, xa);
          }
        }
        if (r_own != m_ref) {
          // (before the row's first finite logit l is 0, or NaN after a NaN one: kept)
          if (r_own != -INFINITY) l *= fast_exp2(r_own - m_ref);
          r_own = m_ref;
        }
        // one warpgroup: the P buffer is free once the PV before is done (with
        // two, the QK into this S buffer has waited for it)
        if (NW == 1 && gt >= 1 && !tc::mbar_wait(p_free, (gt - 1) & 1, abort_flag)) { ok = false; break; }
        const float eref = (m_ref == -INFINITY) ? 0.f : m_ref;
        const float2 ner = make_float2(-eref, -eref), sl2 = make_float2(p.scale_log2, p.scale_log2);
        float2 acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = make_float2(0.f, 0.f);
        auto second_pass = [&](const uint32_t (&x)[32], int c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 xe = make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
            const float2 v = GEN ? add2(xe, ner) : fma2(xe, sl2, ner);
            const float2 pe = make_float2(fast_exp2(v.x), fast_exp2(v.y));
            acc[e & 3] = add2(acc[e & 3], pe);
            pk[e] = pack2<F16>(pe.x, pe.y);
          }
          tc::tmem_st16(pa + c * 16, pk);
        };
        if constexpr (NARROW) {
          uint32_t zero[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) zero[e] = 0;
#pragma unroll 1
          for (int c = 1; c < 4; ++c) tc::tmem_st16(pa + ((wq + c) & 3) * 16, zero);
          second_pass(xb, wq);
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tc::tmem_ld32(sa + (c + 1) * 32, xa);
            second_pass(xb, c);
            tmem_loaded(xa);
            if (c < 2) tc::tmem_ld32(sa + (c + 2) * 32, xb);
            second_pass(xa, c + 1);
            if (c < 2) tmem_loaded(xb);
          }
        }
        acc[0] = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
        l += acc[0].x + acc[0].y;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        if (NW == 1) tc::mbar_arrive_relaxed(s_free);  // the next QK may overwrite S
        tc::mbar_arrive_relaxed(p_full + sb);
        advance();
      }
      if (!ok) break;
      // ---- epilogue: both warpgroups' row sums against the final reference
      const int gl = g + count - 1;  // the piece's last tile
      g += count;
      if (NW == 2 && (gl & 1) != w) {
        if (!tc::mbar_wait(refb + (gl & 1), (gl >> 1) & 1, abort_flag)) { ok = false; break; }
        m_ref = refv[(gl & 1) * 128 + row];
      }
      const ChunkPiece un = piece_at<C>(p, pi);
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
        // (two sets of sums: a warpgroup may write the next piece's while another
        // still reads these)
        float* rs = rsum + (kk & 1) * 256;
        rs[w * 128 + row] = (r_own == m_ref || r_own == -INFINITY) ? l : l * fast_exp2(r_own - m_ref);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        tc::mbar_arrive(sumx);
        if (!tc::mbar_wait(sumx, kk & 1, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        lt = rs[row] + rs[128 + row];
      } else {
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        lt = l;
      }
      const bool empty = lt == 0.f;  // (a row with a NaN stays NaN)
      const float inv = empty ? 0.f : 1.f / lt;
      const float lse2 = empty ? -INFINITY : m_ref + __log2f(lt);
      const int q_len = chunk_qlen(p, un.b);
      const int64_t qbase = p.cu_q ? (int64_t)p.cu_q[un.b] : 0, ob = p.cu_q ? 0 : un.b;
      if constexpr (NARROW) {
        // The four quarters' rows, each over its quarter of every tile's keys, are
        // joined by their log-sum-exp, 8 rows at a time through the
        // warpgroup's staging memory.
        float* so = reinterpret_cast<float*>(smem + C::kStageOff + w * 8192);  // [4 quarters][8 rows][kHalfD]
        float* sl = reinterpret_cast<float*>(smem + C::kNarOff) + w * 128;     // [4 quarters][32 rows]
        const int n_rows = min(p.rt_tokens, q_len - un.rt * p.rt_tokens) * p.gp;
        const int wtid = 32 * wq + lane, c4 = 4 * (wtid % (kHalfD / 4)), rr = wtid / (kHalfD / 4);
        auto step = [&] {
          tc::mbar_arrive(narb + w);
          const bool go = tc::mbar_wait(narb + w, nsteps & 1, abort_flag);
          ++nsteps;
          return go;
        };
        for (int r0 = 0; r0 < n_rows && ok; r0 += 8) {
          if (!(ok = step())) break;  // the staging memory is free
          if (r0 == 0) sl[wq * 32 + lane] = lse2;
          if (lane >= r0 && lane < r0 + 8) {
            float* dst = so + (wq * 8 + lane - r0) * kHalfD;
#pragma unroll
            for (int c = 0; c < kHalfD / 32; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(dst + c * 32 + e) =
                    make_float4(__uint_as_float(ro[c][e]) * inv, __uint_as_float(ro[c][e + 1]) * inv,
                                __uint_as_float(ro[c][e + 2]) * inv, __uint_as_float(ro[c][e + 3]) * inv);
          }
          if (!(ok = step())) break;
          const int r1 = r0 + rr;
          if (rr < 8 && r1 < n_rows) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) top = fmaxf(top, sl[q * 32 + r1]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (top == -INFINITY) top = 0.f;  // no quarter keeps a key: all weights 0
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float f = fast_exp2(sl[q * 32 + r1] - top);
              const float4 v = *reinterpret_cast<const float4*>(so + (q * 8 + rr) * kHalfD + c4);
              sum += f;
              o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
            }
            const float f = sum == 0.f ? 0.f : 1.f / sum;
            const float ls = sum == 0.f ? -INFINITY : top + __log2f(sum);
            o.x *= f; o.y *= f; o.z *= f; o.w *= f;
            if (un.slot >= 0) {
              const int64_t at = (int64_t)un.slot * kChunkRows + r1;
              *reinterpret_cast<float4*>(p.part_o + at * D + w * kHalfD + c4) = o;
              if (w == 0 && c4 == 0) p.part_lse[at] = ls;
            } else {
              const int t1 = fast_div(r1, p.div_gp), h1 = un.hg * p.gp + r1 - t1 * p.gp;
              const int64_t qrow = qbase + un.rt * p.rt_tokens + t1;
              *reinterpret_cast<uint2*>(p.o + ob * p.o_sb + qrow * p.o_ss + (int64_t)h1 * p.o_sh + w * kHalfD + c4) =
                  make_uint2(pack2<F16>(o.x, o.y), pack2<F16>(o.z, o.w));
              if (w == 0 && c4 == 0) p.lse[ob * p.lse_sb + (int64_t)h1 * p.lse_sh + qrow * p.lse_ss] = ls * kLn2;
            }
          }
        }
        // (with two warpgroups the next piece's row-sum barrier keeps its staging
        // after these reads)
        if (NW == 1 && ok) ok = step();
        if (!ok) break;
      } else {
        const int tok = fast_div(row, p.div_gp), i = un.rt * p.rt_tokens + tok;
        const bool exists = tok < p.rt_tokens && i < q_len;
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
          uint16_t* obase = p.o + ob * p.o_sb + (int64_t)un.hg * p.gp * p.o_sh;
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
          if (w == 0 && exists)
            p.lse[ob * p.lse_sb + (int64_t)(un.hg * p.gp + row - tok * p.gp) * p.lse_sh + (qbase + i) * p.lse_ss] = lse2 * kLn2;
        }
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

template <int D, int NW, int NP, bool NARROW, bool GEN, bool F16>
cudaError_t launch_v(const ChunkParams& p, bool overlap, cudaStream_t st) {
  using C = CCfg<D, NW, NP>;
  // setmaxnreg.inc would wait forever if the block were launched with fewer
  // registers than the split assumes: launch only when the build matches.
  static std::atomic<int> launch_regs{-1};
  int regs = launch_regs.load(std::memory_order_relaxed);
  cudaError_t e;
  if (regs < 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, chunk_kernel<D, NW, NP, NARROW, GEN, F16>)) != cudaSuccess) return e;
    regs = fa.numRegs;
    launch_regs.store(regs, std::memory_order_relaxed);
  }
  if (regs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  if ((e = ensure_smem_attr<chunk_kernel<D, NW, NP, NARROW, GEN, F16>>(C::kSmem)) != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  const bool packed = p.cu_q != nullptr;
  const int heads_kv = p.Hq / p.G;
  if (!encode_map(&mq, p.q, D, p.Hq, packed ? p.tot_q : p.Sq, packed ? 1 : p.n_seq, p.q_sh, p.q_ss, p.q_sb, p.gp,
                  p.rt_tokens, F16) ||
      !encode_map(&mk, p.k, D, heads_kv, p.cache_rows, p.cache_outer, p.k_sh, p.k_ss, p.k_sb, 1, p.box_rows, F16) ||
      !encode_map(&mv, p.v, D, heads_kv, p.cache_rows, p.cache_outer, p.v_sh, p.v_ss, p.v_sb, 1, p.box_rows, F16))
    return cudaErrorInvalidValue;
  return launch_overlapped(chunk_kernel<D, NW, NP, NARROW, GEN, F16>, (unsigned)p.grid, C::kThreads, C::kSmem, overlap, st, p, mq, mk, mv);
}

template <int D, int NW, int NP, bool NARROW, bool F16>
cudaError_t launch_g(const ChunkParams& p, bool overlap, cudaStream_t st) {
  return (p.softcap > 0.f || p.alibi) ? launch_v<D, NW, NP, NARROW, true, F16>(p, overlap, st)
                                      : launch_v<D, NW, NP, NARROW, false, F16>(p, overlap, st);
}

// (CCfg, ChunkParams::narrow and ::pair say which form is for what)
template <bool F16>
cudaError_t launch_t(const ChunkParams& p, bool overlap, cudaStream_t st) {
  if (p.d == 64) {
    if (p.narrow) return p.pair ? launch_g<64, 1, 1, true, F16>(p, overlap, st) : launch_g<64, 2, 1, true, F16>(p, overlap, st);
    return p.pair ? launch_g<64, 1, 1, false, F16>(p, overlap, st) : launch_g<64, 2, 1, false, F16>(p, overlap, st);
  }
  if (p.narrow) return launch_g<128, 2, 1, true, F16>(p, overlap, st);
  return p.box_rows <= 16 ? launch_g<128, 2, 2, false, F16>(p, overlap, st)
                          : launch_g<128, 2, 1, false, F16>(p, overlap, st);
}

}  // namespace

// The fp16 instantiations build in their own translation unit (chunk_f16.cu
// includes this file with MFA_CHUNK_F16_UNIT defined), in parallel.
#ifndef MFA_CHUNK_F16_UNIT
cudaError_t launch_chunk_attn(const ChunkParams& p, bool overlap, cudaStream_t st) { return launch_t<false>(p, overlap, st); }
#else
cudaError_t launch_chunk_attn_f16(const ChunkParams& p, bool overlap, cudaStream_t st) {
  return launch_t<true>(p, overlap, st);
}
#endif

}  // namespace mfa
