// chunk_q8_sm103.cu -- fa_fwd_chunk_q8's attention kernel for many query rows per K/V
// head, on the 5th-generation tensor cores of sm_103a (tcgen05 + TMEM + TMA).
//
// The tile scheme is that of chunk_sm103.cu: 128 rows of (token, q-head) pairs by 128
// keys, S = Q K^T into TMEM, the weights packed back over S, O += P V, two softmax
// warpgroups on alternate key tiles, pieces of work from the planner's list.  The
// cache is in 8 bits (q8_device.cuh), and three things differ:
//  - K and V tiles come as codes, by TMA into a ring of raw tiles, and a warpgroup
//    widens them to fp16, which is exact, into the swizzled tiles that the products
//    read.  One conversion serves 128 rows.  Beside the products' operands (96 KB per
//    pair of tiles) shared memory takes 32 KB of codes in, 32 KB out and 64 KB of fp16
//    in, and the conversion shares the issue slots with the softmax: this is the bound;
//  - Q enters in fp16 after a power of two per row (its largest element at 2^7 .. 2^8),
//    written by the same warps;
//  - the scales, one per 16 keys or more, join in the softmax: with K's scale 2^a and
//    V's 2^b the logit in log2 units is x = 2^a f <q, code>, y = x + b, the weight
//    w = 2^(y - ref) multiplies V's codes and the row sum adds w 2^-b.  The maximum of
//    16 keys is one of raw products (2^a f > 0), so this costs no instruction per
//    element.  Weights reach 2^7 .. 2^15 (chunk_q8.cu).
//
// A NaN in V would reach every row of the tile (0 times NaN): in a tile that some row
// does not see whole, the widening writes 0 for it and marks the piece, and the
// epilogue of a marked piece looks the NaNs of the keys that each row sees up in the
// cache.  Rows past the sequence's end are written as 0.
//
// Warp roles (16 warps): 0 copies codes, 1 issues QK, 2 looks up pages and scales, 3 issues
// PV, 4 .. 11 softmax, 12 .. 15 widen.  512 threads launch at 128 registers, split 72 / 184
// / 72.  Every mbarrier wait is bounded as in chunk_sm103.cu.
//
// Measured (32 heads on 8, d 128, pages of 64 keys): 2048 tokens over 32768 keys 1255 us
// (849 TFLOP/s; the 16-bit cache 682 us), 4 x 512 over 4096 keys 194 us, 64 x 16 over 4016
// keys 197 us (2.8 TB/s).  With eight pieces of the conversion's loads ahead; one at a time
// takes 334 us for the second.  A second warpgroup for the conversion (20 warps of fewer
// registers) took 207, 256 rows to a CTA 219, codes by plain loads straight into
// registers more than 230, a half of the columns of every tile to each softmax warpgroup 203.
// Without conversion and softmax the copies and products alone take 138, with either 165 .. 173.
#include <algorithm>
#include <atomic>
#include <climits>

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk.h"
#include "chunk_device.cuh"
#include "fa_device.cuh"
#include "host_util.h"
#include "q8_device.cuh"
#include "rope_common.cuh"
#include "tc_sm103.cuh"

namespace mfa {

namespace {

constexpr float kTop = 7.f, kRaise = 15.f;  // log2 of the weights at the top
constexpr int kGroups = kKeysPerTile / 16;  // keys with one scale, at least
constexpr int kScaleRing = 32;              // tiles whose scales are held
constexpr int kPlaceRing = 16;              // tiles whose places in the cache are held
constexpr int kRowRing = 8;                 // pieces whose row factors are held (Q is two ahead, S buffers three)

template <int D>
struct TCfg {
  static constexpr int kThreads = 512;
  static constexpr int kLaunchRegs = 128, kOtherRegs = 72, kWidenRegs = 72, kSoftmaxRegs = 184;
  static_assert(128 * kOtherRegs + 128 * kWidenRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs, "the register split must fit the launch");
  static constexpr uint32_t kCols = 512, kOCol = 384;  // TMEM: three S buffers, each overwritten by its P, and O
  static constexpr int NB = 3;
  // (more of them at d = 64 are slower: 8 x 512 tokens of 12 heads over 4608 keys 150 us, with
  // four and six 165; at d = 128 two or three raw tiles are the same)
  static constexpr int NS = D == 128 ? 2 : 3;          // tiles of K, and of V
  static constexpr int NR = 3;                         // raw tiles of both
  static constexpr int kRawBytes = 128 * D, kTileBytes = 2 * kRawBytes;
  static constexpr int kHalfStep = 16384;  // D / 64 halves of 128 rows by 128 bytes
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kTileBytes;
  static constexpr int kVOff = kKOff + NS * kTileBytes;
  static constexpr int kRawOff = kVOff + NS * kTileBytes;
  static constexpr int kAuxOff = kRawOff + NR * kRawBytes;    // barriers and flags
  static constexpr int kRefOff = kAuxOff + 1024;              // row references [2][128]
  static constexpr int kSumOff = kRefOff + 2 * 128 * 4;       // row sums [2][2][128]
  static constexpr int kFacOff = kSumOff + 2 * 2 * 128 * 4;   // row factors [kRowRing][128]
  static constexpr int kScaOff = kFacOff + kRowRing * 128 * 4;  // {2^a, b, 2^-b, of the tile: first key, 1 if not whole, first and last key seen, 0 ..} [kScaleRing][kGroups]
  static constexpr int kPlaOff = kScaOff + kScaleRing * kGroups * 16;  // {page (-1: not seen), row in it} [kPlaceRing][kGroups]
  static constexpr int kOwnOff = kPlaOff + kPlaceRing * kGroups * 8;
  static constexpr int kSmem = kOwnOff + 32 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// The piece this CTA takes in round r, as in chunk_sm103.cu.
__device__ __forceinline__ int round_of(const ChunkParams& p, int r) {
  if (p.direct) return r;
  const int c = (r & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
  return r * (int)gridDim.x + c;
}
template <class C>
__device__ __forceinline__ ChunkPiece piece_of(const ChunkParams& p, int i) {
  const int4* src = p.direct ? reinterpret_cast<const int4*>(smem_base() + C::kOwnOff) + 2 * i : reinterpret_cast<const int4*>(p.pieces + i);
  const int4 a = src[0], b = src[1];
  ChunkPiece w;
  w.b = a.x; w.rt = a.y; w.hg = a.z; w.kt0 = a.w;
  w.count = b.x; w.slot = b.y;
  return w;
}
// Next round at or after r whose piece has key tiles, or -1.
template <class C>
__device__ __forceinline__ int next_with_keys(const ChunkParams& p, int n_pieces, int r, ChunkPiece& w) {
  for (;; ++r) {
    const int i = round_of(p, r);
    if (i >= n_pieces) return -1;
    w = piece_of<C>(p, i);
    if (w.count > 0) return r;
  }
}

// A piece's sequence, and where its list of tiles jumps.
struct Geo {
  int q_len, kv_len, prefix, off;
  int kt0, first, gap;
  // keys that some row of the tile sees: at or below need_hi, and at or above need_lo
  // or among the first `sinks`; keys all_lo .. all_hi are seen by every row
  int need_lo, need_hi, all_lo, all_hi, sinks;
  __device__ __forceinline__ int first_key(int it) const {
    const int tile = kt0 + it;
    return (tile + (tile >= first ? gap : 0)) * kKeysPerTile;
  }
};
__device__ __forceinline__ Geo geo_of(const ChunkParams& p, const ChunkPiece& w) {
  Geo g;
  g.q_len = chunk_qlen(p, w.b);
  g.kv_len = p.kv_len[w.b];
  g.prefix = p.prefix ? p.prefix[w.b] : 0;
  g.off = g.kv_len - g.q_len;
  const SinkTiles t = row_tile_sinks(p, make_int4(0, g.q_len, g.kv_len, g.prefix), w.rt);
  g.kt0 = w.kt0;
  g.first = t.first;
  g.gap = t.gap;
  const int i0 = w.rt * p.rt_tokens, i1 = min(i0 + p.rt_tokens, g.q_len) - 1;
  chunk_row_keys(p, i0, g.off, g.kv_len, g.prefix, g.need_lo, g.all_hi);
  chunk_row_keys(p, i1, g.off, g.kv_len, g.prefix, g.all_lo, g.need_hi);
  g.sinks = p.wl >= 0 ? p.sinks : 0;
  return g;
}

// GEN: soft-cap and / or ALiBi.
template <int D, bool GEN>
__global__ void __launch_bounds__(512, 1) chunk_q8_tc_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tmk,
                                                             const __grid_constant__ CUtensorMap tmv) {
  using C = TCfg<D>;
  constexpr int NS = C::NS, NR = C::NR, NB = C::NB;
  unsigned char* smem = smem_base();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kAuxOff);
  uint64_t* raw_full = bars;               // [NR] codes landed
  uint64_t* raw_empty = raw_full + NR;     // [NR] codes read (4 warps)
  uint64_t* k_full = raw_empty + NR;       // [NS] widened (4 warps)
  uint64_t* k_empty = k_full + NS;         // [NS] QK done
  uint64_t* v_full = k_empty + NS;         // [NS]
  uint64_t* v_empty = v_full + NS;         // [NS]
  uint64_t* q_full = v_empty + NS;         // [kRowRing] Q and its factors written (4 warps)
  uint64_t* q_empty = q_full + kRowRing;   // [1] a piece's QKs done
  uint64_t* s_full = q_empty + 1;          // [NB] S written
  uint64_t* p_full = s_full + NB;          // [NB] P written, O rescaled (128 threads)
  uint64_t* p_free = p_full + NB;          // [NB] PV done
  uint64_t* o_full = p_free + NB;          // [1] a piece's last PV done
  uint64_t* drained = o_full + 1;          // [2] all MMAs of an issuer done
  uint64_t* sumx = drained + 2;            // [1] row sums posted (256 threads)
  uint64_t* refb = sumx + 1;               // [2] row references posted (128 threads)
  uint64_t* sc_full = refb + 2;            // [kScaleRing] scales written
  uint64_t* pl_full = sc_full + kScaleRing;   // [kPlaceRing] places written
  uint64_t* pl_empty = pl_full + kPlaceRing;  // [kPlaceRing] places read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pl_empty + kPlaceRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* nan_piece = abort_flag + 1;  // [kRowRing] the busy piece whose partly seen tiles hold a NaN, + 1
  static_assert((2 * NR + 4 * NS + kRowRing + 1 + 3 * NB + 1 + 2 + 1 + 2 + kScaleRing + 2 * kPlaceRing) * 8 + 8 + 4 * kRowRing <= 1024, "barriers");
  float* s_fac = reinterpret_cast<float*>(smem + C::kFacOff);
  float4* s_sca = reinterpret_cast<float4*>(smem + C::kScaOff);
  int2* s_pla = reinterpret_cast<int2*>(smem + C::kPlaOff);

  if (tid == 0) {
    for (int k = 0; k < NR; ++k) {
      tc::mbar_init(raw_full + k, 1);
      tc::mbar_init(raw_empty + k, 4);
    }
    for (int k = 0; k < NS; ++k) {
      tc::mbar_init(k_full + k, 4);
      tc::mbar_init(k_empty + k, 1);
      tc::mbar_init(v_full + k, 4);
      tc::mbar_init(v_empty + k, 1);
    }
    for (int k = 0; k < kRowRing; ++k) {
      tc::mbar_init(q_full + k, 4);
      nan_piece[k] = 0;
    }
    for (int k = 0; k < NB; ++k) {
      tc::mbar_init(s_full + k, 1);
      tc::mbar_init(p_full + k, 128);
      tc::mbar_init(p_free + k, 1);
    }
    tc::mbar_init(o_full, 1);
    tc::mbar_init(q_empty, 1);
    for (int k = 0; k < 2; ++k) {
      tc::mbar_init(drained + k, 1);
      tc::mbar_init(refb + k, 128);
    }
    tc::mbar_init(sumx, 256);
    for (int k = 0; k < kScaleRing; ++k) tc::mbar_init(sc_full + k, 1);
    for (int k = 0; k < kPlaceRing; ++k) {
      tc::mbar_init(pl_full + k, 1);
      tc::mbar_init(pl_empty + k, 1);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::kCols);
    tc::tmem_relinquish();
  }
  wait_for_previous();
  if (p.direct && tid == 128) *reinterpret_cast<ChunkPiece*>(smem + C::kOwnOff) = q8_own_piece(p, blockIdx.x);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const int n_pieces = p.direct ? 1 : p.counts->n_pieces;

  // (one register limit to a branch: where two met, the compiler would take the lower)
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
  if (warp == 0) {
    // ------------------------------------------------------------ codes
    // Raw tiles K_0, K_1, V_0, K_2, V_1 .. through the ring (V's place is free once a
    // product of two tiles back is done, which K does not have to wait for): box x of a
    // tile (its rows x * box_rows ..) is sent by lane x.
    if (lane == 0) {
      tc::tma_prefetch_desc(&tmk);
      tc::tma_prefetch_desc(&tmv);
    }
    int s = 0, g = 0;
    uint32_t phase = 1;
    bool ok = true, withhold = p.debug_flags & FA_DEBUG_WITHHOLD;  // test only: the first tile of K is never sent
    const int box0 = lane << p.box_shift >> 4;                     // this lane's box: its first group of 16 keys
    ChunkPiece w;
    for (int r = next_with_keys<C>(p, n_pieces, 0, w); ok && r >= 0; r = next_with_keys<C>(p, n_pieces, r + 1, w)) {
      const int head = w.hg * p.gp / p.G;
      int2 at = make_int2(-1, 0), at_v = at;
      uint32_t bytes = 0, bytes_v = 0;
      for (int i = 0; ok && i <= w.count; ++i) {
        // K of tile i, and V of the tile before it
        at_v = at;
        bytes_v = bytes;
        if (i < w.count) {
          const int e = g % kPlaceRing;
          ok = __all_sync(0xffffffffu, tc::mbar_wait(pl_full + e, (g / kPlaceRing) & 1, abort_flag));
          if (!ok) break;
          at = box0 < kGroups ? s_pla[e * kGroups + box0] : make_int2(-1, 0);
          bytes = __popc(__ballot_sync(0xffffffffu, at.x >= 0)) * p.box_rows * (uint32_t)D;
          if (lane == 0) tc::mbar_arrive(pl_empty + e);
          ++g;
        }
        for (int v = i < w.count ? 0 : 1; v < (i > 0 ? 2 : 1); ++v) {
          bool go = true;
          if (lane == 0) {
            go = tc::mbar_wait(raw_empty + s, phase, abort_flag);
            if (go) tc::mbar_arrive_expect_tx(raw_full + s, v ? bytes_v : bytes);
          }
          ok = __shfl_sync(0xffffffffu, go, 0);
          if (!ok) break;
          unsigned char* dst = smem + C::kRawOff + s * C::kRawBytes + lane * p.box_rows * D;
          if (v == 0 && at.x >= 0 && !withhold) tc::tma_load_4d(dst, &tmk, raw_full + s, 0, head, at.y, at.x);
          if (v == 1 && at_v.x >= 0) tc::tma_load_4d(dst, &tmv, raw_full + s, 0, head, at_v.y, at_v.x);
          withhold = false;
          if (++s == NR) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    }
    if (!ok && lane == 0) fail(p, abort_flag, 1);
    if (lane == 0 && *abort_flag) {
      // let the copies under way land: each stage's next full phase, up to a limit
      for (int k = 0; k < NR; ++k) tc::mbar_wait_drain(raw_full + k, k < s ? phase ^ 1 : phase, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ pages and scales
    // Four tiles at a time, ahead of the copies, by a lane for each group of 16 keys: its page
    // and row (-1: no row of the tile sees its box) and its scales.  The softmax is less than
    // 16 tiles behind the copies (by the rings between), so the place of a tile's scales,
    // kScaleRing behind, is free when that of its pages is.
    bool ok = true;
    int g = 0;
    const int x = lane & 7, tt = lane >> 3;
    ChunkPiece w;
    for (int r = next_with_keys<C>(p, n_pieces, 0, w); ok && r >= 0; r = next_with_keys<C>(p, n_pieces, r + 1, w)) {
      const Geo geo = geo_of(p, w);
      const int head = w.hg * p.gp / p.G, box_keys = p.box_rows;
      const int32_t* table = p.block_table ? p.block_table + (int64_t)w.b * p.bt_stride : nullptr;
      // (the group of tile i0 + tt, and the next four tiles' asked for)
      auto key_of = [&](int i0) {
        if (i0 + tt >= w.count) return -1;
        const int key = geo.first_key(i0 + tt) + 16 * x, box = key & ~(box_keys - 1);  // (a box is copied whole)
        return box <= geo.need_hi && (box + box_keys > geo.need_lo || box < geo.sinks) && key < geo.kv_len ? key : -1;
      };
      auto page_of = [&](int key) { return key < 0 ? -1 : table ? __ldg(table + fast_div(key, p.div_page)) : w.b; };
      int key = key_of(0), page = page_of(key);
      for (int i0 = 0; ok && i0 < w.count; i0 += 4) {
        const int n = min(4, w.count - i0);
        const int key_n = key_of(i0 + 4), page_n = page_of(key_n);
        bool good = key >= 0;
        if (good && (page < 0 || page >= p.num_pages)) {
          chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)page);
          good = false;
        }
        const int row = good ? key - fast_div(key, p.div_page) * p.page_size : 0;
        float ks = 1.f, vs = 1.f;
        if (good) {
          const int64_t b = row >> p.block_shift;
          ks = __ldg(p.ks + page * p.ks_sb + b * p.ks_ss + head * p.ks_sh);
          vs = __ldg(p.vs + page * p.vs_sb + b * p.vs_ss + head * p.vs_sh);
        }
        const int to = g + i0 + tt;
        bool go = true;
        if (tt < n && to >= kPlaceRing) go = tc::mbar_wait(pl_empty + to % kPlaceRing, ((to - kPlaceRing) / kPlaceRing) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, go);
        if (!ok) break;
        if (tt < n) {
          s_pla[(to % kPlaceRing) * kGroups + x] = make_int2(good ? page : -1, row);
          const int ve = scale_exponent(vs), key0 = geo.first_key(i0 + tt);
          // not whole: some row does not see all of the tile, or it goes past the end
          const bool part = key0 + kKeysPerTile - 1 > geo.all_hi || (key0 < geo.all_lo && key0 + kKeysPerTile - 1 >= geo.sinks);
          const int about = x == 0 ? key0 : x == 1 ? (int)part : x == 2 ? geo.need_lo : x == 3 ? geo.need_hi : 0;
          s_sca[(to % kScaleRing) * kGroups + x] = make_float4(pow2f(scale_exponent(ks)), (float)ve, pow2f(-ve), __int_as_float(about));
        }
        __syncwarp();
        if (x == 0 && tt < n) {
          tc::mbar_arrive(pl_full + to % kPlaceRing);
          tc::mbar_arrive(sc_full + to % kScaleRing);
        }
        key = key_n;
        page = page_n;
      }
      g += w.count;
    }
    if (!ok && lane == 0) fail(p, abort_flag, 7);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK issuer
    if (lane == 0) {
      constexpr uint32_t idS = tc::idesc_bf16_f32(128, 128, false, false, true);
      const uint32_t sQ = tc::smem_u32(smem + C::kQOff), sK = tc::smem_u32(smem + C::kKOff);
      bool ok = true;
      int g = 0, kk = 0;  // tiles and busy pieces so far
      ChunkPiece w;
      for (int r = next_with_keys<C>(p, n_pieces, 0, w); ok && r >= 0; r = next_with_keys<C>(p, n_pieces, r + 1, w), ++kk) {
        if (!tc::mbar_wait(q_full + kk % kRowRing, (kk / kRowRing) & 1, abort_flag)) { ok = false; break; }
        for (int i = 0; i < w.count; ++i, ++g) {
          const int s = g % NS, sb = g % NB;
          if (!tc::mbar_wait(k_full + s, (g / NS) & 1, abort_flag) ||
              (g >= NB && !tc::mbar_wait(p_free + sb, ((g - NB) / NB) & 1, abort_flag))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t qd = tc::sdesc_sw128(sQ, 16, 1024), kd = tc::sdesc_sw128(sK + s * C::kTileBytes, 16, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = ((ks >> 2) * C::kHalfStep + (ks & 3) * 32) >> 4;
            tc::mma_ss(tbase + sb * 128, qd + o, kd + o, idS, ks > 0 ? 1u : 0u);
          }
          tc::mma_commit(s_full + sb);
          tc::mma_commit(k_empty + s);
        }
        if (!ok) break;
        tc::mma_commit(q_empty);
      }
      if (!ok) fail(p, abort_flag, 2);
      tc::mma_commit(drained);
      tc::mbar_wait_drain(drained, 0, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0) {
      constexpr uint32_t idO = tc::idesc_bf16_f32(128, D, false, true, true);
      const uint32_t sV = tc::smem_u32(smem + C::kVOff);
      bool ok = true;
      int g = 0;
      ChunkPiece w;
      for (int r = next_with_keys<C>(p, n_pieces, 0, w); ok && r >= 0; r = next_with_keys<C>(p, n_pieces, r + 1, w)) {
        for (int i = 0; i < w.count; ++i, ++g) {
          const int s = g % NS, pb = g % NB;
          if (!tc::mbar_wait(p_full + pb, (g / NB) & 1, abort_flag) || !tc::mbar_wait(v_full + s, (g / NS) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t vd = tc::sdesc_sw128(sV + s * C::kTileBytes, C::kHalfStep, 1024);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_ts(tbase + C::kOCol, tbase + pb * 128 + ks * 8, vd + (uint32_t)(ks * 2048 >> 4), idO, (i > 0 || ks > 0) ? 1u : 0u);
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
  }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kWidenRegs));
    // ------------------------------------------------------------ Q, and the widening
    const int cw = warp - 12;
    // 8 codes to 16 bytes: a thread's piece is one of the row's D / 8, in every kRows-th
    // row, a multiple of 8: its place in the swizzle stays
    constexpr int kPieces = D / 8, kRows = 128 / kPieces;
    const int t = 32 * cw + lane, c = t % kPieces, row0 = t / kPieces;
    const unsigned char* const src0 = smem + C::kRawOff + t * 8;
    unsigned char* const dst0 = smem + (c >> 3) * C::kHalfStep + row0 * 128 + (((c & 7) ^ (row0 & 7)) << 4);
    bool ok = true;
    int g = 0, kk = 0, rs = 0;  // tiles and busy pieces so far, raw tile
    uint32_t rphase = 0;
    ChunkPiece w;
    for (int r = next_with_keys<C>(p, n_pieces, 0, w); ok && r >= 0; r = next_with_keys<C>(p, n_pieces, r + 1, w), ++kk) {
      {
        // Q: D / 8 lanes per row, 16 bytes each, kAhead loads in flight
        constexpr int kQLanes = D / 8, kPer = 32 / kQLanes, kSteps = 128 / (4 * kPer), kAhead = 4;
        const int64_t qbase = p.cu_q ? (int64_t)p.cu_q[w.b] : 0, qb = p.cu_q ? 0 : w.b;
        const int i0 = w.rt * p.rt_tokens, qc = lane % kQLanes, q_len = chunk_qlen(p, w.b);
        float* fac = s_fac + (kk % kRowRing) * 128;
#pragma unroll 1
        for (int s0 = 0; ok && s0 < kSteps; s0 += kAhead) {
          uint4 u[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int row = ((s0 + k) * 4 + cw) * kPer + lane / kQLanes, tok = fast_div(row, p.div_gp);
            u[k] = make_uint4(0, 0, 0, 0);
            if (tok < p.rt_tokens && i0 + tok < q_len)
              u[k] = *reinterpret_cast<const uint4*>(p.q + qb * p.q_sb + (qbase + i0 + tok) * p.q_ss +
                                                     (int64_t)(w.hg * p.gp + row - tok * p.gp) * p.q_sh + 8 * qc);
          }
          if (s0 == 0 && kk > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(q_empty, (kk - 1) & 1, abort_flag));
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int row = ((s0 + k) * 4 + cw) * kPer + lane / kQLanes;
            const uint32_t v[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
            float x[8], top = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = p.f16 ? unpack2<true>(v[e]) : unpack2<false>(v[e]);
              x[2 * e] = y.x;
              x[2 * e + 1] = y.y;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(fmaf(x[e], 0.f, x[e])));  // (finite ones)
#pragma unroll
            for (int o = 1; o < kQLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e = q_exponent(top);
            const float down = pow2f(-e);
            *reinterpret_cast<uint4*>(smem + C::kQOff + (qc >> 3) * C::kHalfStep + row * 128 + (((qc & 7) ^ (row & 7)) << 4)) =
                make_uint4(pack2<true>(x[0] * down, x[1] * down), pack2<true>(x[2] * down, x[3] * down),
                           pack2<true>(x[4] * down, x[5] * down), pack2<true>(x[6] * down, x[7] * down));
            // (never so small that a scale of K makes it 0, which times a masked -inf would be NaN; 2^-36 of a logit at most)
            if (qc == 0) fac[row] = GEN ? pow2f(e) : fmaxf(pow2f(e) * p.scale_log2, 0x1p-100f);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(q_full + kk % kRowRing);
      }
      // (the raw tiles come as K_0, K_1, V_0, K_2, V_1 .. V_n-1)
#pragma unroll 1
      for (int m = 0; ok && m < 2 * w.count; ++m) {
        const bool is_v = m > 0 && (!(m & 1) || m == 2 * w.count - 1);
        const int gt = g + (is_v ? (m == 2 * w.count - 1 ? w.count - 1 : m / 2 - 1) : (m + 1) / 2), s = gt % NS;
        uint64_t* const full = is_v ? v_full : k_full;
        uint64_t* const empty = is_v ? v_empty : k_empty;
        ok = tc::mbar_wait(raw_full + rs, rphase, abort_flag) && (gt < NS || tc::mbar_wait(empty + s, ((gt - NS) / NS) & 1, abort_flag)) &&
             (!is_v || tc::mbar_wait(sc_full + gt % kScaleRing, (gt / kScaleRing) & 1, abort_flag));
        ok = __all_sync(0xffffffffu, ok);  // (the warp stays together)
        if (!ok) break;
        const unsigned char* src = src0 + rs * C::kRawBytes;
        unsigned char* dst = dst0 + (is_v ? C::kVOff : C::kKOff) + s * C::kTileBytes;
        auto widen = [](uint2 u) {
          return make_uint4(e4m3x2_to_f16x2((uint16_t)u.x), e4m3x2_to_f16x2((uint16_t)(u.x >> 16)), e4m3x2_to_f16x2((uint16_t)u.y),
                            e4m3x2_to_f16x2((uint16_t)(u.y >> 16)));
        };
        const float4* sca = s_sca + (gt % kScaleRing) * kGroups;
        if (!is_v || !__float_as_int(sca[1].w)) {
          constexpr int kAhead = 8;
#pragma unroll
          for (int n0 = 0; n0 < kPieces; n0 += kAhead) {
            uint2 u[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n) u[n] = *reinterpret_cast<const uint2*>(src + (n0 + n) * 1024);
#pragma unroll
            for (int n = 0; n < kAhead; ++n) *reinterpret_cast<uint4*>(dst + (n0 + n) * kRows * 128) = widen(u[n]);
          }
        } else {
          const int key = __float_as_int(sca[0].w), need_lo = __float_as_int(sca[2].w), need_hi = __float_as_int(sca[3].w);
          const int sinks = p.wl >= 0 ? p.sinks : 0;
          bool nans = false;
#pragma unroll 2
          for (int n = 0; n < kPieces; ++n) {
            const int j = key + row0 + n * kRows;
            const bool seen = j <= need_hi && (j >= need_lo || j < sinks);
            uint2 u = *reinterpret_cast<const uint2*>(src + n * 1024);
            const uint32_t mx = seen ? nan_codes(u.x) : 0xffffffffu, my = seen ? nan_codes(u.y) : 0xffffffffu;  // (a key that no row sees: 0)
            nans |= seen && (mx | my) != 0;
            u.x &= ~mx;
            u.y &= ~my;
            *reinterpret_cast<uint4*>(dst + n * kRows * 128) = widen(u);
          }
          if (nans) nan_piece[kk % kRowRing] = kk + 1;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(raw_empty + rs);
        if (++rs == NR) {
          rs = 0;
          rphase ^= 1;
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full + s);
      }
      g += w.count;
    }
    if (!ok && lane == 0) fail(p, abort_flag, 6);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int wg = (warp - 4) >> 2, wq = warp & 3;  // warpgroup, TMEM lane quarter
    const int row = 32 * wq + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(32 * wq) << 16);
    float* refv = reinterpret_cast<float*>(smem + C::kRefOff);  // [2 tile parity][128]
    float* rsum = reinterpret_cast<float*>(smem + C::kSumOff);  // [2][2 warpgroups][128]
    constexpr int kHalfD = D / 2;
    const int sinks = p.wl >= 0 ? p.sinks : 0;
    bool ok = true;
    int g = 0, kk = 0;
    int sb = wg;       // buffer of this warpgroup's next tile (tiles come two apart) and the parity of its use
    uint32_t use = 0;
    auto advance = [&] {
      sb += 2;
      if (sb >= NB) {
        sb -= NB;
        use ^= 1;
      }
    };
    for (int r = 0; ok; ++r) {
      const int pi = round_of(p, r);
      if (pi >= n_pieces) break;
      int kt0, first, gap, count, jlo_r, jhi_r, place = 0;
      float alibi_l2 = 0.f;
      bool active;
      {
        const ChunkPiece un = piece_of<C>(p, pi);
        if (un.count < 0) continue;
        const Geo geo = geo_of(p, un);
        kt0 = geo.kt0; first = geo.first; gap = geo.gap;
        count = un.count;
        const int tok = fast_div(row, p.div_gp), i = un.rt * p.rt_tokens + tok, h = un.hg * p.gp + row - tok * p.gp;
        const bool exists = tok < p.rt_tokens && i < geo.q_len;
        if (count == 0) {
          if (wg == 0 && exists) {
            const int64_t qrow = (p.cu_q ? p.cu_q[un.b] : 0) + i, ob = p.cu_q ? 0 : un.b;
            uint16_t* o = p.o + ob * p.o_sb + qrow * p.o_ss + (int64_t)h * p.o_sh;
#pragma unroll
            for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(o + c) = make_uint4(0, 0, 0, 0);
            p.lse[ob * p.lse_sb + (int64_t)h * p.lse_sh + qrow * p.lse_ss] = -INFINITY;
          }
          continue;
        }
        chunk_row_keys(p, i, geo.off, geo.kv_len, geo.prefix, jlo_r, jhi_r);
        if (!exists) { jlo_r = 0; jhi_r = INT_MAX; }  // whatever it computes is not stored
        active = __any_sync(0xffffffffu, exists);
        if (GEN) {
          place = i + geo.off;
          if (p.alibi && exists) alibi_l2 = __ldg(p.alibi + h) * kLog2e;
        }
      }
      ok = tc::mbar_wait(q_full + kk % kRowRing, (kk / kRowRing) & 1, abort_flag);
      if (!ok) break;
      const float fac = s_fac[(kk % kRowRing) * 128 + row];
      float m_ref = -INFINITY;  // reference after the last tile seen
      float r_own = -INFINITY;  // reference this warpgroup's row sum is against
      float l = 0.f;
      const int it0 = (g & 1) == wg ? 0 : 1;  // the piece's first tile that is this warpgroup's
      if (!active) {
        // no row of this warp exists: keep step on the barriers
        for (int it = it0; ok && it < count; it += 2) {
          const int gt = g + it;
          ok = tc::mbar_wait(s_full + sb, use, abort_flag) &&
               (gt < 1 || tc::mbar_wait(refb + ((gt - 1) & 1), ((gt - 1) >> 1) & 1, abort_flag));
          tc::mbar_arrive(refb + (gt & 1));
          tc::mbar_arrive_relaxed(p_full + sb);
          advance();
        }
      } else
      for (int it = it0; it < count; it += 2) {
        const int gt = g + it, tile = kt0 + it;
        const int j0 = (tile + (tile >= first ? gap : 0)) * kKeysPerTile;
        // some row of the warp does not see the whole tile
        const bool part = __any_sync(0xffffffffu, (jlo_r > j0 && sinks < j0 + kKeysPerTile) || jhi_r < j0 + kKeysPerTile - 1);
        const float4* sca = s_sca + (gt % kScaleRing) * kGroups;
        if (!tc::mbar_wait(sc_full + gt % kScaleRing, (gt / kScaleRing) & 1, abort_flag) ||
            !tc::mbar_wait(s_full + sb, use, abort_flag)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        // as in chunk_sm103.cu: four runs of 32 columns, from the last to the first for
        // the maximum and back for the exponentials
        const uint32_t sa = lane_base + sb * 128;
        uint32_t xa[32], xb[32];
        float mx = -INFINITY;
        auto first_pass = [&](uint32_t (&x)[32], int c, bool keep) {
          const float4 s0 = sca[2 * c], s1 = sca[2 * c + 1];
          const float f0 = s0.x * fac, f1 = s1.x * fac;
          if constexpr (GEN) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * (e < 16 ? f0 : f1));
            if (p.softcap > 0.f) {
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
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) - alibi_l2 * fabsf(dist - (float)e));
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) + (e < 16 ? s0.y : s1.y));
          }
          if (part) {
            // the row sees keys clo .. clo + span of the run, and the first n_sink
            // (the scale is positive, so a raw -inf stays -inf through it)
            const bool none = jhi_r < jlo_r;
            const int clo = none ? (1 << 20) : jlo_r - j0 - 32 * c;
            const unsigned span = none ? 0u : (unsigned)(jhi_r - jlo_r);
            const int n_sink = min(sinks - 1, jhi_r) + 1 - j0 - 32 * c;
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = ((unsigned)(e - clo) <= span || e < n_sink) ? x[e] : __float_as_uint(-INFINITY);
          }
          if ((GEN || part) && keep) tc::tmem_st32(sa + c * 32, x);
          float m[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = max3f(__uint_as_float(x[8 * k]), __uint_as_float(x[8 * k + 1]), __uint_as_float(x[8 * k + 2]));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            m[k] = max3f(m[k], __uint_as_float(x[8 * k + 3]), __uint_as_float(x[8 * k + 4]));
            m[k] = fmaxf(max3f(m[k], __uint_as_float(x[8 * k + 5]), __uint_as_float(x[8 * k + 6])), __uint_as_float(x[8 * k + 7]));
          }
          const float m0 = fmaxf(m[0], m[1]), m1 = fmaxf(m[2], m[3]);
          mx = GEN ? max3f(mx, m0, m1) : max3f(mx, fmaf(m0, f0, s0.y), fmaf(m1, f1, s1.y));
        };
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
        if (GEN || part) tc::tmem_wait_st();
        // the reference after tile gt - 1
        if (gt >= 1 && !tc::mbar_wait(refb + ((gt - 1) & 1), ((gt - 1) >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        const float m_prev = (it == 0) ? -INFINITY : refv[((gt - 1) & 1) * 128 + row];
        const bool upd = mx > m_prev + kRaise;
        m_ref = upd ? mx - kTop : m_prev;
        refv[(gt & 1) * 128 + row] = m_ref;
        tc::mbar_arrive(refb + (gt & 1));
        if (it != 0 && __any_sync(0xffffffffu, upd && m_prev != -INFINITY)) {
          // O holds the PV of tile gt - 1 (against m_prev) once that PV is done
          const int pb = sb > 0 ? sb - 1 : NB - 1;
          if (!tc::mbar_wait(p_free + pb, sb > 0 ? use : use ^ 1, abort_flag)) { ok = false; break; }
          tc::fence_after_sync();
          const float f = (upd && m_prev != -INFINITY) ? fast_exp2(m_prev - m_ref) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            const uint32_t a = lane_base + C::kOCol + c * 32;
            tc::tmem_ld32(a, xa);
            tmem_loaded(xa);
#pragma unroll
            for (int e = 0; e < 32; ++e) xa[e] = __float_as_uint(__uint_as_float(xa[e]) * f);
            tc::tmem_st32(a, xa);
          }
        }
        if (r_own != m_ref) {
          if (r_own != -INFINITY) l *= fast_exp2(r_own - m_ref);
          r_own = m_ref;
        }
        const float eref = (m_ref == -INFINITY) ? 0.f : m_ref;
        auto second_pass = [&](const uint32_t (&x)[32], int c) {
          const float4 s0 = sca[2 * c], s1 = sca[2 * c + 1];
          uint32_t pk[16];
          float2 acc[2][2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 sq = q ? s1 : s0;
            const float f = sq.x * fac, b = GEN ? -eref : sq.y - eref;
            const float2 f2 = make_float2(f, f), b2 = make_float2(b, b);
            acc[q][0] = acc[q][1] = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 8 * q; e < 8 * q + 8; ++e) {
              const float2 xe = make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
              const float2 v = GEN ? add2(xe, b2) : fma2(xe, f2, b2);
              const float2 pe = make_float2(fast_exp2(v.x), fast_exp2(v.y));
              acc[q][e & 1] = add2(acc[q][e & 1], pe);
              pk[e] = pack2<true>(pe.x, pe.y);
            }
          }
          tc::tmem_st16(sa + c * 16, pk);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 a = add2(acc[q][0], acc[q][1]);
            l = fmaf(a.x + a.y, q ? s1.z : s0.z, l);
          }
        };
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {
          tc::tmem_ld32(sa + (c + 1) * 32, xa);
          second_pass(xb, c);
          tmem_loaded(xa);
          if (c < 2) tc::tmem_ld32(sa + (c + 2) * 32, xb);
          second_pass(xa, c + 1);
          if (c < 2) tmem_loaded(xb);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive_relaxed(p_full + sb);
        advance();
      }
      if (!ok) break;
      // ---- epilogue: both warpgroups' row sums against the final reference
      const int gl = g + count - 1;  // the piece's last tile
      g += count;
      if ((gl & 1) != wg) {
        if (!tc::mbar_wait(refb + (gl & 1), (gl >> 1) & 1, abort_flag)) { ok = false; break; }
        m_ref = refv[(gl & 1) * 128 + row];
      }
      const ChunkPiece un = piece_of<C>(p, pi);
      // (O is read before this warpgroup's row sum is posted: chunk_sm103.cu)
      if (!tc::mbar_wait(o_full, kk & 1, abort_flag)) { ok = false; break; }
      tc::fence_after_sync();
      uint32_t ro[kHalfD / 32][32];
#pragma unroll
      for (int c = 0; c < kHalfD / 32; ++c) tc::tmem_ld32(lane_base + C::kOCol + wg * kHalfD + c * 32, ro[c]);
      float* rs = rsum + (kk & 1) * 256;
      rs[wg * 128 + row] = (r_own == m_ref || r_own == -INFINITY) ? l : l * fast_exp2(r_own - m_ref);
      tc::tmem_wait_ld();
      const bool marked = nan_piece[kk % kRowRing] == kk + 1;  // (read before this piece's ring entry can be written again)
      tc::fence_before_sync();
      tc::mbar_arrive(sumx);
      if (!tc::mbar_wait(sumx, kk & 1, abort_flag)) { ok = false; break; }
      tc::fence_after_sync();
      const float lt = rs[row] + rs[128 + row];
      const bool empty = lt == 0.f;  // (a row with a NaN stays NaN)
      const float inv = empty ? 0.f : 1.f / lt;
      const float lse2 = empty ? -INFINITY : m_ref + __log2f(lt);
      const int q_len = chunk_qlen(p, un.b);
      const int64_t qbase = p.cu_q ? (int64_t)p.cu_q[un.b] : 0, ob = p.cu_q ? 0 : un.b;
      const int tok = fast_div(row, p.div_gp), i = un.rt * p.rt_tokens + tok, h = un.hg * p.gp + row - tok * p.gp;
      const bool exists = tok < p.rt_tokens && i < q_len;
#pragma unroll
      for (int c = 0; c < kHalfD / 32; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e) ro[c][e] = __float_as_uint(__uint_as_float(ro[c][e]) * inv);
      if (marked && exists) {
        // the NaNs in V of the keys that this row sees
        uint32_t nan[kHalfD / 32];
#pragma unroll
        for (int c = 0; c < kHalfD / 32; ++c) nan[c] = 0;
        const int hk = un.hg * p.gp / p.G;
        const Geo geo = geo_of(p, un);
        for (int it = 0; it < count; ++it) {
          const int tile = kt0 + it, j0 = (tile + (tile >= first ? gap : 0)) * kKeysPerTile;
          // (in a tile that every row sees whole the products bring them)
          if (j0 + kKeysPerTile - 1 <= geo.all_hi && (j0 >= geo.all_lo || j0 + kKeysPerTile - 1 < sinks)) continue;
          for (int j = j0; j < j0 + kKeysPerTile; ++j) {
            if (j > jhi_r || (j < jlo_r && j >= sinks)) continue;
            const int pg_i = fast_div(j, p.div_page), pg = p.block_table ? p.block_table[(int64_t)un.b * p.bt_stride + pg_i] : un.b;
            if (pg < 0 || pg >= p.num_pages) continue;
            const uint8_t* v = p.v8 + pg * p.v_sb + (int64_t)(j - pg_i * p.page_size) * p.v_ss + hk * p.v_sh + wg * kHalfD;
#pragma unroll
            for (int c = 0; c < kHalfD / 32; ++c)
#pragma unroll 1
              for (int e = 0; e < 32; ++e)
                if ((v[32 * c + e] & 0x7f) == 0x7f) nan[c] |= 1u << e;
          }
        }
#pragma unroll
        for (int c = 0; c < kHalfD / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((nan[c] >> e) & 1) ro[c][e] = 0x7fffffffu;
      }
      if (exists) {
        if (un.slot >= 0) {
          float* dst = p.part_o + ((int64_t)un.slot * kChunkRows + row) * D + wg * kHalfD;
#pragma unroll
          for (int c = 0; c < kHalfD / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(dst + c * 32 + e) = make_uint4(ro[c][e], ro[c][e + 1], ro[c][e + 2], ro[c][e + 3]);
          if (wg == 0) p.part_lse[(int64_t)un.slot * kChunkRows + row] = lse2;
        } else {
          uint16_t* dst = p.o + ob * p.o_sb + (qbase + i) * p.o_ss + (int64_t)h * p.o_sh + wg * kHalfD;
#pragma unroll
          for (int c = 0; c < kHalfD / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = __uint_as_float(ro[c][e + 2 * k]), b = __uint_as_float(ro[c][e + 2 * k + 1]);
                u[k] = p.f16 ? pack2<true>(a, b) : pack2<false>(a, b);
              }
              *reinterpret_cast<uint4*>(dst + c * 32 + e) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          if (wg == 0) p.lse[ob * p.lse_sb + (int64_t)h * p.lse_sh + (qbase + i) * p.lse_ss] = lse2 * kLn2;
        }
      }
      ++kk;
    }
    if (!ok) fail(p, abort_flag, 4 + wg);
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tbase, C::kCols);
}

template <int D, bool GEN>
cudaError_t launch_tc(const ChunkParams& p, bool overlap, cudaStream_t st) {
  using C = TCfg<D>;
  // setmaxnreg.inc would wait forever if the block were launched with fewer
  // registers than the split assumes: launch only when the build matches.
  static std::atomic<int> launch_regs{-1};
  int regs = launch_regs.load(std::memory_order_relaxed);
  cudaError_t e;
  if (regs < 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, chunk_q8_tc_kernel<D, GEN>)) != cudaSuccess) return e;
    regs = fa.numRegs;
    launch_regs.store(regs, std::memory_order_relaxed);
  }
  if (regs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  if ((e = ensure_smem_attr<chunk_q8_tc_kernel<D, GEN>>(C::kSmem)) != cudaSuccess) return e;
  CUtensorMap mk, mv;
  const int heads = p.Hq / p.G;
  if (!encode_codes(&mk, p.k8, D, heads, p.cache_rows, p.cache_outer, p.k_sh, p.k_ss, p.k_sb, p.box_rows, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_codes(&mv, p.v8, D, heads, p.cache_rows, p.cache_outer, p.v_sh, p.v_ss, p.v_sb, p.box_rows, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  return launch_overlapped(chunk_q8_tc_kernel<D, GEN>, (unsigned)p.grid, C::kThreads, C::kSmem, overlap, st, p, mk, mv);
}

}  // namespace

cudaError_t launch_chunk_q8_tc(const ChunkParams& p, bool overlap, cudaStream_t st) {
  const bool gen = p.softcap > 0.f || p.alibi;
  if (p.d == 64) return gen ? launch_tc<64, true>(p, overlap, st) : launch_tc<64, false>(p, overlap, st);
  return gen ? launch_tc<128, true>(p, overlap, st) : launch_tc<128, false>(p, overlap, st);
}

}  // namespace mfa
