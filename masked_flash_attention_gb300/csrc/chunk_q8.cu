// chunk_q8.cu -- fa_fwd_chunk_q8's attention kernel for few query rows per K/V
// head: single tokens, speculated ones, short pieces of prompts, over a cache
// in 8 bits (q8_device.cuh).
//
// Bound: HBM, one byte per cached element.  A CTA runs one piece of a query tile's
// keys (the planner of chunk.cu); of each 128-key tile its eight warps take 16 keys
// each.  A warp streams its keys through a ring of its own, by two TMA copies for 16
// keys, and waits for nobody else.  With two CTAs per SM 128 KB are in flight.
// Measured (64 single tokens over 128 .. 8192 keys, window 4096, soft-cap, 32 heads on 8,
// d 128, pages of 16): 103 us (4.3 TB/s) with the planner and the join, which are 10 of it.
// With three stages of copies it was 114, the copies alone 90 (a head's 16 rows of a page
// are 128 bytes each, 1 KB apart), the products alone 75; four sums instead of one for S
// changed nothing, two tiles at a time, with barriers of their own for K and V, took 134.
//
// Products are m16n8k16 in fp16 with fp32 sums, S^T = K Q^T and O^T = V^T P^T, so that
// the 16 rows of an operand are keys or columns and eight query rows fill the other.
// e4m3 is exact in fp16.  A row of Q is scaled by a power of two into fp16 (its
// largest element to 2^7 .. 2^8, so what fp16 rounds off is below 2^-32 of it),
// whatever its own type.  The order of columns in a product is free as long as both
// sides agree, so a lane's 16-byte loads of a key are its operands of four steps; for
// V the bytes of two keys are interleaved (two byte permutes for eight values)
// before they widen.
//
// The scales: with K's scale 2^a and V's 2^b of a key's block, the logit is
// x = 2^a scale <q, code>, and with y = x log2 e + b the weight w = 2^(y - ref)
// multiplies V's codes themselves, while the row sum adds w 2^-b:
//     O = sum w code / sum w 2^-b.
// ref follows the maximum of y with 7 below it and is raised when y is more than
// 15 above, so weights reach 2^7 .. 2^15 at the top and fp16 keeps all eleven
// bits of those down to 2^-21 of the largest (the sum is of unrounded ones).
// The warps' results are joined by their ref through shared memory.
//
// Sixteen keys that the masks hide from every row of the tile are never read.  A key
// that some rows see and others do not, or one behind the sequence's end in its
// block, is multiplied by a weight of 0; where 16 keys with such a one among them hold a
// NaN in V, it is left out of the products and set in the rows that the masks let see it,
// whatever its key's weight, and in no others.
#include <climits>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk.h"
#include "chunk_device.cuh"
#include "fa_device.cuh"
#include "host_util.h"
#include "mma_sync.cuh"
#include "q8_device.cuh"
#include "rope_common.cuh"
#include "tc_sm103.cuh"

namespace mfa {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch = 16;                   // tiles that a warp looks up at once
constexpr float kTop = 7.f, kRaise = 15.f;  // log2 of the weights at the top

// NT: 8-row tiles of a query tile, 1 or 2.
template <int D, int NT>
struct QCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = 2 * 16 * D;        // K and V of 16 keys
  // (d = 128, two and three: the decoding step at the top 109 and 114 us, 16 rows of 64
  // sequences over 4000 keys 133 and 147, before the NaNs of V left the loop of the
  // products (103 and 131 since): what shared memory leaves is L1)
  static constexpr int kStages = 2 * 128 / D;
  static constexpr int kQStride = 2 * D + 16;           // bytes of a Q row
  static constexpr int kOStride = D + 36;               // floats of a row of the join: eight runs of D / 8 + 4, and 4
  // (the join's rows take the ring's place)
  static constexpr int kRing = kWarps * (kStages * kStageBytes > kRows * kOStride * 4 ? kStages * kStageBytes : kRows * kOStride * 4);
  static constexpr int kQOff = (kRing + 127) / 128 * 128;
  static constexpr int kRowOff = kQOff + kRows * kQStride;           // per row: factor, keys, place, slope
  static constexpr int kSumOff = kRowOff + kRows * 5 * 4;            // ref and sum [kWarps][kRows]
  static constexpr int kInfoOff = kSumOff + kWarps * kRows * 8;      // {page, row, first key, exponents} [kWarps][2 kBatch]
  static constexpr int kBarOff = kInfoOff + kWarps * 2 * kBatch * 16;         // [kWarps][kStages], abort flag
  static constexpr int kOwnOff = kBarOff + kWarps * kStages * 8 + 16;
  static constexpr int kGeoOff = kOwnOff + 32;  // what only the look-ups need of the piece
  static constexpr int kSmem = kGeoOff + 48 + 1024;                  // (the ring starts on a 1024-byte boundary)
  static_assert(kQ8Ctas * kSmem <= 226 * 1024, "shared memory budget");
};

// GEN: soft-cap and / or ALiBi.
template <int D, int NT, bool GEN>
__global__ void __launch_bounds__(kThreads, kQ8Ctas)
    chunk_q8_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv) {
  using C = QCfg<D, NT>;
  constexpr int NST = C::kStages, kRows = C::kRows;
  constexpr int NP = D / 64;  // 16-byte pieces of a key of K per lane
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + warp * NST * C::kStageBytes;
  // where this lane's operands stand in 16 rows of D bytes, which TMA swizzles by 16-byte
  // pieces (128- and 64-byte patterns): K's piece 4 q + t of key g, V's columns (D / 8) g
  // of keys 2 t and 2 t + 1; eight keys later is 8 D bytes on
  int k_at[NP], v_at[2];
  if constexpr (D == 128) {
    k_at[0] = g * 128 + ((t ^ g) << 4);
    k_at[NP - 1] = g * 128 + (((4 + t) ^ g) << 4);
    v_at[0] = 2 * t * 128 + ((g ^ (2 * t)) << 4);
    v_at[1] = (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) << 4);
  } else {
    k_at[0] = g * 64 + ((t ^ (g >> 1)) << 4);
    v_at[0] = 2 * t * 64 + (((g >> 1) ^ t) << 4) + 8 * (g & 1);
    v_at[1] = v_at[0] + 64;
  }
  float* s_fac = reinterpret_cast<float*>(smem + C::kRowOff);  // logit per dot product (GEN: without scale)
  int* s_lo = reinterpret_cast<int*>(s_fac + kRows);
  int* s_hi = s_lo + kRows;
  int* s_place = s_hi + kRows;
  float* s_slope = reinterpret_cast<float*>(s_place + kRows);
  float2* s_sum = reinterpret_cast<float2*>(smem + C::kSumOff);
  int4* s_info = reinterpret_cast<int4*>(smem + C::kInfoOff) + warp * 2 * kBatch;
  volatile int* s_geo = reinterpret_cast<volatile int*>(smem + C::kGeoOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * NST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + kWarps * NST * 8);
  float* s_o = reinterpret_cast<float*>(smem);
  ChunkPiece* own = reinterpret_cast<ChunkPiece*>(smem + C::kOwnOff);

  if (tid == 0) {
    *abort_flag = 0;
    for (int k = 0; k < kWarps * NST; ++k) tc::mbar_init(reinterpret_cast<uint64_t*>(smem + C::kBarOff) + k, 1);
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmk);
    tc::tma_prefetch_desc(&tmv);
  }
  wait_for_previous();
  if (p.direct && tid == 0) *own = q8_own_piece(p, blockIdx.x);
  __syncthreads();
  uint32_t phases = 0;  // parity of each stage's next full phase
  bool withhold = p.debug_flags & FA_DEBUG_WITHHOLD;  // test only: the first copy of K is never sent
  const int n_pieces = p.direct ? 1 : p.counts->n_pieces;

  for (int round = 0;; ++round) {
    // one piece per round of the grid, every other round in reverse CTA order
    const int at = p.direct ? round
                            : round * (int)gridDim.x + ((round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (at >= n_pieces) break;
    int count, all_lo, all_hi, sinks;  // all_lo .. all_hi: the keys that every row sees
    {
    const ChunkPiece w = p.direct ? *own : p.pieces[at];
    if (w.count < 0) continue;
    count = w.count;
    const int q_len = chunk_qlen(p, w.b), kv_len = p.kv_len[w.b], prefix = p.prefix ? p.prefix[w.b] : 0, off = kv_len - q_len;
    const int i0 = w.rt * p.rt_tokens, i1 = min(i0 + p.rt_tokens, q_len) - 1;
    const int head0 = w.hg * p.gp;
    const int64_t qbase = p.cu_q ? (int64_t)p.cu_q[w.b] : 0, qb = p.cu_q ? 0 : w.b;
    // the keys that some row sees: at or below need_hi, and at or above need_lo or
    // among the first `sinks` (both ends of a row's keys move right with the row)
    sinks = p.wl >= 0 ? p.sinks : 0;
    int need_lo, need_hi;
    chunk_row_keys(p, i0, off, kv_len, prefix, need_lo, all_hi);
    chunk_row_keys(p, i1, off, kv_len, prefix, all_lo, need_hi);
    if (tid == 0) {
      const SinkTiles geo = row_tile_sinks(p, make_int4(0, q_len, kv_len, prefix), w.rt);
      const int v[9] = {w.kt0, w.count, geo.first, geo.gap, need_lo, need_hi, sinks, w.b, head0 / p.G};
      for (int k = 0; k < 9; ++k) s_geo[k] = v[k];
    }

    // ---- Q, scaled into fp16: a row per warp and 8-row tile
    for (int r = warp; r < kRows; r += kWarps) {
      const int tok = fast_div(r, p.div_gp), i = i0 + tok, h = head0 + r - tok * p.gp;
      const bool exists = tok < p.rt_tokens && i < q_len;
      float x[D / 32];
      if (exists) {
        const uint16_t* src = p.q + qb * p.q_sb + (qbase + i) * p.q_ss + (int64_t)h * p.q_sh + lane * (D / 32);
        if constexpr (D == 128) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          const float2 a = p.f16 ? unpack2<true>(u.x) : unpack2<false>(u.x), b = p.f16 ? unpack2<true>(u.y) : unpack2<false>(u.y);
          x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
        } else {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(src);
          const float2 a = p.f16 ? unpack2<true>(u) : unpack2<false>(u);
          x[0] = a.x; x[1] = a.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[e] = 0.f;
      }
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) top = fmaxf(top, fabsf(fmaf(x[e], 0.f, x[e])));  // (finite ones)
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = q_exponent(top);
      const float down = pow2f(-e);
      uint32_t o[D / 64];
#pragma unroll
      for (int k = 0; k < D / 64; ++k) o[k] = pack2<true>(x[2 * k] * down, x[2 * k + 1] * down);
      unsigned char* dst = smem + C::kQOff + r * C::kQStride + lane * (D / 16);
      if constexpr (D == 128) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
      else *reinterpret_cast<uint32_t*>(dst) = o[0];
      if (lane == 0) {
        int lo = 0, hi = INT_MAX;  // whatever a row that does not exist computes is not stored
        if (exists) chunk_row_keys(p, i, off, kv_len, prefix, lo, hi);
        s_fac[r] = GEN ? pow2f(e) : pow2f(e) * p.scale_log2;
        s_lo[r] = lo;
        s_hi[r] = hi;
        s_place[r] = i + off;
        s_slope[r] = (GEN && p.alibi && exists) ? __ldg(p.alibi + h) * kLog2e : 0.f;
      }
    }
    }
    __syncthreads();

    // ---- the warp's 16 keys of each tile of the piece.  16 tiles are looked up at once,
    // one by each lane, and the pages of the 16 after them asked for; what is found goes
    // to shared memory (two sets: the copies run ahead of the products).
    int next_page = -1;
    auto first_key = [&](int v) {
      const int tile = s_geo[0] + v;
      return (tile + (tile >= s_geo[2] ? s_geo[3] : 0)) * kKeysPerTile + 16 * warp;
    };
    auto ask = [&](int v) {
      const int j0 = first_key(v);
      // no row sees these keys
      if (lane >= kBatch || v >= s_geo[1] || j0 > s_geo[5] || (j0 + 15 < s_geo[4] && j0 >= s_geo[6])) return -1;
      if (!p.block_table) return s_geo[7];
      const int pg = __ldg(p.block_table + (int64_t)s_geo[7] * p.bt_stride + fast_div(j0, p.div_page));
      if (pg < 0 || pg >= p.num_pages) {
        chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)pg);
        return -1;
      }
      return pg;
    };
    auto look_up = [&](int v) {
      const int page = next_page, j0 = first_key(v + lane), h = s_geo[8];
      const int r = p.block_table ? j0 - fast_div(j0, p.div_page) * p.page_size : j0;
      int ex = 0;
      if (page >= 0) {
        const int64_t b = r >> p.block_shift;
        const int ke = scale_exponent(__ldg(p.ks + page * p.ks_sb + b * p.ks_ss + h * p.ks_sh));
        const int ve = scale_exponent(__ldg(p.vs + page * p.vs_sb + b * p.vs_ss + h * p.vs_sh));
        ex = (ke & 0xff) | ((ve & 0xff) << 8);
      }
      if (lane < kBatch) s_info[(v + lane) % (2 * kBatch)] = make_int4(page, r, j0, ex);
      next_page = ask(v + kBatch + lane);
      __syncwarp();
    };
    next_page = ask(lane);
    auto issue = [&](int v, int stage) {
      if (v >= count) return;
      if (v % kBatch == 0) look_up(v);
      if (lane == 0) {
        const int4 at = s_info[v % (2 * kBatch)];
        if (at.x >= 0) {
          const int h = s_geo[8];
          unsigned char* dst = ring + stage * C::kStageBytes;
          tc::mbar_arrive_expect_tx(full + stage, C::kStageBytes);
          if (!withhold) tc::tma_load_4d(dst, &tmk, full + stage, 0, h, at.y, at.x);
          tc::tma_load_4d(dst + 16 * D, &tmv, full + stage, 0, h, at.y, at.x);
          withhold = false;
        }
      }
    };

    // O^T: rows 2 t + r of tile m, columns (D / 8) g + 2 i and, two on, + 1
    float o[NT][D / 16][4];
    float ref[NT][2], l[NT][2], fac[NT][2];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[m][i][c] = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ref[m][r] = -INFINITY;
        l[m][r] = 0.f;
        fac[m][r] = s_fac[8 * m + 2 * t + r];
      }
    }
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) issue(s, s);
    int stage = 0;
#pragma unroll 1
    for (int v = 0; v < count; ++v) {
      __syncwarp();  // the stage before is read
      issue(v + NST - 1, stage == 0 ? NST - 1 : stage - 1);
      const unsigned char* src = ring + stage * C::kStageBytes;
      const int st = stage;
      if (++stage == NST) stage = 0;
      const int4 info = s_info[v % (2 * kBatch)];
      if (info.x < 0) continue;  // no row sees these keys
      const int ke = (int)(int8_t)info.w, ve = (int)(int8_t)(info.w >> 8), j0 = info.z;
      if (!__all_sync(0xffffffffu, tc::mbar_wait(full + st, (phases >> st) & 1, abort_flag))) {  // (the warp stays together)
        if (!*abort_flag) {
          *abort_flag = 1;
          chunk_error(p, FA_ERR_DEVICE_TIMEOUT, 1u);
        }
        // let the copies under way land: every stage asked for, up to a limit
        for (int k = 0; k < NST; ++k)
          if (v + k < count && s_info[(v + k) % (2 * kBatch)].x >= 0)
            tc::mbar_wait_drain(full + (st + k) % NST, (phases >> ((st + k) % NST)) & 1, 100000000ull);
        break;
      }
      phases ^= 1u << st;

      // ---- S^T = K Q^T: keys j0 + g (first two) and j0 + g + 8, rows 2 t and 2 t + 1
      float s[NT][4];
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[m][c] = 0.f;
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(src + k_at[q]);
        const uint4 k1 = *reinterpret_cast<const uint4*>(src + k_at[q] + 8 * D);
        const uint32_t kw[2][4] = {{k0.x, k0.y, k0.z, k0.w}, {k1.x, k1.y, k1.z, k1.w}};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 qb[NT];
#pragma unroll
          for (int m = 0; m < NT; ++m)
            qb[m] = *reinterpret_cast<const uint4*>(smem + C::kQOff + (8 * m + g) * C::kQStride + 128 * q + 32 * t + 16 * half);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t u0 = kw[0][2 * half + e], u1 = kw[1][2 * half + e];
            const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)u0), e4m3x2_to_f16x2((uint16_t)u1),
                                   e4m3x2_to_f16x2((uint16_t)(u0 >> 16)), e4m3x2_to_f16x2((uint16_t)(u1 >> 16))};
#pragma unroll
            for (int m = 0; m < NT; ++m) mma_bf16<true>(s[m], a, e ? qb[m].z : qb[m].x, e ? qb[m].w : qb[m].y);
          }
        }
      }

      // ---- logits in log2 units plus V's exponent, masks, the reference
      const float kf = pow2f(ke), vf = (float)ve, per_v = pow2f(-ve);
      bool raise = false;
      // some row does not see all 16 keys (the same for all lanes)
      const bool part = j0 + 15 > all_hi || (j0 < all_lo && j0 + 15 >= sinks);
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 8 * m + 2 * t + r;
          const float f = fac[m][r] * kf;
          float &x0 = s[m][r], &x1 = s[m][2 + r];
          if constexpr (GEN) {
            x0 *= f;
            x1 *= f;
            if (p.softcap > 0.f) {
              const float k = 2.f * p.scale_log2 * p.inv_softcap, c1 = p.softcap * kLog2e;
              if (p.softcap <= kPlainSoftcap) {
                x0 = fmaf(-2.f * c1, fast_rcp(1.f + fast_exp2(x0 * k)), c1);
                x1 = fmaf(-2.f * c1, fast_rcp(1.f + fast_exp2(x1 * k)), c1);
              } else {
                x0 = wide_softcap(x0, k, c1, p);
                x1 = wide_softcap(x1, k, c1, p);
              }
            } else {
              x0 *= p.scale_log2;
              x1 *= p.scale_log2;
            }
            if (p.alibi) {
              const float slope = s_slope[row];
              const int dist = s_place[row] - j0 - g;
              x0 -= slope * (float)abs(dist);
              x1 -= slope * (float)abs(dist - 8);
            }
            x0 += vf;
            x1 += vf;
          } else {
            x0 = fmaf(x0, f, vf);
            x1 = fmaf(x1, f, vf);
          }
          if (part) {
            const int lo = s_lo[row], hi = s_hi[row], j = j0 + g;
            if (!(j <= hi && (j >= lo || j < sinks))) x0 = -INFINITY;
            if (!(j + 8 <= hi && (j + 8 >= lo || j + 8 < sinks))) x1 = -INFINITY;
          }
          raise |= fmaxf(x0, x1) > ref[m][r] + kRaise;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float top = fmaxf(s[m][r], s[m][2 + r]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            if (top > ref[m][r] + kRaise) {
              const float up = top - kTop;
              if (ref[m][r] != -INFINITY) {
                const float f = fast_exp2(ref[m][r] - up);
                l[m][r] *= f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  o[m][i][r] *= f;
                  o[m][i][2 + r] *= f;
                }
              }
              ref[m][r] = up;
            }
          }
      }

      // ---- weights: P^T of keys and rows, turned to rows and keys in registers
      uint32_t pb[NT][2];
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        float e[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float base = ref[m][r] == -INFINITY ? 0.f : ref[m][r];
          e[r] = fast_exp2(s[m][r] - base);
          e[2 + r] = fast_exp2(s[m][2 + r] - base);
          l[m][r] = fmaf(e[r] + e[2 + r], per_v, l[m][r]);
        }
        pb[m][0] = movmatrix_t(pack2<true>(e[0], e[1]));
        pb[m][1] = movmatrix_t(pack2<true>(e[2], e[3]));
      }

      // ---- O^T += V^T P^T
      uint32_t vw[4][D / 32];  // this lane's columns of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const unsigned char* at_v = src + 16 * D + v_at[n & 1] + (n >> 1) * 8 * D;
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(at_v);
          vw[n][0] = u.x; vw[n][1] = u.y; vw[n][2] = u.z; vw[n][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(at_v);
          vw[n][0] = u.x; vw[n][1] = u.y;
        }
      }
      bool apart = false;
      if (part) {
        uint32_t nan = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t x = nan_codes(vw[n][i]);
            vw[n][i] &= ~x;
            nan |= x;
          }
        apart = __any_sync(0xffffffffu, nan != 0);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t sel = i & 1 ? 0x7362 : 0x5140;  // columns 2 i and 2 i + 1 of two keys
        const uint32_t x0 = __byte_perm(vw[0][i / 2], vw[1][i / 2], sel), x1 = __byte_perm(vw[2][i / 2], vw[3][i / 2], sel);
        const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)x0), e4m3x2_to_f16x2((uint16_t)(x0 >> 16)), e4m3x2_to_f16x2((uint16_t)x1),
                               e4m3x2_to_f16x2((uint16_t)(x1 >> 16))};
#pragma unroll
        for (int m = 0; m < NT; ++m) mma_bf16<true>(o[m][i], a, pb[m][0], pb[m][1]);
      }
      if (apart) {
        // the NaNs by what the masks admit, not by the weights: a visible key's may be 0 in fp16
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          float e[4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = 8 * m + 2 * t + r, lo = s_lo[row], hi = s_hi[row], j = j0 + g;
            e[r] = j <= hi && (j >= lo || j < sinks) ? 1.f : 0.f;
            e[2 + r] = j + 8 <= hi && (j + 8 >= lo || j + 8 < sinks) ? 1.f : 0.f;
          }
          const uint32_t s0 = movmatrix_t(pack2<true>(e[0], e[1])), s1 = movmatrix_t(pack2<true>(e[2], e[3]));
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            // (V is read again, by volatile loads: kept from before it would cost registers on the way here)
            const unsigned char* at_v = src + 16 * D + 4 * (i / 2);
            auto word = [&](int at) { return *reinterpret_cast<const volatile uint32_t*>(at_v + at); };
            const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
            const uint32_t x0 = nan_codes(__byte_perm(word(v_at[0]), word(v_at[1]), sel));
            const uint32_t x1 = nan_codes(__byte_perm(word(v_at[0] + 8 * D), word(v_at[1] + 8 * D), sel));
            const uint32_t one = 0x3c003c00;  // 1 where V is NaN
            const uint32_t a[4] = {one & __byte_perm(x0, 0, 0x1100), one & __byte_perm(x0, 0, 0x3322), one & __byte_perm(x1, 0, 0x1100),
                                   one & __byte_perm(x1, 0, 0x3322)};
            float hit[4] = {0.f, 0.f, 0.f, 0.f};
            mma_bf16<true>(hit, a, s0, s1);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (hit[c] > 0.f) o[m][i][c] = __int_as_float(0x7fffffff);
          }
        }
      }
    }

    // ---- the warps' rows, joined
    __syncthreads();  // the ring is read
    if (*abort_flag) break;
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 8 * m + 2 * t + r;
        float sum = l[m][r];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (g == 0) s_sum[warp * kRows + row] = make_float2(ref[m][r], sum);
        float* dst = s_o + (warp * kRows + row) * C::kOStride + (D / 8 + 4) * g;
#pragma unroll
        for (int i = 0; i < D / 16; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[m][i][r], o[m][i][2 + r], o[m][i + 1][r], o[m][i + 1][2 + r]);
      }
    __syncthreads();
    const ChunkPiece w = p.direct ? *own : p.pieces[at];
    const int q_len = chunk_qlen(p, w.b), i0 = w.rt * p.rt_tokens, head0 = w.hg * p.gp;
    const int64_t qbase = p.cu_q ? (int64_t)p.cu_q[w.b] : 0, qb = p.cu_q ? 0 : w.b;
    for (int e = tid; e < kRows * (D / 4); e += kThreads) {
      const int row = e / (D / 4), d = 4 * (e % (D / 4));
      const int tok = fast_div(row, p.div_gp), i = i0 + tok, h = head0 + row - tok * p.gp;
      if (tok >= p.rt_tokens || i >= q_len) continue;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_sum[k * kRows + row].x);
      float sum = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = s_sum[k * kRows + row];
        if (ml.y == 0.f) continue;  // (no key seen)
        // (no reference but a sum: a NaN logit before any other)
        const float f = ml.x == -INFINITY ? ml.y : fast_exp2(ml.x - top);
        const float4 v = *reinterpret_cast<const float4*>(s_o + (k * kRows + row) * C::kOStride + d + 4 * (d / (D / 8)));
        sum = fmaf(f, ml.y, sum);
        x.x = fmaf(f, v.x, x.x); x.y = fmaf(f, v.y, x.y); x.z = fmaf(f, v.z, x.z); x.w = fmaf(f, v.w, x.w);
      }
      const bool empty = sum == 0.f;
      const float inv = empty ? 0.f : 1.f / sum;
      const float lse2 = empty ? -INFINITY : top + __log2f(sum);
      x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
      if (w.slot >= 0) {
        const int64_t to = (int64_t)w.slot * kRows + row;
        *reinterpret_cast<float4*>(p.part_o + to * D + d) = x;
        if (d == 0) p.part_lse[to] = lse2;
      } else {
        const uint2 u = p.f16 ? make_uint2(pack2<true>(x.x, x.y), pack2<true>(x.z, x.w))
                              : make_uint2(pack2<false>(x.x, x.y), pack2<false>(x.z, x.w));
        *reinterpret_cast<uint2*>(p.o + qb * p.o_sb + (qbase + i) * p.o_ss + (int64_t)h * p.o_sh + d) = u;
        if (d == 0) p.lse[qb * p.lse_sb + (int64_t)h * p.lse_sh + (qbase + i) * p.lse_ss] = lse2 * kLn2;
      }
    }
    tc::fence_proxy_async_smem();  // the next piece's copies overwrite the rows
    __syncthreads();
  }
}

template <int D, int NT, bool GEN>
cudaError_t launch(const ChunkParams& p, bool overlap, cudaStream_t st) {
  using C = QCfg<D, NT>;
  const cudaError_t e = ensure_smem_attr<chunk_q8_kernel<D, NT, GEN>>(C::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  const CUtensorMapSwizzle swz = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!encode_codes(&mk, p.k8, D, p.Hq / p.G, p.cache_rows, p.cache_outer, p.k_sh, p.k_ss, p.k_sb, 16, swz) ||
      !encode_codes(&mv, p.v8, D, p.Hq / p.G, p.cache_rows, p.cache_outer, p.v_sh, p.v_ss, p.v_sb, 16, swz))
    return cudaErrorInvalidValue;
  return launch_overlapped(chunk_q8_kernel<D, NT, GEN>, (unsigned)p.grid, kThreads, C::kSmem, overlap, st, p, mk, mv);
}
template <int D, int NT>
cudaError_t launch(const ChunkParams& p, bool overlap, cudaStream_t st) {
  return (p.softcap > 0.f || p.alibi) ? launch<D, NT, true>(p, overlap, st) : launch<D, NT, false>(p, overlap, st);
}

}  // namespace

cudaError_t launch_chunk_q8(const ChunkParams& p, bool overlap, cudaStream_t st) {
  if (p.d == 64) return p.form == 1 ? launch<64, 1>(p, overlap, st) : launch<64, 2>(p, overlap, st);
  return p.form == 1 ? launch<128, 1>(p, overlap, st) : launch<128, 2>(p, overlap, st);
}

}  // namespace mfa
