// chunk_q8.cu -- fa_fwd_chunk_q8's attention kernel for few query rows per K/V
// head: single tokens, speculated ones, short pieces of prompts, over a cache
// in 8 bits (q8_device.cuh).
//
// Bound: HBM, one byte per cached element.  A CTA runs one piece of a query tile's
// keys (the planner of chunk.cu); of each 128-key tile its eight warps take 16 keys
// each, and every lane copies with cp.async exactly the bytes that it will feed
// to the matrix instructions itself, so a warp streams its keys through a private
// ring without any barrier.  With two CTAs per SM 190 KB are in flight.
//
// Products are m16n8k16 in fp16 with fp32 sums.  e4m3 is exact in fp16.  A row of
// Q is scaled by a power of two into fp16 (its largest element to 2^7 .. 2^8, so
// what fp16 rounds off is below 2^-32 of it), whatever its own type.  The order of
// columns in a product is free as long as both sides agree, so a lane's 16-byte
// loads of a key are its operands of four steps; for P V the bytes of two keys
// are interleaved (two byte permutes for eight values) before they widen.
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
// A key that the masks hide from every row of the tile is never read.  One that
// some rows see and others do not is multiplied by a weight of 0 for these; where
// such a key's V holds a NaN, its product is made apart, so that it reaches the
// rows that see it and no others.
#include <climits>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chunk.h"
#include "chunk_logit.cuh"
#include "fa_device.cuh"
#include "host_util.h"
#include "mma_sync.cuh"
#include "q8_device.cuh"
#include "rope_common.cuh"

namespace mfa {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kTop = 7.f, kRaise = 15.f;  // log2 of the weights at the top

// MT: 16-row tiles of a query tile.
template <int D, int MT>
struct QCfg {
  static constexpr int kRows = 16 * MT;
  static constexpr int kCtas = MT == 1 ? 2 : 1;         // per SM
  static constexpr int kStageBytes = 2 * 16 * D;        // K and V of 16 keys
  static constexpr int kStages = (MT == 1 ? 3 : 6) * 128 / D;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kQStride = 2 * D + 16;           // bytes of a Q row
  static constexpr int kOStride = D + 4 * (D / 32);     // floats of a row of the join
  static constexpr int kQOff = kRing;
  static constexpr int kRowOff = kQOff + kRows * kQStride;           // per row: factor, keys, place, slope
  static constexpr int kSumOff = kRowOff + kRows * 5 * 4;            // ref and sum [kWarps][kRows]
  static constexpr int kExpOff = kSumOff + kWarps * kRows * 8;       // scales' exponents [kWarps][64]
  static constexpr int kOwnOff = kExpOff + kWarps * 64 * 4;
  static constexpr int kSmem = kOwnOff + 32;
  static_assert(kWarps * kRows * kOStride * 4 <= kRing, "the join's rows take the ring's place");
  static_assert(kSmem <= (kCtas == 1 ? 227 * 1024 : 113 * 1024), "shared memory budget");
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool real) {
  const uint32_t n = real ? BYTES : 0;  // zero-filled otherwise
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// No planner: the piece of CTA i (count -1: the sequence has no such tile), and the check of its lengths.
__device__ __forceinline__ ChunkPiece own_piece(const ChunkParams& p, int i) {
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

// GEN: soft-cap and / or ALiBi.
template <int D, int MT, bool GEN>
__global__ void __launch_bounds__(kThreads, QCfg<D, MT>::kCtas) chunk_q8_kernel(const __grid_constant__ ChunkParams p) {
  using C = QCfg<D, MT>;
  constexpr int NST = C::kStages, kRows = C::kRows;
  constexpr int NP = D / 64;                  // 16-byte pieces of a key of K per lane
  constexpr int kVBytes = D / 8;              // bytes of a key of V per lane
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + warp * NST * C::kStageBytes;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  float* s_fac = reinterpret_cast<float*>(smem + C::kRowOff);  // logit per dot product (GEN: without scale)
  int* s_lo = reinterpret_cast<int*>(s_fac + kRows);
  int* s_hi = s_lo + kRows;
  int* s_place = s_hi + kRows;
  float* s_slope = reinterpret_cast<float*>(s_place + kRows);
  float2* s_sum = reinterpret_cast<float2*>(smem + C::kSumOff);
  int* s_exp = reinterpret_cast<int*>(smem + C::kExpOff) + warp * 64;
  float* s_o = reinterpret_cast<float*>(smem);
  ChunkPiece* own = reinterpret_cast<ChunkPiece*>(smem + C::kOwnOff);

  wait_for_previous();
  if (p.direct) {
    if (tid == 0) *own = own_piece(p, blockIdx.x);
    __syncthreads();
  }
  const int n_pieces = p.direct ? 1 : p.counts->n_pieces;

  for (int round = 0;; ++round) {
    // one piece per round of the grid, every other round in reverse CTA order
    const int at = p.direct ? round
                            : round * (int)gridDim.x + ((round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (at >= n_pieces) break;
    const ChunkPiece w = p.direct ? *own : p.pieces[at];
    if (w.count < 0) continue;
    const int q_len = chunk_qlen(p, w.b), kv_len = p.kv_len[w.b], prefix = p.prefix ? p.prefix[w.b] : 0, off = kv_len - q_len;
    const int i0 = w.rt * p.rt_tokens, i1 = min(i0 + p.rt_tokens, q_len) - 1;
    const int head0 = w.hg * p.gp, hk = head0 / p.G;
    const int64_t qbase = p.cu_q ? (int64_t)p.cu_q[w.b] : 0, qb = p.cu_q ? 0 : w.b;
    const SinkTiles geo = row_tile_sinks(p, make_int4(0, q_len, kv_len, prefix), w.rt);
    // the keys that some row sees: at or below need_hi, and at or above need_lo or among the first `sinks`
    const int sinks = p.wl >= 0 ? p.sinks : 0;
    int need_lo, need_hi, lo_, hi_;
    chunk_row_keys(p, i0, off, kv_len, prefix, need_lo, hi_);
    chunk_row_keys(p, i1, off, kv_len, prefix, lo_, need_hi);

    // ---- Q: two rows per warp and 16-row tile, scaled into fp16
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
      const int e = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23) - 127 - 7, -100), 120) : 0;
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
    __syncthreads();

    // ---- the warp's 16 keys of tile v of the piece
    auto first_key = [&](int v) {
      const int tile = w.kt0 + v;
      return (tile + (tile >= geo.first ? geo.gap : 0)) * kKeysPerTile + 16 * warp;
    };
    auto needed = [&](int j0) { return j0 <= need_hi && (j0 + 15 >= need_lo || j0 < sinks); };
    // The pages of 32 tiles are looked up at once, one by each lane, and those of
    // the 32 after them asked for; the scales' exponents go to shared memory (two sets:
    // the copies run ahead of the products).
    int page = -1, next_page = -1;
    auto ask = [&](int v) {
      const int j0 = first_key(v);
      if (v >= w.count || !needed(j0)) return -1;
      if (!p.block_table) return w.b;
      const int pg = __ldg(p.block_table + (int64_t)w.b * p.bt_stride + fast_div(j0, p.div_page));
      if (pg < 0 || pg >= p.num_pages) {
        chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)pg);
        return -1;
      }
      return pg;
    };
    auto look_up = [&](int v) {
      page = next_page;
      const int j0 = first_key(v + lane);
      int ex = 0;
      if (page >= 0) {
        const int r = p.block_table ? j0 - fast_div(j0, p.div_page) * p.page_size : j0;
        const int64_t b = r >> p.block_shift;
        const int ke = scale_exponent(__ldg(p.ks + page * p.ks_sb + b * p.ks_ss + hk * p.ks_sh));
        const int ve = scale_exponent(__ldg(p.vs + page * p.vs_sb + b * p.vs_ss + hk * p.vs_sh));
        ex = (ke & 0xff) | ((ve & 0xff) << 8) | (1 << 16);  // (bit 16: there are keys)
      }
      s_exp[(v + lane) & 63] = ex;
      next_page = ask(v + 32 + lane);
      __syncwarp();
    };
    next_page = ask(lane);
    auto issue = [&](int v, int stage) {
      if (v < w.count) {
        if ((v & 31) == 0) look_up(v);
        const int pg = __shfl_sync(0xffffffffu, page, v & 31);
        if (pg >= 0) {
          const int j0 = first_key(v);
          const int r = p.block_table ? j0 - fast_div(j0, p.div_page) * p.page_size : j0;
          const uint8_t* kp = p.k8 + pg * p.k_sb + r * p.k_ss + hk * p.k_sh;
          const uint8_t* vp = p.v8 + pg * p.v_sb + r * p.v_ss + hk * p.v_sh;
          const uint32_t dst = ring_at + stage * C::kStageBytes;
          auto real = [&](int m) {
            const int j = j0 + m;
            return j <= need_hi && (j >= need_lo || j < sinks);
          };
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int m = g + 8 * n;
            const bool ok = real(m);
#pragma unroll
            for (int q = 0; q < NP; ++q)
              copy_async<16>(dst + ((n * NP + q) * 32 + lane) * 16, ok ? kp + m * p.k_ss + 64 * q + 16 * t : p.k8, ok);
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int m = 2 * t + (n & 1) + 8 * (n >> 1);
            const bool ok = real(m);
            copy_async<kVBytes>(dst + 16 * D + (n * 32 + lane) * kVBytes, ok ? vp + m * p.v_ss + kVBytes * g : p.v8, ok);
          }
        }
      }
      cp_async_commit();
    };

    float o[MT][D / 8][4];
    float ref[MT][2], l[MT][2], fac[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[m][i][c] = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ref[m][r] = -INFINITY;
        l[m][r] = 0.f;
        fac[m][r] = s_fac[16 * m + 8 * r + g];
      }
    }
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) issue(s, s);
    int stage = 0;
#pragma unroll 1
    for (int v = 0; v < w.count; ++v) {
      issue(v + NST - 1, stage == 0 ? NST - 1 : stage - 1);
      cp_async_wait<NST - 1>();
      const unsigned char* src = ring + stage * C::kStageBytes;
      if (++stage == NST) stage = 0;
      const int ex = s_exp[v & 63];
      if (!(ex >> 16)) continue;  // no row sees these keys
      const int ke = (int)(int8_t)ex, ve = (int)(int8_t)(ex >> 8);
      const int j0 = first_key(v);

      // ---- S = Q K^T: keys j0 + 2 t, + 1 (first tile) and + 8, + 9 (second)
      float s[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[m][n][c] = 0.f;
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(src + (q * 32 + lane) * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(src + ((NP + q) * 32 + lane) * 16);
        const uint32_t kw[2][4] = {{k0.x, k0.y, k0.z, k0.w}, {k1.x, k1.y, k1.z, k1.w}};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 qa[MT], qc[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const unsigned char* row = smem + C::kQOff + (16 * m + g) * C::kQStride + 128 * q + 32 * t + 16 * half;
            qa[m] = *reinterpret_cast<const uint4*>(row);
            qc[m] = *reinterpret_cast<const uint4*>(row + 8 * C::kQStride);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t u = kw[n][2 * half + e];
              const uint32_t b0 = e4m3x2_to_f16x2((uint16_t)u), b1 = e4m3x2_to_f16x2((uint16_t)(u >> 16));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                const uint32_t a[4] = {e ? qa[m].z : qa[m].x, e ? qc[m].z : qc[m].x, e ? qa[m].w : qa[m].y, e ? qc[m].w : qc[m].y};
                mma_bf16<true>(s[m][n], a, b0, b1);
              }
            }
        }
      }

      // ---- logits in log2 units plus V's exponent, masks, the reference
      const float kf = pow2f(ke), vf = (float)ve, per_v = pow2f(-ve);
      bool raise = false, part = false;
      float mx[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 16 * m + 8 * r + g;
          const float f = fac[m][r] * kf;
          if constexpr (GEN) {
            const float k = 2.f * p.scale_log2 * p.inv_softcap, c1 = p.softcap * kLog2e;
            const float slope = s_slope[row];
            const int place = s_place[row];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float x = s[m][n][2 * r + c] * f;
                if (p.softcap > 0.f)
                  x = p.softcap <= kPlainSoftcap ? fmaf(-2.f * c1, fast_rcp(1.f + fast_exp2(x * k)), c1) : wide_softcap(x, k, c1, p);
                else
                  x *= p.scale_log2;
                if (p.alibi) x -= slope * (float)abs(place - (j0 + 8 * n + 2 * t + c));
                s[m][n][2 * r + c] = x + vf;
              }
          } else {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) s[m][n][2 * r + c] = fmaf(s[m][n][2 * r + c], f, vf);
          }
          const int lo = s_lo[row], hi = s_hi[row];
          const bool cut = (lo > j0 && sinks < j0 + 16) || hi < j0 + 15;
          part |= cut;
          if (cut) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int j = j0 + 8 * n + 2 * t + c;
                if (!(j <= hi && (j >= lo || j < sinks))) s[m][n][2 * r + c] = -INFINITY;
              }
          }
          mx[m][r] = fmaxf(fmaxf(s[m][0][2 * r], s[m][0][2 * r + 1]), fmaxf(s[m][1][2 * r], s[m][1][2 * r + 1]));
          raise |= mx[m][r] > ref[m][r] + kRaise;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float top = mx[m][r];
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > ref[m][r] + kRaise) {
              const float up = top - kTop;
              if (ref[m][r] != -INFINITY) {
                const float f = fast_exp2(ref[m][r] - up);
                l[m][r] *= f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                  o[m][i][2 * r] *= f;
                  o[m][i][2 * r + 1] *= f;
                }
              }
              ref[m][r] = up;
            }
          }
      }

      // ---- weights
      uint32_t pa[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float base = ref[m][r] == -INFINITY ? 0.f : ref[m][r];
          float e[4];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) e[2 * n + c] = fast_exp2(s[m][n][2 * r + c] - base);
          l[m][r] = fmaf((e[0] + e[1]) + (e[2] + e[3]), per_v, l[m][r]);
          pa[m][r] = pack2<true>(e[0], e[1]);
          pa[m][2 + r] = pack2<true>(e[2], e[3]);
        }
      }

      // ---- O += P V: column i of lane group n is d = (D / 8) n + i
      uint32_t vw[4][D / 32];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const unsigned char* at_v = src + 16 * D + (n * 32 + lane) * kVBytes;
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(at_v);
          vw[n][0] = u.x; vw[n][1] = u.y; vw[n][2] = u.z; vw[n][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(at_v);
          vw[n][0] = u.x; vw[n][1] = u.y;
        }
      }
      bool apart = false;
      if (__any_sync(0xffffffffu, part)) {
        uint32_t nan = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) nan |= (vw[n][i] & 0x7f7f7f7fu) + 0x01010101u;
        apart = __any_sync(0xffffffffu, (nan & 0x80808080u) != 0);
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t x[2][2];  // [keys][columns 4 i, + 1 and + 2, + 3]
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          x[n][0] = __byte_perm(vw[2 * n][i], vw[2 * n + 1][i], 0x5140);
          x[n][1] = __byte_perm(vw[2 * n][i], vw[2 * n + 1][i], 0x7362);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t b0 = e4m3x2_to_f16x2((uint16_t)(x[0][e >> 1] >> (16 * (e & 1))));
          uint32_t b1 = e4m3x2_to_f16x2((uint16_t)(x[1][e >> 1] >> (16 * (e & 1))));
          if (apart) {
            // 1 where V is NaN, and V without those
            const uint32_t n0 = half2_bits(__hneu2(bits_half2(b0), bits_half2(b0)));
            const uint32_t n1 = half2_bits(__hneu2(bits_half2(b1), bits_half2(b1)));
            b0 &= ~__hneu2_mask(bits_half2(b0), bits_half2(b0));
            b1 &= ~__hneu2_mask(bits_half2(b1), bits_half2(b1));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              float hit[4] = {0.f, 0.f, 0.f, 0.f};
              mma_bf16<true>(hit, pa[m], n0, n1);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (hit[c] > 0.f) o[m][4 * i + e][c] = __int_as_float(0x7fffffff);
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) mma_bf16<true>(o[m][4 * i + e], pa[m], b0, b1);
        }
      }
    }

    // ---- the warps' rows, joined
    __syncthreads();  // the ring is read
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * m + 8 * r + g;
        float sum = l[m][r];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (t == 0) s_sum[warp * kRows + row] = make_float2(ref[m][r], sum);
        // this lane's columns: lane groups 2 t and 2 t + 1, D / 8 each, in runs of 32 padded by 4
        float* dst = s_o + (warp * kRows + row) * C::kOStride;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < D / 8; i += 4) {
            const int d = (2 * t + c) * (D / 8) + i;
            *reinterpret_cast<float4*>(dst + d + 4 * (d / 32)) =
                make_float4(o[m][i][2 * r + c], o[m][i + 1][2 * r + c], o[m][i + 2][2 * r + c], o[m][i + 3][2 * r + c]);
          }
      }
    __syncthreads();
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
        const float4 v = *reinterpret_cast<const float4*>(s_o + (k * kRows + row) * C::kOStride + d + 4 * (d / 32));
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
    __syncthreads();  // the next piece overwrites the rows
  }
}

template <int D, int MT, bool GEN>
cudaError_t launch(const ChunkParams& p, bool overlap, cudaStream_t st) {
  using C = QCfg<D, MT>;
  const cudaError_t e = ensure_smem_attr<chunk_q8_kernel<D, MT, GEN>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_overlapped(chunk_q8_kernel<D, MT, GEN>, (unsigned)p.grid, kThreads, C::kSmem, overlap, st, p);
}
template <int D, int MT>
cudaError_t launch(const ChunkParams& p, bool overlap, cudaStream_t st) {
  return (p.softcap > 0.f || p.alibi) ? launch<D, MT, true>(p, overlap, st) : launch<D, MT, false>(p, overlap, st);
}

}  // namespace

cudaError_t launch_chunk_q8(const ChunkParams& p, bool overlap, cudaStream_t st) {
  if (p.d == 64) return p.form == 1 ? launch<64, 1>(p, overlap, st) : launch<64, 2>(p, overlap, st);
  return p.form == 1 ? launch<128, 1>(p, overlap, st) : launch<128, 2>(p, overlap, st);
}

}  // namespace mfa
