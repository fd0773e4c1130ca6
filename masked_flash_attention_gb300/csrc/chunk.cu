// chunk.cu -- fa_fwd_chunk: attention of a chunk of new tokens per sequence over
// a paged (or padded) KV cache.  This file holds the entry points, the planner
// kernel, which cuts the step into pieces of work from the sequences' actual
// lengths, and the kernel that joins the pieces of a unit; the attention itself
// is chunk_sm103.cu.
//
// A unit is one query tile of one head group; units are independent and cover a
// run of key tiles that the pair rules leave.  A serving step's units differ
// widely (prompts' pieces beside single tokens, caches of any length), and may
// be far fewer than the SMs, so the planner chooses one length T in key tiles,
// cuts units longer than T into even pieces, and lists all pieces longest first;
// the attention kernel's CTAs take them in rounds.  The pieces of a cut unit
// leave normalised fp32 rows and their log-sum-exp, which are joined by
// O = sum 2^(L_k - L) O_k, 2^L = sum 2^(L_k), in the order of the keys: the
// result does not depend on scheduling.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "chunk.h"
#include "fa_device.cuh"

namespace mfa {
namespace {

constexpr int kPlanThreads = 256;  // (512 and 1024 took longer, over their barriers)
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBins = 256;
constexpr int kSeqSmem = 1024, kTileSmem = 1280;  // sequences and row tiles kept in shared memory, more in the workspace
constexpr int kTailFlag = 1 << 30;                // in a row tile's second word: its units are cut as tail
// Cost model, in key tiles (about 0.8 us of a CTA): what a piece costs beside
// its tiles (its start, Q, the epilogue), what leaving a partial and joining it
// costs more, and what there being any to join does.
constexpr float kPieceCost = 3.f, kPartialCost = 1.5f, kJoinCost = 4.f;
constexpr int kMaxTailCut = 8;
constexpr int kMaxSeqTiles = 1 << 22;  // row tiles of one sequence

// Block-wide exclusive prefix sum; `total` gets the sum.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    const int y = s_warp[w];
    if (w < warp) before += y;
    total += y;
  }
  __syncthreads();
  return x - v + before;
}

// One CTA cuts the step into pieces (see the head of this file).  It runs before
// everything else and its code once, from a cold instruction cache, so it is kept
// short: loops not unrolled, one warp-wide step where one will do (64 single
// tokens: 5.7 us, of which 1.2 the first loads; unrolled, with 1024 threads, 7.6).
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ int4 s_seq[kSeqSmem];
  __shared__ int4 s_tile[kTileSmem];
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[kPlanWarps];
  __shared__ float s_cost[32];
  __shared__ int s_T[32];
  __shared__ int s_nmax[kPlanWarps];
  __shared__ unsigned int s_work[kPlanWarps];
  __shared__ int s_slots, s_splits, s_bin, s_before;
  let_dependents_start();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int4* const seqs = p.n_seq <= kSeqSmem ? s_seq : p.seqs;
  if (tid == 0) {
    s_slots = s_splits = 0;
  }

  // ---- row tiles per sequence; sequences whose lengths do not fit get none
  int R = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < p.n_seq; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int nt = 0;
    int4 q = make_int4(0, 0, 0, 0);
    if (s < p.n_seq) {
      if (chunk_seq(p, s, q)) nt = (q.y + p.rt_tokens - 1) / p.rt_tokens;
      else chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)s);
    }
    int total;
    q.x = R + block_scan(nt, s_warp, total);
    if (s < p.n_seq) seqs[s] = q;
    // (a sum that overlapping cu_seqlens_q grow stays in 32 bits: total is at most
    // 256 * kMaxSeqTiles, and past max_rtiles nothing depends on R)
    R = min(R + total, p.max_rtiles + 1);
  }
  if (R > p.max_rtiles) {  // overlapping cu_seqlens_q: more tiles than the workspace lists
    if (tid == 0) chunk_error(p, FA_ERR_DEVICE_BOUNDS, (uint32_t)p.n_seq);
    R = p.max_rtiles;
  }
  int4* const tiles = R <= kTileSmem ? s_tile : p.rtiles;
  __syncthreads();

  // ---- key tiles of each row tile
  int nmax = 0;
  unsigned int work = 0;
#pragma unroll 1
  for (int r = tid; r < R; r += kPlanThreads) {
    int lo = 0, hi = p.n_seq;  // the last sequence whose first tile is at or before r
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seqs[mid].x <= r) lo = mid;
      else hi = mid;
    }
    const int4 q = seqs[lo];
    int kt0, n;
    row_tile_keys(p, q, r - q.x, kt0, n);
    tiles[r] = make_int4(lo, r - q.x, kt0, n);
    nmax = max(nmax, n);
    work += n;
  }
  nmax = __reduce_max_sync(0xffffffffu, nmax);
  work = __reduce_add_sync(0xffffffffu, work);
  if (lane == 0) {
    s_nmax[warp] = nmax;
    s_work[warp] = work;
  }
  s_hist[tid] = 0;
  __syncthreads();
  float fwork = 0.f;
#pragma unroll 1
  for (int w = 0; w < kPlanWarps; ++w) {
    nmax = max(nmax, s_nmax[w]);
    fwork += (float)s_work[w];
  }
  fwork *= p.n_hg;
  const float P = (float)p.grid;
  const int units = R * p.n_hg;

  // ---- the length T, of 32 candidates: whole units; t0 tiles, which would fill
  // one round of the grid evenly, up to twice as many (room for the units' odd
  // lengths), and the same for two, three and four rounds
  int T = max(nmax, 1);
  if (p.max_slots > 0 && nmax > 1) {
    const float t0 = fwork / P;
#pragma unroll 1
    for (int j = warp; j < 32; j += kPlanWarps) {
      float f;
      if (j <= 16) f = 1.f + (j - 1) / 16.f;
      else if (j <= 24) f = (1.f + (j - 17) / 8.f) / 2.f;
      else if (j <= 28) f = (1.f + (j - 25) / 4.f) / 3.f;
      else f = (1.f + (j - 29) / 4.f) / 4.f;
      const int t = j == 0 ? nmax : min(max(1, (int)ceilf(f * t0)), nmax);
      float cost = 3e38f;
      if (j == 0 || t < nmax) {
        int m = 0, part = 0, longest = 0;
        const float per_t = 1.f / t;
#pragma unroll 1
        for (int r = lane; r < R; r += 32) {
          // (quotients rounded up as floats: a cost may be off by a piece)
          const float n = (float)tiles[r].w;
          const int k = n <= t ? 1 : (int)ceilf(n * per_t);
          m += k;
          if (k > 1) part += k;
          longest = max(longest, (int)ceilf(__fdividef(n, (float)k)));
        }
        m = __reduce_add_sync(0xffffffffu, m) * p.n_hg;
        part = __reduce_add_sync(0xffffffffu, part) * p.n_hg;
        longest = __reduce_max_sync(0xffffffffu, longest);
        const float total = fwork + kPieceCost * m + kPartialCost * part;
        cost = fmaxf(longest + kPieceCost + (part ? kPartialCost : 0.f),
                     (total + (ceilf(m / P) * P - m) * total / m) / P) + (part ? kJoinCost : 0.f);
        if (part > p.max_slots) cost = 3e38f;
      }
      if (lane == 0) {
        s_cost[j] = cost;
        s_T[j] = t;
      }
    }
    __syncthreads();
    float best = s_cost[lane];
    int at = lane;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      const float c = __shfl_xor_sync(0xffffffffu, best, o);
      const int w = __shfl_xor_sync(0xffffffffu, at, o);
      if (c < best || (c == best && w < at)) {
        best = c;
        at = w;
      }
    }
    T = s_T[at];
  }
  int shift = 0;
#pragma unroll 1
  while ((T >> shift) >= kBins) ++shift;
  auto bin_of = [&](int len) { return kBins - 1 - (len >> shift); };

  // ---- whole units that leave a last round mostly empty: as many row tiles as
  // that round holds, the shortest ones (in their order where they are equally
  // long), are cut in `cut` and fill it
  int cut = 1;
  const int last = units % p.grid;  // units of the last round
  if (T >= nmax && nmax > 1 && units > p.grid && last > 0 && 2 * last <= p.grid) {
    const int tails = (last + p.n_hg - 1) / p.n_hg;  // row tiles
    cut = min(min(p.grid / (tails * p.n_hg), kMaxTailCut), p.max_slots / (tails * p.n_hg));
    if (cut >= 2) {
#pragma unroll 1
      for (int r = tid; r < R; r += kPlanThreads) atomicAdd(&s_hist[bin_of(tiles[r].w)], 1);
      __syncthreads();
      const int mine = s_hist[tid];
      int total;
      const int before = block_scan(mine, s_warp, total);
      if (before < R - tails + 1 && before + mine >= R - tails + 1) {  // holds the first tail tile
        s_bin = tid;
        s_before = before;
      }
      s_hist[tid] = 0;
      __syncthreads();
      // of that bin's tiles, in their order, the first `whole` stay
      const int bin = s_bin, whole = R - tails - s_before;
      int seen = 0;
      bool worth = false;
#pragma unroll 1
      for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
        const int r = r0 + tid;
        const int b = r < R ? bin_of(tiles[r].w) : -1;
        const int rank = seen + block_scan(b == bin ? 1 : 0, s_warp, total);
        if (r < R && (b > bin || (b == bin && rank >= whole))) {
          tiles[r].y |= kTailFlag;
          // (the round ends with its longest piece)
          worth |= tiles[r].w * (1.f - 1.f / cut) > kPartialCost + kJoinCost;
        }
        seen += total;
      }
      if (!__syncthreads_or(worth)) cut = 1;
    } else {
      cut = 1;
    }
  }
  auto pieces_of = [&](int4 t) {
    if (t.w > T) return (t.w + T - 1) / T;
    return (cut > 1 && (t.y & kTailFlag)) ? max(1, min(cut, t.w)) : 1;
  };

  // ---- list the pieces, longest first (a counting sort by length)
#pragma unroll 1
  for (int r = tid; r < R; r += kPlanThreads) {
    const int4 t = tiles[r];
    const int k = pieces_of(t), len = t.w / k, more = t.w - len * k;
    if (more) atomicAdd(&s_hist[bin_of(len + 1)], more * p.n_hg);
    atomicAdd(&s_hist[bin_of(len)], (k - more) * p.n_hg);
  }
  __syncthreads();
  int total;
  const int start = block_scan(s_hist[tid], s_warp, total);
  s_hist[tid] = start;
  __syncthreads();
#pragma unroll 1
  for (int u = tid; u < units; u += kPlanThreads) {
    const int r = fast_div(u, p.div_hg), hg = u - r * p.n_hg;
    const int4 t = tiles[r];
    const int k = pieces_of(t), len = t.w / k, more = t.w - len * k, rt = t.y & ~kTailFlag;
    int slot0 = -1;
    if (k > 1) {
      slot0 = atomicAdd(&s_slots, k);
      ChunkSplit sp;
      sp.b = t.x; sp.rt = rt; sp.hg = hg; sp.slot0 = slot0; sp.n = k;
      sp.pad[0] = sp.pad[1] = sp.pad[2] = 0;
      p.splits[atomicAdd(&s_splits, 1)] = sp;
    }
    int at = t.z;
#pragma unroll 1
    for (int i = 0; i < k; ++i) {
      const int c = len + (i < more ? 1 : 0);
      int4* dst = reinterpret_cast<int4*>(p.pieces + atomicAdd(&s_hist[bin_of(c)], 1));
      dst[0] = make_int4(t.x, rt, hg, at);
      dst[1] = make_int4(c, k > 1 ? slot0 + i : -1, 0, 0);
      at += c;
    }
  }
  __syncthreads();
  if (tid == 0) {
    ChunkCounts c;
    c.n_pieces = total; c.n_slots = s_slots; c.n_splits = s_splits; c.n_rtiles = R;
    *p.counts = c;
  }
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

// A group of D / 4 threads per row of a split unit: the weights of its pieces
// from their log-sum-exps, then the weighted sum of their rows, four columns per
// thread.  Bound by the latency of its loads (a few L2 reads one behind the
// other), so the rows get as many threads as there are and the first pieces'
// rows are asked for before the weights are known.
template <int D, bool F16>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes;  // threads per row, rows per block
  constexpr int kAhead = 4;
  const int c = threadIdx.x % kLanes;
  wait_for_previous();
  const int n_rows = p.counts->n_splits * kChunkRows;
  for (int w = blockIdx.x * kRows + threadIdx.x / kLanes; w < n_rows; w += gridDim.x * kRows) {
    const ChunkSplit sp = p.splits[w / kChunkRows];
    const int row = w % kChunkRows;
    const int tok = fast_div(row, p.div_gp), i = sp.rt * p.rt_tokens + tok;
    if (tok >= p.rt_tokens || i >= chunk_qlen(p, sp.b)) continue;
    const float* po = p.part_o + ((int64_t)sp.slot0 * kChunkRows + row) * D + 4 * c;
    const float* pl = p.part_lse + (int64_t)sp.slot0 * kChunkRows + row;
    float4 v[kAhead];
    float ls[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool have = k < sp.n;
      v[k] = have ? *reinterpret_cast<const float4*>(po + (int64_t)k * kChunkRows * D) : make_float4(0.f, 0.f, 0.f, 0.f);
      ls[k] = have ? pl[k * kChunkRows] : -INFINITY;
    }
    float mx = fmaxf(fmaxf(ls[0], ls[1]), fmaxf(ls[2], ls[3]));
    for (int k = kAhead; k < sp.n; ++k) mx = fmaxf(mx, pl[k * kChunkRows]);
    const float ref = mx == -INFINITY ? 0.f : mx;  // no piece has a key of the row: all weights 0
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float l, float4 x) {
      const float f = fast_exp2(l - ref);
      sum += f;
      o.x += f * x.x; o.y += f * x.y; o.z += f * x.z; o.w += f * x.w;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) add(ls[k], v[k]);
#pragma unroll 4
    for (int k = kAhead; k < sp.n; ++k)
      add(pl[k * kChunkRows], *reinterpret_cast<const float4*>(po + (int64_t)k * kChunkRows * D));
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int h = sp.hg * p.gp + row - tok * p.gp;
    const int64_t qrow = (p.cu_q ? p.cu_q[sp.b] : 0) + i, ob = p.cu_q ? 0 : sp.b;
    *reinterpret_cast<uint2*>(p.o + ob * p.o_sb + qrow * p.o_ss + (int64_t)h * p.o_sh + 4 * c) =
        make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
    if (c == 0)
      p.lse[ob * p.lse_sb + (int64_t)h * p.lse_sh + qrow * p.lse_ss] = sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * kLn2;
  }
}

// Arguments checked, geometry and workspace laid out (offsets from `base`,
// which may be null for a plan).
int plan_chunk(const fa_tensor* q, const fa_tensor* k, const fa_tensor* v, const fa_tensor* out, const fa_tensor* lse,
               const fa_tensor* cu_q, const fa_tensor* seqlens_k, const fa_tensor* block_table,
               const fa_tensor* prefix, int32_t wl, int32_t wr, float softcap, float scale, int32_t causal,
               const fa_opts* opts, ChunkParams* P, fa_plan* pub) {
  if (!q || !k || !v || !out || !lse || !seqlens_k || !opts) return FA_ERR_INVALID_ARG;
  memset(P, 0, sizeof(*P));
  memset(pub, 0, sizeof(*pub));
  ChunkParams& p = *P;
  int rc;
  const int nd = cu_q ? 3 : 4;
  if ((rc = check_bf16(q, nd)) || (rc = check_bf16(out, nd)) || (rc = check_bf16(k, 4)) || (rc = check_bf16(v, 4)))
    return rc;
  int64_t n_seq, Sq;
  if (cu_q) {
    if (cu_q->ndim != 1 || cu_q->shape[0] < 1) return FA_ERR_INVALID_ARG;
    n_seq = cu_q->shape[0] - 1;
    if ((rc = check_i32_vec(cu_q, n_seq + 1))) return rc;
    Sq = opts->max_seqlen_q;
    if (Sq < 0 || (Sq == 0 && q->shape[0] > 0)) return FA_ERR_INVALID_ARG;
    p.cu_q = static_cast<const int32_t*>(cu_q->data);
    p.tot_q = q->shape[0];
    p.q_sb = q->stride[0]; p.q_ss = q->stride[0]; p.q_sh = q->stride[1];
    p.o_sb = 0; p.o_ss = out->stride[0]; p.o_sh = out->stride[1];
  } else {
    n_seq = q->shape[0];
    Sq = q->shape[1];
    p.q_sb = q->stride[0]; p.q_ss = q->stride[1]; p.q_sh = q->stride[2];
    p.o_sb = out->stride[0]; p.o_ss = out->stride[1]; p.o_sh = out->stride[2];
  }
  const int64_t Hq = q->shape[nd - 2], d = q->shape[nd - 1], Hkv = k->shape[2], Sk = opts->max_seqlen_k;
  if ((d != 64 && d != 128) || k->shape[3] != d || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (n_seq > INT32_MAX / 64 || Sq > INT32_MAX / 64 || Sk < 0 || Sk > INT32_MAX / 64 || Hq > INT32_MAX / 1024)
    return FA_ERR_INVALID_ARG;
  for (int i = 0; i < nd; ++i) {
    if (out->shape[i] != q->shape[i]) return FA_ERR_INVALID_ARG;
    if (out->shape[i] > 1 && out->stride[i] == 0) return FA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 4; ++i)
    if (v->shape[i] != k->shape[i]) return FA_ERR_INVALID_ARG;
  if (k->dtype != q->dtype || v->dtype != q->dtype || out->dtype != q->dtype) return FA_ERR_INVALID_ARG;
  if ((rc = check_i32_vec(seqlens_k, n_seq))) return rc;
  if (prefix && ((rc = check_i32_vec(prefix, n_seq)) || !causal)) return FA_ERR_INVALID_ARG;
  // ---- LSE
  if (!lse->data || lse->dtype != FA_DTYPE_F32 || (reinterpret_cast<uintptr_t>(lse->data) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  if (cu_q) {
    if (lse->ndim != 2 || lse->shape[0] != Hq || lse->shape[1] != p.tot_q) return FA_ERR_INVALID_ARG;
    p.lse_sb = 0; p.lse_sh = lse->stride[0]; p.lse_ss = lse->stride[1];
  } else {
    if (lse->ndim != 3 || lse->shape[0] != n_seq || lse->shape[1] != Hq || lse->shape[2] != Sq)
      return FA_ERR_INVALID_ARG;
    p.lse_sb = lse->stride[0]; p.lse_sh = lse->stride[1]; p.lse_ss = lse->stride[2];
  }
  // ---- cache
  if (block_table) {
    const int64_t page = k->shape[1];
    if (!block_table->data || block_table->dtype != FA_DTYPE_I32 || block_table->ndim != 2 ||
        block_table->shape[0] != n_seq || block_table->stride[1] != 1 || block_table->stride[0] < 0 ||
        block_table->shape[1] < 1 || page < 1 || page > INT32_MAX / 2 || k->shape[0] > INT32_MAX)
      return FA_ERR_INVALID_ARG;
    if (Sk > block_table->shape[1] * page || (Sk > 0 && k->shape[0] == 0)) return FA_ERR_INVALID_ARG;
    p.block_table = static_cast<const int32_t*>(block_table->data);
    p.bt_stride = block_table->stride[0];
    p.page_size = (int32_t)page;
    p.num_pages = (int32_t)k->shape[0];
    // rows per copy: the largest power of two that divides a page and a tile
    p.box_rows = (int32_t)std::min<int64_t>(page & -page, kKeysPerTile);
  } else {
    // a padded cache is one page per sequence
    if (k->shape[0] != n_seq || Sk > k->shape[1]) return FA_ERR_INVALID_ARG;
    p.page_size = INT32_MAX / 2;
    p.num_pages = (int32_t)n_seq;
    p.box_rows = kKeysPerTile;
  }
  while ((1 << p.box_shift) < p.box_rows) ++p.box_shift;
  p.div_page = make_fastdiv((uint32_t)p.page_size);
  p.cache_rows = k->shape[1];
  p.cache_outer = k->shape[0];
  // TMA reads q and the cache: no stride of 0 along more than one element
  const fa_tensor* in[3] = {q, k, v};
  for (const fa_tensor* t : in)
    for (int i = 0; i < t->ndim; ++i)
      if (t->shape[i] > 1 && t->stride[i] == 0) return FA_ERR_UNSUPPORTED;
  p.k_sb = k->stride[0]; p.k_ss = k->stride[1]; p.k_sh = k->stride[2];
  p.v_sb = v->stride[0]; p.v_ss = v->stride[1]; p.v_sh = v->stride[2];
  // ---- scalars
  if (wl < -1 || wr < -1 || !(softcap >= 0.f) || !std::isfinite(softcap) || !std::isfinite(scale))
    return FA_ERR_INVALID_ARG;
  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)d);
  p.q = static_cast<const uint16_t*>(q->data);
  p.k = static_cast<const uint16_t*>(k->data);
  p.v = static_cast<const uint16_t*>(v->data);
  p.o = static_cast<uint16_t*>(out->data);
  p.lse = static_cast<float*>(lse->data);
  p.kv_len = static_cast<const int32_t*>(seqlens_k->data);
  p.prefix = prefix ? static_cast<const int32_t*>(prefix->data) : nullptr;
  p.n_seq = (int32_t)n_seq;
  p.Sq = (int32_t)Sq;
  p.Sk = (int32_t)Sk;
  p.Hq = (int32_t)Hq;
  p.G = (int32_t)(Hq / Hkv);
  p.d = (int32_t)d;
  p.f16 = q->dtype == FA_DTYPE_F16;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.softcap = softcap;
  p.inv_softcap = softcap > 0.f ? 1.f / softcap : 0.f;
  p.alibi = static_cast<const float*>(opts->alibi_slopes);
  p.causal = causal ? 1 : 0;
  // (lengths stay below 2^25, so a wider window is no window; sums with it stay in 32 bits)
  p.wl = std::min(wl, 1 << 30);
  p.wr = std::min(wr, 1 << 30);
  p.debug_flags = opts->debug_flags;
  // q-heads packed into a query tile: as many of a K/V head's as divide them
  // and leave at most an eighth of the tile empty
  p.gp = 1;
  for (int g = 1; g <= p.G && g <= kChunkRows; ++g)
    if (p.G % g == 0 && g * (kChunkRows / g) >= 112) p.gp = g;
  p.rt_tokens = kChunkRows / p.gp;
  p.n_hg = p.Hq / p.gp;
  // few rows in every sequence: query tiles of at most 32 rows, and the kernel
  // form that deals each key tile's keys to the tile's four quarters
  p.narrow = Sq > 0 && Sq * p.gp <= 32;
  if (p.narrow) p.rt_tokens = 32 / p.gp;
  // d = 64: two CTAs per SM overlap their units' ends, which short units need;
  // one CTA with two softmax warpgroups keeps the tensor cores fed better along
  // long ones (two and one: 8 x 512 tokens, 12 heads, over 512 keys 24.0 and 26.6
  // us, over 4096 keys 95 and 87; 64 single tokens over up to 1500 keys 44 and 48)
  p.pair = d == 64 && Sk <= (p.narrow ? 2048 : 1024);
  p.div_gp = make_fastdiv((uint32_t)p.gp);
  p.div_hg = make_fastdiv((uint32_t)p.n_hg);

  // ---- bounds of the work, workspace
  int64_t rtiles = n_seq * ((Sq + p.rt_tokens - 1) / p.rt_tokens);
  if (cu_q) rtiles = std::min(rtiles, p.tot_q / p.rt_tokens + n_seq);
  const int64_t longest = cu_q ? std::min(Sq, p.tot_q) : Sq;
  if (rtiles * p.n_hg > (1 << 27) || (longest + p.rt_tokens - 1) / p.rt_tokens > kMaxSeqTiles) return FA_ERR_INVALID_ARG;
  const int64_t units = rtiles * p.n_hg, n_kt = std::max<int64_t>(1, (Sk + kKeysPerTile - 1) / kKeysPerTile);
  const int64_t ctas = (int64_t)sm_count() * (p.pair ? 2 : 1);
  // partials: at most two rounds of the grid, and no more than all tiles alone;
  // none where no sequence has more than 8 key tiles: such units then need no
  // planner either (below).  One token over 700 keys, 6 tiles, in a graph: cut in
  // six and joined 13.3 us, whole with the planner 14.0, whole without it 10.2.
  // None either for more tiles than 32-bit sums hold, on which the planner's bound
  // on the partials rests (there are thousands of units then).
  const int64_t slots = n_kt > 8 && rtiles * n_kt <= INT32_MAX ? std::min<int64_t>(2 * ctas, units * n_kt) : 0;
  const int64_t pieces = units + slots;
  p.max_rtiles = (int32_t)rtiles;
  p.max_slots = (int32_t)slots;
  p.grid = (int32_t)std::min<int64_t>(ctas, std::max<int64_t>(1, pieces));
  // Few short units: no planner, each CTA works out its own piece, one per row
  // tile that a sequence may have and head group (one token that sees 60 keys: 7.3
  // us in a graph, with the planner 10.8).  More units than CTAs are left to
  // the planner's order: 8 x 1024 tokens of 12 heads, 768 units of 1 to 8 tiles,
  // took 42 us in turn, 34 us longest first.
  const int64_t all = n_seq * ((Sq + p.rt_tokens - 1) / p.rt_tokens) * p.n_hg;
  p.direct = slots == 0 && all <= ctas ? (int32_t)all : 0;
  if (p.direct) p.grid = p.direct;
  size_t off = kWsHeadBytes;
  unsigned char* base = static_cast<unsigned char*>(opts->workspace);
  auto take = [&](size_t bytes) {
    unsigned char* at = base + off;
    off = align_up(off + bytes);
    return at;
  };
  p.ws = reinterpret_cast<WsHeader*>(base);
  p.counts = reinterpret_cast<ChunkCounts*>(take(sizeof(ChunkCounts)));
  p.seqs = reinterpret_cast<int4*>(take((size_t)n_seq * sizeof(int4)));
  p.rtiles = reinterpret_cast<int4*>(take((size_t)rtiles * sizeof(int4)));
  p.pieces = reinterpret_cast<ChunkPiece*>(take((size_t)pieces * sizeof(ChunkPiece)));
  p.splits = reinterpret_cast<ChunkSplit*>(take((size_t)(slots / 2) * sizeof(ChunkSplit)));
  p.part_lse = reinterpret_cast<float*>(take((size_t)slots * kChunkRows * 4));
  p.part_o = reinterpret_cast<float*>(take((size_t)slots * kChunkRows * d * 4));

  pub->path = FA_PATH_PREFILL;
  pub->n_seq = p.n_seq;
  pub->n_heads_sched = p.n_hg;
  pub->n_row_tiles = (int32_t)((Sq + p.rt_tokens - 1) / p.rt_tokens);
  pub->rows_per_tile = p.rt_tokens;
  pub->keys_per_tile = kKeysPerTile;
  pub->n_k_tiles = (int32_t)n_kt;
  pub->n_splits = p.max_slots;
  pub->n_items = units;
  pub->n_kernels = units > 0 ? 1 + (p.direct == 0) + (slots > 0) : 0;
  pub->workspace_bytes = off;
  return FA_OK;
}

template <int D, bool F16>
cudaError_t launch_join(const ChunkParams& p, bool overlap, cudaStream_t st) {
  const int64_t rows = (int64_t)p.max_slots / 2 * kChunkRows;
  const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(rows / (1024 / D), sm_count() * 8));
  return launch_overlapped(chunk_join_kernel<D, F16>, blocks, 256, 0, overlap, st, p);
}

}  // namespace
}  // namespace mfa

using namespace mfa;

extern "C" {

int fa_fwd_chunk(const fa_tensor* q, const fa_tensor* k_cache, const fa_tensor* v_cache, const fa_tensor* out,
                 const fa_tensor* lse, const fa_tensor* cu_seqlens_q, const fa_tensor* seqlens_k,
                 const fa_tensor* block_table, const fa_tensor* prefix_lens, int32_t window_left,
                 int32_t window_right, float softcap, float scale, int32_t causal, const fa_opts* opts) {
  ChunkParams p;
  fa_plan pub;
  int rc = plan_chunk(q, k_cache, v_cache, out, lse, cu_seqlens_q, seqlens_k, block_table, prefix_lens, window_left,
                      window_right, softcap, scale, causal, opts, &p, &pub);
  if (rc != FA_OK) return rc;
  if (!opts->workspace || (reinterpret_cast<uintptr_t>(opts->workspace) % kAlign) != 0 ||
      opts->workspace_bytes < pub.workspace_bytes)
    return FA_ERR_WORKSPACE;
  if ((rc = check_device()) != FA_OK) return rc;
  TraceRange tr("mfa.fwd_chunk");
  cudaStream_t st = static_cast<cudaStream_t>(opts->stream);
  cudaError_t e = cudaSuccess;
  auto record = [&](void* ev) {
    if (e == cudaSuccess && ev) e = cudaEventRecord(static_cast<cudaEvent_t>(ev), st);
  };
  const bool any = pub.n_items > 0;
  // (events between the kernels would be recorded late if these overlapped)
  const bool overlap = !opts->event_begin && !opts->event_attn_end;
  if (any && !p.direct) {
    chunk_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
    e = cudaGetLastError();
  }
  record(opts->event_begin);
  if (any && e == cudaSuccess) e = p.f16 ? launch_chunk_attn_f16(p, overlap && !p.direct, st) : launch_chunk_attn(p, overlap && !p.direct, st);
  record(opts->event_attn_end);
  if (any && e == cudaSuccess && p.max_slots > 0) {
    if (p.d == 64) e = p.f16 ? launch_join<64, true>(p, overlap, st) : launch_join<64, false>(p, overlap, st);
    else e = p.f16 ? launch_join<128, true>(p, overlap, st) : launch_join<128, false>(p, overlap, st);
  }
  record(opts->event_end);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

int fa_fwd_chunk_plan(const fa_tensor* q, const fa_tensor* k_cache, const fa_tensor* v_cache, const fa_tensor* out,
                      const fa_tensor* lse, const fa_tensor* cu_seqlens_q, const fa_tensor* seqlens_k,
                      const fa_tensor* block_table, const fa_tensor* prefix_lens, int32_t window_left,
                      int32_t window_right, float softcap, float scale, int32_t causal, const fa_opts* opts,
                      fa_plan* plan_out) {
  ChunkParams p;
  fa_plan pub;
  int rc = plan_chunk(q, k_cache, v_cache, out, lse, cu_seqlens_q, seqlens_k, block_table, prefix_lens, window_left,
                      window_right, softcap, scale, causal, opts, &p, &pub);
  if (rc == FA_OK && plan_out) *plan_out = pub;
  return rc;
}

}  // extern "C"
