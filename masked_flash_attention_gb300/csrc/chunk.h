// chunk.h -- parameters of fa_fwd_chunk, shared by its planner, its attention
// kernel and its combine kernel.
#pragma once

#include <cstdint>

#include "fa_internal.h"

namespace mfa {

constexpr int kChunkRows = 128;  // rows of a query tile (tcgen05 M)

// A piece of work: one query tile of one group of q-heads over a run of key
// tiles (two 16-byte words in the workspace).
struct ChunkPiece {
  int32_t b, rt, hg;   // sequence, row tile, head group
  int32_t kt0, count;  // key tiles kt0 .. kt0 + count - 1
  int32_t slot;        // where its partial rows go; -1: it holds all the unit's keys
  int32_t pad[2];
};
static_assert(sizeof(ChunkPiece) == 32, "two 16-byte loads");

// A unit whose keys were split: its pieces' partials are slots slot0 .. slot0 + n - 1.
struct ChunkSplit {
  int32_t b, rt, hg, slot0, n, pad[3];
};

struct ChunkCounts {
  int32_t n_pieces, n_slots, n_splits, n_rtiles;
};

// A query tile's 128 rows are (token, q-head) pairs: `rt_tokens` tokens of `gp`
// q-heads that share a K/V head, row = token * gp + head, so that a K/V tile
// is read once for all of them and a few tokens still fill the tile.
struct ChunkParams {
  uint16_t* o;
  float* lse;
  int64_t o_sb, o_ss, o_sh, lse_sb, lse_sh, lse_ss;
  const int32_t* cu_q;         // nullable
  const int32_t* kv_len;       // [n_seq]
  const int32_t* prefix;       // nullable [n_seq]
  const int32_t* block_table;  // nullable: padded cache
  int64_t bt_stride;
  int32_t page_size, num_pages, box_rows, box_shift;  // rows per TMA box = 2^box_shift
  FastDiv div_page;
  int32_t n_seq, Sq, Sk;  // Sq/Sk: fixed or maximum lengths
  int64_t tot_q;
  int32_t Hq, G, gp, rt_tokens, n_hg;  // G = Hq / Hkv; n_hg = Hq / gp
  FastDiv div_gp, div_hg;
  int32_t narrow;  // no unit has more than 32 rows
  int32_t pair;    // d = 64: two CTAs with one softmax warpgroup each per SM
  int32_t d, f16;
  float scale, scale_log2, softcap, inv_softcap;
  const float* alibi;
  int32_t causal, wl, wr;
  uint32_t debug_flags;
  // workspace
  WsHeader* ws;
  ChunkCounts* counts;
  int4* seqs;         // [n_seq] {first row tile, q_len, kv_len, prefix} (many sequences)
  int4* rtiles;       // [max_rtiles] {sequence, row tile, first key tile, key tiles} (many row tiles)
  ChunkPiece* pieces;
  ChunkSplit* splits;
  float* part_o;      // [max_slots][128][d]
  float* part_lse;    // [max_slots][128] log2 units
  int32_t max_rtiles, max_slots, grid;
  int32_t direct;  // > 0: this many pieces, one per CTA, which works it out itself (no planner)
  // layouts for the tensor maps (element strides)
  const uint16_t *q, *k, *v;
  int64_t q_sb, q_ss, q_sh, k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;
  int64_t cache_rows, cache_outer;  // page_size x num_pages, or cap x n_seq
};

// `overlap`: the kernel may start while the one before it on the stream runs
// (programmatic dependent launch; it waits for that one's results itself).
cudaError_t launch_chunk_attn(const ChunkParams& p, bool overlap, cudaStream_t st);      // bf16
cudaError_t launch_chunk_attn_f16(const ChunkParams& p, bool overlap, cudaStream_t st);  // fp16

#ifdef __CUDACC__
// Launch with or without overlap of the preceding kernel's end.
template <typename... Args>
inline cudaError_t launch_overlapped(void (*kern)(Args...), unsigned grid, unsigned block, size_t smem, bool overlap,
                                     cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, args...);
}

// Lets a dependent kernel that may overlap start; waits for the kernel before
// (at once when it did not overlap).
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

#ifdef __CUDACC__
__device__ __forceinline__ int chunk_qlen(const ChunkParams& p, int b) {
  return p.cu_q ? (p.cu_q[b + 1] - p.cu_q[b]) : p.Sq;
}

// Keys [lo, hi] that query row i (token) of a sequence may see: the pair rules
// of fa_fwd, with the first `prefix` keys exempt from the causal one.
__device__ __forceinline__ void chunk_row_keys(const ChunkParams& p, int i, int off, int kv_len, int prefix, int& lo,
                                               int& hi) {
  lo = 0;
  hi = kv_len - 1;
  if (p.causal) hi = min(hi, max(i + off, prefix - 1));
  if (p.wl >= 0) lo = max(lo, i + off - p.wl);
  if (p.wr >= 0) hi = min(hi, i + off + p.wr);
}

__device__ __forceinline__ void chunk_error(const ChunkParams& p, uint32_t code, uint32_t info) {
  if (atomicCAS(&p.ws->error, 0u, code) == 0u) atomicExch(&p.ws->error_info, info);
}

// Sequence s's lengths {-, q_len, kv_len, prefix}; false when they do not fit
// the sizes the host planned for (nothing indexes with them then).
__device__ __forceinline__ bool chunk_seq(const ChunkParams& p, int s, int4& q) {
  const int64_t c0 = p.cu_q ? p.cu_q[s] : 0, c1 = p.cu_q ? p.cu_q[s + 1] : p.Sq, q_len = c1 - c0;
  q.z = p.kv_len[s];
  q.w = p.prefix ? p.prefix[s] : 0;
  if (c0 < 0 || q_len < 0 || q_len > p.Sq || (p.cu_q && c1 > p.tot_q) || q.z < 0 || q.z > p.Sk || q.w < 0) return false;
  q.y = (int)q_len;
  return true;
}

// Key tiles that some row of row tile rt of a sequence sees: kt0 .. kt0 + count - 1.
__device__ __forceinline__ void row_tile_keys(const ChunkParams& p, int4 seq, int rt, int& kt0, int& count) {
  const int q_len = seq.y, kv = seq.z, pre = seq.w, off = kv - q_len;
  const int i0 = rt * p.rt_tokens, i1 = min(i0 + p.rt_tokens, q_len) - 1;
  int lo0, hi0, lo1, hi1;  // both ends move right with the row
  chunk_row_keys(p, i0, off, kv, pre, lo0, hi0);
  chunk_row_keys(p, i1, off, kv, pre, lo1, hi1);
  kt0 = count = 0;
  if (p.debug_flags & FA_DEBUG_NO_SKIP) {
    count = (kv + kKeysPerTile - 1) / kKeysPerTile;
    return;
  }
  if (lo0 > hi1) return;
  kt0 = lo0 / kKeysPerTile;
  count = hi1 / kKeysPerTile - kt0 + 1;
}
#endif

}  // namespace mfa
