// Packed sequences: what the attention kernels share when the rows of q, k
// and v are several sequences one after the other.
//
// A sequence is treated as a tensor of its own.  Every TMA map a kernel uses is
// made once per sequence, with the sequence's first row as its base and its
// length as the row count (tensormap.replace, in the plan kernel of varlen.cu),
// so rows of a neighbour are out of range: they arrive as
// zeros, exactly as rows past the end of an unpacked tensor do, and neither a
// value nor a NaN of one sequence can reach another.  With pointers moved and
// Nq = Nkv = length (localize below) the kernels' index arithmetic is that of
// an unpacked call with one batch.
//
// The host does not know the lengths.  It launches as many (sequence, tile)
// slots as `n` sequences of `T` rows in all can have; the plan kernel fills the
// slots, heaviest tile first, and a block whose slot is empty returns at once.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace ffpa {

// One slot's sequence and 128-row tile.
struct VarTile {
  int seq;   // -1: empty slot
  int tile;  // query tile; its work in a causal call is tile + 1 key tiles
  int start, len;
};

// A packed call's launches overlap where they do not depend on one another (each is
// launched as a programmatic dependent of the one before):
//   forward   the attention kernel starts while the plan runs and waits for it
//             (var_wait) before it reads its tile;
//   backward  the preprocess runs beside the plan; the first gradient kernel follows
//             both; the others read nothing of its results, so they start as its
//             blocks leave.  The last block of each ends only after the launch
//             before has (var_end), so that the end of the last launch is the end
//             of all: one block, because a block that waits holds its SM.
__device__ __forceinline__ void var_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void var_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void var_end() {
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) var_wait();
}

__device__ __forceinline__ VarTile var_tile(const VarParams& v, int slot) {
  const int4 t = __ldcg(v.tiles + slot);  // written by a launch that this one overlaps
  return VarTile{t.x, t.y, t.z, t.w};
}

__device__ __forceinline__ const CUtensorMap* var_map(const VarParams& v, const VarTile& t, int which) {
  return v.maps + static_cast<int64_t>(t.seq) * kVarMaps + which;
}

// One warp, ahead of the block's first barrier and so of its first TMA load: makes the
// sequence's first `n` maps, which the plan kernel wrote, visible to this block's loads
// (a map per lane).  No load that uses a map may be in flight meanwhile, and a map in
// global memory takes no prefetch.tensormap, which is for the param and const spaces.
__device__ __forceinline__ void var_acquire(const VarParams& v, const VarTile& t, int n) {
  const int lane = threadIdx.x & 31;
  if (lane < n)
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(
                     reinterpret_cast<uint64_t>(var_map(v, t, lane)))
                 : "memory");
}

__device__ __forceinline__ void* var_rows(const void* base, int64_t rows, int64_t row_stride) {
  return const_cast<uint16_t*>(static_cast<const uint16_t*>(base) + rows * row_stride);  // 16-bit elements
}

// The call's parameters as an unpacked call over one sequence would have them.
__device__ __forceinline__ void localize(FwdParams& p, const VarTile& t) {
  p.Nq = p.Nkv = t.len;
  p.q_tiles = (t.len + kTileRows - 1) / kTileRows;
  p.q = var_rows(p.q, t.start, p.q_sn);
  p.out = var_rows(p.out, t.start, p.o_sn);
  if (p.lse) p.lse += t.start;
}

__device__ __forceinline__ void localize(BwdParams& p, const VarTile& t) {
  p.Nq = p.Nkv = t.len;
  p.q_tiles = p.kv_tiles = (t.len + kTileRows - 1) / kTileRows;
  p.q = var_rows(p.q, t.start, p.q_sn);
  p.k = var_rows(p.k, t.start, p.k_sn);
  p.v = var_rows(p.v, t.start, p.v_sn);
  p.dout = var_rows(p.dout, t.start, p.do_sn);
  p.dq = var_rows(p.dq, t.start, p.dq_sn);
  p.dk = var_rows(p.dk, t.start, p.dk_sn);
  p.dv = var_rows(p.dv, t.start, p.dv_sn);
  p.delta += t.start;
  p.lse2 += t.start;
}

// The backward's masked tiles.  With a bias and 64-bit addresses in it, the general
// per-score code of a masked 128 x 128 tile takes about 8 us (D = 64, 14,000 cycles
// for a thread's 128 scores), which short sequences pay on nearly every tile.  A
// packed call has no bias, and its masks leave one span of a thread's scores:
// those of columns base + lo .. base + hi - 1.
struct VarSpan {
  int lo, hi;
};
// Stationary row `srow` is a query (DQ) or a key; the columns are the other side.
template <bool DQ>
__device__ __forceinline__ VarSpan var_span(const BwdParams& p, int srow, int base) {
  if (DQ) return {0, srow < p.Nq ? (p.causal ? min(p.Nkv, srow + 1) : p.Nkv) - base : 0};
  return {p.causal ? srow - base : 0, srow < p.Nkv ? p.Nq - base : 0};
}
// A row without keys has lse -inf and no weights: 2^(x - inf) = 0.
__device__ __forceinline__ float var_lse(float l2) { return l2 == -INFINITY ? INFINITY : l2; }

// Distance between the heads of lse, delta and lse2.
template <bool VAR, class P>
__device__ __forceinline__ int stat_rows(const P& p) {
  return VAR ? p.var.total : p.Nq;
}

}  // namespace ffpa
