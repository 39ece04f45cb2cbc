// Attention of drafted tokens over a paged cache (one token per request is the
// decode case) on sm_103a.
//
// Request b has n = seq_lens[b] tokens in the cache, the last m of them its
// drafted tokens.  Row i of the m attends to every position before the drafts
// and, of the drafts, to those its mask row marks (no mask: those up to
// itself).  Query heads of a GQA group share their kv head's keys, so a kv head
// of a request has group * m rows.
//
// What bounds it: reading K and V once, 4 D bytes per key and kv head.  A tile
// of 128 query rows would be mostly padding, so the operands are swapped: keys
// and head-dimension columns are the MMA's M, the rows its N (16, 32, 48, 64 or 96):
//   S^T [128 keys, N]  = K_tile (K-major A) . Q^T (K-major B)
//   O^T [128 columns, N] += V_tile^T (MN-major A) . P^T (K-major B)
// O^T of all D columns stays in TMEM (ceil(D / 128) N columns of 512), the S^T
// buffers above it, and the tensor work follows the rows there are.
//
// Work is cut evenly, not per request: the 128-key tiles of all (request, kv
// head, row tile) units form one line, and block c of G takes tiles
// [W c / G, W (c + 1) / G).  A unit that lies in one block is finished there;
// one that crosses blocks leaves fp32 partials (O unnormalised, max, sum), at
// most two per block, and the merge kernel joins them.  Lengths are read on
// the device only.
//
// Pages: a key tile is 128 / page boxes of `page` rows (a page of 128 rows or
// more is read in boxes of 128).  The box that holds the last valid rows starts
// earlier by as many rows as it lacks: rows before the page are out of range
// and arrive as zeros, so nothing behind the length, NaN included, is ever
// read.  Boxes past the length, and pages with a bad number, use a page index
// out of range: zeros.  The scores of such rows are -inf.
//
// bf16 P goes to shared memory as two terms, the rounded weight and its rounding
// residual, each with its own product: for N <= 64 the matrix pipe has the
// time (an MMA of these shapes takes 46 to 57 cycles, 64 of them per V tile of D =
// 512, against 10,000 cycles for the tile's bytes), and O then carries P to
// about 2^-16.  At N = 96 the residual's 24 KB are worth more as a third ring
// slot, and fp16 weights, rounded to 2^-11, need none.
//
// Warps: 0 and 2 TMA producers (even and odd ring slots; the lanes of a warp issue
// a slot's boxes), 1 TMEM owner and MMA issuer, from 4 on softmax, correction
// and epilogue: a warpgroup per 32 rows, 16 at N = 16 and 48 (thread = key of S^T,
// then column of O^T).  Every wait is bounded.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace ffpa {
namespace {

// P of a key tile: two halves of 64 keys, each N rows of 128 bytes; and as much
// again for the rounding residual where it is kept.
constexpr int p_bytes(int N) { return 2 * N * 128; }
constexpr bool keeps_residual(int N, bool bf16) { return bf16 && N <= 64; }
constexpr int kMaxSlots = 6;
constexpr float kRescaleLog2 = 8.0f;  // rescale O only when a row's max grows by > 2^8
// The largest weight of a row is 2^kTop when its reference is set: fp16 ends at
// 2^16 above and, in steps of 2^-24, below, so its weights are moved up by 2^6
// (at most 2^14 before the next rescale); bf16 has fp32's range.
template <bool BF16>
constexpr float kTop = BF16 ? 0.f : 6.f;
constexpr int kMergeThreads = 128;

// One request as the device sees it: n cached tokens, the last m of them drafts.
struct Request {
  int n, m;
};

__device__ __forceinline__ Request request(const TreeParams& p, int b) {
  Request r;
  r.n = __ldg(p.seq_lens + b);
  r.m = p.draft_lens ? __ldg(p.draft_lens + b) : p.T;
  const int cap = p.max_pages * p.page;
  if (r.n < 0 || r.n > cap || r.m < 0 || r.m > p.T || (r.m > r.n && (r.n > 0 || p.draft_lens))) {
    record_error(p.status, FFPA_DEV_LENGTHS);
    r.n = max(0, min(r.n, cap));
    r.m = max(0, min(r.m, p.T));
  }
  r.m = min(r.m, r.n);  // an empty entry of a padded batch: no rows
  return r;
}
template <int N>
__device__ __forceinline__ int row_tiles(const TreeParams& p, const Request& r) {
  return (p.group * r.m + N - 1) / N;
}
__device__ __forceinline__ int key_tiles(const Request& r) { return r.m > 0 ? (r.n + kTileRows - 1) / kTileRows : 0; }
template <int N>
__device__ __forceinline__ int64_t request_work(const TreeParams& p, const Request& r) {
  return static_cast<int64_t>(p.Hkv) * row_tiles<N>(p, r) * key_tiles(r);
}

// The requests' work, all of it and before the run of requests that this thread
// takes; `sums` has threads / 32 entries.
struct WorkSum {
  int64_t before_run, run, total;
  int first, last;  // requests of this thread's run
  Request r;        // the first of them
};
template <int N>
__device__ __forceinline__ WorkSum sum_work(const TreeParams& p, int64_t* sums, int threads) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.B + threads - 1) / threads;
  WorkSum w;
  w.first = min(p.B, tid * per);
  w.last = min(p.B, w.first + per);
  w.run = 0;
  w.r = {0, 0};
  if (w.first < w.last) {
    w.r = request(p, w.first);
    w.run = request_work<N>(p, w.r);
    for (int b = w.first + 1; b < w.last; ++b) w.run += request_work<N>(p, request(p, b));
  }
  int64_t incl = w.run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  w.before_run = incl - w.run;
  w.total = 0;
  for (int i = 0; i < threads / 32; ++i) {
    if (i < warp) w.before_run += sums[i];
    w.total += sums[i];
  }
  return w;
}

// First tile of block c of `blocks`.
__device__ __forceinline__ int64_t block_start(int64_t total, int blocks, int c) { return total * c / blocks; }

// The units of one block, in order.  Every role walks its own copy.
template <int N>
struct Walk {
  int64_t left;        // tiles of the line still to take
  int b, sub;          // request; kv head * row tiles + row tile
  int tile;            // first key tile of the current segment
  Request r;
  int rt, tiles;       // row tiles per kv head and key tiles of the request
  int hk, row0;        // kv head, first row of the row tile
  int end;             // one past the segment's last key tile

  __device__ __forceinline__ void shape(const TreeParams& p) {
    rt = row_tiles<N>(p, r);
    tiles = key_tiles(r);
  }
  __device__ __forceinline__ void place() {
    hk = sub / rt;
    row0 = (sub % rt) * N;
    end = static_cast<int>(min(static_cast<int64_t>(tiles), tile + left));
  }
  // `offset`: the block's first tile within the request's work
  __device__ __forceinline__ void begin(const TreeParams& p, int request_index, const Request& rq, int64_t offset,
                                        int64_t count) {
    left = count;
    b = request_index;
    r = rq;
    shape(p);
    sub = static_cast<int>(offset / tiles);
    tile = static_cast<int>(offset - static_cast<int64_t>(sub) * tiles);
    place();
  }
  // to the next segment; false when the block's tiles are used up
  __device__ __forceinline__ bool next(const TreeParams& p) {
    left -= end - tile;
    if (left <= 0) return false;
    tile = 0;
    if (++sub == rt * p.Hkv) {
      sub = 0;
      do {
        ++b;
        if (b >= p.B) return false;
        r = request(p, b);
        shape(p);
      } while (tiles == 0 || rt == 0);
    }
    place();
    return true;
  }
  __device__ __forceinline__ bool whole() const { return tile == 0 && end == tiles; }
};

struct Bars {
  int full, empty, q_full, s_full, s_free, p_ready, pv_done, o_free, drain, count;
};
__host__ __device__ constexpr Bars bar_layout() {
  return Bars{0, kMaxSlots, 2 * kMaxSlots, 2 * kMaxSlots + 1, 2 * kMaxSlots + 3, 2 * kMaxSlots + 5,
              2 * kMaxSlots + 6, 2 * kMaxSlots + 7, 2 * kMaxSlots + 8, 2 * kMaxSlots + 9};
}

constexpr int kStats = 12 * 32;  // floats of one copy of the exchanged statistics: 12 softmax warps at most
constexpr int kMiscBytes = 256 /* barriers, TMEM base, start */ + 128 /* work sums */ + 3 * 128 * 4 /* vis */ +
                           96 * 8 * 2 /* rows in out and lse */ + kStats * 4 * 3 /* statistics, twice; one warp's own */;
static_assert(kMiscBytes % 128 == 0, "tile alignment");
__host__ __device__ constexpr int q_bytes(int n_chunks, int N) { return n_chunks * N * 128; }
__host__ __device__ constexpr int fixed_bytes(int n_chunks, int N, bool bf16) {
  // D = 64: a V slot holds one chunk, and the second half of its M = 128 operand
  // is the 16 KB after it, past the ring for the last slot
  return q_bytes(n_chunks, N) + (keeps_residual(N, bf16) ? 2 : 1) * p_bytes(N) + kMiscBytes + 1024 +
         (n_chunks == 1 ? kChunkBytes : 0);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16)
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ void store1(void* base, int64_t at, float x) {
  if constexpr (BF16)
    static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(base)[at] = __float2half_rn(x);
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tst.shared.b16 [%0], h;\n\t}" ::"r"(addr), "r"(v) : "memory");
}
// Asynchronous 16-byte copy to shared memory; zeros where `real` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
// All `threads` threads meet; true if every one of them passes true.
__device__ __forceinline__ bool bar_and(uint32_t id, uint32_t threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// C consecutive TMEM columns of this thread's lane (C = 16 or 32)
template <int C>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[C]) {
  if constexpr (C == 32)
    tmem_ld32(taddr, r);
  else
    tmem_ld16(taddr, r);
  tmem_ld_wait();
}
template <int C>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[C]) {
  if constexpr (C == 32)
    tmem_st32(taddr, r);
  else
    tmem_st16(taddr, r);
}

struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// Reduces each of the C columns over the 32 lanes; lane l returns column l mod
// C.  At every step a lane keeps half of its columns and trades the others with
// the lane that keeps those: 31 exchanges for all C columns.
template <int C, class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[C], int lane, Op op) {
  if constexpr (C == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], 16));
  }
#pragma unroll
  for (int h = (C == 32 ? 16 : 8); h >= 1; h >>= 1) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, h));
    }
  }
  return v[0];
}

// Rows of a softmax warpgroup, and the block's threads.
template <int N>
constexpr int tree_rows() {
  return N == 16 || N == 48 ? 16 : 32;
}
template <int N>
constexpr int tree_threads() {
  return 128 + 128 * (N / tree_rows<N>());
}
// Blocks per SM the registers allow for: two for N <= 32 (launched as two where
// the shared memory of a small D allows it, see launch_n).
template <int N>
constexpr int tree_residency() {
  return N <= 32 ? 2 : 1;
}

template <int N, bool BF16>
__global__ void __launch_bounds__(tree_threads<N>(), tree_residency<N>())
    tree_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                const __grid_constant__ TreeParams p) {
  typedef typename std::conditional<BF16, __nv_bfloat16, __half>::type T;
  constexpr int kThreads = tree_threads<N>();
  constexpr int kSoftWarps = kThreads / 32 - 4;
  constexpr int C = tree_rows<N>();        // rows per softmax thread
  constexpr int kSBuf = N == 96 ? 1 : 2;   // S^T buffers: TMEM has room for one next to a 96-row O^T
  constexpr bool kLo = keeps_residual(N, BF16);
  constexpr Bars bl = bar_layout();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NC = p.n_chunks, slots = p.slots;
  const uint32_t slot_bytes = p.slot_bytes;
  const uint32_t ring = smem_u32(smem), p_hi = ring + slots * slot_bytes, p_lo = p_hi + p_bytes(N);
  const uint32_t q_sm = kLo ? p_lo + p_bytes(N) : p_lo;
  uint8_t* misc = smem + slots * slot_bytes + (kLo ? 2 : 1) * p_bytes(N) + q_bytes(NC, N);
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + bl.count);
  Walk<N>* start = reinterpret_cast<Walk<N>*>(misc + 176);  // the block's first segment (left == 0: none)
  int* pieces = reinterpret_cast<int*>(misc + 252);         // of the unit that this block's start is the first inside
  int64_t* sums = reinterpret_cast<int64_t*>(misc + 256);
  uint32_t* vis = reinterpret_cast<uint32_t*>(misc + 256 + 128);       // [3][128] draft -> rows that see it, C rows each
  int64_t* row_off = reinterpret_cast<int64_t*>(vis + 3 * 128);        // [N] offset of the row in out (0: padding)
  int64_t* row_lse = row_off + 96;                                     // [N] index of the row in lse
  float* stat = reinterpret_cast<float*>(row_lse + 96);                // [2][warps][32] exchanged statistics
  float* bcast = stat + 2 * kStats;                                    // [warps][32] per-row values of one warp
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  static_assert(bl.count * 8 + 4 <= 176 && 176 + sizeof(Walk<N>) <= 252, "barrier area");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* status = p.status;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(bar(bl.full + i), 1);
      mbar_init(bar(bl.empty + i), 1);
    }
    mbar_init(bar(bl.q_full), kSoftWarps);
    for (int i = 0; i < kSBuf; ++i) {
      mbar_init(bar(bl.s_full + i), 1);
      mbar_init(bar(bl.s_free + i), kSoftWarps);
    }
    mbar_init(bar(bl.p_ready), kSoftWarps);
    mbar_init(bar(bl.pv_done), 1);
    mbar_init(bar(bl.o_free), kSoftWarps);
    mbar_init(bar(bl.drain), 1);
    fence_mbar_init();
    start->left = 0;
    *pieces = 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  tc_fence_before();
  {
    const WorkSum w = sum_work<N>(p, sums, kThreads);  // contains a __syncthreads
    if (w.total > 0) {
      const int blocks = static_cast<int>(min(static_cast<int64_t>(gridDim.x), w.total));
      const int c = blockIdx.x;
      if (c < blocks) {
        const int64_t w0 = block_start(w.total, blocks, c), w1 = block_start(w.total, blocks, c + 1);
        if (w0 >= w.before_run && w0 < w.before_run + w.run) {
          int64_t at = w.before_run;
          int b = w.first;
          Request r = w.r;
          while (w0 >= at + request_work<N>(p, r)) {
            at += request_work<N>(p, r);
            r = request(p, ++b);
          }
          Walk<N> first;
          first.begin(p, b, r, w0 - at, w1 - w0);
          *start = first;
          // For the merge kernel: a unit that begins in the block before and goes on in
          // this one is joined from here; its pieces are that block's and those of the
          // blocks that start inside it, w_c < unit_end <=> c < unit_end blocks / total.
          if (first.tile > 0 && first.tile <= w0 - block_start(w.total, blocks, c - 1)) {
            const int64_t unit_end = w0 - first.tile + first.tiles;
            *pieces = static_cast<int>((unit_end * blocks + w.total - 1) / w.total) - c + 1;
          }
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0) p.joins[blockIdx.x] = make_int4(*pieces, start->b, start->sub, start->r.m);
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const bool any = start->left > 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge kernel's blocks may take free room
  const uint32_t s_tm = p.tmem_cols - kSBuf * N;  // the S^T buffers above O^T
  const int kslots = (NC + 1) / 2;    // ring slots of one key tile of K, or of V

  if (any && (warp == 0 || warp == 2)) {
    // ------------------------------------------------------------ TMA producers
    // Loads in the order of use: K of tile 0; then K of tile t + 1, V of tile t.
    // Warp 0 takes the loads of the even slots, warp 2 those of the odd ones.  A parity
    // wait tells apart a barrier's current phase and the one before, and the releases of
    // different slots may land in any order, so every load of a slot is the same warp's:
    // it has then waited for each of the slot's releases.
    const int pi = warp >> 1;
    const int box = min(p.page, kTileRows), pieces = kTileRows / box;
    bool ok = true;
    uint32_t it = 0;
    // one key tile of K or V: lane l issues box l of each slot (piece l mod pieces, chunk l / pieces)
    auto load_tile = [&](const CUtensorMap* m, const Walk<N>& w, int t) {
      const int piece = lane % pieces, ch = lane / pieces;
      const int pos = t * kTileRows + piece * box;  // first position of the box
      int row = 0, page = p.n_pages;                // out of range: zeros
      if (ch < 2 && pos < w.r.n) {
        page = __ldg(p.table + static_cast<int64_t>(w.b) * p.table_stride + pos / p.page);
        if (page < 0 || page >= p.n_pages) {
          record_error(status, FFPA_DEV_LENGTHS);
          page = p.n_pages;
        }
        row = pos % p.page + min(0, w.r.n - pos - box);  // the last box ends at the last valid row
      }
      for (int s2 = 0; s2 < kslots && ok; ++s2, ++it) {
        const uint32_t s = it % slots, rd = it / slots;
        if (static_cast<int>(s & 1) != pi) continue;
        ok = mbar_wait<false>(bar(bl.empty + s), (rd & 1) ^ 1, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int cn = min(2, NC - 2 * s2);
        if (lane == 0) mbar_expect_tx(bar(bl.full + s), cn * kChunkBytes);
        __syncwarp();
        if (ch < cn)
          tma_load_4d(ring + s * slot_bytes + ch * kChunkBytes + piece * box * 128, m, bar(bl.full + s),
                      (2 * s2 + ch) * kChunk, row, w.hk, page);
      }
    };
    Walk<N> w = *start;
    do {
      load_tile(&map_k, w, w.tile);
      for (int t = w.tile; t < w.end && ok; ++t) {
        if (t + 1 < w.end) load_tile(&map_k, w, t + 1);
        load_tile(&map_v, w, t);
      }
    } while (ok && w.next(p));
    // the last release of each of this warp's slots (commit arrivals are not
    // ordered with one another and must not land after the block is gone)
    if (lane == 0)
      for (uint32_t s = pi; s < static_cast<uint32_t>(slots) && s < it && ok; s += 2) {
        const uint32_t rounds = (it - 1 - s) / slots;  // full ones before the slot's last load
        mbar_wait<false>(bar(bl.empty + s), rounds & 1, status);
      }
  } else if (any && warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = idesc_f16(BF16, 128, N, false, false);
    constexpr uint32_t idesc_o = idesc_f16(BF16, 128, N, true, false);
    const uint64_t dk = sdesc_sw128(ring, 16, 1024), dv = sdesc_sw128(ring, kChunkBytes, 1024);
    const uint64_t dq = sdesc_sw128(q_sm, 16, 1024);
    const uint64_t dhi = sdesc_sw128(p_hi, 16, 1024), dlo = sdesc_sw128(p_lo, 16, 1024);
    bool ok = true;
    uint32_t it = 0, tc = 0, unit = 0;  // ring loads, S^T tiles and units so far
    auto scores = [&]() {
      if (tc >= kSBuf) {
        ok = mbar_wait<false>(bar(bl.s_free + tc % kSBuf), ((tc - kSBuf) / kSBuf) & 1, status);
        if (!ok) return;
        tc_fence_after();
      }
      const uint32_t d = tbase + s_tm + (tc % kSBuf) * N;
      for (int s2 = 0; s2 < kslots; ++s2, ++it) {
        const uint32_t s = it % slots;
        ok = mbar_wait<false>(bar(bl.full + s), (it / slots) & 1, status);
        if (!ok) return;
        tc_fence_after();
        const int cn = min(2, NC - 2 * s2);
        for (int i = 0; i < cn; ++i) {
          const uint64_t a = sdesc_advance(dk, s * slot_bytes + i * kChunkBytes);
          const uint64_t b = sdesc_advance(dq, (2 * s2 + i) * N * 128);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss(d, sdesc_advance(a, kk * 32), sdesc_advance(b, kk * 32), idesc_s, (s2 | i | kk) != 0);
        }
        umma_commit(bar(bl.empty + s));
      }
      umma_commit(bar(bl.s_full + tc % kSBuf));
      ++tc;
    };
    Walk<N> w = *start;
    uint32_t pv = 0;  // P V products so far
    do {
      ok = mbar_wait<false>(bar(bl.q_full), unit & 1, status);
      if (!ok) break;
      tc_fence_after();
      scores();
      for (int t = w.tile; t < w.end && ok; ++t, ++pv) {
        if (t + 1 < w.end) scores();
        if (!ok) break;
        if (t == w.tile && unit > 0) {  // the epilogue of the unit before has read O^T
          ok = mbar_wait<false>(bar(bl.o_free), (unit - 1) & 1, status);
          if (!ok) break;
        }
        ok = mbar_wait<false>(bar(bl.p_ready), pv & 1, status);
        if (!ok) break;
        tc_fence_after();
        for (int s2 = 0; s2 < kslots && ok; ++s2, ++it) {
          const uint32_t s = it % slots;
          ok = mbar_wait<false>(bar(bl.full + s), (it / slots) & 1, status);
          if (!ok) break;
          tc_fence_after();
          // columns 128 s2 .. of O^T; at an odd chunk count the last slot's second
          // half is stale shared memory: it reaches only O^T rows past D
          const uint64_t a = sdesc_advance(dv, s * slot_bytes);
          const uint32_t d = tbase + s2 * N;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_ss(d, sdesc_advance(a, ks * 2048), sdesc_advance(dhi, (ks >> 2) * (N * 128) + (ks & 3) * 32), idesc_o,
                    t > w.tile || ks > 0);
          if constexpr (kLo)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_ss(d, sdesc_advance(a, ks * 2048), sdesc_advance(dlo, (ks >> 2) * (N * 128) + (ks & 3) * 32), idesc_o,
                    1u);
          umma_commit(bar(bl.empty + s));
        }
        if (!ok) break;
        umma_commit(bar(bl.pv_done));
      }
      ++unit;
    } while (ok && w.next(p));
    umma_commit(bar(bl.drain));
    mbar_wait<false>(bar(bl.drain), 0, status);
  } else if (any && warp >= 4) {
    // ------------------------------------------------------------ softmax / correction / epilogue
    const int st = tid - 128;           // softmax thread
    const int wg = st >> 7;             // its rows: C wg .. C wg + C - 1 of the row tile
    const int t = st & 127;             // TMEM lane: key of S^T, column of O^T
    const int sw = warp - 4;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t nb = 1 + wg;         // named barrier of this warpgroup
    constexpr uint32_t kAll = kSoftWarps * 32;
    float* my_stat = stat + sw * 32;
    float* my_bcast = bcast + sw * 32;
    const float* wg_stat = stat + wg * 4 * 32;
    const int box = min(p.page, kTileRows);
    constexpr float kLn2 = 0.6931471805599453f;
    bool ok = true;
    uint32_t tc = 0;
    // Q rows of a row tile, K-major with the 128-byte swizzle, padding rows zero:
    // warp sw copies rows sw, sw + kSoftWarps, ..; the copies are asynchronous
    auto issue_q = [&](const Walk<N>& w) {
      const int m = w.r.m;
      for (int r = sw; r < N; r += kSoftWarps) {
        const int rr = w.row0 + r;
        const bool real = rr < p.group * m;
        const uint4* src = reinterpret_cast<const uint4*>(p.q);
        if (real)
          src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + w.b * p.q_sb +
                                               (w.hk * p.group + rr / m) * p.q_sh + (rr % m) * p.q_sn);
        for (int gq = lane; gq < 8 * NC; gq += 32)
          cp_async16(q_sm + (gq >> 3) * (N * 128) + r * 128 + (((gq & 7) ^ (r & 7)) << 4), real ? src + gq : src, real);
      }
    };
    auto finish_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bl.q_full));
    };
    Walk<N> w = *start, after = w;
    bool more = true;
    issue_q(w);
    finish_q();
    while (more) {
      const int m = w.r.m, n = w.r.n, prefix = n - m, rows = p.group * m;
      // ---- the unit: row offsets, draft visibility (its Q is on the way)
      if (!bar_and(4, kAll, ok)) break;  // the epilogue before has read the tables
      if (st < N) {
        const int rr = w.row0 + st;
        int64_t off = 0;
        int64_t li = 0;
        if (rr < rows) {
          const int h = w.hk * p.group + rr / m, i = rr % m;
          off = w.b * p.o_sb + h * p.o_sh + i * p.o_sn;
          li = (static_cast<int64_t>(w.b) * p.Hq + h) * p.T + i;
        }
        row_off[st] = off;
        row_lse[st] = li;
      }
      if (w.end * kTileRows > prefix) {  // this segment has drafts among its keys
        // item (draft j, C rows g): a bit for each row that sees the draft
        for (int it = st; it < (N / C) * m; it += kAll) {
          const int j = it % m, g = it / m;
          uint32_t bits = 0;
          for (int x = 0; x < C; ++x) {
            const int rr = w.row0 + g * C + x;
            if (rr >= rows) break;
            const int i = rr % m;
            const bool see = p.mask ? __ldg(p.mask + w.b * p.mask_sb + static_cast<int64_t>(i) * p.T + j) != 0 : j <= i;
            if (see) bits |= 1u << x;
          }
          vis[g * 128 + j] = bits;
        }
      }
      if (!bar_and(4, kAll, ok)) break;  // tables written

      float l[C];  // this key's share of the rows' sums
#pragma unroll
      for (int x = 0; x < C; ++x) l[x] = 0.f;
      float m_used = -INFINITY;  // lane x mod C: reference maximum of row x (log2 domain), the same in all warps
      for (int tile = w.tile; tile < w.end; ++tile, ++tc) {
        if (ok) ok = mbar_wait<false>(bar(bl.s_full + tc % kSBuf), (tc / kSBuf) & 1, status);
        ok = __all_sync(0xffffffffu, ok);
        float s[C];
        if (ok) {
          tc_fence_after();
          uint32_t v[C];
          tmem_load<C>(tbase + lane_off + s_tm + (tc % kSBuf) * N + wg * C, v);
#pragma unroll
          for (int x = 0; x < C; ++x) s[x] = __uint_as_float(v[x]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bl.s_free + tc % kSBuf));
        } else {
#pragma unroll
          for (int x = 0; x < C; ++x) s[x] = 0.f;
        }
        if ((tile + 1) * kTileRows > prefix) {
          // position of this thread's key: a box that the length cuts ends at the last valid row
          const int r = t % box, base = tile * kTileRows + t - r;
          const int shift = max(0, base + box - n);
          const int pos = base + r - shift;
          uint32_t see = 0xffffffffu;
          if (r < shift)
            see = 0u;
          else if (pos >= prefix)
            see = vis[wg * 128 + pos - prefix];
#pragma unroll
          for (int x = 0; x < C; ++x)
            if (!((see >> x) & 1u)) s[x] = -INFINITY;
        }
        // row maxima: over the warp's 32 keys, then over the four warps.  Tiles take the
        // two copies in turn: a warp that writes a copy again has passed the barrier of the
        // tile between, where every warp arrives after it has read the copy.
        const int at = (tc & 1) * kStats;
        {
          float mx[C];
#pragma unroll
          for (int x = 0; x < C; ++x) mx[x] = s[x];
          my_stat[at + lane] = reduce_columns<C>(mx, lane, MaxOp()) * p.scale_log2;
        }
        // A warp that gave up on a wait keeps taking part in the barriers: all
        // softmax warps leave together at the next unit.
        ok = bar_and(nb, 128, ok);
        float alpha = 1.f;
        {
          const float* x = wg_stat + at + lane;
          const float m_tile = fmaxf(fmaxf(x[0], x[32]), fmaxf(x[64], x[96]));
          if (m_used == -INFINITY) {
            m_used = m_tile - kTop<BF16>;
          } else if (m_tile - kTop<BF16> > m_used + kRescaleLog2) {
            alpha = ex2(m_used - (m_tile - kTop<BF16>));
            m_used = m_tile - kTop<BF16>;
          }
          my_bcast[lane] = m_used == -INFINITY ? 0.f : m_used;
          __syncwarp();
        }
        const bool rescale = __any_sync(0xffffffffu, alpha != 1.f);  // the same in the four warps
        if (rescale) {
#pragma unroll
          for (int x = 0; x < C; ++x) l[x] *= __shfl_sync(0xffffffffu, alpha, x);
        }
        if (tc > 0) {  // the product before has read P and written O^T
          if (ok) ok = mbar_wait<false>(bar(bl.pv_done), (tc - 1) & 1, status);
          ok = __all_sync(0xffffffffu, ok);
        }
        if (rescale && tile > w.tile && ok) {
          tc_fence_after();
          for (int blk = 0; blk < kslots; ++blk) {
            uint32_t v[C];
            const uint32_t a = tbase + lane_off + blk * N + wg * C;
            tmem_load<C>(a, v);
#pragma unroll
            for (int x = 0; x < C; ++x)
              v[x] = __float_as_uint(__uint_as_float(v[x]) * __shfl_sync(0xffffffffu, alpha, x));
            tmem_store<C>(a, v);
          }
          tmem_st_wait();
        }
        // P and its rounding residual of this key: row wg C + x of the key's half,
        // granule (t mod 64) / 8 under the 128-byte swizzle
        const uint32_t key_at = (t >> 6) * (N * 128) + wg * C * 128 + (t & 7) * 2, gran = (t & 63) >> 3;
#pragma unroll
        for (int x = 0; x < C; x += 4) {
          const float4 ref = *reinterpret_cast<const float4*>(my_bcast + x);
          const float e[4] = {ex2(fmaf(s[x], p.scale_log2, -ref.x)), ex2(fmaf(s[x + 1], p.scale_log2, -ref.y)),
                              ex2(fmaf(s[x + 2], p.scale_log2, -ref.z)), ex2(fmaf(s[x + 3], p.scale_log2, -ref.w))};
#pragma unroll
          for (int u = 0; u < 4; u += 2) {
            l[x + u] += e[u];
            l[x + u + 1] += e[u + 1];
            const uint32_t hi = pack2<BF16>(e[u], e[u + 1]);
            const uint32_t at0 = key_at + (x + u) * 128 + ((gran ^ ((x + u) & 7)) << 4);
            const uint32_t at1 = key_at + (x + u + 1) * 128 + ((gran ^ ((x + u + 1) & 7)) << 4);
            st_shared_u16(p_hi + at0, hi);
            st_shared_u16(p_hi + at1, hi >> 16);
            if constexpr (kLo) {
              const float2 r = unpack2<BF16>(hi);
              const uint32_t lo = pack2<BF16>(e[u] - r.x, e[u + 1] - r.y);
              st_shared_u16(p_lo + at0, lo);
              st_shared_u16(p_lo + at1, lo >> 16);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bl.p_ready));
      }
      // ---- the unit's end: row sums, then O^T to out or to a partial.  Every
      // score of the unit has been computed, so the next unit's Q may replace
      // this one's while the last product runs.
      after = w;
      more = after.next(p);
      if (more) issue_q(after);
      if (ok) ok = mbar_wait<false>(bar(bl.pv_done), (tc - 1) & 1, status);
      ok = __all_sync(0xffffffffu, ok);
      my_stat[lane] = reduce_columns<C>(l, lane, SumOp());  // pv_done: every warp has read the last tile's maxima
      ok = bar_and(nb, 128, ok);
      if (more) finish_q();
      const float sum = (wg_stat[lane] + wg_stat[32 + lane]) + (wg_stat[64 + lane] + wg_stat[96 + lane]);
      tc_fence_after();
      const int mine = rows - w.row0 - wg * C;  // of this warpgroup's rows, those that are not padding
      if (w.whole()) {
        my_bcast[lane] = sum > 0.f ? 1.f / sum : 0.f;
        __syncwarp();
        for (int blk = 0; blk < kslots; ++blk) {
          uint32_t v[C];
          tmem_load<C>(tbase + lane_off + blk * N + wg * C, v);
          const int d = blk * 128 + t;
          if (d < p.D) {
#pragma unroll
            for (int x = 0; x < C; ++x) {
              const int64_t off = row_off[wg * C + x] + d;
              const float y = __uint_as_float(v[x]) * my_bcast[x];
              if (x < mine) store1<BF16>(p.out, off, y);
            }
          }
        }
        if ((warp & 3) == 0 && lane < C && p.lse && lane < mine)
          p.lse[row_lse[wg * C + lane]] = sum > 0.f ? (m_used + __log2f(sum)) * kLn2 : -INFINITY;
      } else {
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.tile > 0 ? 0 : 1);
        float* part = p.part_o + (slot * N + wg * C) * p.D;
        for (int blk = 0; blk < kslots; ++blk) {
          uint32_t v[C];
          tmem_load<C>(tbase + lane_off + blk * N + wg * C, v);
          const int d = blk * 128 + t;
          if (d < p.D) {
#pragma unroll
            for (int x = 0; x < C; ++x)
              if (x < mine) part[x * p.D + d] = __uint_as_float(v[x]);
          }
        }
        if ((warp & 3) == 0 && lane < C) {
          float* ml = p.part_ml + (slot * N + wg * C + lane) * 2;
          ml[0] = m_used;
          ml[1] = sum;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bl.o_free));
      w = after;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, p.tmem_cols);
  }
}

// Joins the partials of the units that cross blocks.  Such a unit begins in a
// block c - 1 (its slot 1) and goes on in the blocks from c on (their slots 0);
// attention block c leaves its place and number of pieces in joins[c].  A warp takes
// Q x 128 columns of a row:
//   O = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c
// This form is for many units, each of few pieces.  Latency bounds it: the place,
// the maxima and sums, then 16 / Q partial rows in flight at a time.
template <int N, bool BF16, int Q>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kDeep = 16 / Q;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x + 1;
  const int4 join = p.joins[c];
  const int pieces = join.x, b = join.y, sub = join.z, m = join.w;
  if (pieces == 0) return;
  const int parts = (p.D + 128 * Q - 1) / (128 * Q);  // warps of a row
  const int item = blockIdx.y * (kMergeThreads / 32) + warp, x = item / parts, d0 = 128 * Q * (item % parts) + 4 * lane;
  const int rt = (p.group * m + N - 1) / N;
  const int rr = (sub % rt) * N + x;
  if (x >= N || rr >= p.group * m) return;
  auto slot = [&](int k) { return (2 * static_cast<int64_t>(c - 1 + k) + (k == 0 ? 1 : 0)) * N + x; };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float M = -INFINITY;
  for (int k = lane; k < pieces; k += 32) M = fmaxf(M, ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
  float4 o[Q];  // columns d0 + 128 q ..
#pragma unroll
  for (int q = 0; q < Q; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < pieces; k0 += 32) {
    float f = 0.f;
    if (k0 + lane < pieces) {
      const float2 s = ml[slot(k0 + lane)];
      f = ex2(s.x - ref);
      sum = fmaf(f, s.y, sum);
    }
    const int n = min(32, pieces - k0);
    for (int k1 = 0; k1 < n; k1 += kDeep) {
      float4 y[kDeep][Q];
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          y[k][q] = *reinterpret_cast<const float4*>(p.part_o + slot(min(k0 + k1 + k, pieces - 1)) * p.D +
                                                     min(d0 + 128 * q, p.D - 4));
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        if (k1 + k >= n) break;
        const float fk = __shfl_sync(0xffffffffu, f, (k1 + k) & 31);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          o[q].x = fmaf(fk, y[k][q].x, o[q].x);
          o[q].y = fmaf(fk, y[k][q].y, o[q].y);
          o[q].z = fmaf(fk, y[k][q].z, o[q].z);
          o[q].w = fmaf(fk, y[k][q].w, o[q].w);
        }
      }
    }
  }
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, e);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int h = (sub / rt) * p.group + rr / m, i = rr % m;
  typedef typename std::conditional<BF16, __nv_bfloat16, __half>::type T;
  T* orow = static_cast<T*>(p.out) + b * p.o_sb + h * p.o_sh + i * p.o_sn;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int d = d0 + 128 * q;
    if (d < p.D) {
      uint2 w;
      w.x = pack2<BF16>(o[q].x * inv, o[q].y * inv);
      w.y = pack2<BF16>(o[q].z * inv, o[q].w * inv);
      *reinterpret_cast<uint2*>(orow + d) = w;
    }
  }
  constexpr float kLn2 = 0.6931471805599453f;
  if (d0 == 0 && p.lse)
    p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + i] = sum > 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
}

// The form for few units of many pieces (one long request: up to a piece per block).
// Block (u, y) takes 128 columns of a row of the u-th unit to join; its warps share
// out the pieces, eight partial rows in flight each, and add up in shared memory.
constexpr int kDeepThreads = 512;
template <int N, bool BF16>
__global__ void __launch_bounds__(kDeepThreads) tree_merge_deep_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kWarps = kDeepThreads / 32, kDeep = 8;
  __shared__ int found[kWarps];
  __shared__ int4 place;
  __shared__ int first;
  __shared__ float weight[kDeepThreads];
  __shared__ float part_max[kWarps], part_sum[kWarps];
  __shared__ float4 acc[kWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the u-th block with pieces to join (at most kDeepThreads blocks, see launch_merge)
  int4 join = make_int4(0, 0, 0, 0);
  if (tid < p.blocks) join = p.joins[tid];
  const uint32_t have = __ballot_sync(0xffffffffu, join.x > 0);
  if (lane == 0) found[warp] = __popc(have);
  if (tid == 0) place = make_int4(0, 0, 0, 0);
  __syncthreads();
  int before = __popc(have & ((1u << lane) - 1u));
  for (int w = 0; w < warp; ++w) before += found[w];
  if (join.x > 0 && before == static_cast<int>(blockIdx.x)) {
    place = join;
    first = tid;
  }
  __syncthreads();
  const int pieces = place.x, b = place.y, sub = place.z, m = place.w;
  if (pieces == 0) return;
  const int c = first, parts = (p.D + 127) / 128;
  const int x = blockIdx.y / parts, d = 128 * (blockIdx.y % parts) + 4 * lane;
  const int rt = (p.group * m + N - 1) / N;
  const int rr = (sub % rt) * N + x;
  if (rr >= p.group * m) return;
  auto slot = [&](int k) { return (2 * static_cast<int64_t>(c - 1 + k) + (k == 0 ? 1 : 0)) * N + x; };
  // a piece per thread: the maximum, the weights and the sum
  const float2 s = tid < pieces ? reinterpret_cast<const float2*>(p.part_ml)[slot(tid)] : make_float2(-INFINITY, 0.f);
  float M = s.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) part_max[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_max[w]);
  const float f = ex2(s.x - (M == -INFINITY ? 0.f : M));
  weight[tid] = f;
  float sum = f * s.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part_sum[warp] = sum;
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* src = p.part_o + min(d, p.D - 4);
  for (int k0 = warp; k0 < pieces; k0 += kDeep * kWarps) {
    float4 y[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      y[i] = *reinterpret_cast<const float4*>(src + slot(min(k0 + i * kWarps, pieces - 1)) * p.D);
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      if (k0 + i * kWarps >= pieces) break;
      const float w = weight[k0 + i * kWarps];
      o.x = fmaf(w, y[i].x, o.x);
      o.y = fmaf(w, y[i].y, o.y);
      o.z = fmaf(w, y[i].z, o.z);
      o.w = fmaf(w, y[i].w, o.w);
    }
  }
  acc[warp][lane] = o;
  __syncthreads();
  if (warp > 0) return;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += part_sum[w];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const float4 y = acc[w][lane];
    o.x += y.x;
    o.y += y.y;
    o.z += y.z;
    o.w += y.w;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int h = (sub / rt) * p.group + rr / m, i = rr % m;
  if (d < p.D) {
    typedef typename std::conditional<BF16, __nv_bfloat16, __half>::type T;
    uint2 w;
    w.x = pack2<BF16>(o.x * inv, o.y * inv);
    w.y = pack2<BF16>(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + b * p.o_sb + h * p.o_sh + i * p.o_sn + d) = w;
  }
  constexpr float kLn2 = 0.6931471805599453f;
  if (d == 0 && p.lse)
    p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + i] = sum > 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
}

template <int N, bool BF16, int Q>
cudaError_t launch_merge_q(const TreeParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int rows = std::min(N, p.group * p.T);  // of a row tile, at most
  const int warps = rows * ((p.D + 128 * Q - 1) / (128 * Q)), per = kMergeThreads / 32;
  cfg.gridDim = dim3(p.blocks - 1, (warps + per - 1) / per, 1);
  cfg.blockDim = dim3(kMergeThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  set_overlap(&attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<N, BF16, Q>, p);
}

// Few units (fewer than a quarter of the blocks: five pieces or more on average)
// take the deep form, as long as its blocks are two waves or so.  Whole calls, wide /
// deep, with as many keys in all (us; * what the rule takes):
//   rows x units     1 x 1      1 x 32     8 x 1     8 x 16     8 x 37     48 x 4     48 x 8
//   D = 64         82 / 21*   25 / 24*   83 / 21*  26 / 24*   31 / 30*   47 / 38*   42 / 38*
//   D = 512        96 / 56*   93 / 93*   97 / 57*  97 / 97*  109 / 113* 113 / 104* 106* / 108
//   D = 1024      151 / 96*   97 / 96*  153 / 97* 100 / 102*  99* / 109 123* / 113 114* / 123
// and with 90 rows, 4 and 16 units: 50 / 41* and 45* / 49 (D = 64), 117* / 110 and
// 108* / 136 (D = 512).  Where the rule errs it costs 9% at most.
template <int N, bool BF16>
cudaError_t launch_merge(const TreeParams& p, cudaStream_t st) {
  const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * ((static_cast<int64_t>(p.group) * p.T + N - 1) / N);
  const int items = std::min(N, p.group * p.T) * ((p.D + 127) / 128);  // of a unit: 128 columns of a row
  if (units * 4 < p.blocks && units * items <= 8 * p.blocks && p.blocks <= kDeepThreads) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(units, p.blocks - 1)), items, 1);
    cfg.blockDim = dim3(kDeepThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    set_overlap(&attr[0]);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_deep_kernel<N, BF16>, p);
  }
  if (p.D <= 128) return launch_merge_q<N, BF16, 1>(p, st);
  if (p.D <= 256) return launch_merge_q<N, BF16, 2>(p, st);
  if (p.D <= 512) return launch_merge_q<N, BF16, 4>(p, st);
  return launch_merge_q<N, BF16, 8>(p, st);
}

template <int N, bool BF16>
cudaError_t launch_n(const TreeParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  const int smem = fixed_bytes(p.n_chunks, N, BF16) + p.slots * p.slot_bytes;
  auto kern = tree_kernel<N, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBlockSmem);
  if (e != cudaSuccess) return e;
  timing_mark(st);
  e = launch_kernel(kern, dim3(p.blocks), tree_threads<N>(), smem, st, mk, mv, p);
  timing_mark(st);
  if (e != cudaSuccess || p.blocks < 2) return e;
  e = launch_merge<N, BF16>(p, st);
  timing_mark(st);
  return e;
}

template <bool BF16>
cudaError_t launch_tree(const TreeParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  switch (p.rows_n) {
    case 16: return launch_n<16, BF16>(p, mk, mv, st);
    case 32: return launch_n<32, BF16>(p, mk, mv, st);
    case 48: return launch_n<48, BF16>(p, mk, mv, st);
    case 64: return launch_n<64, BF16>(p, mk, mv, st);
    default: return launch_n<96, BF16>(p, mk, mv, st);
  }
}

}  // namespace

// The rows of a row tile, the ring and the blocks per SM for `rows` rows per kv head.
//
// Rows: the fewest row tiles (each reads K and V again), then the smallest N.
// O^T takes ceil(D / 128) N columns of TMEM next to the scores, Q and P 2 N D +
// 512 N (1024 N with the residual) bytes of shared memory next to the ring, so
// N = 96 serves D <= 512, N = 64 D <= 768 and N = 48 D <= 1024.
//
// Two blocks per SM for D <= 256 and N <= 32, where a tile's chain (scores,
// softmax, product) takes longer than its bytes.
int tree_shape(TreeParams* p, int64_t rows, bool bf16) {
  const int widest = p->D <= 512 ? 96 : p->D <= 768 ? 64 : 48;
  const int64_t tiles = (rows + widest - 1) / widest;
  int n = widest;
  for (int c : {64, 48, 32, 16})
    if (c < widest && (rows + c - 1) / c == tiles) n = c;
  p->rows_n = n;
  p->slot_bytes = std::min(2, p->n_chunks) * kChunkBytes;
  const int fixed = fixed_bytes(p->n_chunks, n, bf16);
  const bool two = p->D <= 256 && n <= 32;
  // an SM has 228 KB, of which a block's own 1 KB is reserved for the system
  const int room = two ? (233472 - 2 * 1024) / 2 : kMaxBlockSmem;
  p->slots = std::min(kMaxSlots, (room - fixed) / p->slot_bytes);
  p->tmem_cols = two ? 256 : 512;
  return two ? 2 : 1;
}

cudaError_t launch_fwd_tree(const TreeParams& p, const CUtensorMap& mk, const CUtensorMap& mv, bool bf16,
                            cudaStream_t s) {
  return bf16 ? launch_tree<true>(p, mk, mv, s) : launch_tree<false>(p, mk, mv, s);
}

}  // namespace ffpa
