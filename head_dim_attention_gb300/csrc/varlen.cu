// The plan of a packed call: which tile each block takes, and every
// sequence's TMA maps (varlen.cuh).
//
// Block 0 sorts the tiles by their work, heaviest first (the causal tile of
// index t has t + 1 key tiles), with a counting sort over kBins work classes:
// a histogram, a scan from the heaviest class down, and a scatter.  The order
// inside a class is whatever the shared-memory atomics give; it decides only
// when a tile runs, never what it computes.  The other blocks make the maps,
// one warp per (sequence, map): 128 bytes through shared memory, three fields
// replaced, published with the tensormap release that var_acquire pairs with.
//
// The maps start from that of a single row (base, rows and heads are replaced) and
// not from that of all rows, because the encoder gives large tensors another form
// than small ones, and a map of that form over few rows faults: kernels that
// loaded short sequences through such maps ended in an illegal address twice, once
// in about three hundred small calls.  The form of the smallest tensor holds for
// every size: it is what a map gets that is encoded before its sizes are known.
//
// Starts that do not ascend within 0 .. T describe no sequence: such an entry
// counts as length 0 and the status word reports it; no read or write follows
// from it.
#include "varlen.cuh"

namespace ffpa {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kBins = 1024;

struct SeqRange {
  int start, len;
};

__device__ __forceinline__ SeqRange seq_range(const VarPlan& p, int s) {
  const int a = __ldg(p.cu + s), z = __ldg(p.cu + s + 1);
  if (a < 0 || z < a || z > p.total) {
    record_error(p.status, FFPA_DEV_LENGTHS);
    return {0, 0};
  }
  return {a, z - a};
}

__global__ void __launch_bounds__(kPlanThreads) varlen_plan_kernel(const __grid_constant__ VarPlan p) {
  var_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kPlanThreads / 32;
  if (blockIdx.x > 0) {
    // ------------------------------------------------------------ maps
    __shared__ __align__(128) uint8_t stage[kWarps][128];
    const int64_t item = static_cast<int64_t>(blockIdx.x - 1) * kWarps + warp;
    const int s = static_cast<int>(item / p.n_maps), which = static_cast<int>(item % p.n_maps);
    if (s >= p.n_seqs) return;
    const SeqRange r = seq_range(p, s);
    if (r.len == 0) return;  // no tile uses these maps
    const uint32_t sm = smem_u32(stage[warp]);
    reinterpret_cast<uint32_t*>(stage[warp])[lane] = reinterpret_cast<const uint32_t*>(&p.maps[which])[lane];
    __syncwarp();
    if (lane == 0) {
      const uint64_t base = reinterpret_cast<uint64_t>(p.base[which]) + 2ull * static_cast<uint64_t>(r.start) * p.row_stride[which];
      asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(sm), "l"(base) : "memory");
      asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(sm), "r"(r.len) : "memory");
      asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 2, %1;" ::"r"(sm), "r"(p.heads[which]) : "memory");
    }
    __syncwarp();
    const CUtensorMap* dst = p.out_maps + static_cast<int64_t>(s) * kVarMaps + which;
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
            reinterpret_cast<uint64_t>(dst)),
        "r"(sm)
        : "memory");
    return;
  }
  // -------------------------------------------------------------- tiles
  __shared__ int count[kBins];
  __shared__ int warp_sum[kWarps];
  for (int i = tid; i < kBins; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  // work class of a tile: its key tiles, scaled so that the longest possible sequence fits
  auto bin = [&](int tile, int tiles) {
    const int work = p.causal ? tile + 1 : tiles;
    return kBins - 1 - min(work >> p.bin_shift, kBins - 1);  // heaviest first
  };
  // A warp takes 32 sequences at a time; a lane goes through the first kOwn tiles of its
  // own (short sequences come by the thousand), the warp through the rest together,
  // one sequence after the other.  Plan alone, kOwn = 1 / 4 / 8 / 16: 5000 sequences of 3
  // rows 16.4 / 17.0 / 18.3 / 18.3 us, 64 of 300 14.4 / 4.1 / 4.1 / 4.1, 256 of 700
  // 14.4 / 16.4 / 4.1 / 4.1, 1000 of 1000 51 / 52 / 12 / 11, 16 of 8192 12.2 / 12.3 / 12.3 / 12.3.
  auto each_tile = [&](auto&& visit) {
    constexpr int kOwn = 8;
    for (int s0 = 32 * warp; s0 < p.n_seqs; s0 += 32 * kWarps) {
      const int s = s0 + lane;
      const SeqRange r = s < p.n_seqs ? seq_range(p, s) : SeqRange{0, 0};
      const int tiles = (r.len + kTileRows - 1) / kTileRows;
      for (int t = 0; t < min(tiles, kOwn); ++t) visit(s, r, t, tiles);
      for (uint32_t todo = __ballot_sync(0xffffffffu, tiles > kOwn); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        const SeqRange o = {__shfl_sync(0xffffffffu, r.start, src), __shfl_sync(0xffffffffu, r.len, src)};
        const int n = __shfl_sync(0xffffffffu, tiles, src);
        for (int t = kOwn + lane; t < n; t += 32) visit(s0 + src, o, t, n);
      }
    }
  };
  each_tile([&](int, const SeqRange&, int t, int tiles) { atomicAdd(&count[bin(t, tiles)], 1); });
  __syncthreads();
  // exclusive scan over the classes: each thread takes kBins / kPlanThreads of them
  constexpr int kPer = kBins / kPlanThreads;
  int own[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    own[i] = sum;
    sum += count[tid * kPer + i];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = incl - sum, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) count[tid * kPer + i] = before + own[i];
  __syncthreads();
  each_tile([&](int s, const SeqRange& r, int t, int tiles) {
    const int at = atomicAdd(&count[bin(t, tiles)], 1);
    // overlapping ranges (starts that do not ascend) can have more tiles than slots
    if (at < p.slots) p.tiles[at] = make_int4(s, t, r.start, r.len);
  });
  for (int i = all + tid; i < p.slots; i += kPlanThreads) p.tiles[i] = make_int4(-1, 0, 0, 0);
}

}  // namespace

cudaError_t launch_varlen_plan(const VarPlan& p, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(p.n_seqs) * p.n_maps;
  const unsigned blocks = 1 + static_cast<unsigned>((items + kPlanThreads / 32 - 1) / (kPlanThreads / 32));
  return launch_kernel(varlen_plan_kernel, dim3(blocks), kPlanThreads, 0, s, p);
}

}  // namespace ffpa
