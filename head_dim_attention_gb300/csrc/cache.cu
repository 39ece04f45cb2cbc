// A paged cache's bookkeeping and writes: block tables and slot maps from
// request lengths, and new keys and values into their slots.
//
// Plan.  Request b has lens[b] tokens and gets new_lens[b] more:
//   had = ceil(lens / page),  need = ceil((lens + new) / page) - had
//   table[b, had .. had + need) = free[head + sum_{b' < b} need ..]
//   slot of the request's k-th new token, pos = lens + k:
//     table[b, pos / page] * page + pos % page
// Two exclusive scans over the requests, then one independent item per page and
// per token.  The bytes are few (8 per token): launches and dependent reads
// bound it.  One block scans and hands out the pages; the slots follow in the
// same block while they are few, in a grid of their own above that.
//
// Append: one 16-byte vector per thread and step from [1, H, T, D] rows to the
// rows of their slots, both with free strides; bound by HBM, 4 bytes moved per
// element of K or V.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace ffpa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kAppendThreads = 256;

// Exclusive scan of (a, b) over the block's threads; totals returned too.
struct Pair {
  int64_t a, b;
};
__device__ __forceinline__ Pair block_scan(Pair v, Pair* total, Pair* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Pair incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl.a, o), y = __shfl_up_sync(0xffffffffu, incl.b, o);
    if (lane >= o) {
      incl.a += x;
      incl.b += y;
    }
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  Pair before = {incl.a - v.a, incl.b - v.b};
  *total = {0, 0};
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < warp) {
      before.a += sums[i].a;
      before.b += sums[i].b;
    }
    total->a += sums[i].a;
    total->b += sums[i].b;
  }
  __syncthreads();
  return before;
}

// Slot of packed new token t, or -1 behind the last one or without a page; the
// requests' starts `cu` and lengths `lens` in shared memory or where they were written.
__device__ __forceinline__ int64_t token_slot(const PlanParams& p, const int32_t* cu, const int32_t* lens, int64_t t) {
  if (t >= cu[p.B]) return -1;
  int lo = 0, hi = p.B - 1;  // the last request that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  // a request's first new token follows what it had: its length now less its new tokens
  const int64_t pos = static_cast<int64_t>(lens[lo]) - (cu[lo + 1] - t);
  const int64_t block = pos / p.page;
  if (block >= p.max_pages) return -1;
  const int page = p.table[lo * p.table_stride + block];
  return page < 0 ? -1 : static_cast<int64_t>(page) * p.page + pos % p.page;
}

// Lengths, starts and pages; with `slots_too` the slot map as well.
__global__ void __launch_bounds__(kPlanThreads, 1) cache_plan_kernel(const __grid_constant__ PlanParams p, int slots_too) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ Pair sums[kPlanThreads / 32];
  __shared__ int32_t s_cu[kPlanThreads + 1], s_lens[kPlanThreads];  // the last 1024 requests'
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t head = *p.free_head;
  Pair carry = {0, 0};
  bool bad = head < 0 || head > p.n_free;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int len = 0, add = 0;
    if (b < p.B) {
      len = p.lens[b];
      add = p.new_lens[b];
      if (len < 0 || add < 0 || len > INT32_MAX - add) {
        bad = true;
        len = max(0, len);
        add = 0;
      }
    }
    const int had = static_cast<int>((static_cast<int64_t>(len) + p.page - 1) / p.page);
    const int need = static_cast<int>((static_cast<int64_t>(len) + add + p.page - 1) / p.page) - had;
    Pair total;
    const Pair at = block_scan({add, need}, &total, sums);
    if (b < p.B) {
      p.cu[b] = static_cast<int32_t>(min(carry.a + at.a, static_cast<int64_t>(INT32_MAX)));
      p.lens_out[b] = len + add;
      s_cu[tid] = p.cu[b];
      s_lens[tid] = len + add;
    }
    // a request's k-th new page; false without a page or a column for it
    auto take = [&](int request, int col, int64_t f) {
      if (col >= p.max_pages) return false;
      const bool there = f >= 0 && f < p.n_free;
      p.table[request * p.table_stride + col] = there ? p.free_pages[f] : -1;
      return there;
    };
    const int64_t first = head + carry.b + at.b;
    if (need > 0 && !take(b, had, first)) bad = true;
    // prompts take many: the warp shares out the pages past a request's first
    for (uint32_t todo = __ballot_sync(0xffffffffu, need > 1); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int n = __shfl_sync(0xffffffffu, need, src), col = __shfl_sync(0xffffffffu, had, src);
      const int64_t f = __shfl_sync(0xffffffffu, first, src);
      for (int k = 1 + lane; k < n; k += 32) {
        if (col + k >= p.max_pages) {
          bad = true;
          break;
        }
        if (!take(b - lane + src, col + k, f + k)) bad = true;
      }
    }
    carry.a += total.a;
    carry.b += total.b;
  }
  if (tid == 0) {
    p.cu[p.B] = static_cast<int32_t>(min(carry.a, static_cast<int64_t>(INT32_MAX)));
    s_cu[min(p.B, kPlanThreads)] = p.cu[p.B];
    *p.free_head_out = static_cast<int32_t>(max(static_cast<int64_t>(0), min(head + carry.b, static_cast<int64_t>(p.n_free))));
    bad |= carry.a > p.max_new;
  }
  if (bad) record_error(p.status, FFPA_DEV_LENGTHS);
  if (!slots_too) return;
  __syncthreads();
  const bool here = p.B <= kPlanThreads;
  for (int64_t t = tid; t < p.max_new; t += kPlanThreads)
    p.slots[t] = here ? token_slot(p, s_cu, s_lens, t) : token_slot(p, p.cu, p.lens_out, t);
}

__global__ void __launch_bounds__(256) cache_slots_kernel(const __grid_constant__ PlanParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (t < p.max_new) p.slots[t] = token_slot(p, p.cu, p.lens_out, t);
}

__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ AppendParams p) {
  const int vecs = p.D / 8;
  const int64_t items = p.T * p.H * vecs, step = static_cast<int64_t>(gridDim.x) * kAppendThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x; i < items; i += step) {
    const int c = static_cast<int>(i % vecs) * 8;
    const int64_t row = i / vecs;
    const int h = static_cast<int>(row % p.H);
    const int64_t t = row / p.H;
    const int64_t slot = __ldg(p.slots + t);
    if (slot < 0) continue;
    const int64_t page = slot / p.page;
    if (page >= p.n_pages) {
      record_error(p.status, FFPA_DEV_LENGTHS);
      continue;
    }
    const int64_t at = slot % p.page;
    const uint4 k = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k) + h * p.k_sh + t * p.k_sn + c));
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + h * p.v_sh + t * p.v_sn + c));
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.kc) + page * p.kc_sp + h * p.kc_sh + at * p.kc_sn + c) = k;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.vc) + page * p.vc_sp + h * p.vc_sh + at * p.vc_sn + c) = v;
  }
}

}  // namespace

cudaError_t launch_cache_plan(const PlanParams& p, cudaStream_t s) {
  // The slots in the plan's own block, or in a grid of their own behind it: up to 1024
  // tokens 5.1 to 6.2 us and 6.4 to 7.7 (1 to 512 requests), at 2048 6.1 to 8.8 and 6.5
  // to 8.8, at 4096 7.2 to 10.4 and 6.7 to 9.1, at 16384 14 to 25 and 7.8 to 11.6.
  const bool one = p.max_new <= 2 * kPlanThreads;
  cudaError_t e = launch_kernel(cache_plan_kernel, dim3(1), kPlanThreads, 0, s, p, one ? 1 : 0);
  timing_mark(s);
  if (e != cudaSuccess || one) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.max_new + 255) / 256), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  set_overlap(&attr[cfg.numAttrs++]);
  e = cudaLaunchKernelEx(&cfg, cache_slots_kernel, p);
  timing_mark(s);
  return e;
}

cudaError_t launch_cache_append(const AppendParams& p, int sms, cudaStream_t s) {
  const int64_t items = p.T * p.H * (p.D / 8);
  const int64_t blocks = (items + kAppendThreads - 1) / kAppendThreads;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(sms) * 32)));
  return launch_kernel(cache_append_kernel, grid, kAppendThreads, 0, s, p);
}

}  // namespace ffpa
