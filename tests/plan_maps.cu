// The plan kernel of packed sequences, alone: the TMA map it makes of each sequence against
// the map the encoder makes of it, and its tile list.  Nothing is read through the maps.
// The plan's maps all have the form of the encoder's smallest tensor.  The encoder may give
// large tensors another one: those of its maps may differ from the plan's, but all in the
// same bits, and they are larger than all that do not.
// Prints what differs; exit status 0 when nothing else does.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <set>
#include <utility>
#include <vector>

#include "../head_dim_attention_gb300/csrc/internal.h"

using namespace ffpa;

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Tensor {
  char* base;
  int64_t D, heads, row_stride, head_stride;
  int box_rows;
  bool bf16;
};

static EncodeFn encode_fn;
static CUtensorMap encode(const Tensor& t, int64_t first, int64_t rows, int64_t heads) {
  CUtensorMap m;
  const cuuint64_t dims[4] = {(cuuint64_t)t.D, (cuuint64_t)rows, (cuuint64_t)heads, 1};
  const cuuint64_t strides[3] = {(cuuint64_t)t.row_stride * 2, (cuuint64_t)t.head_stride * 2,
                                 (cuuint64_t)(t.head_stride * t.heads) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)t.box_rows, 1, 1}, one[4] = {1, 1, 1, 1};
  const CUresult r = encode_fn(&m, t.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                               t.base + 2 * first * t.row_stride, dims, strides, box, one,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    std::printf("encode failed: %d\n", r);
    std::exit(2);
  }
  return m;
}

struct Map {
  uint64_t w[16] = {};
  Map() = default;
  explicit Map(const CUtensorMap& m) { std::memcpy(w, &m, sizeof w); }
  bool operator==(const Map& o) const { return std::equal(w, w + 16, o.w); }
  Map operator^(const Map& o) const {
    Map r;
    for (int i = 0; i < 16; ++i) r.w[i] = w[i] ^ o.w[i];
    return r;
  }
};

static void ok(cudaError_t e) {
  if (e == cudaSuccess) return;
  std::printf("%s\n", cudaGetErrorString(e));
  std::exit(2);
}

int main() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  ok(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found));
  encode_fn = reinterpret_cast<EncodeFn>(fn);
  const size_t capacity = 1 << 24;
  char *data, *scratch;
  uint32_t* status;
  int32_t* cu;
  ok(cudaMalloc(&data, 1 << 20));
  ok(cudaMalloc(&scratch, capacity));
  ok(cudaMalloc(&status, sizeof *status));
  ok(cudaMalloc(&cu, 4096 * sizeof *cu));
  ok(cudaMemset(status, 0, sizeof *status));
  std::mt19937 gen(7);
  auto draw = [&](int a, int b) { return std::uniform_int_distribution<int>(a, b)(gen); };
  const int edges[] = {63, 64, 65, 127, 128, 129, 255, 256, 257};
  long maps = 0, large = 0, wrong_maps = 0, wrong_tiles = 0;
  int64_t largest_equal = 0, smallest_other = INT64_MAX;  // elements between a map's first and last
  Map form;                                               // what large tensors' maps differ in
  for (int call = 0; call < 2000; ++call) {
    const int n = call % 50 == 0 ? draw(500, 3000) : draw(1, 12);
    std::vector<int> lens(n), first(n + 1, 0);
    for (int& x : lens) {
      const int kind = draw(0, 4);
      x = kind == 0 ? 0 : kind == 1 ? 1 : kind == 2 ? draw(1, 400) : kind == 3 ? edges[draw(0, 8)] : draw(1, 20000);
      if (call % 7 && x > 400) x = 5;
    }
    if (std::all_of(lens.begin(), lens.end(), [](int x) { return x == 0; })) lens[0] = 5;
    for (int s = 0; s < n; ++s) first[s + 1] = first[s] + lens[s];
    const int64_t T = first[n], D = 64 * draw(1, 16);
    VarPlan p;
    p.n_maps = draw(3, kVarMaps);
    Tensor t[kVarMaps];
    for (int w = 0; w < p.n_maps; ++w) {
      const int64_t heads = draw(1, 15);
      const bool token_major = draw(0, 1);
      t[w] = Tensor{data + 512 * draw(0, 1000), D, heads, token_major ? heads * D : D, token_major ? D : T * D,
                    draw(0, 1) ? 64 : 128, draw(0, 1) == 1};
      p.maps[w] = encode(t[w], 0, 1, 1);
      p.heads[w] = static_cast<int>(heads);
      p.base[w] = t[w].base;
      p.row_stride[w] = t[w].row_stride;
    }
    p.cu = cu;
    p.n_seqs = n;
    p.total = static_cast<int>(T);
    p.causal = draw(0, 1);
    p.slots = static_cast<int>(std::min<int64_t>((T + 127ll * n) / 128, T));
    for (p.bin_shift = 0; (T / 128 + 1) >> p.bin_shift >= 1024;) ++p.bin_shift;
    const size_t map_bytes = static_cast<size_t>(n) * kVarMaps * sizeof(CUtensorMap);
    if (map_bytes + p.slots * sizeof(int4) > capacity) return std::printf("scratch too small\n"), 2;
    p.out_maps = reinterpret_cast<CUtensorMap*>(scratch);
    p.tiles = reinterpret_cast<int4*>(scratch + map_bytes);
    p.status = status;
    ok(cudaMemcpy(cu, first.data(), first.size() * sizeof(int32_t), cudaMemcpyHostToDevice));
    ok(launch_varlen_plan(p, nullptr));
    std::vector<CUtensorMap> got(static_cast<size_t>(n) * kVarMaps);
    std::vector<int4> tiles(p.slots);
    ok(cudaMemcpy(got.data(), scratch, map_bytes, cudaMemcpyDeviceToHost));
    ok(cudaMemcpy(tiles.data(), scratch + map_bytes, p.slots * sizeof(int4), cudaMemcpyDeviceToHost));
    int all = 0;
    for (int s = 0; s < n; ++s) {
      all += (lens[s] + 127) / 128;
      for (int w = 0; lens[s] && w < p.n_maps; ++w) {
        const Map want(encode(t[w], first[s], lens[s], t[w].heads)), is(got[static_cast<size_t>(s) * kVarMaps + w]);
        const Map diff = want ^ is;
        const int64_t span = t[w].D + (lens[s] - 1) * t[w].row_stride + (t[w].heads - 1) * t[w].head_stride;
        ++maps;
        bool wrong = false;
        if (diff == Map()) {
          largest_equal = std::max(largest_equal, span);
        } else {
          ++large;
          if (large == 1) form = diff;
          wrong = !(diff == form);
          smallest_other = std::min(smallest_other, span);
        }
        if (wrong && wrong_maps++ < 5)
          std::printf("map differs: %d rows from %d of %lld, D %lld, %lld heads, strides %lld %lld\n", lens[s], first[s],
                      (long long)T, (long long)D, (long long)t[w].heads, (long long)t[w].row_stride,
                      (long long)t[w].head_stride);
      }
    }
    std::set<std::pair<int, int>> seen;
    int work_before = 1 << 30;
    for (int i = 0; i < p.slots; ++i) {
      const int4 x = tiles[i];
      if (i >= all) {
        wrong_tiles += x.x != -1;
        continue;
      }
      const bool good = x.x >= 0 && x.x < n && x.z == first[x.x] && x.w == lens[x.x] && x.y >= 0 && 128 * x.y < x.w &&
                        seen.insert({x.x, x.y}).second;
      const int work = (p.causal ? x.y + 1 : (x.w + 127) / 128) >> p.bin_shift;
      wrong_tiles += !good || work > work_before;  // heaviest first
      work_before = work;
    }
    wrong_tiles += static_cast<int>(seen.size()) != all;
  }
  uint32_t word = 0;
  ok(cudaMemcpy(&word, status, sizeof word, cudaMemcpyDeviceToHost));
  std::printf("%ld maps, %ld of them of large tensors, %ld wrong; sizes %s; %ld wrong tiles; status %u\n", maps, large,
              wrong_maps, largest_equal < smallest_other ? "apart" : "mixed", wrong_tiles, word);
  return wrong_maps || largest_equal >= smallest_other || wrong_tiles || word || maps == large;
}
