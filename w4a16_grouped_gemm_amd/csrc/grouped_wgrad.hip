// The weights' gradient of the experts' product: for each expert e
//   dW[e, n, k] = sum_p dout[p, n] A[r(p), k]
// over e's rows p that hold a slot, with r(p) the row itself or its slot's token.
//
// A workgroup computes a square tile of one expert's dW over all of its rows (or, where the tiles
// are few, a share of them, and a second kernel adds the shares in their order). Both operands
// are column panels: the rows are the steps of the sum. Rows without a slot, whatever they
// hold, are replaced by zeros as they are copied to LDS (global_load_lds); the mfma loop is in gemm_tile.h.
#include "gemm_tile.h"
#include "grouped_gemm.h"
#include "row_ops.h"

#include <algorithm>
#include <climits>
#include <cstdlib>

namespace w4a16 {
namespace {

using namespace tile;

constexpr int kXcds = 8;

// The tile of expert e of this workgroup: XCD x takes a contiguous eighth of each expert's
// tiles, in groups of 8 rows of tiles.
__device__ __forceinline__ bool tile_of(int mtiles, int ntiles, int& e, int& mt, int& nt) {
  const int total = mtiles * ntiles;
  const int chunk = (total + kXcds - 1) / kXcds;
  const int at = (int)(blockIdx.x / kXcds);
  e = at / chunk;
  const int tile = (int)(blockIdx.x % kXcds) * chunk + at % chunk;
  if (tile >= total) return false;
  const int per_group = 8 * ntiles;
  const int first = tile / per_group * 8;
  const int rows = min(8, mtiles - first);
  const int rest = tile % per_group;
  nt = rest / rows;
  mt = first + rest - nt * rows;
  return true;
}

// kTile x kTile values a workgroup, its waves 2 deep and 4 wide.
template <typename T, typename O, int kTile, bool GATHER>
__global__ __launch_bounds__(kThreads, kTile == 256 ? 2 : 4) void wgrad_kernel(WgradParams p, int mtiles, int ntiles) {
  constexpr int MT = kTile / 64, NT = kTile / 128;
  typedef ColumnPanel<kTile> Panel;
  constexpr int kRows = 64 / Panel::kLanes;  // of a copy
  constexpr int kMine = Panel::kMine;
  static_assert(kMine * kRows == 8, "eight rows a wave");
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRingBytes<Panel, Panel, 2>];
  int* const run = reinterpret_cast<int*>(ring);
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int e, mt, nt;
  if (!tile_of(mtiles, ntiles, e, mt, nt)) return;

  // the expert's first and last block
  const int used = p.capacity > 0 ? min(p.capacity, *p.ntpp) >> p.log_block : 0;
  if (threadIdx.x == 0) run[0] = INT_MAX, run[1] = -1;
  __syncthreads();
  int lo = INT_MAX, hi = -1;
  for (int i = (int)threadIdx.x; i < used; i += kThreads)
    if (p.expert_ids[i] == e) lo = min(lo, i), hi = i;
  if (hi >= 0) {
    atomicMin(&run[0], lo);
    atomicMax(&run[1], hi);
  }
  __syncthreads();
  const int last = __builtin_amdgcn_readfirstlane(run[1]);
  const int begun = __builtin_amdgcn_readfirstlane(run[0]);
  __syncthreads();  // the ring's copies go where the run is
  const int first = last < 0 ? 0 : begun << p.log_block;
  const int end = last < 0 ? 0 : (last + 1) << p.log_block;
  const int share = (((end - first + kStep - 1) / kStep + p.cut.splits - 1) / p.cut.splits) * kStep;
  const int begin = min((int64_t)first + (int64_t)share * blockIdx.y, (int64_t)end);
  const int stop = min((int64_t)begin + share, (int64_t)end);
  const int stages = (stop - begin + kStep - 1) / kStep;

  const int m0 = mt * kTile, n0 = nt * kTile;
  floatx16 acc[MT][NT] = {};
  if (stages > 0) {
    // Which rows a wave copies comes by scalar loads: a vector load's wait would be for every copy issued before it
    // too. They are eight of a stage, of one block.
    typedef const __attribute__((address_space(4))) int32_t* scalar_i32;
    const scalar_i32 sorted = (scalar_i32)(uintptr_t)p.sorted, expert_ids = (scalar_i32)(uintptr_t)p.expert_ids;
    struct Rows {
      int32_t slot[8], owner;  // of a wave's rows of a stage, and their block's expert
      bool inside;
    };
    Rows of_m, of_n;
    auto look = [&](Rows& r, int stage) {
      const int row = begin + stage * kStep + 8 * wave, at = min(row, stop - 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) r.slot[i] = sorted[at + i];
      r.owner = expert_ids[at >> p.log_block];
      r.inside = row < stop;
    };
    const int my_row = lane / Panel::kLanes;
    const int64_t row_m = (int64_t)p.N * (int)sizeof(T), row_n = (int64_t)p.K * (int)sizeof(T);
    const uint8_t *at_m[kMine], *at_n[kMine];  // this lane's 16 bytes in the copies of the next stage (GATHER: of token 0)
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int64_t row = begin + 8 * wave + kRows * q + my_row;
      const int column = 8 * (lane % Panel::kLanes ^ (Panel::swizzle(kRows * q + my_row) << 2));
      at_m[q] = static_cast<const uint8_t*>(p.dout) + row * row_m + 2 * (m0 + (column < p.N - m0 ? column : 0));
      at_n[q] = static_cast<const uint8_t*>(p.a) + (GATHER ? 0 : row * row_n) + 2 * (n0 + (column < p.K - n0 ? column : 0));
    }
    auto copy = [&](const Rows& r, const uint8_t* at, uint32_t slot, int q, uint32_t lds) {
      const bool real = (slot < (uint32_t)p.n_slots) & (r.owner == e) & r.inside;
      copy16(real ? (const void*)at : (const void*)kZeros, lds + 1024 * (kMine * wave + q));
    };
    auto slot_of = [&](const Rows& r, int q) {  // of this lane's row
      int32_t slot = r.slot[kRows * q];
#pragma unroll
      for (int i = 1; i < kRows; ++i) slot = my_row == i ? r.slot[kRows * q + i] : slot;
      return (uint32_t)slot;
    };
    look(of_m, 0);
    look(of_n, 0);
    loop<T, Panel, Panel, 2>(
        ring, stages, wave / 4 * 32 * MT, wave % 4 * 32 * NT, lane, acc,
        [&](int q, uint32_t lds, int stage) {
          copy(of_m, at_m[q], slot_of(of_m, q), q, lds);
          at_m[q] += kStep * row_m;
          if (q == kMine - 1) look(of_m, stage + 1);
        },
        [&](int q, uint32_t lds, int stage) {
          const uint32_t slot = slot_of(of_n, q);
          copy(of_n, GATHER ? at_n[q] + (uint64_t)p.by_topk.of(slot) * (uint32_t)row_n : at_n[q], slot, q, lds);
          if (!GATHER) at_n[q] += kStep * row_n;
          if (q == kMine - 1) look(of_n, stage + 1);
        },
        [&] {
          asm volatile(""
                       : "+s"(of_m.slot[0]), "+s"(of_m.slot[1]), "+s"(of_m.slot[2]), "+s"(of_m.slot[3]),
                         "+s"(of_m.slot[4]), "+s"(of_m.slot[5]), "+s"(of_m.slot[6]), "+s"(of_m.slot[7]), "+s"(of_m.owner));
          asm volatile(""
                       : "+s"(of_n.slot[0]), "+s"(of_n.slot[1]), "+s"(of_n.slot[2]), "+s"(of_n.slot[3]),
                         "+s"(of_n.slot[4]), "+s"(of_n.slot[5]), "+s"(of_n.slot[6]), "+s"(of_n.slot[7]), "+s"(of_n.owner));
        });
  }

  const int64_t size = (int64_t)p.E * p.N * p.K;
  if (p.cut.splits > 1) {
    float* partial = p.partial + (int64_t)blockIdx.y * size;
    drain<float>(ring, wave / 4 * 32 * MT, wave % 4 * 32 * NT, wave, lane, acc, [&](int n, int k, float (&v)[4]) {
      if (m0 + n < p.N && n0 + k < p.K) Line<float>::store(partial + ((int64_t)e * p.N + m0 + n) * p.K + n0 + k, v);
    });
  } else {
    drain<O>(ring, wave / 4 * 32 * MT, wave % 4 * 32 * NT, wave, lane, acc, [&](int n, int k, float (&v)[Line<O>::kEach]) {
      if (m0 + n >= p.N || n0 + k >= p.K) return;
      O* dw = static_cast<O*>(p.dw) + ((int64_t)e * p.N + m0 + n) * p.K + n0 + k;
      if (p.accumulate) Line<O>::add(dw, v);
      Line<O>::store(dw, v);
    });
  }
}

// dW (+)= the shares, in their order.
template <typename O>
__global__ __launch_bounds__(256) void join_kernel(const float* partial, O* dw, int64_t size, int32_t splits,
                                                   int32_t accumulate) {
  constexpr int kEach = Line<O>::kEach;
  const int64_t stride = (int64_t)gridDim.x * 256 * kEach;
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kEach; at < size; at += stride) {
    float sums[kEach] = {};
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int i = 0; i < kEach; i += 4) {
        const floatx4 part = *reinterpret_cast<const floatx4*>(partial + s * size + at + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) sums[i + k] += part[k];
      }
    if (accumulate) Line<O>::add(dw + at, sums);
    Line<O>::store(dw + at, sums);
  }
}

template <typename T, typename O, int kTile>
hipError_t launch_tile(const WgradParams& p, hipStream_t stream) {
  const int mtiles = (p.N + kTile - 1) / kTile, ntiles = (p.K + kTile - 1) / kTile;
  const int64_t chunk = ((int64_t)mtiles * ntiles + kXcds - 1) / kXcds;
  const int64_t grid = chunk * kXcds * p.E;
  const dim3 g((unsigned)grid, (unsigned)p.cut.splits), t(kThreads);
  if (p.gather)
    hipLaunchKernelGGL((wgrad_kernel<T, O, kTile, true>), g, t, 0, stream, p, mtiles, ntiles);
  else
    hipLaunchKernelGGL((wgrad_kernel<T, O, kTile, false>), g, t, 0, stream, p, mtiles, ntiles);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch(const WgradParams& p, hipStream_t stream) {
  const hipError_t err = p.cut.tile == 256 ? launch_tile<T, O, 256>(p, stream) : launch_tile<T, O, 128>(p, stream);
  if (err != hipSuccess || p.cut.splits == 1) return err;
  const int64_t size = (int64_t)p.E * p.N * p.K;
  const int64_t grid = std::min<int64_t>((size / Line<O>::kEach + 255) / 256, (int64_t)device_cu_count() * 32);
  hipLaunchKernelGGL((join_kernel<O>), dim3((unsigned)grid), dim3(256), 0, stream, p.partial, static_cast<O*>(p.dw),
                     size, p.cut.splits, p.accumulate);
  return hipGetLastError();
}

}  // namespace

int64_t wgrad_workgroups(int32_t E, int32_t N, int32_t K, int32_t splits) {
  const int64_t tiles = (int64_t)((N + 127) / 128) * ((K + 127) / 128);
  return (tiles + kXcds - 1) / kXcds * kXcds * E * splits;
}

WgradCut wgrad_cut(int32_t E, int32_t N, int32_t K, int32_t capacity) {
  const char* v = getenv("WG");
  auto tiles = [&](int64_t t) { return E * ((N + t - 1) / t) * ((K + t - 1) / t); };
  const int64_t rows = capacity / E;
  WgradCut c;
  c.tile = v ? atoi(v) / 100 : tiles(256) >= 256 ? 256 : 128;
  c.splits = v ? atoi(v) % 100 : (int32_t)std::max<int64_t>(1, std::min<int64_t>({(c.tile == 256 ? 256 : 512) / tiles(c.tile), rows / 256, 16}));
  return c;
}

hipError_t launch_grouped_wgrad(const WgradParams& p, int32_t dtype, int32_t dw_dtype, hipStream_t stream) {
  if (dtype == kBF16)
    return dw_dtype == kFP32 ? launch<bf16_t, float>(p, stream) : launch<bf16_t, bf16_t>(p, stream);
  return dw_dtype == kFP32 ? launch<f16_t, float>(p, stream) : launch<f16_t, f16_t>(p, stream);
}

}  // namespace w4a16
