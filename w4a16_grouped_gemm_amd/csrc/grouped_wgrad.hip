// The weights' gradient of the experts' product: for each expert e
//   dW[e, n, k] = sum_p dout[p, n] A[r(p), k]
// over e's rows p that hold a slot, with r(p) the row itself or its slot's token.
//
// A workgroup computes a square tile of one expert's dW over all of its rows (or, where the tiles
// are few, a share of them, and a second kernel adds the shares in their order). Both operands
// are column panels: the rows are the steps of the sum. Rows without a slot, whatever they
// hold, are replaced by zeros as they are copied to LDS.
// The copies to LDS (global_load_lds) and the mfma loop are in gemm_tile.h.
#include "gemm_tile.h"
#include "grouped_gemm.h"
#include "row_ops.h"

#include <algorithm>
#include <climits>

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

// kTile x kTile values a workgroup, its waves 2 deep and 4 wide. In LDS a row's kTile values of dout
// and of a lie side by side, so that one copy of a wave fetches both.
template <typename T, typename O, int kTile>
__global__ __launch_bounds__(kThreads, kTile == 256 ? 2 : 4) void wgrad_kernel(WgradParams p, int mtiles, int ntiles) {
  constexpr int MT = kTile / 64, NT = kTile / 128;
  constexpr int kPitch = 4 * kTile;
  typedef ColumnPanel<kTile, kPitch> Panel;
  constexpr int kRowLanes = kPitch / 16, kUnitRows = 64 / kRowLanes;
  constexpr int kMine = kStep / kUnitRows / kWaves;  // copies a wave and stage
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * kStep * kPitch];
  __shared__ int run[2];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int e, mt, nt;
  if (!tile_of(mtiles, ntiles, e, mt, nt)) return;

  // the expert's first and last block
  const int used = p.capacity > 0 ? min(p.capacity, *p.ntpp) / p.block_m : 0;
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
  const int first = last < 0 ? 0 : __builtin_amdgcn_readfirstlane(run[0]) * p.block_m;
  const int end = last < 0 ? 0 : (last + 1) * p.block_m;
  const int share = (((end - first + kStep - 1) / kStep + p.splits - 1) / p.splits) * kStep;
  const int begin = min((int64_t)first + (int64_t)share * blockIdx.y, (int64_t)end);
  const int stop = min((int64_t)begin + share, (int64_t)end);
  const int stages = (stop - begin + kStep - 1) / kStep;

  const int m0 = mt * kTile, n0 = nt * kTile;
  floatx16 acc[MT][NT] = {};
  if (stages > 0) {
    // Each lane copies 16 bytes of dout or of a: rows `wave_row` + kUnitRows q + my_row of a stage.
    const int my_row = lane / kRowLanes, part = lane % kRowLanes;
    const bool of_a = part >= kRowLanes / 2;
    const int wave_row = wave * kMine * kUnitRows;
    const int chunk = part % (kRowLanes / 2);
    const uint32_t ld = (uint32_t)(of_a ? p.K : p.N) * (uint32_t)sizeof(T);
    const uint8_t* base = static_cast<const uint8_t*>(of_a ? p.a : p.dout) + (of_a ? n0 : m0) * (int)sizeof(T);
    const int columns = of_a ? p.K - n0 : p.N - m0;
    const bool by_slot = of_a && p.gather;
    const Divisor by_topk = p.by_topk;
    // The slots of the rows to be copied next. A wave's rows of a stage are eight, so in one block.
    int32_t slot[kMine], owner;
    auto look = [&](int stage) {
      const int row = begin + stage * kStep + wave_row;
#pragma unroll
      for (int q = 0; q < kMine; ++q) slot[q] = p.sorted[min(row + kUnitRows * q + my_row, stop - 1)];
      owner = p.expert_ids[min(row, stop - 1) / p.block_m];
    };
    look(0);
    loop<T, Panel, Panel, MT, NT, kMine, 2 * kTile, kStep * kPitch>(
        ring, stages, wave / 4 * 32 * MT, wave % 4 * 32 * NT, lane, acc, [&](int q, uint32_t lds, int stage) {
          const int step = wave_row + kUnitRows * q + my_row, row = begin + stage * kStep + step;
          const bool real = (row < stop) & ((uint32_t)slot[q] < (uint32_t)p.n_slots) & (owner == e);
          const uint32_t from = by_slot ? by_topk.of((uint32_t)slot[q]) : (uint32_t)row;
          const int column = 8 * (chunk ^ (Panel::swizzle(step) << 2));
          const uint8_t* at = base + (uint64_t)from * ld + 2 * (column < columns ? column : 0);
          copy16(real ? (const void*)at : (const void*)kZeros, lds + 1024 * (kMine * wave + q));
          if (q == kMine - 1) look(stage + 1);
        });
  }

  const int64_t size = (int64_t)p.E * p.N * p.K;
  drain(ring, wave / 4 * 32 * MT, wave % 4 * 32 * NT, wave, lane, acc, [&](int n, int k, const float (&v)[8]) {
    if (m0 + n >= p.N || n0 + k >= p.K) return;
    const int64_t at = ((int64_t)e * p.N + m0 + n) * p.K + n0 + k;
    if (p.splits > 1) {
      store(p.partial + (int64_t)blockIdx.y * size + at, v);
      return;
    }
    O* dw = static_cast<O*>(p.dw) + at;
    float sums[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[i] = v[i];
    if (p.accumulate) {
      const Eight<O> old = load8(dw);
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[i] += (float)old.v[i];
    }
    store(dw, sums);
  });
}

// dW (+)= the shares, in their order.
template <typename O>
__global__ __launch_bounds__(256) void join_kernel(const float* partial, O* dw, int64_t size, int32_t splits,
                                                   int32_t accumulate) {
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; at < size; at += (int64_t)gridDim.x * 256 * 8) {
    float sums[8] = {};
    for (int s = 0; s < splits; ++s) {
      const Eight<float> part = load8(partial + s * size + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[i] += part.v[i];
    }
    if (accumulate) {
      const Eight<O> old = load8(dw + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[i] += (float)old.v[i];
    }
    store(dw + at, sums);
  }
}

template <typename T, typename O, int kTile>
hipError_t launch_tile(const WgradParams& p, hipStream_t stream) {
  const int mtiles = (p.N + kTile - 1) / kTile, ntiles = (p.K + kTile - 1) / kTile;
  const int64_t chunk = ((int64_t)mtiles * ntiles + kXcds - 1) / kXcds;
  const int64_t grid = chunk * kXcds * p.E;
  hipLaunchKernelGGL((wgrad_kernel<T, O, kTile>), dim3((unsigned)grid, (unsigned)p.splits), dim3(kThreads), 0, stream,
                     p, mtiles, ntiles);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch(const WgradParams& p, hipStream_t stream) {
  const hipError_t err = launch_tile<T, O, 256>(p, stream);
  if (err != hipSuccess || p.splits == 1) return err;
  const int64_t size = (int64_t)p.E * p.N * p.K;
  const int64_t grid = std::min<int64_t>((size / 8 + 255) / 256, (int64_t)device_cu_count() * 32);
  hipLaunchKernelGGL((join_kernel<O>), dim3((unsigned)grid), dim3(256), 0, stream, p.partial, static_cast<O*>(p.dw),
                     size, p.splits, p.accumulate);
  return hipGetLastError();
}

}  // namespace

int64_t wgrad_workgroups(int32_t E, int32_t N, int32_t K, int32_t splits) {
  const int64_t tiles = (int64_t)((N + 127) / 128) * ((K + 127) / 128);
  return (tiles + kXcds - 1) / kXcds * kXcds * E * splits;
}

int32_t wgrad_splits(int32_t E, int32_t N, int32_t K, int32_t capacity) {
  const int64_t tiles = (int64_t)E * ((N + 255) / 256) * ((K + 255) / 256);
  const int64_t rows = capacity / E;
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>({256 / tiles, rows / 256, 16}));
}

hipError_t launch_grouped_wgrad(const WgradParams& p, int32_t dtype, int32_t dw_dtype, hipStream_t stream) {
  if (dtype == kBF16)
    return dw_dtype == kFP32 ? launch<bf16_t, float>(p, stream) : launch<bf16_t, bf16_t>(p, stream);
  return dw_dtype == kFP32 ? launch<f16_t, float>(p, stream) : launch<f16_t, f16_t>(p, stream);
}

}  // namespace w4a16
