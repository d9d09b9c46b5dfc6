// The experts' product on 16-bit weights, and with the weights read the other
// way the gradient of its rows:
//   out[p, n] = sum_k A[r(p), k] W[e(p), n, k]     (or W[e(p), k, n])
// with e(p) the expert of p's block and r(p) the row itself or its slot's token.
//
// An expert's blocks lie side by side, so a tile takes as many of them as its
// rows hold, whatever block_m is: the workgroup of a run's first block, and
// of every (tile rows / block_m)-th after it, computes the tile, the others'
// workgroups end at once.
// The copies to LDS (global_load_lds) and the mfma loop are in gemm_tile.h.
#include "gemm_tile.h"
#include "grouped_gemm.h"
#include "row_ops.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

using namespace tile;

constexpr int kTileN = 256;

// The tile (block b, columns nt * kTileN on) of this workgroup, from the blocks in use.
// Workgroups go round-robin to the 8 XCDs, each with an L2 of its own: XCD x takes a
// contiguous eighth of the tiles, in groups of `group` blocks with all their columns,
// blocks innermost.
constexpr int kXcds = 8;
__device__ __forceinline__ bool tile_of(int used, int ntiles, int group, int& b, int& nt) {
  const int64_t total = (int64_t)used * ntiles;
  const int64_t chunk = (total + kXcds - 1) / kXcds;
  const int64_t at = (int64_t)blockIdx.x / kXcds;
  const int64_t tile = ((int64_t)blockIdx.x % kXcds) * chunk + at;
  if (at >= chunk || tile >= total) return false;
  const int64_t per_group = (int64_t)group * ntiles;
  const int first = (int)(tile / per_group) * group;
  const int rows = min(group, used - first);
  const int rest = (int)(tile % per_group);
  nt = rest / rows;
  b = first + rest - nt * rows;
  return true;
}

// The blocks of expert e from b on that a tile at b takes, at most `per`; 0 where b belongs
// to a tile that begins before it.
__device__ __forceinline__ int run_of(const int32_t* expert_ids, int used, int b, int e, int per, int lane) {
  int before = 0;  // blocks of e right before b
  for (int at = b - 1;; at -= 64) {
    const int i = at - lane;
    const uint64_t other = ~__ballot(i >= 0 && expert_ids[max(i, 0)] == e);
    if (other) {
      before += __builtin_ctzll(other);
      break;
    }
    before += 64;
  }
  if (before % per) return 0;
  const int i = b + lane;
  const uint64_t other = ~__ballot(lane < per && i < used && expert_ids[min(i, used - 1)] == e);
  return __builtin_ctzll(other);  // per <= 16, so lane 16 is another
}

// A tile of up to 32 WM MT rows and 256 columns; waves lie WM deep, 8 / WM wide.
template <typename T, typename O, bool TRANSPOSED, int WM, int MT>
__device__ __forceinline__ void product(const GroupedParams& p, uint8_t* ring, int first, int rows, int e, int n0) {
  constexpr int WN = kWaves / WM;
  constexpr int NT = kTileN / (32 * WN);
  typedef RowPanel<32 * WM * MT> M;
  typedef std::conditional_t<TRANSPOSED, ColumnPanel<kTileN>, RowPanel<kTileN>> N;
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  floatx16 acc[MT][NT] = {};
  M m;
#pragma unroll
  for (int i = 0; i < M::kMine; ++i) {
    const int row = M::row_of(i, wave, lane);
    const uint32_t slot = row < rows ? (uint32_t)p.sorted[first + row] : ~0u;
    const int64_t from = p.gather ? (int64_t)(slot / (uint32_t)p.topk) : first + row;
    m.set(i, slot < (uint32_t)p.n_slots ? static_cast<const T*>(p.a) + from * p.K : nullptr, p.K, wave, lane);
  }
  const T* w = static_cast<const T*>(p.w) + (int64_t)e * p.N * p.K;
  N n;
  if constexpr (TRANSPOSED) {
    n.set(w + n0, (int64_t)p.N, p.N - n0, p.K, wave, lane);
  } else {
#pragma unroll
    for (int i = 0; i < N::kMine; ++i) {
      const int column = n0 + N::row_of(i, wave, lane);
      n.set(i, column < p.N ? w + (int64_t)column * p.K : nullptr, p.K, wave, lane);
    }
  }
  const int at_m = wave / WN * 32 * MT, at_n = wave % WN * 32 * NT;
  loop<T, M, N>(ring, (p.K + kStep - 1) / kStep, at_m, at_n, lane, acc, [&](uint32_t lds) {
    m.issue(lds, wave);
    n.issue(lds + M::kBytes, wave);
  });
  drain(ring, at_m, at_n, wave, lane, acc, [&](int row, int column, const float (&v)[8]) {
    if (row >= rows || n0 + column >= p.N) return;
    const bool real = (uint32_t)p.sorted[first + row] < (uint32_t)p.n_slots;
    float sums[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[i] = real ? v[i] : 0.f;
    store(static_cast<O*>(p.out) + (int64_t)(first + row) * p.N + n0 + column, sums);
  });
}

// Tiles of 32 WM MT rows; a run's last tile takes the half of them where it has no more.
template <typename T, typename O, bool TRANSPOSED, int WM, int MT>
__global__ __launch_bounds__(kThreads, MT == 4 ? 2 : 4) void grouped_kernel(GroupedParams p, int ntiles, int group) {
  constexpr int kRows = 32 * WM * MT;
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * (kRows + kTileN) * 128];
  const int lane = (int)threadIdx.x & 63;
  const int used = min(p.capacity, *p.ntpp) / p.block_m;
  int b, nt;
  if (!tile_of(used, ntiles, group, b, nt)) return;
  const int e = p.expert_ids[b];
  const int blocks = run_of(p.expert_ids, used, b, e, max(kRows / p.block_m, 1), lane);
  if (blocks == 0) return;
  const int first = b * p.block_m, n0 = nt * kTileN;
  if ((uint32_t)e >= (uint32_t)p.E) {  // no such expert
    const float zero[8] = {};
    for (int64_t i = threadIdx.x; i < (int64_t)blocks * p.block_m * (kTileN / 8); i += kThreads) {
      const int row = (int)(i / (kTileN / 8)), column = n0 + 8 * (int)(i % (kTileN / 8));
      if (column < p.N) store(static_cast<O*>(p.out) + (int64_t)(first + row) * p.N + column, zero);
    }
    return;
  }
  const int rows = blocks * p.block_m;
  if (MT > 1 && rows <= kRows / 2)
    product<T, O, TRANSPOSED, WM, (MT + 1) / 2>(p, ring, first, rows, e, n0);
  else
    product<T, O, TRANSPOSED, WM, MT>(p, ring, first, rows, e, n0);
}

template <typename T, typename O, bool TRANSPOSED>
hipError_t launch(const GroupedParams& p, hipStream_t stream) {
  const int ntiles = (p.N + kTileN - 1) / kTileN;
  const int64_t tiles = (int64_t)(p.capacity / p.block_m) * ntiles;
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid == 0) return hipSuccess;
  const dim3 g((unsigned)grid), t(kThreads);
  hipLaunchKernelGGL((grouped_kernel<T, O, TRANSPOSED, 2, 4>), g, t, 0, stream, p, ntiles, std::max(1, 2048 / p.block_m));
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch(const GroupedParams& p, hipStream_t stream) {
  return p.transposed ? launch<T, O, true>(p, stream) : launch<T, O, false>(p, stream);
}

}  // namespace

int64_t grouped_workgroups(int32_t N, int32_t capacity, int32_t block_m) {
  return (int64_t)(capacity / block_m) * ((N + 127) / 128) + kXcds - 1;
}

hipError_t launch_grouped_gemm(const GroupedParams& p, int32_t dtype, int32_t out_dtype, hipStream_t stream) {
  if (dtype == kBF16)
    return out_dtype == kFP32 ? launch<bf16_t, float>(p, stream) : launch<bf16_t, bf16_t>(p, stream);
  return out_dtype == kFP32 ? launch<f16_t, float>(p, stream) : launch<f16_t, f16_t>(p, stream);
}

}  // namespace w4a16
