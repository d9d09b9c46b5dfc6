// The experts' product on 16-bit weights, and with the weights read the other
// way the gradient of its rows:
//   out[p, n] = sum_k A[r(p), k] W[e(p), n, k]     (or W[e(p), k, n])
// with e(p) the expert of p's block and r(p) the row itself or its slot's token.
//
// An expert's blocks lie side by side, so a tile takes as many of them as its rows hold, whatever
// block_m is.
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

// Tile (row tile, column tile) of this workgroup: row tiles go in groups of kTileGroup with all their columns,
// row tiles innermost. Workgroups go round-robin to the 8 XCDs, each with an L2 of its own, so XCD x
// takes the x-th run of kChunk tiles of every 8 kChunk: about what its 32 compute units work on at once.
constexpr int kXcds = 8;
constexpr int kTileGroup = 8;
constexpr int kChunk = 32;
__device__ __forceinline__ void tile_of(int ntiles, int64_t& row_tile, int& column_tile) {
  const int64_t at = (int64_t)blockIdx.x / kXcds;
  const int64_t tile = (at / kChunk * kXcds + blockIdx.x % kXcds) * kChunk + at % kChunk;
  const int64_t per_group = (int64_t)kTileGroup * ntiles;
  const int64_t group = tile / per_group;
  const int rest = (int)(tile - group * per_group);
  row_tile = group * kTileGroup + rest % kTileGroup;
  column_tile = rest / kTileGroup;
}

// Row tile `target`: the tiles are the runs of blocks of one expert, cut into 1 << log_per
// blocks. Returns how many tiles there are, and of this one its first block and its number of blocks (0 where
// there is none). All threads of the workgroup call it. Counting here needs no launch or memory of its
// own. (A workgroup for every block, of which those inside a tile end at once, costs more: they went to every
// other shader engine and left its compute units idle, 2880 us instead of 1805 at 32768 rows, 16 experts,
// 4096 x 7168.)
struct Scan {
  int last[kWaves];   // last block of a wave's 64 where a run begins, or -1
  int count[kWaves];  // tiles that begin in a wave's blocks
  int found;
};
__device__ __forceinline__ int64_t find_tile(const int32_t* expert_ids, int used, int log_per, int64_t target,
                                             Scan& scan, int& block, int& blocks) {
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const uint64_t up_to = ~0ull >> (63 - lane);  // this lane and those below
  if (threadIdx.x == 0) scan.found = -1;
  int begun = 0;       // where the run at the chunk's start begins
  int64_t before = 0;  // tiles in the chunks before
  for (int chunk = 0; chunk < used; chunk += kThreads) {
    const int b = chunk + (int)threadIdx.x;
    const int e = expert_ids[min(b, used - 1)], previous = expert_ids[max(min(b, used) - 1, 0)];
    const uint64_t begins = __ballot(b < used && (b == 0 || e != previous));
    if (lane == 0) scan.last[wave] = begins ? b + 63 - __builtin_clzll(begins) : -1;
    __syncthreads();
    int start = begun;
    for (int i = 0; i < kWaves; ++i) {
      if (i < wave) start = max(start, scan.last[i]);
      begun = max(begun, scan.last[i]);
    }
    const uint64_t mine = begins & up_to;
    if (mine) start = b - lane + 63 - __builtin_clzll(mine);
    const uint64_t heads = __ballot(b < used && ((b - start) & ((1 << log_per) - 1)) == 0);
    if (lane == 0) scan.count[wave] = __builtin_popcountll(heads);
    __syncthreads();
    int64_t index = before + __builtin_popcountll(heads & up_to) - 1;
    for (int i = 0; i < kWaves; ++i) {
      if (i < wave) index += scan.count[i];
      before += scan.count[i];
    }
    if (index == target && (heads >> lane & 1)) scan.found = b;
  }
  __syncthreads();
  block = __builtin_amdgcn_readfirstlane(scan.found);
  __syncthreads();  // the ring's copies go where the counts are
  blocks = 0;
  if (block >= 0) {
    const int i = block + lane;
    const uint64_t other =
        ~__ballot(lane < 1 << log_per && i < used && expert_ids[min(i, used - 1)] == expert_ids[block]);
    blocks = __builtin_ctzll(other);  // at most 16 to a tile, so lane 16 is another
  }
  return before;
}

// A tile of up to 32 WM MT rows and 256 columns; waves lie WM deep, 8 / WM wide.
template <typename T, typename O, bool TRANSPOSED, int WM, int MT>
__device__ __forceinline__ void product(const GroupedParams& p, uint8_t* ring, int first, int rows, int e, int n0) {
  constexpr int WN = kWaves / WM;
  constexpr int NT = kTileN / (32 * WN);
  typedef RowPanel<32 * WM * MT> M;
  typedef std::conditional_t<TRANSPOSED, ColumnPanel<kTileN>, RowPanel<kTileN>> N;
  int lane = (int)threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // addresses made of it are made here: before the loop around this they would spill
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  floatx16 acc[MT][NT] = {};
  M m;
#pragma unroll
  for (int i = 0; i < M::kMine; ++i) {
    // a row without a slot reads row 0 and is zeroed at the store
    const int row = M::row_of(i, wave, lane);
    const uint32_t slot = row < rows ? (uint32_t)p.sorted[first + row] : ~0u;
    const int64_t from = slot >= (uint32_t)p.n_slots ? 0 : p.gather ? (int64_t)p.by_topk.of(slot) : first + row;
    m.set(i, static_cast<const T*>(p.a) + from * p.K, wave, lane);
  }
  const T* w = static_cast<const T*>(p.w) + (int64_t)e * p.N * p.K;
  N n;
  if constexpr (TRANSPOSED) {
    n.set(w + n0, (int64_t)p.N, p.N - n0, wave, lane);
  } else {
#pragma unroll
    for (int i = 0; i < N::kMine; ++i)
      n.set(i, w + (int64_t)min(n0 + N::row_of(i, wave, lane), p.N - 1) * p.K, wave, lane);
  }
  const int at_m = wave / WN * 32 * MT, at_n = wave % WN * 32 * NT;
  loop<T, M, N>(
      ring, (p.K + kStep - 1) / kStep, at_m, at_n, lane, acc,
      [&](int q, uint32_t slot, int stage) { m.copy(q, slot, p.K - stage * kStep, wave); },
      [&](int q, uint32_t slot, int stage) { n.copy(q, slot, p.K - stage * kStep, wave); }, [] {});
  uint32_t slotted[MT];  // which of 32 rows have a slot
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int row = at_m + 32 * i + (lane & 31);
    slotted[i] = (uint32_t)__ballot(row < rows && (uint32_t)p.sorted[first + min(row, rows - 1)] < (uint32_t)p.n_slots);
  }
  drain(ring, at_m, at_n, wave, lane, acc, [&](int row, int column, const float (&v)[8]) {
    if (row >= rows || n0 + column >= p.N) return;
    const bool real = slotted[(row - at_m) / 32] >> (row & 31) & 1;
    float sums[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[i] = real ? v[i] : 0.f;
    store(static_cast<O*>(p.out) + (int64_t)(first + row) * p.N + n0 + column, sums);
  });
}

// Tiles of 32 WM MT rows; a run's last tile takes the half of them where it has no more.
template <typename T, typename O, bool TRANSPOSED, int WM, int MT>
__global__ __launch_bounds__(kThreads, MT == 4 ? 2 : 4) void grouped_kernel(GroupedParams p, int ntiles, int row_tiles,
                                                                            int log_per) {
  constexpr int kRows = 32 * WM * MT;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRingBytes<RowPanel<kRows>, RowPanel<kTileN>>];
  const int used = min(p.capacity, *p.ntpp) / p.block_m;
  int64_t target;
  int nt;
  tile_of(ntiles, target, nt);
  if (target >= row_tiles) return;
  // more tiles than moe_align's order can have: go round again
  for (; target < used; target += row_tiles) {
    int b, blocks;
    const int64_t total = find_tile(p.expert_ids, used, log_per, target, *reinterpret_cast<Scan*>(ring), b, blocks);
    if (blocks == 0) return;
    const int e = p.expert_ids[b];
    const int first = b * p.block_m, rows = blocks * p.block_m, n0 = nt * kTileN;
    if ((uint32_t)e >= (uint32_t)p.E) {  // no such expert
      const float zero[8] = {};
      for (int i = (int)threadIdx.x; i < rows * (kTileN / 8); i += kThreads) {
        const int row = i / (kTileN / 8), column = n0 + 8 * (i % (kTileN / 8));
        if (column < p.N) store(static_cast<O*>(p.out) + (int64_t)(first + row) * p.N + column, zero);
      }
    } else if (MT > 1 && rows <= kRows / 2) {
      product<T, O, TRANSPOSED, WM, (MT + 1) / 2>(p, ring, first, rows, e, n0);
    } else {
      product<T, O, TRANSPOSED, WM, MT>(p, ring, first, rows, e, n0);
    }
    if (target + row_tiles >= total) return;
    __syncthreads();
  }
}

template <typename T, typename O, bool TRANSPOSED>
hipError_t launch(const GroupedParams& p, hipStream_t stream) {
  constexpr int kRows = 256;
  const int ntiles = (p.N + kTileN - 1) / kTileN, per = std::max(1, kRows / p.block_m);
  const int blocks = p.capacity / p.block_m;
  if (blocks == 0) return hipSuccess;
  // an expert's last tile may be of fewer blocks
  const int row_tiles = (std::min(blocks, blocks / per + p.E) + kTileGroup - 1) / kTileGroup * kTileGroup;
  const int64_t tiles = (int64_t)row_tiles * ntiles;
  const int64_t grid = (tiles + kXcds * kChunk - 1) / (kXcds * kChunk) * (kXcds * kChunk);
  hipLaunchKernelGGL((grouped_kernel<T, O, TRANSPOSED, 2, 4>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p,
                     ntiles, row_tiles, __builtin_ctz(per));
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch(const GroupedParams& p, hipStream_t stream) {
  return p.transposed ? launch<T, O, true>(p, stream) : launch<T, O, false>(p, stream);
}

}  // namespace

int64_t grouped_workgroups(int32_t N, int32_t capacity, int32_t block_m) {
  return ((int64_t)(capacity / block_m) + kTileGroup - 1) * ((N + 127) / 128) + kXcds * kChunk;
}

hipError_t launch_grouped_gemm(const GroupedParams& p, int32_t dtype, int32_t out_dtype, hipStream_t stream) {
  if (dtype == kBF16)
    return out_dtype == kFP32 ? launch<bf16_t, float>(p, stream) : launch<bf16_t, bf16_t>(p, stream);
  return out_dtype == kFP32 ? launch<f16_t, float>(p, stream) : launch<f16_t, f16_t>(p, stream);
}

}  // namespace w4a16
