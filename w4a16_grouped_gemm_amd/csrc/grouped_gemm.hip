// The experts' product on 16-bit weights, and with the weights read the other
// way the gradient of its rows:
//   out[p, n] = sum_k A[r(p), k] W[e(p), n, k]     (or W[e(p), k, n])
// with e(p) the expert of p's block and r(p) the row itself or its slot's token.
//
// Weights and rows go from memory straight to LDS (global_load_lds) and from there to the mfma
// instructions (gemm_tile.h). An expert's blocks lie side by side, so a tile takes as many of them as its rows
// hold, whatever block_m is. Tiles are 256 x 256 where that fills the card: 128 flops a byte copied from L2,
// and at half of that (128 x 128) the copies alone would take the time of the products. Tiles whose blocks fill at most
// half of their rows multiply half. Rows count by blocks here: a block's padding is multiplied as its real rows are,
// also in a tile that a large block of few rows leaves without any.
//
// Measured (one MI355X, bf16): 32768 rows on 16 experts, 4096 x 7168: 1560..1670 us by card, 1.15..1.23 PFLOP/s, with
// transposed weights 1550..1680; one expert of 8192 rows, 8192 x 8192: 804 us, 1.37. The clock is what gives: under
// this load it falls to 1.6 GHz of 2.4 (a timing build without copies, on LDS that stays as it is, keeps 2.4). 48 experts
// of 85 rows, 7168 x 2048: 320..340 us, 4.6 TB/s; of three rows, 4096 x 7168: 420..450 us, 6.1 TB/s (reads
// alone reach 6.9); one token on 8 of 64 experts, 512 x 7168: 12.3 us, 4.8 TB/s.
#include "gemm_tile.h"
#include "grouped_gemm.h"
#include "row_ops.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

using namespace tile;

// Tile (row tile, column tile) of this workgroup: row tiles go in groups of kTileGroup with all their columns,
// row tiles innermost. XCD x takes the x-th run of 1 << log_run tiles of every 8 runs: about what its 32 compute
// units work on at once.
constexpr int kTileGroup = 8;
constexpr int kLogRun = 5;
__device__ __forceinline__ void tile_of(int ntiles, int log_run, int64_t& row_tile, int& column_tile) {
  const int64_t at = (int64_t)blockIdx.x / kXcds;
  const int64_t tile = (((at >> log_run) * kXcds + blockIdx.x % kXcds) << log_run) + (at & ((1 << log_run) - 1));
  const int64_t per_group = (int64_t)kTileGroup * ntiles;
  const int64_t group = tile / per_group;
  const int rest = (int)(tile - group * per_group);
  row_tile = group * kTileGroup + rest % kTileGroup;
  column_tile = rest / kTileGroup;
}

// How a call is cut into tiles.
struct Cut {
  int ntiles, row_tiles;  // of columns; of rows, as many as moe_align's order can have at most
  int log_per, log_cut;   // blocks a tile, or tiles a block
  int log_run;            // as in tile_of
};

// Row tile `target`: the tiles are the runs of blocks of one expert, cut into 1 << log_per
// blocks. All threads of the workgroup call it. Counting here needs no launch or memory of its own. (A workgroup for every
// block, of which those inside a tile end at once, costs more: they went to every other shader engine and left its
// compute units idle, 2880 us instead of 1805 at 32768 rows, 16 experts, 4096 x 7168.)
struct Scan {
  int last[kWaves];   // last of a wave's blocks where a run begins, or -1
  int count[kWaves];  // tiles that begin in a wave's blocks
  int found;
};
struct RowTile {
  int64_t total;  // tiles there are
  int block;      // the first block
  int blocks;     // 0: no such tile
  int expert;
};
__device__ __forceinline__ RowTile find_tile(const GroupedParams& p, int log_per, int64_t target, Scan& scan) {
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int per = 1 << log_per, held = p.capacity / p.block_m;
  const int32_t* expert_ids = p.expert_ids;
  const uint64_t up_to = ~0ull >> (63 - lane);  // this lane and those below
  const int first64 = expert_ids[min(lane, held - 1)];  // on its way together with the count
  const int used = min(p.capacity, *p.ntpp) / p.block_m;
  RowTile t = {0, 0, 0, 0};
  if (used <= 64) {  // a lane a block, every wave by itself
    const int previous = __shfl_up(first64, 1);
    const uint64_t begins = __ballot(lane < used && (lane == 0 || first64 != previous));
    const int start = 63 - __builtin_clzll((begins & up_to) | 1);
    const uint64_t heads = __ballot(lane < used && ((lane - start) & (per - 1)) == 0);
    t.total = __builtin_popcountll(heads);
    if (target >= t.total) return t;
    const uint64_t found = __ballot((heads >> lane & 1) && __builtin_popcountll(heads & up_to) == target + 1);
    t.block = __builtin_ctzll(found);
    const uint64_t after = t.block == 63 ? 0 : (begins | heads) >> (t.block + 1);  // where the next tile begins
    t.blocks = min(after ? __builtin_ctzll(after) + 1 : used - t.block, used - t.block);
    t.expert = __builtin_amdgcn_readlane(first64, t.block);
    return t;
  }
  if (target >= used) return t;
  if (threadIdx.x == 0) scan.found = -1;
  // a wave takes `steps` times 64 blocks that follow each other, the workgroup 8192 at most
  const int steps = min((used + kThreads - 1) / kThreads, 16);
  int begun = 0;  // where the run at the chunk's start begins
  for (int chunk = 0; chunk < used; chunk += kThreads * steps) {
    const int base = chunk + wave * 64 * steps;
    int before = expert_ids[max(min(base, used) - 1, 0)], last = -1;
    uint32_t mine = 0;  // which of this lane's blocks begin a run
    for (int j = 0; j < steps; j += 4) {
      int id[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) id[i] = expert_ids[min(base + 64 * (j + i) + lane, used - 1)];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = base + 64 * (j + i) + lane, below = __shfl_up(id[i], 1);
        mine |= (uint32_t)((b < used) & ((b == 0) | (id[i] != (lane == 0 ? before : below)))) << (j + i);
        before = __builtin_amdgcn_readlane(id[i], 63);
      }
    }
    for (int j = 0; j < steps; ++j) {
      const uint64_t begins = __ballot(mine >> j & 1);
      if (begins) last = base + 64 * j + 63 - __builtin_clzll(begins);
    }
    if (lane == 0) scan.last[wave] = last;
    __syncthreads();
    int start = begun;
    for (int i = 0; i < kWaves; ++i) {
      if (i < wave) start = max(start, scan.last[i]);
      begun = max(begun, scan.last[i]);
    }
    uint32_t heads = 0;
    int count = 0;
    for (int j = 0; j < steps; ++j) {
      const int first = base + 64 * j, b = first + lane;
      const uint64_t begins = __ballot(mine >> j & 1), at = begins & up_to;
      const bool head = b < used && ((b - (at ? first + 63 - __builtin_clzll(at) : start)) & (per - 1)) == 0;
      heads |= (uint32_t)head << j;
      count += __builtin_popcountll(__ballot(head));
      if (begins) start = first + 63 - __builtin_clzll(begins);
    }
    if (lane == 0) scan.count[wave] = count;
    __syncthreads();
    int64_t ahead = t.total;  // tiles before this wave's
    for (int i = 0; i < kWaves; ++i) {
      if (i < wave) ahead += scan.count[i];
      t.total += scan.count[i];
    }
    if (target < ahead || target >= ahead + count) continue;
    for (int j = 0; j < steps; ++j) {
      const uint64_t at = __ballot(heads >> j & 1);
      if ((heads >> j & 1) && ahead + __builtin_popcountll(at & up_to) == target + 1) scan.found = base + 64 * j + lane;
      ahead += __builtin_popcountll(at);
    }
  }
  __syncthreads();
  t.block = __builtin_amdgcn_readfirstlane(scan.found);
  __syncthreads();  // the ring's copies go where the counts are
  if (t.block < 0) return t;
  t.expert = expert_ids[t.block];
  const int i = t.block + lane;
  const uint64_t other = ~__ballot(lane < per && i < used && expert_ids[min(i, used - 1)] == t.expert);
  t.blocks = __builtin_ctzll(other);  // at most 16 to a tile, so lane 16 is another
  return t;
}

// The stages of K in turn, from one that the expert chooses. For tiles of few rows, whose time is the weights' stream: the
// rows of weights that run at a time are K apart and the experts N K, so that at sizes such as 2048 all of them ask the same
// few channels of the memory for the same stage. 48 experts of 85 rows, 4096 x 4096: 406 -> 331 us; 7168 x 2048: 373 ->
// 337; at 4096 x 7168 no difference (549). Tiles of 256 rows gain nothing (1695 -> 1730 us for 16 of 2048 rows),
// and so they begin at stage 0, as do those of weights transposed (602 and 600).
template <bool ON>
struct Turn {
  int K, stages, start;
  __device__ __forceinline__ Turn(int K_, int e)
      : K(K_),
        stages((K_ + kStep - 1) / kStep),
        start(ON && K_ % kStep == 0 ? (int)(3u * (unsigned)e % (unsigned)stages) : 0) {}
  __device__ __forceinline__ int at(int stage) const {
    const int s = stage + start;
    return s < stages ? s : s - stages;
  }
  // steps from that stage on; none past the last one
  __device__ __forceinline__ int left(int stage) const {
    return !ON ? K - stage * kStep : stage < stages ? K - at(stage) * kStep : 0;
  }
  // stages from it to the next
  __device__ __forceinline__ int on(int stage) const { return ON && at(stage) == stages - 1 ? 1 - stages : 1; }
};

// A way to compute tiles: 64 MT rows by 128 NT columns, waves two deep and four wide, kAhead stages in LDS.
template <int MT_, int NT_, int kAhead_>
struct Way {
  static constexpr int MT = MT_, NT = NT_, kAhead = kAhead_;
  static constexpr int kRows = 64 * MT, kTileN = 128 * NT;
  static constexpr int kRing = kRingBytes<RowPanel<kRows>, RowPanel<kTileN>, kAhead>;
  typedef Way<(MT + 1) / 2, NT, kAhead + (MT > 1)> Half;  // half the rows leave room for a stage more
  static_assert(kRing >= kDrainBytes && kRing >= (int)sizeof(Scan), "the sums leave through the ring's place");
};

// Where the wave's copies of rows come from: row i of the tile, or row 0 where it has no slot (zeroed at the store).
template <typename T, typename M>
__device__ __forceinline__ void set_rows(M& m, const GroupedParams& p, int first, int rows, int wave, int lane) {
  const int64_t pitch = (int64_t)p.K * (int)sizeof(T);
  m.base = uniform(static_cast<const uint8_t*>(p.a) + (p.gather ? 0 : first * pitch));
  m.far = p.far ? pitch : 0;
#pragma unroll
  for (int i = 0; i < M::kMine; ++i) {
    const int row = M::row_of(i, wave, lane);
    const uint32_t slot = row < rows ? (uint32_t)p.sorted[first + row] : ~0u;
    m.set(i, slot >= (uint32_t)p.n_slots ? 0 : p.gather ? p.by_topk.of(slot) : (uint32_t)row, pitch, wave, lane);
  }
}

// Of weights: expert e's columns from n0 on; a column past the last is a copy of another, and not stored.
template <typename T, bool TRANSPOSED, typename N>
__device__ __forceinline__ void set_weights(N& n, const GroupedParams& p, int e, int n0, int wave, int lane) {
  const T* w = static_cast<const T*>(p.w) + (int64_t)e * p.N * p.K;
  if constexpr (TRANSPOSED) {
    n.set(w + n0, p.N, p.N - n0, wave, lane);
  } else {
    n.base = uniform(w + (int64_t)n0 * p.K);
    n.far = 0;
#pragma unroll
    for (int i = 0; i < N::kMine; ++i)
      n.set(i, (uint32_t)min(N::row_of(i, wave, lane), p.N - 1 - n0), (int64_t)p.K * (int)sizeof(T), wave, lane);
  }
}

template <typename T, typename O, bool TRANSPOSED, typename W>
__device__ __forceinline__ void product(const GroupedParams& p, uint8_t* ring, int first, int rows, int e, int n0) {
  constexpr int MT = W::MT, NT = W::NT;
  typedef RowPanel<W::kRows> M;
  typedef std::conditional_t<TRANSPOSED, ColumnPanel<W::kTileN>, RowPanel<W::kTileN>> N;
  int lane = (int)threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // addresses made of it are made here: before the loop around this they would spill
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  floatx16 acc[MT][NT] = {};
  M m;
  set_rows<T>(m, p, first, rows, wave, lane);
  N n;
  set_weights<T, TRANSPOSED>(n, p, e, n0, wave, lane);
  const int at_m = wave / 4 * 32 * MT, at_n = wave % 4 * 32 * NT;
  const Turn<(!TRANSPOSED && MT == 2 && NT == 2)> turn(p.K, e);
  m.go(turn.start);
  n.go(turn.start);
  auto copy_of = [&](auto& panel, int q, uint32_t slot, int stage, auto whole) {
    if constexpr (whole)
      panel.copy(q, slot, wave);
    else
      panel.copy(q, slot, turn.left(stage), wave, lane);
    if (q == std::remove_reference_t<decltype(panel)>::kMine - 1) panel.go(turn.on(stage));
  };
  auto copy_m = [&](int q, uint32_t slot, int stage, auto whole) { copy_of(m, q, slot, stage, whole); };
  auto copy_n = [&](int q, uint32_t slot, int stage, auto whole) { copy_of(n, q, slot, stage, whole); };
  prologue<M, N, W::kAhead, M::kBytes>(ring, copy_m, copy_n, [](int) {});
  loop<T, M, N, W::kAhead, M::kBytes>(ring, p.far ? 0 : p.K / kStep - W::kAhead, turn.stages, at_m, at_n, lane, acc,
                                      copy_m, copy_n, [] { return true; }, [](int) {}, [] {});
  uint32_t slotted[MT];  // which of 32 rows have a slot
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int row = at_m + 32 * i + (lane & 31);
    slotted[i] = (uint32_t)__ballot(row < rows && (uint32_t)p.sorted[first + min(row, rows - 1)] < (uint32_t)p.n_slots);
  }
  drain<O>(ring, at_m, at_n, wave, lane, acc, [&](int row, int column, u32x4 v) {
    if (row >= rows || n0 + column >= p.N) return;
    if (!(slotted[(row - at_m) / 32] >> (row & 31) & 1)) v = u32x4{0, 0, 0, 0};
    Line<O>::store(static_cast<O*>(p.out) + (int64_t)(first + row) * p.N + n0 + column, v);
  });
}

// A run's last tile takes half of the rows where it has no more.
template <typename T, typename O, bool TRANSPOSED, typename W>
__global__ __launch_bounds__(kThreads, W::kRing > 80 * 1024 ? 2 : 4) void grouped_kernel(GroupedParams p, Cut c) {
  constexpr int kRows = W::kRows, kTileN = W::kTileN;
  static_assert(W::MT == 1 || W::Half::kRing <= W::kRing, "both ways are in one ring");
  __shared__ __attribute__((aligned(16))) uint8_t ring[W::kRing];
  int64_t target;
  int nt;
  tile_of(c.ntiles, c.log_run, target, nt);
  if (target >= c.row_tiles) return;
  // more tiles than moe_align's order can have: go round again
  for (;; target += c.row_tiles) {
    const RowTile tile = find_tile(p, c.log_per, target >> c.log_cut, *reinterpret_cast<Scan*>(ring));
    if (tile.blocks == 0) return;
    const int e = tile.expert;
    const int first = tile.block * p.block_m + (int)(target & ((1 << c.log_cut) - 1)) * kRows;
    const int rows = min(tile.blocks * p.block_m, kRows), n0 = nt * kTileN;
    if ((uint32_t)e >= (uint32_t)p.E) {  // no such expert
      constexpr int kEach = Line<O>::kEach, kLanes = kTileN / kEach;
      const u32x4 zero = {0, 0, 0, 0};
      for (int i = (int)threadIdx.x; i < rows * kLanes; i += kThreads) {
        const int row = i / kLanes, column = n0 + kEach * (i % kLanes);
        if (column < p.N) Line<O>::store(static_cast<O*>(p.out) + (int64_t)(first + row) * p.N + column, zero);
      }
    } else if (W::MT > 1 && rows <= kRows / 2) {
      product<T, O, TRANSPOSED, typename W::Half>(p, ring, first, rows, e, n0);
    } else {
      product<T, O, TRANSPOSED, W>(p, ring, first, rows, e, n0);
    }
    if (target + c.row_tiles >= tile.total << c.log_cut) return;
    __syncthreads();
  }
}

// Few rows an expert, or little work at all: a tile of 32 rows by 32 NT columns, shared by the waves along K.
template <typename T, typename O, bool TRANSPOSED, int NT, int kAhead>
__global__ __launch_bounds__(kThreads) void narrow_kernel(GroupedParams p, Cut c) {
  constexpr int kRows = 32, kTileN = 32 * NT, kSteps = 128;
  typedef RowPanel<kRows, kSteps> M;
  typedef std::conditional_t<TRANSPOSED, ColumnPanel<kTileN, kSteps>, RowPanel<kTileN, kSteps>> N;
  constexpr int kRing = kAhead * (M::kBytes + N::kBytes), kSums = kSumsBytes<1, NT>;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRing > kSums ? kRing : kSums];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int64_t target;
  int nt;
  tile_of(c.ntiles, c.log_run, target, nt);
  if (target >= c.row_tiles) return;
  for (;; target += c.row_tiles) {
    const RowTile tile = find_tile(p, c.log_per, target >> c.log_cut, *reinterpret_cast<Scan*>(ring));
    if (tile.blocks == 0) return;
    const int e = tile.expert;
    const int first = tile.block * p.block_m + (int)(target & ((1 << c.log_cut) - 1)) * kRows;
    const int rows = min(tile.blocks * p.block_m, kRows), n0 = nt * kTileN;
    floatx16 acc[1][NT] = {};
    const bool known = (uint32_t)e < (uint32_t)p.E;
    if (known) {
      M m;
      set_rows<T>(m, p, first, rows, wave, lane);
      N n;
      set_weights<T, TRANSPOSED>(n, p, e, n0, wave, lane);
      const int whole = p.far ? 0 : p.K / kSteps - (kAhead - 1);
      shared_loop<T, M, N, kAhead, true>(ring, whole, (p.K + kSteps - 1) / kSteps, wave, lane, acc,
                                         [&](uint32_t slot, int stage, auto kind) {
        const int left = p.K - stage * kSteps;
#pragma unroll
        for (int i = 0; i < M::kMine; ++i)
          if constexpr (kind)
            m.copy(i, slot, wave);
          else
            m.copy(i, slot, left, wave, lane);
#pragma unroll
        for (int i = 0; i < N::kMine; ++i)
          if constexpr (kind)
            n.copy(i, slot + M::kBytes, wave);
          else
            n.copy(i, slot + M::kBytes, left, wave, lane);
        m.go(1);
        n.go(1);
      });
    }
    shared_drain(ring, wave, lane, acc, [&](int row, int column, floatx4 v) {
      if (row >= rows || n0 + column >= p.N) return;
      const bool real = known && (uint32_t)p.sorted[first + row] < (uint32_t)p.n_slots;
      const floatx4 none = {0.f, 0.f, 0.f, 0.f};
      Four<O>::store(static_cast<O*>(p.out) + (int64_t)(first + row) * p.N + n0 + column, real ? v : none);
    });
    if (target + c.row_tiles >= tile.total << c.log_cut) return;
    __syncthreads();
  }
}

Cut cut(const GroupedParams& p, int rows, int columns) {
  const int per = std::max(1, rows / p.block_m), pieces = std::max(1, p.block_m / rows), blocks = p.capacity / p.block_m;
  Cut c;
  c.ntiles = (p.N + columns - 1) / columns;
  // What moe_align's order can have at most: an expert's last tile may be of fewer rows. (By capacity alone, one token on
  // 8 of 64 experts had 900 workgroups without a tile beside its 128: 18.6 us instead of 13.)
  const int tiles = p.n_slots / std::max(rows, p.block_m) + std::min(p.E, p.n_slots);
  c.row_tiles = (std::min(blocks, tiles) * pieces + kTileGroup - 1) / kTileGroup * kTileGroup;
  c.log_per = __builtin_ctz((unsigned)per);
  c.log_cut = __builtin_ctz((unsigned)pieces);
  // a launch has less than 2^32 threads; a workgroup goes on with every row_tiles-th row tile
  c.row_tiles = std::min(c.row_tiles, ((1 << 20) - (kXcds << kLogRun)) / c.ntiles * kTileGroup);
  const int64_t all = (int64_t)c.row_tiles * c.ntiles;
  c.log_run = 0;  // few tiles go to all XCDs
  while (c.log_run < kLogRun && (kXcds << (c.log_run + 1)) <= all) ++c.log_run;
  return c;
}
dim3 grid_of(const Cut& c) {
  const int64_t all = (int64_t)c.row_tiles * c.ntiles, turn = kXcds << c.log_run;
  return dim3((unsigned)((all + turn - 1) / turn * turn));
}

template <typename T, typename O, bool TRANSPOSED, typename W>
hipError_t launch_tiles(const GroupedParams& p, hipStream_t stream) {
  const Cut c = cut(p, W::kRows, W::kTileN);
  hipLaunchKernelGGL((grouped_kernel<T, O, TRANSPOSED, W>), grid_of(c), dim3(kThreads), 0, stream, p, c);
  return hipGetLastError();
}

template <typename T, typename O, bool TRANSPOSED, int NT, int kAhead>
hipError_t launch_narrow(const GroupedParams& p, hipStream_t stream) {
  const Cut c = cut(p, 32, 32 * NT);
  hipLaunchKernelGGL((narrow_kernel<T, O, TRANSPOSED, NT, kAhead>), grid_of(c), dim3(kThreads), 0, stream, p, c);
  return hipGetLastError();
}

template <typename T, typename O, bool TRANSPOSED>
hipError_t launch(const GroupedParams& p, hipStream_t stream) {
  const GroupedTile tile = grouped_tile(p.E, p.N, p.n_slots, TRANSPOSED);
  if (tile.rows == 256) return launch_tiles<T, O, TRANSPOSED, Way<4, 2, 2>>(p, stream);
  if (tile.rows == 128) return launch_tiles<T, O, TRANSPOSED, Way<2, 1, 2>>(p, stream);
  if constexpr (TRANSPOSED) {
    if (tile.rows == 64) return launch_tiles<T, O, true, Way<1, 1, 3>>(p, stream);
  } else {
    if (tile.columns == 32) return launch_narrow<T, O, false, 1, 7>(p, stream);
  }
  return launch_narrow<T, O, TRANSPOSED, 2, 3>(p, stream);
}

template <typename T, typename O>
hipError_t launch(const GroupedParams& p, hipStream_t stream) {
  return p.transposed ? launch<T, O, true>(p, stream) : launch<T, O, false>(p, stream);
}

}  // namespace

// Which way, by the tiles that the call is expected to have without padding. The counts are on the device, so an
// expert's rows are taken as n_slots over E, their mean where every routed expert is resident; on a slice of the experts that counts
// the others' slots too, and larger tiles may be taken than the slice's rows fill. Results do not
// depend on the way but for the order of their sums. Measured, us by (256 x 256, 128 x 128, 64 x 128, 32 x 64) tiles,
// bf16, K last: one expert of 4096 rows, 4096 x 4096: 110, 141, 190, 351; 8 experts of 256, 2048 x 2048: 56, 33,
// 40, 59; 48 of 85, 7168 x 2048: 320, 374, 435, 899; one of 512 rows, 2048 x 2048: 44, 21, 19, 12.5; 10 of 100, 1384 x 1000
// transposed: 24, 15.7, 17.3, 22; 384 of 11, 512 x 7168: 489, 475, 475, 477, and 7168 x 512 transposed: 689, 634, 619, 821;
// 48 of 3 (384 routed), 4096 x 7168: 464, 463, 464, 451, and 7168 x 4096 transposed 509, 483, 481, 498; 8 experts of one
// row, 512 x 7168: 79, 42, 42, 19, and by 32 x 32 tiles 10.5 (of 512 rows above: 20).
GroupedTile grouped_tile(int32_t E, int32_t N, int32_t n_slots, bool transposed) {
  const int64_t experts = std::min(E, n_slots), rows = (n_slots + experts - 1) / experts;
  auto tiles = [&](int64_t r, int64_t columns) {
    return experts * ((rows + r / 2 - 1) / r + (rows <= r / 2)) * ((N + columns - 1) / columns);
  };
  if (rows <= 48) {  // an expert's rows are one tile or two: what counts is the weights' stream
    if (transposed && tiles(64, 128) >= 64) return {64, 128};
  } else {
    if (tiles(256, 256) >= 112 && N > 128) return {256, 256};
    if (tiles(128, 128) >= 96) return {128, 128};
  }
  // fewer workgroups than compute units: stages ahead for each instead (16 rows, 2048 x 8192: five 21.5 us, seven 17.3)
  if (!transposed && tiles(32, 64) < 128) return {32, 32};
  return {32, 64};
}

hipError_t launch_grouped_gemm(const GroupedParams& p, int32_t dtype, int32_t out_dtype, hipStream_t stream) {
  if (p.capacity < p.block_m) return hipSuccess;  // no whole block
  if (dtype == kBF16)
    return out_dtype == kFP32 ? launch<bf16_t, float>(p, stream) : launch<bf16_t, bf16_t>(p, stream);
  return out_dtype == kFP32 ? launch<f16_t, float>(p, stream) : launch<f16_t, f16_t>(p, stream);
}

}  // namespace w4a16
