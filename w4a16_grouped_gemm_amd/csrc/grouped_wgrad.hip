// The weights' gradient of the experts' product: for each expert e
//   dW[e, n, k] = sum_p dout[p, n] A[r(p), k]
// over e's rows p that hold a slot, with r(p) the row itself or its slot's token.
//
// A workgroup computes a square tile of one expert's dW over all of its rows (or, where the tiles
// are few, a share of them, and a second kernel adds the shares in their order). Both operands
// are column panels: the rows are the steps of the sum. Rows without a slot, whatever they
// hold, are replaced by zeros as they are copied to LDS (global_load_lds); the mfma loop is in gemm_tile.h.
//
// Measured (one MI355X): 32768 rows, 16 experts, 4096 x 7168: aligned rows to bf16 1620..1770 us by card, gathered ones to
// fp32 1740..1880, 1.02..1.18 PFLOP/s; 131072 rows
// 6130..6290 us, 1.25. Bound as the product by the clock that the load leaves, and by a tile's start and its
// store, 128 or 256 KB, which take as long as four or five of its 32 stages. 4 experts of 1388 rows, 264 x 712: 14.7
// us, a chain of a dozen dependent steps.
#include "gemm_tile.h"
#include "grouped_gemm.h"
#include "row_ops.h"

#include <algorithm>
#include <climits>

namespace w4a16 {
namespace {

using namespace tile;

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

// The rows [begin, stop) of expert e that this workgroup (of blockIdx.y's share) goes through: from the expert's first
// block to its last. scratch: two ints of LDS. All threads of the workgroup call it.
struct Span {
  int begin, stop;
};
__device__ __forceinline__ Span span_of(const WgradParams& p, int e, int* scratch) {
  const int used = p.capacity > 0 ? min(p.capacity, *p.ntpp) >> p.log_block : 0;
  if (threadIdx.x == 0) scratch[0] = INT_MAX, scratch[1] = -1;
  __syncthreads();
  int lo = INT_MAX, hi = -1;
  int i = (int)threadIdx.x;
  if (i < used && p.expert_ids[i] == e) lo = hi = i;
  for (i += kThreads; i < used; i += 8 * kThreads) {  // many blocks: eight loads on their way together
    int id[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) id[j] = p.expert_ids[min(i + j * kThreads, used - 1)];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (id[j] == e) lo = min(lo, min(i + j * kThreads, used - 1)), hi = max(hi, min(i + j * kThreads, used - 1));
  }
  if (hi >= 0) {
    atomicMin(&scratch[0], lo);
    atomicMax(&scratch[1], hi);
  }
  __syncthreads();
  const int first = __builtin_amdgcn_readfirstlane(scratch[0]), last = __builtin_amdgcn_readfirstlane(scratch[1]);
  __syncthreads();  // the ring's copies go where the run is
  if (last < 0) return {0, 0};
  const int rows = (last + 1 - first) << p.log_block, begin = first << p.log_block;
  const int share = ((rows + kStep - 1) / kStep + p.cut.splits - 1) / p.cut.splits * kStep;
  const int at = (int)min((int64_t)share * blockIdx.y, (int64_t)rows);
  return {begin + at, begin + min(at + share, rows)};
}

// Four sums of dW (one workgroup's share of them) to where they go.
template <typename O>
__device__ __forceinline__ void put4(const WgradParams& p, int e, int n, int k, floatx4 v) {
  if (n >= p.N || k >= p.K) return;
  const int64_t at = ((int64_t)e * p.N + n) * p.K + k;
  if (p.cut.splits > 1) {
    Four<float>::store(p.partial + (int64_t)blockIdx.y * p.E * p.N * p.K + at, v);
    return;
  }
  O* dw = static_cast<O*>(p.dw) + at;
  if (p.accumulate) v += Four<O>::load(dw);
  Four<O>::store(dw, v);
}

// Few weights: 64 x 64 values a workgroup, shared by its waves along the rows, 128 of them a stage.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void narrow_wgrad_kernel(WgradParams p, int mtiles, int ntiles) {
  constexpr int kTile = 64, kSteps = 128, kAhead = 4, kTable = 4096;
  typedef ColumnPanel<kTile, kSteps> Panel;
  static_assert(Panel::kMine == 2, "two copies of eight rows a wave and panel");
  __shared__ __attribute__((aligned(16))) uint8_t ring[kAhead * 2 * Panel::kBytes];
  static_assert(sizeof(ring) >= kSumsBytes<2, 2>, "the waves' shares take the ring's place");
  __shared__ int32_t table[kTable];  // of kTable rows: the row of a, or -1 where the row adds nothing
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int e, mt, nt;
  if (!tile_of(mtiles, ntiles, e, mt, nt)) return;
  const Span span = span_of(p, e, table);
  const int m0 = mt * kTile, n0 = nt * kTile;
  floatx16 acc[2][2] = {};
  const int my_row = lane / Panel::kLanes;
  const int64_t row_m = (int64_t)p.N * (int)sizeof(T), row_n = (int64_t)p.K * (int)sizeof(T);
  for (int base = span.begin; base < span.stop; base += kTable) {
    const int rows = min(span.stop - base, kTable), stages = (rows + kSteps - 1) / kSteps;
    // the copies go up to kAhead - 1 stages past the last
    const int filled = min((stages + kAhead) * kSteps, kTable);
    for (int i = (int)threadIdx.x; i < filled; i += kThreads) {
      const int row = base + min(i, rows - 1);
      const uint32_t slot = (uint32_t)p.sorted[row];
      const bool real = i < rows && slot < (uint32_t)p.n_slots && p.expert_ids[row >> p.log_block] == e;
      table[i] = !real ? -1 : p.gather ? (int32_t)p.by_topk.of(slot) : row;
    }
    __syncthreads();
    const uint8_t *at_m[2], *at_n[2];  // this lane's 16 bytes of the chunk's first row of dout, of row 0 of a
    int32_t from[2];                   // its rows of a, of the stage to be copied next
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int row = 16 * wave + 8 * q + my_row;
      const int column = 8 * (lane % Panel::kLanes ^ (Panel::swizzle(row) << 2));
      at_m[q] = static_cast<const uint8_t*>(p.dout) + (int64_t)(base + row) * row_m +
                2 * (m0 + (column < p.N - m0 ? column : 0));
      at_n[q] = static_cast<const uint8_t*>(p.a) + 2 * (n0 + (column < p.K - n0 ? column : 0));
      from[q] = table[row];
    }
    shared_loop<T, Panel, Panel, kAhead, false>(ring, 0, stages, wave, lane, acc,
                                                [&](uint32_t lds, int stage, std::false_type) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool real = from[q] >= 0;
        const uint8_t* n = at_n[q] + (uint64_t)(uint32_t)from[q] * (uint32_t)row_n;
        copy16(real ? (const void*)at_m[q] : (const void*)kZeros, lds + 1024 * (2 * wave + q));
        copy16(real ? (const void*)n : (const void*)kZeros, lds + Panel::kBytes + 1024 * (2 * wave + q));
        at_m[q] += kSteps * row_m;
        const int next = (stage + 1) * kSteps + 16 * wave + 8 * q + my_row;
        from[q] = next < filled ? table[next] : -1;
      }
    });
  }
  shared_drain(ring, wave, lane, acc, [&](int n, int k, floatx4 v) { put4<O>(p, e, m0 + n, n0 + k, v); });
}

// Many weights: kTile x kTile values a workgroup, its waves 2 deep and 4 wide.
template <typename T, typename O, int kTile, bool GATHER>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(WgradParams p, int mtiles, int ntiles) {
  constexpr int MT = kTile / 64, NT = kTile / 128;
  constexpr int kAhead = kTile == 256 ? 2 : 4;
  typedef ColumnPanel<kTile> Panel;
  constexpr int kRows = 64 / Panel::kLanes;  // of a copy
  constexpr int kMine = Panel::kMine;
  static_assert(kMine * kRows == 8, "eight rows a wave");
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRingBytes<Panel, Panel, kAhead>];
  static_assert(sizeof(ring) >= kDrainBytes, "the sums leave through the ring's place");
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int e, mt, nt;
  if (!tile_of(mtiles, ntiles, e, mt, nt)) return;
  const Span span = span_of(p, e, reinterpret_cast<int*>(ring));
  const int begin = span.begin, stop = span.stop, stages = (stop - begin + kStep - 1) / kStep;
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
    Rows rows, next;   // of the stage that is being copied, and of the one after it
    uint32_t from[8];  // where the rows begin in a, in bytes (GATHER; not used where 32 bits do not hold them)
    bool real;         // all eight have a slot
    const int64_t row_m = (int64_t)p.N * (int)sizeof(T), row_n = (int64_t)p.K * (int)sizeof(T);
    auto look = [&](Rows& r, int stage) {
      const int row = begin + stage * kStep + 8 * wave, at = min(row, stop - 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) r.slot[i] = sorted[at + i];
      r.owner = expert_ids[at >> p.log_block];
      r.inside = row < stop;
    };
    auto arrive = [&] {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        most = max(most, (uint32_t)rows.slot[i]);
        from[i] = GATHER ? p.by_topk.of((uint32_t)rows.slot[i]) * (uint32_t)row_n : 0;
      }
      real = (most < (uint32_t)p.n_slots) & (rows.owner == e) & rows.inside & !p.far;
    };
    const int my_row = lane / Panel::kLanes;
    auto mine = [&](const auto* of) {  // of this lane's row
      if constexpr (kRows == 2) return my_row ? of[1] : of[0];
      // by the bits of my_row: a chain over its values becomes an array in memory
      const auto low = my_row & 1 ? of[1] : of[0], high = my_row & 1 ? of[3] : of[2];
      return my_row & 2 ? high : low;
    };
    // of the next stage's first row of the workgroup (GATHER: of token 0), and this lane's 16 bytes from there
    const uint8_t* base_m = uniform(static_cast<const uint8_t*>(p.dout) + begin * row_m + 2 * m0);
    const uint8_t* base_n = uniform(static_cast<const uint8_t*>(p.a) + (GATHER ? 0 : begin * row_n) + 2 * n0);
    uint32_t offset_m[kMine], offset_n[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int row = 8 * wave + kRows * q + my_row;
      const int column = 8 * (lane % Panel::kLanes ^ (Panel::swizzle(kRows * q + my_row) << 2));
      offset_m[q] = (uint32_t)row * (uint32_t)row_m + 2 * (m0 + column < p.N ? column : 0);
      offset_n[q] = (GATHER ? 0 : (uint32_t)row * (uint32_t)row_n) + 2 * (n0 + column < p.K ? column : 0);
    }
    auto copy = [&](const uint8_t* at, uint32_t slot, int q, uint32_t lds) {
      const bool some = (slot < (uint32_t)p.n_slots) & (rows.owner == e) & rows.inside;
      copy16(some ? (const void*)at : (const void*)kZeros, lds + 1024 * (kMine * wave + q));
    };
    auto copy_m = [&](int q, uint32_t lds, int, auto whole) {
      if constexpr (whole)
        copy16(base_m, offset_m[q], lds + 1024 * (kMine * wave + q));
      else
        copy(base_m + offset_m[q], (uint32_t)mine(&rows.slot[kRows * q]), q, lds);
      if (q == kMine - 1) base_m += kStep * row_m;
    };
    auto copy_n = [&](int q, uint32_t lds, int, auto whole) {
      if constexpr (whole) {
        copy16(base_n, GATHER ? offset_n[q] + mine(&from[kRows * q]) : offset_n[q], lds + 1024 * (kMine * wave + q));
      } else {
        const uint32_t slot = (uint32_t)mine(&rows.slot[kRows * q]);
        const uint8_t* at = base_n + offset_n[q];
        copy(GATHER ? at + (uint64_t)p.by_topk.of(slot) * (uint64_t)row_n : at, slot, q, lds);
      }
      if (!GATHER && q == kMine - 1) base_n += kStep * row_n;
    };
    look(rows, 0);
    prologue<Panel, Panel, kAhead, Panel::kBytes>(ring, copy_m, copy_n, [&](int stage) { look(rows, stage); });
    arrive();
    loop<T, Panel, Panel, kAhead, Panel::kBytes>(
        ring, stages, stages, wave / 4 * 32 * MT, wave % 4 * 32 * NT, lane, acc, copy_m, copy_n, [&] { return real; },
        [&](int stage) { look(next, stage); },
        [&] {
          rows = next;
          arrive();
        });
  }

  const int at_m = wave / 4 * 32 * MT, at_n = wave % 4 * 32 * NT;
  if (p.cut.splits > 1 || (p.accumulate && sizeof(O) == 2)) {  // 32-bit sums to a share, or to be added to what is there
    drain<float>(ring, at_m, at_n, wave, lane, acc, [&](int n, int k, u32x4 v) {
      put4<O>(p, e, m0 + n, n0 + k, __builtin_bit_cast(floatx4, v));
    });
    return;
  }
  drain<O>(ring, at_m, at_n, wave, lane, acc, [&](int n, int k, u32x4 v) {
    if (m0 + n >= p.N || n0 + k >= p.K) return;
    O* dw = static_cast<O*>(p.dw) + ((int64_t)e * p.N + m0 + n) * p.K + n0 + k;
    if constexpr (sizeof(O) == 4) {
      if (p.accumulate)
        v = __builtin_bit_cast(u32x4, __builtin_bit_cast(floatx4, v) + *reinterpret_cast<const floatx4*>(dw));
    }
    Line<O>::store(dw, v);
  });
}

// dW (+)= the shares, in their order.
template <typename O>
__global__ __launch_bounds__(256) void join_kernel(const float* partial, O* dw, int64_t size, int32_t splits,
                                                   int32_t accumulate) {
  const int64_t stride = (int64_t)gridDim.x * 256 * 4;
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < size; at += stride) {
    floatx4 sums = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) sums += Four<float>::load(partial + s * size + at);
    if (accumulate) sums += Four<O>::load(dw + at);
    Four<O>::store(dw + at, sums);
  }
}

template <typename T, typename O, int kTile>
hipError_t launch_tile(const WgradParams& p, hipStream_t stream) {
  const int mtiles = (p.N + kTile - 1) / kTile, ntiles = (p.K + kTile - 1) / kTile;
  const int64_t chunk = ((int64_t)mtiles * ntiles + kXcds - 1) / kXcds;
  const int64_t grid = chunk * kXcds * p.E;
  const dim3 g((unsigned)grid, (unsigned)p.cut.splits), t(kThreads);
  if constexpr (kTile == 64)
    hipLaunchKernelGGL((narrow_wgrad_kernel<T, O>), g, t, 0, stream, p, mtiles, ntiles);
  else if (p.gather)
    hipLaunchKernelGGL((wgrad_kernel<T, O, kTile, true>), g, t, 0, stream, p, mtiles, ntiles);
  else
    hipLaunchKernelGGL((wgrad_kernel<T, O, kTile, false>), g, t, 0, stream, p, mtiles, ntiles);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch(const WgradParams& p, hipStream_t stream) {
  const hipError_t err = p.cut.tile == 256   ? launch_tile<T, O, 256>(p, stream)
                         : p.cut.tile == 128 ? launch_tile<T, O, 128>(p, stream)
                                             : launch_tile<T, O, 64>(p, stream);
  if (err != hipSuccess || p.cut.splits == 1) return err;
  const int64_t size = (int64_t)p.E * p.N * p.K;
  const int64_t grid = std::min<int64_t>((size / 4 + 255) / 256, (int64_t)device_cu_count() * 32);
  hipLaunchKernelGGL((join_kernel<O>), dim3((unsigned)grid), dim3(256), 0, stream, p.partial, static_cast<O*>(p.dw),
                     size, p.cut.splits, p.accumulate);
  return hipGetLastError();
}

}  // namespace

int64_t wgrad_workgroups(int32_t E, int32_t N, int32_t K, WgradCut cut) {
  const int64_t tiles = (int64_t)((N + cut.tile - 1) / cut.tile) * ((K + cut.tile - 1) / cut.tile);
  return (tiles + kXcds - 1) / kXcds * kXcds * E * cut.splits;
}

// Measured, us by (256 x 256, 128 x 128, 64 x 64) tiles with shares as below, bf16, K last: 8 experts of 250 rows,
// 1000 x 2000: 24, 38, 98; 8 of 4096, 512 x 512: 76 (without shares 88), 46 (54), 61; 4 of 1388, 264 x 712: 33 (36),
// 24, 17; one of 4096, 512 x 1024: 30 (81), 25 (48), 21 (25); one of 4096, 256 x 256: 29 (80), 20 (43), 15 (21);
// 64 of 64, 1024 x 1024: 50, 96, 317.
WgradCut wgrad_cut(int32_t E, int32_t N, int32_t K, int32_t capacity) {
  auto tiles = [&](int64_t t) { return E * ((N + t - 1) / t) * ((K + t - 1) / t); };
  WgradCut c;
  c.tile = tiles(256) >= 128 ? 256 : tiles(64) <= 256 ? 64 : 128;
  // shares fill the card where tiles do not; each is of 512 rows at least
  c.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>({256 / tiles(c.tile), capacity / E / 512, 16}));
  return c;
}

hipError_t launch_grouped_wgrad(const WgradParams& p, int32_t dtype, int32_t dw_dtype, hipStream_t stream) {
  if (dtype == kBF16)
    return dw_dtype == kFP32 ? launch<bf16_t, float>(p, stream) : launch<bf16_t, bf16_t>(p, stream);
  return dw_dtype == kFP32 ? launch<f16_t, float>(p, stream) : launch<f16_t, f16_t>(p, stream);
}

}  // namespace w4a16
