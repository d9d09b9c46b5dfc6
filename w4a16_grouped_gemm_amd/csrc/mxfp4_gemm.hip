// The experts' product on 4-bit floating point operands with a scale per 32.
//
// out[p, n] = sum_k A[r(p), k] W[e, n, k] on v_mfma_scale_f32_16x16x128_f8f6f4,
// which multiplies 4-bit operands, applies both operands' block scales and
// adds in fp32. The weights are the instruction's first operand and the
// activation rows its second, so a lane's four results are four
// neighbouring output columns of one row.
#include "internal.h"
#include "rows.h"

#include <algorithm>

namespace w4a16 {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

// J, R: which byte of `ws` and `as` holds the weights' and the rows' scale.
template <int J, int R>
__device__ __forceinline__ floatx4 mfma_fp4(i32x4 w, i32x4 a, floatx4 c, int ws, int as) {
  const i32x8 w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, a8, c, 4, 4, J, ws, R, as);
}

template <int R>
__device__ __forceinline__ floatx4 mfma_fp4(int j, i32x4 w, i32x4 a, floatx4 c, int ws, int as) {
  switch (j) {
    case 0: return mfma_fp4<0, R>(w, a, c, ws, as);
    case 1: return mfma_fp4<1, R>(w, a, c, ws, as);
    case 2: return mfma_fp4<2, R>(w, a, c, ws, as);
    default: return mfma_fp4<3, R>(w, a, c, ws, as);
  }
}

// j and r are constants wherever this is used, so one call remains.
__device__ __forceinline__ floatx4 mfma_fp4(int j, int r, i32x4 w, i32x4 a, floatx4 c, int ws, int as) {
  switch (r) {
    case 0: return mfma_fp4<0>(j, w, a, c, ws, as);
    case 1: return mfma_fp4<1>(j, w, a, c, ws, as);
    case 2: return mfma_fp4<2>(j, w, a, c, ws, as);
    default: return mfma_fp4<3>(j, w, a, c, ws, as);
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, floatx4 v) {
  struct Four {
    T v[4];
  } r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = (T)v[i];
  *reinterpret_cast<__attribute__((aligned(4 * sizeof(T)))) Four*>(p) = r;
}

// Weight streaming: a workgroup of four waves takes 4 / SPLIT units, a unit
// being one row block (16 RB rows) times 64 columns; SPLIT waves share a unit's
// steps of K = 128 and add up through LDS in wave order. Weights and rows go
// from memory straight to the registers that the MFMAs read, D steps ahead.
// TAIL: K may end inside a step, and what lies past it is zeroed, or the scales
// are not aligned to 4 bytes: scales are then read one by one instead of the four
// of a row and step at once.
template <typename T, int RB, int SPLIT, int D, bool TAIL>
__global__ __launch_bounds__(256) void fp4_stream_kernel(Fp4GemmParams p) {
  constexpr int kUnits = 4 / SPLIT;
  __shared__ floatx4 part[SPLIT > 1 ? (SPLIT - 1) * kUnits : 1][RB * 4][SPLIT > 1 ? 64 : 1];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int split = wave % SPLIT, local = wave / SPLIT;
  const int nblocks = fp4_nblocks(p.N), steps = fp4_steps(p.K);
  const int used = min(p.capacity, *p.ntpp) / (16 * RB);
  const int64_t units = (int64_t)used * nblocks;
  for (int64_t u0 = (int64_t)blockIdx.x * kUnits; u0 < units; u0 += (int64_t)gridDim.x * kUnits) {
    const int64_t u = u0 + local;
    const bool active = u < units;
    const int b = (int)(u / nblocks), nb = (int)(u - (int64_t)b * nblocks);
    const int e = active ? p.expert_ids[b] : -1;
    const bool known = (uint32_t)e < (uint32_t)p.E;
    floatx4 acc[RB][4] = {};
    bool real[RB] = {};
    if (known) {
      const uint8_t* aq[RB];
      const uint8_t* as[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const int row = b * 16 * RB + 16 * r + (lane & 15);
        const uint32_t slot = (uint32_t)p.sorted[row];
        real[r] = slot < (uint32_t)p.n_slots;
        const int64_t src = !real[r] ? 0 : p.gather ? (int64_t)(slot / (uint32_t)p.topk) : row;
        aq[r] = p.a_q + src * (p.K / 2);
        as[r] = p.a_s + src * (p.K / 32);
      }
      const uint8_t* wu = p.packed + ((int64_t)e * nblocks + nb) * steps * kFp4UnitBytes;
      i32x4 w[D][4], a[D][RB];
      int ws[D], sc[D][RB];
      // a step past the last repeats it, so that the loop has no branch but its own
      auto fetch = [&](int d, int step) {
        step = min(step, steps - 1);
        const uint8_t* at = wu + (int64_t)step * kFp4UnitBytes;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[d][j] = *reinterpret_cast<const i32x4*>(at + 1024 * j + 16 * lane);
        ws[d] = *reinterpret_cast<const int*>(at + 4096 + 4 * lane);
        const int block = step * 4 + (lane >> 4);  // of 32 values
        const bool in = !TAIL || block < p.K / 32;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          a[d][r] = *reinterpret_cast<const i32x4*>(aq[r] + (in ? 16 * block : 0));
          sc[d][r] = TAIL ? as[r][in ? block : 0] : *reinterpret_cast<const int*>(as[r] + 4 * step);
          if (TAIL && !in) a[d][r] = i32x4{0, 0, 0, 0}, sc[d][r] = 0;
        }
      };
      auto compute = [&](int d) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const int scale = TAIL ? sc[d][r] : (int)((uint32_t)sc[d][r] >> (8 * (lane >> 4)));
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][j] = mfma_fp4(j, 0, w[d][j], a[d][r], acc[r][j], ws[d], scale);
        }
      };
#pragma unroll
      for (int d = 0; d < D; ++d) {
        fetch(d, split + d * SPLIT);
        __builtin_amdgcn_sched_barrier(0);
      }
      int step = split;
      for (; step + (D - 1) * SPLIT < steps; step += D * SPLIT) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          compute(d);
          fetch(d, step + (D + d) * SPLIT);
          __builtin_amdgcn_sched_barrier(0);  // keeps the fetches in step order, so that a wait is for the oldest
        }
      }
#pragma unroll
      for (int d = 0; d < D - 1; ++d)
        if (step + d * SPLIT < steps) compute(d);
    }
    if (SPLIT > 1) {
      if (split > 0) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[local * (SPLIT - 1) + split - 1][4 * r + j][lane] = acc[r][j];
      }
      __syncthreads();
      if (split == 0) {
        for (int k = 0; k < SPLIT - 1; ++k)
#pragma unroll
          for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][j] += part[local * (SPLIT - 1) + k][4 * r + j][lane];
      }
      __syncthreads();
    }
    if (split == 0 && active) {
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        T* out = static_cast<T*>(p.out) + (int64_t)(b * 16 * RB + 16 * r + (lane & 15)) * p.N;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = nb * kNBlock + 16 * j + 4 * (lane >> 4);
          const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
          if (n < p.N) store4(out + n, real[r] ? acc[r][j] : zero);
        }
      }
    }
  }
}

// A barrier that orders LDS only: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The tile (row block b, 256-column tile nt) of this workgroup, from the row
// blocks in use. Workgroups go round-robin to the 8 XCDs, each with an L2 of
// its own: XCD x takes a contiguous eighth of the tiles, in groups of kGroupRows
// row blocks with all their columns, row blocks innermost.
constexpr int kXcds = 8;
constexpr int kGroupRows = 8;
__device__ __forceinline__ bool tile_of(int used, int ntiles, int& b, int& nt) {
  const int64_t total = (int64_t)used * ntiles;
  const int64_t chunk = (total + kXcds - 1) / kXcds;
  const int64_t at = (int64_t)blockIdx.x / kXcds;
  const int64_t tile = ((int64_t)blockIdx.x % kXcds) * chunk + at;
  if (at >= chunk || tile >= total) return false;
  const int64_t per_group = (int64_t)kGroupRows * ntiles;
  const int first = (int)(tile / per_group) * kGroupRows;
  const int rows = min(kGroupRows, used - first);
  const int rest = (int)(tile % per_group);
  nt = rest / rows;
  b = first + rest - nt * rows;
  return true;
}

// Many rows per expert: a workgroup of four waves computes 16 RB rows times 256
// columns, a wave all of its rows times 64 columns. A wave's weights are its own
// and go from memory to registers; the rows are shared, so each wave fetches its
// part of them and all read them from LDS, in the order the MFMA takes. Both are
// fetched D steps of K = 128 ahead; one barrier per step. Row scales lie in LDS
// so that a lane reads those of its row in all RB row blocks at once, and the
// MFMA picks the byte.
template <typename T, int RB, int D>
__global__ __launch_bounds__(256, 2) void fp4_tile_kernel(Fp4GemmParams p, int ntiles) {
  constexpr int BM = 16 * RB;
  constexpr int kMine = RB / 4;  // row blocks that a wave fetches
  constexpr int kAhead = 2;      // row blocks read from LDS before their use
  __shared__ i32x4 rows_lds[D][RB][64];
  __shared__ uint8_t scales_lds[D][4][16][RB];  // k block of 32, row of 16, row block
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nblocks = fp4_nblocks(p.N), steps = p.K / kFp4StepK;
  int b, nt;
  if (!tile_of(min(p.capacity, *p.ntpp) / BM, ntiles, b, nt)) return;
  const int nb = nt * 4 + wave;
  const int e = p.expert_ids[b];
  const bool known = (uint32_t)e < (uint32_t)p.E;
  floatx4 acc[RB][4] = {};

  if (known) {
    // rows without a slot read row 0 and are zeroed at the store
    auto source = [&](int row) -> int64_t {
      const uint32_t slot = (uint32_t)p.sorted[row];
      if (slot >= (uint32_t)p.n_slots) return 0;
      return p.gather ? (int64_t)(slot / (uint32_t)p.topk) : row;
    };
    const uint8_t* aq[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      aq[i] = p.a_q + source(b * BM + 16 * (wave * kMine + i) + (lane & 15)) * (p.K / 2) + 16 * (lane >> 4);
    const int mine = tid & (BM - 1);  // the row whose scales this thread fetches, as others may
    const uint8_t* as = p.a_s + source(b * BM + mine) * (p.K / 32);
    // a wave past the last column block repeats it and stores nothing
    const uint8_t* wp = p.packed + ((int64_t)e * nblocks + min(nb, nblocks - 1)) * steps * kFp4UnitBytes;

    i32x4 w[D][4], a[D][kMine];
    int ws[D];
    uint32_t sc[D];
    // a step past the last repeats it, so that no load is behind a branch
    auto fetch_rows = [&](int slot, int step) {
      step = min(step, steps - 1);
#pragma unroll
      for (int i = 0; i < kMine; ++i) a[slot][i] = *reinterpret_cast<const i32x4*>(aq[i] + 64 * step);
      sc[slot] = *reinterpret_cast<const uint32_t*>(as + 4 * step);
    };
    auto fetch_weights = [&](int slot, int step) {
      const uint8_t* u = wp + (int64_t)min(step, steps - 1) * kFp4UnitBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[slot][j] = *reinterpret_cast<const i32x4*>(u + 1024 * j + 16 * lane);
      ws[slot] = *reinterpret_cast<const int*>(u + 4096 + 4 * lane);
    };
    auto publish = [&](int slot) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) rows_lds[slot][wave * kMine + i][lane] = a[slot][i];
#pragma unroll
      for (int k = 0; k < 4; ++k) scales_lds[slot][k][mine & 15][mine >> 4] = (uint8_t)(sc[slot] >> (8 * k));
    };
    // step s, in ring slot d: the slot written here was last read a barrier ago
    auto compute = [&](int d, int s) {
      const int next = (d + 1) % D;
      publish(next);
      fetch_rows(next, s + 1 + D);
      uint32_t rs[RB / 4];
      __builtin_memcpy(rs, scales_lds[d][lane >> 4][lane & 15], sizeof(rs));
      i32x4 av[kAhead + 1];
#pragma unroll
      for (int r = 0; r < kAhead; ++r) av[r] = rows_lds[d][r][lane];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        if (r + kAhead < RB) av[(r + kAhead) % (kAhead + 1)] = rows_lds[d][r + kAhead][lane];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[r][j] = mfma_fp4(j, r & 3, w[d][j], av[r % (kAhead + 1)], acc[r][j], ws[d], (int)rs[r / 4]);
        __builtin_amdgcn_sched_barrier(0);
      }
      fetch_weights(d, s + D);
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
      fetch_rows(d, d);
      fetch_weights(d, d);
      __builtin_amdgcn_sched_barrier(0);
    }
    publish(0);
    fetch_rows(0, D);
    lds_barrier();
    int s = 0;
    for (; s + D <= steps; s += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) compute(d, s + d);
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (s + d < steps) compute(d, s + d);
  }

  // A row block at a time through LDS, so that a store covers whole 128-byte
  // lines: 16 rows of 64 columns, rows 16 bytes apart from a bank conflict.
  constexpr int kPitch = 64 * (int)sizeof(T) + 16;
  constexpr int kChunks = 64 * (int)sizeof(T) / 16;  // of a row
  constexpr int kRowsAtOnce = 64 / kChunks;
  __shared__ __attribute__((aligned(16))) uint8_t tile_lds[4][16 * kPitch];
  uint8_t* tile = tile_lds[wave];
  uint64_t real[(BM + 63) / 64];  // which rows have a slot
#pragma unroll
  for (int i = 0; i < BM / 64; ++i) real[i] = __ballot(known && (uint32_t)p.sorted[b * BM + 64 * i + lane] < (uint32_t)p.n_slots);
  const int col = nb * kNBlock + lane % kChunks * (16 / (int)sizeof(T));
#pragma unroll
  for (int r = 0; r < RB; ++r) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      store4(reinterpret_cast<T*>(tile + (lane & 15) * kPitch) + 16 * j + 4 * (lane >> 4), acc[r][j]);
#pragma unroll
    for (int i = 0; i < 16 / kRowsAtOnce; ++i) {
      const int row = 16 * r + i * kRowsAtOnce + lane / kChunks;
      i32x4 v = *reinterpret_cast<const i32x4*>(tile + (row & 15) * kPitch + 16 * (lane % kChunks));
      if (!((real[16 * r / 64] >> (row & 63)) & 1)) v = i32x4{0, 0, 0, 0};
      T* out = static_cast<T*>(p.out) + (int64_t)(b * BM + row) * p.N + col;
      if (col < p.N) __builtin_nontemporal_store(v, reinterpret_cast<i32x4*>(out));
    }
  }
}

// K is whole steps of 128 and a row's scale bytes of a step are an aligned dword.
bool whole_steps(const Fp4GemmParams& p) {
  return p.K % kFp4StepK == 0 && (reinterpret_cast<uintptr_t>(p.a_s) & 3) == 0;
}

template <typename T, int RB, int SPLIT, int D>
hipError_t launch_stream(const Fp4GemmParams& p, hipStream_t stream) {
  const int64_t units = (int64_t)(p.capacity / (16 * RB)) * fp4_nblocks(p.N);
  const int64_t groups = (units * SPLIT + 3) / 4;
  if (groups == 0) return hipSuccess;
  const int grid = (int)std::min<int64_t>(groups, (int64_t)device_cu_count() * 8);
  if (!whole_steps(p))
    hipLaunchKernelGGL((fp4_stream_kernel<T, RB, SPLIT, D, true>), dim3(grid), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((fp4_stream_kernel<T, RB, SPLIT, D, false>), dim3(grid), dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <typename T, int RB, int D>
hipError_t launch_tile(const Fp4GemmParams& p, hipStream_t stream) {
  const int ntiles = (fp4_nblocks(p.N) + 3) / 4;
  const int64_t tiles = (int64_t)(p.capacity / (16 * RB)) * ntiles;
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp4_tile_kernel<T, RB, D>), dim3((unsigned)grid), dim3(256), 0, stream, p, ntiles);
  return hipGetLastError();
}

template <typename T>
hipError_t launch(int32_t block_m, const Fp4GemmParams& p, hipStream_t stream) {
  if (whole_steps(p) && block_m == 128) return launch_tile<T, 8, 2>(p, stream);
  if (whole_steps(p) && block_m == 64) return launch_tile<T, 4, 2>(p, stream);
  switch (block_m) {
    case 16: return launch_stream<T, 1, 4, 4>(p, stream);
    case 32: return launch_stream<T, 2, 4, 3>(p, stream);
    case 64: return launch_stream<T, 4, 1, 2>(p, stream);
    case 128: return launch_stream<T, 8, 1, 1>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_fp4_gemm(int32_t block_m, const Fp4GemmParams& p, int32_t out_dtype, hipStream_t stream) {
  if (out_dtype == kBF16) return launch<bf16_t>(block_m, p, stream);
  if (out_dtype == kFP16) return launch<f16_t>(block_m, p, stream);
  return launch<float>(block_m, p, stream);
}

}  // namespace w4a16
