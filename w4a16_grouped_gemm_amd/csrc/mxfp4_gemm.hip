// The experts' product on 4-bit floating point operands with a scale per 32.
//
// out[p, n] = sum_k A[r(p), k] W[e, n, k] on v_mfma_scale_f32_16x16x128_f8f6f4,
// which multiplies 4-bit operands, applies both operands' block scales and
// adds in fp32. The weights are the instruction's first operand and the
// activation rows its second, so a lane's four results are four
// neighbouring output columns of one row.
#include "row_ops.h"
#include "rows.h"

#include <algorithm>

namespace w4a16 {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// 16 x 16 x 128. j: which byte of `ws` holds the weights' scales; the rows' are in byte 0.
// j (c and h below) is a constant wherever this is used, so one of the calls remains.
__device__ __forceinline__ floatx4 mfma_fp4(int j, i32x4 w, i32x4 a, floatx4 c, int ws, int as) {
#define MFMA(J) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w), widen(a), c, 4, 4, J, ws, 0, as)
  switch (j) {
    case 0: MFMA(0);
    case 1: MFMA(1);
    case 2: MFMA(2);
    default: MFMA(3);
  }
#undef MFMA
}

// 32 x 32 x 64. The weights' scales are in byte 2 c of `ws`, the rows' in byte 2 h of `as`.
__device__ __forceinline__ floatx16 mfma_fp4_32(int c, int h, i32x4 w, i32x4 a, floatx16 acc, int ws, int as) {
#define MFMA(C, H) \
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(w), widen(a), acc, 4, 4, 2 * C, ws, 2 * H, as)
  if (c == 0 && h == 0) MFMA(0, 0);
  if (c == 0) MFMA(0, 1);
  if (h == 0) MFMA(1, 0);
  MFMA(1, 1);
#undef MFMA
}

// A buffer of less than 4 GiB, read at a byte offset per lane plus one that all share.
struct Buffer {
  __amdgpu_buffer_rsrc_t rsrc;
  __device__ __forceinline__ Buffer(const uint8_t* base, int64_t bytes)
      : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, (int)(uint32_t)bytes, 0x00020000)) {}
  template <Policy P = kCached>
  __device__ __forceinline__ i32x4 load4(uint32_t lane_offset, int offset) const {
    constexpr int kAux = P == kStreamed ? 2 : 0;  // the non-temporal bit
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)lane_offset, offset, kAux));
  }
  __device__ __forceinline__ uint32_t load(uint32_t lane_offset, int offset) const {
    return __builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)lane_offset, offset, 0);
  }
};

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
// being 16 RB rows of a row block times 64 columns; SPLIT waves share a unit's
// steps of K = 128 and add up through LDS in wave order. Weights and rows go
// from memory straight to the registers that the MFMAs read, D steps ahead.
// TAIL: K may end inside a step, and what lies past it is zeroed, or the scales
// are not aligned to 4 bytes: scales are then read one by one instead of the four
// of a row and step at once.
//
// Bound by the weights' bytes, which are read once and never again, so past the
// caches' retention: 128 tokens, top-8 of 384 experts, the 48 resident ones of 4096 x
// 7168 (some 45 in use), 699 MB in 103 us, 6.8 TB/s of the 6.9 that such reads reach. A unit's share of memory is one
// contiguous run of 4352 bytes a step, which is why the weights are laid out by
// step inside a column block.
template <typename T, int RB, int SPLIT, int D, bool TAIL>
__global__ __launch_bounds__(256) void fp4_stream_kernel(Fp4GemmParams p) {
  constexpr int kUnits = 4 / SPLIT;
  __shared__ floatx4 part[SPLIT > 1 ? (SPLIT - 1) * kUnits : 1][RB * 4][SPLIT > 1 ? 64 : 1];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int split = wave % SPLIT, local = wave / SPLIT;
  const int nblocks = fp4_nblocks(p.N), steps = fp4_steps(p.K);
  const int per_block = p.block_m / (16 * RB);
  const int used = min(p.capacity, *p.ntpp) / p.block_m * per_block;
  const int64_t units = (int64_t)used * nblocks;
  for (int64_t u0 = (int64_t)blockIdx.x * kUnits; u0 < units; u0 += (int64_t)gridDim.x * kUnits) {
    const int64_t u = u0 + local;
    const bool active = u < units;
    const int b = (int)(u / nblocks), nb = (int)(u - (int64_t)b * nblocks);
    const int e = active ? p.expert_ids[b / per_block] : -1;
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
        for (int j = 0; j < 4; ++j) w[d][j] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(at + 1024 * j + 16 * lane));
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
          for (int j = 0; j < 4; ++j) acc[r][j] = mfma_fp4(j, w[d][j], a[d][r], acc[r][j], ws[d], scale);
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
constexpr int kGroupRows = 4;
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

// Many rows per expert: a workgroup of four waves computes BM rows times 256
// columns, a wave all of its rows times 64 columns, on 32 x 32 x 64 MFMAs. A
// wave's weights are its own and go from memory to registers; the rows are shared,
// so each wave fetches its part of them and all read them from LDS. Both are
// fetched two steps of K = 128 ahead. The loop goes by turns of two steps with a
// barrier each; a step past the last repeats the last one's weights with zero rows.
//
// Rows are fetched with four neighbouring lanes on a row's 64 bytes, since the
// vector cache takes one line of four lanes at a time, and lie in LDS as they
// come, row by row, the 16-byte chunk c of row r in place c ^ (r / 2 % 4): eight
// rows' chunks c then cover 128 bytes modulo 128, while rows r and r + 8 lie on the
// same places modulo 256. Bank conflicts are 37% of the LDS's active cycles at 48 x
// 128 rows and 38% at 32768 (K 7168 and 2048). Row scales, a dword a step, are fetched
// for G steps at once (4 where K allows it: a load of one row's scales per lane
// takes the cache 64 lines).
//
// 32768 rows (16 experts) by 7168 columns, K 2048: 317 us on inputs that change from
// call to call, 3.0 PFLOP/s of the 9.4 that the instruction reaches by itself (300 us
// where they stay the same; the first twenty calls after a pause take up to 381); 48 x
// 128 rows by 4096, K 7168: 137-143 us, 5.7 TB/s. The loads of a step (24 KB a workgroup), the reads from LDS and the MFMAs
// are each about half of its time, and the two workgroups of a compute unit
// overlap them in part. A loop of 32 x 32 x 64 MFMAs reaches 8.9 PFLOP/s with one wave
// a SIMD, one of 16 x 16 x 128 7.6. The accumulators of 128 x 64 values are half of a
// wave's registers; 128 x 128 left room for one wave a SIMD: 391 against 364 us.
template <typename T, int BM, int G, Policy W>
__global__ __launch_bounds__(256, 2) void fp4_tile_kernel(Fp4GemmParams p, int ntiles) {
  constexpr int D = 2;
  constexpr int kBlocks = BM / 32;  // row blocks
  constexpr int kMine = BM / 64;    // 16-row parts that a wave fetches
  constexpr int kAhead = 2;         // row fragments read from LDS before their use
  __shared__ i32x4 rows_lds[2][D][BM][4];  // turn, step, row, chunk
  __shared__ uint32_t scales_lds[2][G][BM];  // group, step, row: the scales of its four k blocks
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nblocks = fp4_nblocks(p.N), last = p.K / kFp4StepK - 1;
  int b, nt;
  if (!tile_of(min(p.capacity, *p.ntpp) / BM, ntiles, b, nt)) return;
  const int nb = nt * 4 + wave;
  const int e = p.expert_ids[b];
  const bool known = (uint32_t)e < (uint32_t)p.E;
  floatx16 acc[kBlocks][2] = {};

  if (known) {
    // rows without a slot read row 0 and are zeroed at the store
    auto source = [&](int row) -> uint32_t {
      const uint32_t slot = (uint32_t)p.sorted[b * BM + row];
      if (slot >= (uint32_t)p.n_slots) return 0;
      return p.gather ? slot / (uint32_t)p.topk : (uint32_t)(b * BM + row);
    };
    const Buffer a_q(p.a_q, (int64_t)p.a_rows * (p.K / 2)), a_s(p.a_s, (int64_t)p.a_rows * (p.K / 32));
    uint32_t aq[kMine];
    i32x4* put[kMine];  // in ring slot 0
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int row = 16 * (wave * kMine + i) + (lane >> 2);
      aq[i] = source(row) * (uint32_t)(p.K / 2) + 16 * (lane & 3);
      put[i] = &rows_lds[0][0][row][(lane & 3) ^ (row >> 1 & 3)];
    }
    const bool scaler = wave < BM / 64;  // this wave fetches scales, a row a thread
    const uint32_t as = scaler ? source(tid) * (uint32_t)(p.K / 32) : 0;
    // a wave past the last column block repeats it and stores nothing
    const Buffer wp(p.packed + ((int64_t)e * nblocks + min(nb, nblocks - 1)) * (last + 1) * kFp4UnitBytes,
                    (int64_t)(last + 1) * kFp4UnitBytes);
    // of a 16 x 128 part: this lane's column and k block in the first half of K
    const uint32_t part = (lane & 15) + 16 * (lane >> 5), odd = lane >> 4 & 1;
    const uint32_t wcodes = 1024 * odd + 16 * part, wscales = 4096 + 4 * part;

    i32x4 w[D][2][2], a[D][kMine];
    uint32_t ws[D][2], sc[G];
    // what lies past the end repeats the last, so that no load is behind a branch
    auto fetch_rows = [&](int slot, int step) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) a[slot][i] = a_q.load4(aq[i], 64 * min(step, last));
    };
    auto publish_rows = [&](int turn) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int keep = D * turn + d <= last ? -1 : 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) put[i][((turn & 1) * D + d) * BM * 4] = a[d][i] & keep;
      }
    };
    auto fetch_scales = [&](int group) {
      if (G == 4) {  // last + 1 is a multiple of 4
        const i32x4 got = a_s.load4(as, 4 * G * min(group, last / G));
#pragma unroll
        for (int g = 0; g < G; ++g) sc[g] = (uint32_t)got[g];
      } else {
#pragma unroll
        for (int g = 0; g < G; ++g) sc[g] = a_s.load(as, 4 * min(G * group + g, last));
      }
    };
    auto publish_scales = [&](int group) {
#pragma unroll
      for (int g = 0; g < G; ++g) scales_lds[group & 1][g][tid] = sc[g];
    };
    auto fetch_weights = [&](int slot, int step) {
      const int at = min(step, last) * kFp4UnitBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < 2; ++c) w[slot][h][c] = wp.load4<W>(wcodes + 2048 * c + 512 * h, at);
        ws[slot][h] = wp.load(wscales + 128 * h, at);
      }
    };
    auto compute = [&](int d, int turn) {
      const int s = D * turn + d;
      // bytes 0 and 2: of the rows' scales, this lane's k block in each half of K; of the
      // columns', this lane's two columns
      uint32_t rs[kBlocks], cs[2];
#pragma unroll
      for (int r = 0; r < kBlocks; ++r) rs[r] = scales_lds[s / G & 1][s % G][32 * r + (lane & 31)] >> (8 * (lane >> 5));
#pragma unroll
      for (int h = 0; h < 2; ++h) cs[h] = ws[d][h] >> (8 * odd);
      constexpr int kFragments = 2 * kBlocks;  // (half of K, row block)
      i32x4 av[kAhead + 1];
      auto fragment = [&](int f) {
        const int row = 32 * (f % kBlocks) + (lane & 31), chunk = 2 * (f / kBlocks) + (lane >> 5);
        av[f % (kAhead + 1)] = rows_lds[turn & 1][d][row][chunk ^ (row >> 1 & 3)];
      };
#pragma unroll
      for (int f = 0; f < kAhead; ++f) fragment(f);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = 0; f < kFragments; ++f) {
        if (f + kAhead < kFragments) fragment(f + kAhead);
        const int h = f / kBlocks, r = f % kBlocks;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          acc[r][c] = mfma_fp4_32(c, h, w[d][h][c], av[f % (kAhead + 1)], acc[r][c], (int)cs[h], (int)rs[r]);
        __builtin_amdgcn_sched_barrier(0);
      }
      fetch_weights(d, s + D);
      __builtin_amdgcn_sched_barrier(0);
    };
    if (scaler) fetch_scales(0);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      fetch_rows(d, d);
      fetch_weights(d, d);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (scaler) {
      publish_scales(0);
      fetch_scales(1);
    }
    publish_rows(0);
#pragma unroll
    for (int d = 0; d < D; ++d) fetch_rows(d, D + d);
    lds_barrier();
    // No load is on its way when the loop is entered: the compiler's waits in it would
    // else count for this order of loads, rows last, as well and drain every turn.
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    for (int turn = 0; D * turn <= last; ++turn) {
      // the next turn's rows and scales, into what was last read a barrier ago
      publish_rows(turn + 1);
#pragma unroll
      for (int d = 0; d < D; ++d) fetch_rows(d, D * (turn + 2) + d);
      if (scaler && D * turn % G == 0) {
        publish_scales(D * turn / G + 1);
        fetch_scales(D * turn / G + 2);
      }
#pragma unroll
      for (int d = 0; d < D; ++d) compute(d, turn);
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // A row block at a time through LDS, so that a store covers whole 128-byte
  // lines: 32 rows of 64 columns, 16 bytes between rows, so that rows begin on the same
  // place modulo 256 no nearer than 16 apart (modulo 128, no nearer than 8).
  constexpr int kPitch = 64 * (int)sizeof(T) + 16;
  constexpr int kChunks = 64 * (int)sizeof(T) / 16;  // of a row
  constexpr int kRowsAtOnce = 64 / kChunks;
  __shared__ __attribute__((aligned(16))) uint8_t tile_lds[4][32 * kPitch];
  uint8_t* tile = tile_lds[wave];
  uint64_t real[BM / 64];  // which rows have a slot
#pragma unroll
  for (int i = 0; i < BM / 64; ++i)
    real[i] = __ballot(known && (uint32_t)p.sorted[b * BM + 64 * i + lane] < (uint32_t)p.n_slots);
  const int col = nb * kNBlock + lane % kChunks * (16 / (int)sizeof(T));
#pragma unroll
  for (int r = 0; r < kBlocks; ++r) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int g = 0; g < 4; ++g)  // a lane's values are columns 8 g + 4 (lane / 32) + 0..3 of row lane % 32
        store4(reinterpret_cast<T*>(tile + (lane & 31) * kPitch) + 32 * c + 8 * g + 4 * (lane >> 5),
               floatx4{acc[r][c][4 * g], acc[r][c][4 * g + 1], acc[r][c][4 * g + 2], acc[r][c][4 * g + 3]});
#pragma unroll
    for (int i = 0; i < 32 / kRowsAtOnce; ++i) {
      const int row = 32 * r + i * kRowsAtOnce + lane / kChunks;
      i32x4 v = *reinterpret_cast<const i32x4*>(tile + (row & 31) * kPitch + 16 * (lane % kChunks));
      if (!((real[32 * r / 64] >> (row & 63)) & 1)) v = i32x4{0, 0, 0, 0};
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
  const int64_t units = (int64_t)(p.capacity / p.block_m) * (p.block_m / (16 * RB)) * fp4_nblocks(p.N);
  const int64_t groups = (units * SPLIT + 3) / 4;
  if (groups == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(groups, (int64_t)device_cu_count() * 64)), threads(256);
  if (!whole_steps(p))
    hipLaunchKernelGGL((fp4_stream_kernel<T, RB, SPLIT, D, true>), grid, threads, 0, stream, p);
  else
    hipLaunchKernelGGL((fp4_stream_kernel<T, RB, SPLIT, D, false>), grid, threads, 0, stream, p);
  return hipGetLastError();
}

template <typename T, int BM, int G>
hipError_t launch_tile(const Fp4GemmParams& p, hipStream_t stream) {
  const int ntiles = (fp4_nblocks(p.N) + 3) / 4;
  const int64_t tiles = (int64_t)(p.capacity / BM) * ntiles;
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid == 0) return hipSuccess;
  if (grid >= 1 << 24) return hipErrorInvalidValue;  // a launch has less than 2^32 threads
  const dim3 g((unsigned)grid), t(256);
  // Weights that one row block of their expert reads are streamed, what several read is
  // kept in the caches: 48 x 128 rows take 139 us so and 147 us cached, 16 x 2048 rows
  // (with the activation) 358 us cached and 418 us streamed. The counts are on the
  // device, so an expert's rows are taken as n_slots over E: their mean where every
  // routed expert is resident. On a slice of the experts n_slots counts the others'
  // slots too, and a call of one row block an expert may read its weights cached.
  if (p.n_slots <= (int64_t)p.E * BM * 3 / 2)
    hipLaunchKernelGGL((fp4_tile_kernel<T, BM, G, kStreamed>), g, t, 0, stream, p, ntiles);
  else
    hipLaunchKernelGGL((fp4_tile_kernel<T, BM, G, kCached>), g, t, 0, stream, p, ntiles);
  return hipGetLastError();
}

template <typename T, int BM>
hipError_t launch_tile(const Fp4GemmParams& p, hipStream_t stream) {
  if (p.K / kFp4StepK % 4 == 0) return launch_tile<T, BM, 4>(p, stream);
  return launch_tile<T, BM, 2>(p, stream);
}

template <typename T>
hipError_t launch(const Fp4GemmParams& p, hipStream_t stream) {
  if (p.block_m == 16) return launch_stream<T, 1, 4, 3>(p, stream);
  if (p.block_m == 32) return launch_stream<T, 2, 4, 3>(p, stream);
  // Tiles that the call is expected to have: its slots, half a block of padding an expert.
  // On a slice of the experts that is more than there are (the other experts' slots count
  // too, up to the capacity), and the rule then takes tiles earlier than the figures below say.
  const int64_t rows = std::min<int64_t>(p.capacity, (int64_t)p.n_slots + (int64_t)p.E * (p.block_m / 2));
  const int64_t tiles = rows * ((fp4_nblocks(p.N) + 3) / 4) / p.block_m;
  // A tile goes through K alone, the streaming kernel's four waves share it. One expert,
  // 128-row blocks, streaming against tiles: 32 tiles at K 7168 25 against 31 us, 56 tiles 44
  // against 32; 32 tiles at K 2048 11 against 13, 56 tiles 18 against 13. 64-row blocks:
  // 32 tiles at K 7168 14 against 20 us, 64 tiles 24 against 20.
  // The tile kernel's offsets into the rows are 32 bits.
  if (tiles >= 48 && whole_steps(p) && (int64_t)p.a_rows * (p.K / 2) < (int64_t)1 << 32)
    return p.block_m == 128 ? launch_tile<T, 128>(p, stream) : launch_tile<T, 64>(p, stream);
  // K that ends inside a step: 64 rows a wave once there are many (2080 by 4096 columns:
  // 500 rows 16 against 15 us, 4000 rows 69 against 113).
  if (tiles >= 128) return launch_stream<T, 4, 1, 2>(p, stream);
  return launch_stream<T, 2, 4, 3>(p, stream);
}

}  // namespace

hipError_t launch_fp4_gemm(const Fp4GemmParams& p, int32_t out_dtype, hipStream_t stream) {
  if (out_dtype == kBF16) return launch<bf16_t>(p, stream);
  if (out_dtype == kFP16) return launch<f16_t>(p, stream);
  return launch<float>(p, stream);
}

}  // namespace w4a16
