// Launchers of the experts' product on 16-bit weights and of its weights' gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

// Division of numbers below 2^31 by d <= 2^16: with 2^l >= d and m = ceil(2^(31+l) / d) <= 2^32,
// n / d = floor(n m / 2^(31+l)), since n (m d - 2^(31+l)) < 2^31 2^l.
struct Divisor {
  uint32_t m;
  int32_t l;
  static Divisor by(uint32_t d) {
    int32_t l = 0;
    while ((1u << l) < d) ++l;
    return {(uint32_t)(((uint64_t)1 << (31 + l)) / d + (((uint64_t)1 << (31 + l)) % d != 0)), l};
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return __umulhi(2 * n, m) >> l; }
};

struct GroupedParams {
  const void* a;          // rows [a_rows, K]
  const void* w;          // [E, N, K], or [E, K, N] with `transposed`
  void* out;              // [capacity, N]
  const int32_t* sorted;  // as moe_align writes them
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int32_t E, N, K;
  int32_t gather;         // row of aligned row p: sorted[p] / topk, else p
  Divisor by_topk;
  int32_t n_slots, capacity, block_m;
  int32_t transposed;
  int32_t far;            // token rows that 32 bits of bytes do not reach
};
// The tile that a call goes by, a rule on sizes alone; n_slots at least 1.
struct GroupedTile {
  int32_t rows, columns;
};
GroupedTile grouped_tile(int32_t E, int32_t N, int32_t n_slots, bool transposed);
hipError_t launch_grouped_gemm(const GroupedParams& p, int32_t dtype, int32_t out_dtype, hipStream_t stream);

// How the weights' gradient is cut, a rule on sizes alone: tiles of tile x tile values, and how many workgroups share an
// expert's rows.
struct WgradCut {
  int32_t tile, splits;
};
struct WgradParams {
  const void* dout;       // [capacity, N]
  const void* a;          // rows [a_rows, K]
  void* dw;               // [E, N, K]
  float* partial;         // [splits, E, N, K] where there are several
  const int32_t* sorted;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int32_t E, N, K;
  int32_t gather;
  Divisor by_topk;
  int32_t n_slots, capacity;
  int32_t far;            // token rows that 32 bits of bytes do not reach
  int32_t log_block;      // of block_m, to base 2
  int32_t accumulate;
  WgradCut cut;
};
WgradCut wgrad_cut(int32_t E, int32_t N, int32_t K, int32_t capacity);
// Workgroups of 512 threads that the call launches; a launch has less than 2^32 threads.
int64_t wgrad_workgroups(int32_t E, int32_t N, int32_t K, WgradCut cut);
hipError_t launch_grouped_wgrad(const WgradParams& p, int32_t dtype, int32_t dw_dtype, hipStream_t stream);

}  // namespace w4a16
