// Launchers of the experts' product on 16-bit weights and of its weights' gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

struct GroupedParams {
  const void* a;          // rows [a_rows, K]
  const void* w;          // [E, N, K], or [E, K, N] with `transposed`
  void* out;              // [capacity, N]
  const int32_t* sorted;  // as moe_align writes them
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int32_t E, N, K;
  int32_t gather;         // row of aligned row p: sorted[p] / topk, else p
  int32_t topk, n_slots, capacity, block_m;
  int32_t transposed;
};
// Workgroups that a call launches at most, of 512 threads; a launch has less than 2^32 threads.
int64_t grouped_workgroups(int32_t N, int32_t capacity, int32_t block_m);
hipError_t launch_grouped_gemm(const GroupedParams& p, int32_t dtype, int32_t out_dtype, hipStream_t stream);

struct WgradParams {
  const void* dout;       // [capacity, N]
  const void* a;          // rows [a_rows, K]
  void* dw;               // [E, N, K]
  float* partial;         // [splits, E, N, K] where splits > 1
  const int32_t* sorted;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int32_t E, N, K;
  int32_t gather;
  int32_t topk, n_slots, capacity, block_m;
  int32_t accumulate;
  int32_t splits;         // wgrad_splits
};
// How many workgroups share an expert's rows, a rule on sizes alone.
int32_t wgrad_splits(int32_t E, int32_t N, int32_t K, int32_t capacity);
int64_t wgrad_workgroups(int32_t E, int32_t N, int32_t K, int32_t splits);
hipError_t launch_grouped_wgrad(const WgradParams& p, int32_t dtype, int32_t dw_dtype, hipStream_t stream);

}  // namespace w4a16
