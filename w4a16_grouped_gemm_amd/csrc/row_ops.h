// Launchers and layouts of the row operators and of 4-bit floating point; the layer's own are in internal.h.
#pragma once

#include "internal.h"

namespace w4a16 {

// Element types of the row operators (w4a16_dtype of the C ABI).
enum Dtype { kBF16 = 0, kFP16 = 1, kFP32 = 2 };

// Token rows into the aligned order and back (permute.hip); n = T * topk slots.
hipError_t launch_permute(const void* x, int32_t dtype, int32_t T, int32_t topk, int32_t H, const int32_t* sorted,
                          int32_t capacity, const int32_t* ntpp, void* xp, int32_t* slot_rows, hipStream_t stream);
hipError_t launch_unpermute(const void* y, int32_t y_dtype, int32_t rows, int32_t T, int32_t topk, int32_t H,
                            const int32_t* slot_rows, const float* weights, void* out, int32_t out_dtype,
                            hipStream_t stream);
hipError_t launch_unpermute_backward(const void* dout, int32_t out_dtype, const void* y, int32_t y_dtype, int32_t rows,
                                     int32_t T, int32_t topk, int32_t H, const int32_t* slot_rows,
                                     const float* weights, const int32_t* sorted, int32_t capacity,
                                     const int32_t* ntpp, void* dy, float* dweights, hipStream_t stream);

// Packed 4-bit floating point weights: one 4352-byte unit per (expert e, n-block
// nb of 64 columns, step of K = 128), e-major, then nb, then step, so that an
// n-block streams all of K contiguously. Lane l of a wave owns, for each 16-column
// block j = 0..3, the 16 bytes at 1024 j + 16 l: the 32 codes of column
// 64 nb + 16 j + (l & 15) from k = 128 step + 32 (l >> 4) on, in the canonical
// order, which is the operand of v_mfma_scale_f32_16x16x128_f8f6f4; and the
// dword at 4096 + 4 l, whose byte j is that block's scale. Columns past N and
// values past K are zero codes with scale byte 0.
constexpr int kFp4StepK = 128;
constexpr int kFp4UnitBytes = 4352;
__host__ __device__ inline int32_t fp4_nblocks(int32_t N) { return (N + kNBlock - 1) / kNBlock; }
__host__ __device__ inline int32_t fp4_steps(int32_t K) { return (K + kFp4StepK - 1) / kFp4StepK; }

hipError_t launch_fp4_quantize(const void* x, int32_t dtype, int32_t rows, int32_t K, const int32_t* num_rows,
                               uint8_t* q, uint8_t* s, hipStream_t stream);
hipError_t launch_fp4_silu_mul_quantize(const void* gu, int32_t dtype, int32_t rows, int32_t I,
                                        const int32_t* num_rows, uint8_t* q, uint8_t* s, hipStream_t stream);
hipError_t launch_fp4_dequantize(const uint8_t* q, const uint8_t* s, int32_t rows, int32_t K, const int32_t* num_rows,
                                 void* out, int32_t dtype, hipStream_t stream);
hipError_t launch_fp4_repack(const uint8_t* w_q, const uint8_t* w_s, int32_t E, int32_t N, int32_t K, uint8_t* packed,
                             hipStream_t stream);

struct Fp4GemmParams {
  const uint8_t* a_q;     // activation codes [a_rows, K / 2]
  const uint8_t* a_s;     // activation scales [a_rows, K / 32]
  const uint8_t* packed;  // packed weights, all experts
  const int32_t* sorted;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  void* out;              // [capacity, N]
  int32_t E, N, K;
  int32_t a_rows;
  int32_t gather;         // A row of aligned row p: sorted[p] / topk, else p
  int32_t topk, n_slots, capacity, block_m;
};
hipError_t launch_fp4_gemm(const Fp4GemmParams& p, int32_t out_dtype, hipStream_t stream);

}  // namespace w4a16
