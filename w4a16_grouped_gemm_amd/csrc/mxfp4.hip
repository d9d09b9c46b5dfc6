// Rows to 4-bit floating point with one power-of-two scale per 32 values, and back.
//
// A quad of lanes owns one block of 32: each lane holds eight values, the
// block's largest magnitude is two DPP steps away, and the scale's exponent is
// that magnitude's exponent less 2. Dividing by a power of two is exact, so the
// only rounding is the conversion's (nearest, ties to even, saturating at 6).
//
// Bound by memory: each value is read once, 17 / 32 byte is written for it. 16384 x
// 7168 bf16 to codes 47 us (6.3 TB/s), back 42 us (7.0 TB/s); the activation of 32768
// rows of 2 x 2048 bf16 54 us (5.7 TB/s). Both ways together took 133 us with cached
// accesses, 105 us with streamed loads, 90 us with streamed stores too and a grid of up
// to 256 blocks a compute unit.
#include "row_ops.h"
#include "rows.h"

#include <algorithm>

namespace w4a16 {
namespace {

constexpr int kThreads = 256;

template <int CTRL>
__device__ __forceinline__ uint32_t quad_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, quad_dpp<0xB1>(v));  // lane ^ 1
  return max(v, quad_dpp<0x4E>(v));  // lane ^ 2
}

// Eight values of a lane's quarter block -> eight codes in a dword and the
// block's scale byte. Magnitudes compare as integers, so that infinities and
// NaN come out on top: such a block is marked 255.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], uint32_t& scale) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  const int32_t exponent = (int32_t)(quad_max(most) >> 23);
  const bool finite = exponent != 255;
  const int32_t byte = max(exponent - 2, 0);
  const float inverse = __uint_as_float((uint32_t)(254 - byte) << 23);  // byte <= 252 where finite: a normal number
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = finite ? x[i] * inverse : 0.f;
  uint32_t code = 0;
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[0], v[1], 1.f, 0);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[2], v[3], 1.f, 1);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[4], v[5], 1.f, 2);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[6], v[7], 1.f, 3);
  scale = finite ? (uint32_t)byte : 255u;
  return code;
}

// silu(g) * u. For g < -87 the reciprocal is below the normal numbers and the result zero.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.f + __expf(-g)) * u;
}

__device__ __forceinline__ int64_t live_rows(int32_t rows, const int32_t* num_rows) {
  return num_rows ? max(0, min(rows, *num_rows)) : rows;
}

// Groups of eight values, kUnroll of them per thread side by side, a block of
// threads apart; the loads of all come before the first use.
constexpr int kUnroll = 4;

// SILU: x is [rows, 2 K] and row r's values are silu(x[r, c]) * x[r, K + c].
template <typename T, bool SILU>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* x, int32_t rows, int32_t K,
                                                            const int32_t* num_rows, uint8_t* q, uint8_t* s) {
  const uint32_t per_row = (uint32_t)K / 8;
  const int64_t total = live_rows(rows, num_rows) * (int64_t)per_row;  // a multiple of 4: quads are whole
  for (int64_t g0 = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; g0 < total;
       g0 += (int64_t)gridDim.x * kThreads * kUnroll) {
    Eight<T> a[kUnroll], b[SILU ? kUnroll : 1];
    const int64_t r0 = SILU ? g0 / per_row : 0;
    const uint32_t c0 = SILU ? (uint32_t)(g0 - r0 * per_row) : 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t g = g0 + u * kThreads;
      if (g >= total) continue;
      if (SILU) {
        const uint32_t c = c0 + u * kThreads, down = c / per_row;  // rows further down
        const T* at = x + 2 * (r0 + down) * K + 8 * (c - down * per_row);
        a[u] = load8<kStreamed>(at);
        b[u] = load8<kStreamed>(at + K);
      } else {
        a[u] = load8<kStreamed>(x + 8 * g);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t g = g0 + u * kThreads;
      if (g >= total) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = SILU ? silu_mul((float)a[u].v[i], (float)b[u].v[i]) : (float)a[u].v[i];
      uint32_t scale;
      reinterpret_cast<uint32_t*>(q)[g] = quantize8(v, scale);
      if ((g & 3) == 0) s[g >> 2] = (uint8_t)scale;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* q, const uint8_t* s, int32_t rows,
                                                              int32_t K, const int32_t* num_rows, T* out) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const int64_t total = live_rows(rows, num_rows) * (K / 8);
  for (int64_t g0 = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; g0 < total;
       g0 += (int64_t)gridDim.x * kThreads * kUnroll) {
    uint32_t code[kUnroll], byte[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t g = g0 + u * kThreads;
      if (g >= total) continue;
      code[u] = reinterpret_cast<const uint32_t*>(q)[g];
      byte[u] = s[g >> 2];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t g = g0 + u * kThreads;
      if (g >= total) continue;
      // 2^-127 is below the normal numbers
      const float scale = __uint_as_float(byte[u] == 255 ? 0x7FC00000u : byte[u] ? byte[u] << 23 : 0x00400000u);
      const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u], 1.f, 0),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u], 1.f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u], 1.f, 2),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u], 1.f, 3)};
      Eight<T> r;
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = (T)(v[i >> 1][i & 1] * scale);
      store8<kStreamed>(out + 8 * g, r);
    }
  }
}

// One thread per lane of a packed unit (see row_ops.h).
__global__ __launch_bounds__(kThreads) void repack_fp4_kernel(const uint8_t* w_q, const uint8_t* w_s, int32_t N,
                                                              int32_t K, int64_t units, uint8_t* packed) {
  const int32_t nblocks = fp4_nblocks(N), steps = fp4_steps(K);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < units * 64; i += (int64_t)gridDim.x * kThreads) {
    const int64_t unit = i >> 6;
    const int lane = (int)(i & 63);
    const int32_t step = (int32_t)(unit % steps);
    const int32_t nb = (int32_t)(unit / steps % nblocks);
    const int64_t e = unit / steps / nblocks;
    const int32_t k = step * kFp4StepK + 32 * (lane >> 4);
    uint8_t* dst = packed + unit * kFp4UnitBytes;
    uint32_t scales = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t n = nb * kNBlock + 16 * j + (lane & 15);
      uint4 codes = {0, 0, 0, 0};
      if (n < N && k < K) {
        const int64_t row = e * N + n;
        codes = *reinterpret_cast<const uint4*>(w_q + (row * K + k) / 2);
        scales |= (uint32_t)w_s[(row * K + k) / 32] << (8 * j);
      }
      *reinterpret_cast<uint4*>(dst + 1024 * j + 16 * lane) = codes;
    }
    *reinterpret_cast<uint32_t*>(dst + 4096 + 4 * lane) = scales;
  }
}

// Blocks for `items` of work of `each` per thread, up to `per_cu` a compute unit.
int grid_for(int64_t items, int each, int per_cu) {
  const int64_t per_block = (int64_t)kThreads * each;
  return (int)std::min<int64_t>((items + per_block - 1) / per_block, (int64_t)device_cu_count() * per_cu);
}

template <bool SILU>
hipError_t quantize(const void* x, int32_t dtype, int32_t rows, int32_t K, const int32_t* num_rows, uint8_t* q,
                    uint8_t* s, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const dim3 grid(grid_for((int64_t)rows * (K / 8), kUnroll, 256)), block(kThreads);
  if (dtype == kBF16)
    hipLaunchKernelGGL((quantize_kernel<bf16_t, SILU>), grid, block, 0, stream, static_cast<const bf16_t*>(x), rows, K,
                       num_rows, q, s);
  else if (dtype == kFP16)
    hipLaunchKernelGGL((quantize_kernel<f16_t, SILU>), grid, block, 0, stream, static_cast<const f16_t*>(x), rows, K,
                       num_rows, q, s);
  else
    hipLaunchKernelGGL((quantize_kernel<float, SILU>), grid, block, 0, stream, static_cast<const float*>(x), rows, K,
                       num_rows, q, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_quantize(const void* x, int32_t dtype, int32_t rows, int32_t K, const int32_t* num_rows,
                               uint8_t* q, uint8_t* s, hipStream_t stream) {
  return quantize<false>(x, dtype, rows, K, num_rows, q, s, stream);
}

hipError_t launch_fp4_silu_mul_quantize(const void* gu, int32_t dtype, int32_t rows, int32_t I,
                                        const int32_t* num_rows, uint8_t* q, uint8_t* s, hipStream_t stream) {
  return quantize<true>(gu, dtype, rows, I, num_rows, q, s, stream);
}

hipError_t launch_fp4_dequantize(const uint8_t* q, const uint8_t* s, int32_t rows, int32_t K, const int32_t* num_rows,
                                 void* out, int32_t dtype, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const dim3 grid(grid_for((int64_t)rows * (K / 8), kUnroll, 256)), block(kThreads);
  if (dtype == kBF16)
    hipLaunchKernelGGL((dequantize_kernel<bf16_t>), grid, block, 0, stream, q, s, rows, K, num_rows,
                       static_cast<bf16_t*>(out));
  else if (dtype == kFP16)
    hipLaunchKernelGGL((dequantize_kernel<f16_t>), grid, block, 0, stream, q, s, rows, K, num_rows,
                       static_cast<f16_t*>(out));
  else
    hipLaunchKernelGGL((dequantize_kernel<float>), grid, block, 0, stream, q, s, rows, K, num_rows,
                       static_cast<float*>(out));
  return hipGetLastError();
}

hipError_t launch_fp4_repack(const uint8_t* w_q, const uint8_t* w_s, int32_t E, int32_t N, int32_t K, uint8_t* packed,
                             hipStream_t stream) {
  const int64_t units = (int64_t)E * fp4_nblocks(N) * fp4_steps(K);
  hipLaunchKernelGGL(repack_fp4_kernel, dim3(grid_for(units * 64, 1, 32)), dim3(kThreads), 0, stream, w_q, w_s, N, K,
                     units, packed);
  return hipGetLastError();
}

}  // namespace w4a16
