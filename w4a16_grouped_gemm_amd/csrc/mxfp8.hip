// Activation checkpoints: rows in 8-bit floating point (four exponent bits,
// three mantissa bits) with one power-of-two scale per 32 values, and the
// activation between the experts' products with a backward pass that reads them.
//
// A quad of lanes owns a block of 32, eight values a lane. The scale is the
// smallest power of two that brings the block's largest magnitude to 448, the
// format's largest, or below, so no value saturates; dividing by it is exact,
// and the conversion (nearest, ties to even) is the only rounding.
//
// All of it is bound by memory: each value is read and written once, in streams of 8 or 16 bytes a lane.
// Measured (one MI355X, bf16): 16384 rows of 7168 quantised in 56 us and back in 57 (6.3 TB/s; reads alone reach
// 6.9, a copy 4.9); the activation of 32768 rows of 2 x 2048 89 us (6.1 TB/s), its gradient 106 (6.3 TB/s), 98 and 120
// where every wave has a gate so far out that the products go by mantissas and exponents; a few rows 3 us, a
// launch's own time.
#include "row_ops.h"
#include "rows.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

constexpr int kThreads = 256;

typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ __forceinline__ uint32_t quad_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, quad_dpp<0xB1>(v));  // lane ^ 1
  return max(v, quad_dpp<0x4E>(v));  // lane ^ 2
}

struct Codes {
  uint32_t v[2];  // eight codes
  uint32_t scale;
  uint32_t most;  // the block's largest magnitude, as bits
};

// Eight values of a lane's quarter block -> their codes and the block's scale byte. Magnitudes
// compare as integers, so that infinities and NaN come out on top: such a block is marked 255.
__device__ __forceinline__ Codes encode8(const float (&x)[8]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  most = quad_max(most);
  const bool finite = most < 0x7F800000u;
  // 448 is 1.75 * 2^8: a mantissa above 1.75 (0x600000) takes the next power of two
  const int32_t byte = max((int32_t)((most + 0x1FFFFFu) >> 23) - 8, 0);
  const float inverse = __uint_as_float((uint32_t)(254 - byte) << 23);  // byte <= 247 where finite: a normal number
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = finite ? x[i] * inverse : 0.f;
  Codes c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int word = 0;
    word = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], word, false);
    word = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], word, true);
    c.v[i] = (uint32_t)word;
  }
  c.scale = finite ? (uint32_t)byte : 255u;
  c.most = most;
  return c;
}

__device__ __forceinline__ float scale_of(uint32_t byte) {
  // 2^-127 is below the normal numbers
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte ? byte << 23 : 0x00400000u);
}

__device__ __forceinline__ void decode8(const uint32_t (&code)[2], float scale, float (&out)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[i], false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[i], true);
    out[4 * i] = lo[0] * scale;
    out[4 * i + 1] = lo[1] * scale;
    out[4 * i + 2] = hi[0] * scale;
    out[4 * i + 3] = hi[1] * scale;
  }
}

constexpr float kLog2E = 1.44269504f, kLog2ELow = 1.92596299e-8f;

// 1 / d, with the instruction's error taken out by one step of Newton's.
__device__ __forceinline__ float reciprocal(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
}

// 1 / (1 + exp(-g)), as sig * 2^power, and 1 less that, neither by a difference. exp(-g) is 2^whole times m = 2^part, the
// part with the product's rounding error and the constant's put back, so that m holds to a few units in the last place
// at any g; where whole is positive, both terms of the sum are taken 2^-whole times.
// FAR: any g. exp(g) leaves fp32's numbers at g = -87, and products with it come back into them where the other factors
// are large. Below -400 it counts as zero: under 2^-577, no product of a gate and two more fp32 values with it rounds to
// anything else. Else |g| is up to 87, and power is 0.
template <bool FAR>
__device__ __forceinline__ void sigmoid(float g, float& sig, int& power, float& rest) {
  const float x = FAR ? __builtin_amdgcn_fmed3f(-g, -400.f, 400.f) : -g;
  const float whole = __builtin_rintf(x * kLog2E);
  const float part = __builtin_fmaf(x, kLog2ELow, __builtin_fmaf(x, kLog2E, -whole));  // within 0.51: good to 2^-25
  const float m = __builtin_amdgcn_exp2f(part);
  const int down = max((int)whole, 0);
  const float over = __builtin_amdgcn_ldexpf(m, (int)whole - down);
  const float inverse = reciprocal(__builtin_amdgcn_ldexpf(1.f, -down) + over);
  sig = !FAR ? __builtin_amdgcn_ldexpf(inverse, -down) : x < 400.f ? inverse : 0.f;
  power = FAR ? -down : 0;
  rest = over * inverse;
}

// x = mantissa * 2^power. FAR: the mantissa in [0.5, 1), so that the only step that can leave fp32's numbers is the
// product's last, and the bits are those of the plain product where that does not leave them.
struct Parts {
  float mantissa;
  int power;
};
template <bool FAR>
__device__ __forceinline__ Parts parts(float x) {
  return FAR ? Parts{__builtin_amdgcn_frexp_mantf(x), __builtin_amdgcn_frexp_expf(x)} : Parts{x, 0};
}
template <bool FAR>
__device__ __forceinline__ float times_power(float x, int power) {
  return FAR ? __builtin_amdgcn_ldexpf(x, power) : x;
}

template <bool FAR>
__device__ __forceinline__ float silu_mul(float gate, float up) {
  float sig, rest;
  int power;
  sigmoid<FAR>(gate, sig, power, rest);
  const Parts g = parts<FAR>(gate), u = parts<FAR>(up);
  return times_power<FAR>(g.mantissa * sig * u.mantissa, g.power + u.power + power);
}

// dgate = dh up sig (1 + gate (1 - sig)), dup = dh gate sig, h = gate sig up
template <bool FAR>
__device__ __forceinline__ void gradient(float gate, float up, float dh, float& dgate, float& dup, float& h) {
  float sig, rest;
  int power;
  sigmoid<FAR>(gate, sig, power, rest);
  const Parts g = parts<FAR>(gate), u = parts<FAR>(up), d = parts<FAR>(dh);
  const float silu = g.mantissa * sig, slope = __builtin_fmaf(gate * sig, rest, sig);
  dgate = times_power<FAR>(d.mantissa * u.mantissa * slope, d.power + u.power + power);
  dup = times_power<FAR>(d.mantissa * silu, d.power + g.power + power);
  h = times_power<FAR>(silu * u.mantissa, g.power + u.power + power);
}

__device__ __forceinline__ int64_t live_rows(int32_t rows, const int32_t* num_rows) {
  return num_rows ? max(0, min(rows, *num_rows)) : rows;
}

__device__ __forceinline__ void store_codes(uint8_t* q, int64_t at, const Codes& c) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(u32x2{c.v[0], c.v[1]}, reinterpret_cast<u32x2*>(q + at));
}

__device__ __forceinline__ void load_codes(const uint8_t* q, int64_t at, uint32_t (&code)[2]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(q + at));
  code[0] = v[0];
  code[1] = v[1];
}

// Groups of eight values, kUnroll of them per thread, a block of threads apart; the loads of all
// come before the first use.
constexpr int kUnroll = 4;

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* x, int32_t rows, int32_t K,
                                                            const int32_t* num_rows, uint8_t* q, uint8_t* s) {
  const int64_t total = live_rows(rows, num_rows) * (int64_t)(K / 8);  // a multiple of 4: quads are whole
  for (int64_t g0 = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; g0 < total;
       g0 += (int64_t)gridDim.x * kThreads * kUnroll) {
    Eight<T> a[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (g0 + u * kThreads < total) a[u] = load8<kStreamed>(x + 8 * (g0 + u * kThreads));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t g = g0 + u * kThreads;
      if (g >= total) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)a[u].v[i];
      const Codes c = encode8(v);
      store_codes(q, 8 * g, c);
      if ((g & 3) == 0) s[g >> 2] = (uint8_t)c.scale;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* q, const uint8_t* s, int32_t rows,
                                                              int32_t K, const int32_t* num_rows, T* out) {
  const int64_t total = live_rows(rows, num_rows) * (int64_t)(K / 8);
  for (int64_t g0 = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; g0 < total;
       g0 += (int64_t)gridDim.x * kThreads * kUnroll) {
    uint32_t code[kUnroll][2], byte[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t g = g0 + u * kThreads;
      if (g >= total) continue;
      load_codes(q, 8 * g, code[u]);
      byte[u] = s[g >> 2];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t g = g0 + u * kThreads;
      if (g >= total) continue;
      float v[8];
      decode8(code[u], scale_of(byte[u]), v);
      Eight<T> r;
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = (T)v[i];
      store8<kStreamed>(out + 8 * g, r);
    }
  }
}

// Where a thread's group of eight columns lies: row r, columns c on of [rows, I].
struct Place {
  int64_t row;
  int32_t column;
};
__device__ __forceinline__ Place place_of(int64_t group, uint32_t per_row) {
  const int64_t row = group / per_row;
  return {row, 8 * (int32_t)(group - row * per_row)};
}

// h = silu(gate) * up, and gate and up in 8 bits.
template <typename T>
__global__ __launch_bounds__(kThreads) void silu_mul_kernel(const T* gu, int32_t rows, int32_t I,
                                                            const int32_t* num_rows, T* h, uint8_t* q, uint8_t* s) {
  const uint32_t per_row = (uint32_t)I / 8;
  const int64_t total = live_rows(rows, num_rows) * (int64_t)per_row;
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < total; g += (int64_t)gridDim.x * kThreads) {
    const Place at = place_of(g, per_row);
    const int64_t gate_at = 2 * at.row * I + at.column, up_at = gate_at + I;
    const Eight<T> a = load8<kStreamed>(gu + gate_at), b = load8<kStreamed>(gu + up_at);
    float gate[8], up[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gate[i] = (float)a.v[i];
      up[i] = (float)b.v[i];
    }
    const Codes cg = encode8(gate), cu = encode8(up);
    Eight<T> r;
    if (!__any(cg.most > __float_as_uint(87.f))) {  // by the wave: some lanes one way and some the other take both ways' time
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = (T)silu_mul<false>(gate[i], up[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = (T)silu_mul<true>(gate[i], up[i]);
    }
    store8<kStreamed>(h + at.row * I + at.column, r);
    store_codes(q, gate_at, cg);
    store_codes(q, up_at, cu);
    if ((g & 3) == 0) {
      s[gate_at / 32] = (uint8_t)cg.scale;
      s[up_at / 32] = (uint8_t)cu.scale;
    }
  }
}

// From the checkpoint: dgate = dh up sig (1 + gate (1 - sig)), dup = dh gate sig, and h again.
template <typename T>
__global__ __launch_bounds__(kThreads) void silu_mul_backward_kernel(const uint8_t* q, const uint8_t* s, const T* dh,
                                                                     int32_t rows, int32_t I, const int32_t* num_rows,
                                                                     T* dgu, T* h) {
  const uint32_t per_row = (uint32_t)I / 8;
  const int64_t total = live_rows(rows, num_rows) * (int64_t)per_row;
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < total; g += (int64_t)gridDim.x * kThreads) {
    const Place at = place_of(g, per_row);
    const int64_t gate_at = 2 * at.row * I + at.column, up_at = gate_at + I;
    uint32_t gate_code[2], up_code[2];
    load_codes(q, gate_at, gate_code);
    load_codes(q, up_at, up_code);
    const uint32_t gate_scale = s[gate_at / 32], up_scale = s[up_at / 32];
    const Eight<T> d = load8<kStreamed>(dh + at.row * I + at.column);
    float gate[8], up[8];
    decode8(gate_code, scale_of(gate_scale), gate);
    decode8(up_code, scale_of(up_scale), up);
    uint32_t most = 0;  // of dh, as bits
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint((float)d.v[i]) & 0x7FFFFFFFu);
    // |gate| up to 448 / 8, |up| and |dh| below 2^63: no product leaves fp32's numbers before the result does
    const bool far = gate_scale > 127 - 3 || up_scale > 127 + 54 || most >= __float_as_uint(0x1p63f);
    auto each = [&](auto kind) {
      Eight<T> dg, du, again;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float dgate, dup, h_again;
        gradient<kind>(gate[i], up[i], (float)d.v[i], dgate, dup, h_again);
        dg.v[i] = (T)dgate;
        du.v[i] = (T)dup;
        again.v[i] = (T)h_again;
      }
      // a line's parts are stored together (32768 rows of 2 x 2048 far gates, fp32: 228 us instead of 368)
      if (kind) __builtin_amdgcn_sched_barrier(0);
      store8<kStreamed>(dgu + gate_at, dg);
      store8<kStreamed>(dgu + up_at, du);
      if (h) store8<kStreamed>(h + at.row * I + at.column, again);
    };
    if (!__any(far))
      each(std::false_type());
    else
      each(std::true_type());
  }
}

// Blocks for `items` of work of `each` per thread, up to `per_cu` a compute unit.
dim3 grid_for(int64_t items, int each, int per_cu) {
  const int64_t per_block = (int64_t)kThreads * each;
  return dim3((unsigned)std::min<int64_t>((items + per_block - 1) / per_block, (int64_t)device_cu_count() * per_cu));
}

// f with a value of the type that `dtype` names.
template <typename F>
hipError_t typed(int32_t dtype, F f) {
  if (dtype == kBF16)
    f(bf16_t());
  else if (dtype == kFP16)
    f(f16_t());
  else
    f(float());
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize(const void* x, int32_t dtype, int32_t rows, int32_t K, const int32_t* num_rows,
                               uint8_t* q, uint8_t* s, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return typed(dtype, [&](auto t) {
    typedef decltype(t) T;
    hipLaunchKernelGGL((quantize_kernel<T>), grid_for((int64_t)rows * (K / 8), kUnroll, 256), dim3(kThreads), 0, stream,
                       static_cast<const T*>(x), rows, K, num_rows, q, s);
  });
}

hipError_t launch_fp8_dequantize(const uint8_t* q, const uint8_t* s, int32_t rows, int32_t K, const int32_t* num_rows,
                                 void* out, int32_t dtype, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return typed(dtype, [&](auto t) {
    typedef decltype(t) T;
    hipLaunchKernelGGL((dequantize_kernel<T>), grid_for((int64_t)rows * (K / 8), kUnroll, 256), dim3(kThreads), 0,
                       stream, q, s, rows, K, num_rows, static_cast<T*>(out));
  });
}

hipError_t launch_fp8_silu_mul(const void* gu, int32_t dtype, int32_t rows, int32_t I, const int32_t* num_rows, void* h,
                               uint8_t* q, uint8_t* s, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return typed(dtype, [&](auto t) {
    typedef decltype(t) T;
    hipLaunchKernelGGL((silu_mul_kernel<T>), grid_for((int64_t)rows * (I / 8), 1, 256), dim3(kThreads), 0, stream,
                       static_cast<const T*>(gu), rows, I, num_rows, static_cast<T*>(h), q, s);
  });
}

hipError_t launch_fp8_silu_mul_backward(const uint8_t* q, const uint8_t* s, const void* dh, int32_t dtype, int32_t rows,
                                        int32_t I, const int32_t* num_rows, void* dgu, void* h, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return typed(dtype, [&](auto t) {
    typedef decltype(t) T;
    hipLaunchKernelGGL((silu_mul_backward_kernel<T>), grid_for((int64_t)rows * (I / 8), 1, 256), dim3(kThreads), 0,
                       stream, q, s, static_cast<const T*>(dh), rows, I, num_rows, static_cast<T*>(dgu),
                       static_cast<T*>(h));
  });
}

}  // namespace w4a16
