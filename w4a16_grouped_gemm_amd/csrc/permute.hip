// Token rows into the aligned order of moe_align and back, with gradients.
//
//   permute            xp[p] = x[sorted[p] / topk], zero for padding rows
//   unpermute          out[t] = sum_j w[t, j] * y[slot_rows[t, j]]   (fp32, j order)
//   its gradients      dy[p] = w[s] * dout[s / topk], dw[t, j] = <dout[t], y[slot_rows[t, j]]>
//   permute's gradient is unpermute with weights of 1.
//
// All of it is bound by memory: one token row against its (at most topk) expert
// rows. slot_rows, the inverse of the aligned order, lets the kernels go token by
// token, so that a token's row is read or written once; small permutes go row by row
// and read it once for each slot. Rows are moved eight
// elements a thread; the last hidden % 8 columns go one a thread, so that the
// loop over whole groups has no branches.
#include "row_ops.h"
#include "rows.h"

#include <algorithm>

namespace w4a16 {
namespace {

constexpr int kThreads = 256;

// slot_rows[i] = -1 for the n slots, then slot_rows[sorted[p]] = p for the real rows.
__global__ __launch_bounds__(kThreads) void slot_fill_kernel(int32_t* slot_rows, int32_t n) {
  const int32_t i = (int32_t)(blockIdx.x * kThreads + threadIdx.x);
  if (i < n) slot_rows[i] = -1;
}

__global__ __launch_bounds__(kThreads) void slot_scatter_kernel(const int32_t* sorted, int32_t capacity,
                                                                const int32_t* ntpp, int32_t n, int32_t* slot_rows) {
  const int32_t p = (int32_t)(blockIdx.x * kThreads + threadIdx.x);
  if (p >= min(capacity, *ntpp)) return;
  const uint32_t s = (uint32_t)sorted[p];
  if (s < (uint32_t)n) slot_rows[s] = p;
}

template <Policy P = kCached, typename T>
__device__ __forceinline__ void zero_row(T* row, int32_t H, int32_t thread, int32_t threads) {
  const int32_t whole = H & ~7;
  for (int32_t c = 8 * thread; c < whole; c += 8 * threads) store8<P>(row + c, Eight<T>{});
  if (thread < H - whole) row[whole + thread] = (T)0.f;
}

// The padding rows among the 32 aligned rows from `first` on, eight rows a wave.
constexpr int kPadRows = 32;
template <typename T>
__device__ __forceinline__ void zero_padding(T* rows, const int32_t* sorted, int32_t first, int32_t capacity,
                                             const int32_t* ntpp, int32_t n, int32_t H) {
  constexpr int kWaveRows = kPadRows / (kThreads / 64);
  const int lane = (int)threadIdx.x & 63;
  const int32_t p0 = first + kWaveRows * ((int32_t)threadIdx.x >> 6);
  const bool pad = lane < kWaveRows && p0 + lane < min(capacity, *ntpp) && (uint32_t)sorted[p0 + lane] >= (uint32_t)n;
  for (uint64_t m = __ballot(pad); m; m &= m - 1) zero_row<kStreamed>(rows + (int64_t)(p0 + __builtin_ctzll(m)) * H, H, lane, 64);
}

// Few slots, one launch: block 0 writes slot_rows, the others one aligned row each.
template <typename T>
__global__ __launch_bounds__(kThreads) void permute_by_row_kernel(const T* x, T* xp, const int32_t* sorted,
                                                                  int32_t capacity, const int32_t* ntpp, int32_t n,
                                                                  int32_t topk, int32_t H, int32_t* slot_rows) {
  const int32_t live = min(capacity, *ntpp);
  if (blockIdx.x == 0) {
    for (int32_t i = (int32_t)threadIdx.x; i < n; i += kThreads) slot_rows[i] = -1;
    __syncthreads();
    for (int32_t p = (int32_t)threadIdx.x; p < live; p += 8 * kThreads) {
      uint32_t slot[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) slot[k] = p + k * kThreads < live ? (uint32_t)sorted[p + k * kThreads] : ~0u;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (slot[k] < (uint32_t)n) slot_rows[slot[k]] = p + k * kThreads;
    }
    return;
  }
  const int32_t p = (int32_t)blockIdx.x - 1;
  if (p >= live) return;
  const uint32_t s = (uint32_t)sorted[p];
  T* dst = xp + (int64_t)p * H;
  if (s >= (uint32_t)n) return zero_row(dst, H, (int32_t)threadIdx.x, kThreads);
  const T* src = x + (int64_t)(s / (uint32_t)topk) * H;
  const int32_t whole = H & ~7;
  for (int32_t c = 8 * (int32_t)threadIdx.x; c < whole; c += 8 * kThreads) store8(dst + c, load8(src + c));
  if ((int32_t)threadIdx.x < H - whole) dst[whole + threadIdx.x] = src[whole + threadIdx.x];
}

// Lane j of every wave holds the row of token t's slot j, topk <= 32; which of them are rows.
__device__ __forceinline__ uint64_t token_rows(const int32_t* slot_rows, int64_t t, int32_t topk, int32_t rows,
                                               int32_t& row) {
  const int lane = (int)threadIdx.x & 63;
  row = lane < topk ? slot_rows[t * topk + lane] : -1;
  return __ballot((uint32_t)row < (uint32_t)rows);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Many slots, slot_rows known: a token's row is read once and written to all of its
// rows. The first `pads` blocks zero the padding rows. The rows written are
// streamed: 32768 rows of 7168 bf16 take 109 us so and 187 us with cached stores,
// 149 us row by row (4.9, 2.8 and 3.6 TB/s).
template <typename T>
__global__ __launch_bounds__(kThreads) void permute_by_token_kernel(const T* x, T* xp, const int32_t* sorted,
                                                                    int32_t capacity, const int32_t* ntpp, int32_t n,
                                                                    int32_t pads, int32_t topk, int32_t H,
                                                                    const int32_t* slot_rows) {
  if ((int32_t)blockIdx.x < pads)
    return zero_padding(xp, sorted, (int32_t)blockIdx.x * kPadRows, capacity, ntpp, n, H);
  const int64_t t = (int32_t)blockIdx.x - pads;
  int32_t row;
  const uint64_t has = token_rows(slot_rows, t, topk, capacity, row);
  if (!has) return;
  const T* src = x + t * H;
  const int32_t whole = H & ~7;
  for (int32_t c = 8 * (int32_t)threadIdx.x; c < whole; c += 8 * kThreads) {
    const Eight<T> v = load8(src + c);
    for (uint64_t m = has; m; m &= m - 1)
      store8<kStreamed>(xp + (int64_t)__builtin_amdgcn_readlane(row, __builtin_ctzll(m)) * H + c, v);
  }
  const int32_t c = whole + (int32_t)threadIdx.x;
  if (c < H) {
    const T v = src[c];
    for (uint64_t m = has; m; m &= m - 1) xp[(int64_t)__builtin_amdgcn_readlane(row, __builtin_ctzll(m)) * H + c] = v;
  }
}

// The next K slots of `has` in ascending order, removed from it.
template <int K>
__device__ __forceinline__ void take(uint64_t& has, int (&j)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    j[k] = __builtin_ctzll(has);
    has &= has - 1;
  }
}

// f(width, left) over the slots of `has`, eight at a time and the rest by
// halves: the rows of one group are loaded side by side, and no row twice.
template <int K>
struct Width {
  static constexpr int value = K;
};
template <typename F>
__device__ __forceinline__ void in_groups(uint64_t has, F f) {
  int left = __builtin_popcountll(has);
  for (; left >= 8; left -= 8) f(Width<8>{}, has);
  if (left & 4) f(Width<4>{}, has);
  if (left & 2) f(Width<2>{}, has);
  if (left & 1) f(Width<1>{}, has);
}

// One block per token and `cols` columns, a multiple of 8. Bound by reading y once:
// 32768 rows of 7168 bf16 into 4096 tokens take 94 us, 5.6 TB/s; the rows of up to eight
// slots are in flight at once, and the columns past whole groups are apart, for
// with a test for them inside the loop the loads came one at a time (137 us).
template <typename TY, typename TO>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(const TY* y, int32_t rows, const int32_t* slot_rows,
                                                             const float* weights, TO* out, int32_t topk, int32_t H,
                                                             int32_t cols) {
  const int32_t chunks = (H + cols - 1) / cols;
  const int64_t t = (int32_t)blockIdx.x / chunks;
  const int32_t c0 = ((int32_t)blockIdx.x - (int32_t)t * chunks) * cols;
  const int32_t c1 = min(H, c0 + cols);
  const int lane = (int)threadIdx.x & 63;
  int32_t row;
  const uint64_t has = token_rows(slot_rows, t, topk, rows, row);
  const float weight = weights && ((has >> lane) & 1) ? weights[t * topk + lane] : 1.f;
  TO* dst = out + t * H;
  const int32_t whole = c1 & ~7;
  for (int32_t c = c0 + 8 * (int32_t)threadIdx.x; c < whole; c += 8 * kThreads) {
    float sum[8] = {};
    in_groups(has, [&](auto width, uint64_t& left) {
      constexpr int K = decltype(width)::value;
      int j[K];
      take<K>(left, j);
      Eight<TY> v[K];
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = load8<kStreamed>(y + (int64_t)__builtin_amdgcn_readlane(row, j[k]) * H + c);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float wt = lane_value(weight, j[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += wt * (float)v[k].v[i];
      }
    });
    Eight<TO> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = (TO)sum[i];
    store8(dst + c, r);
  }
  const int32_t c = whole + (int32_t)threadIdx.x;
  if (c < c1) {
    float sum = 0.f;
    for (uint64_t m = has; m; m &= m - 1) {
      const int j = __builtin_ctzll(m);
      sum += lane_value(weight, j) * (float)y[(int64_t)__builtin_amdgcn_readlane(row, j) * H + c];
    }
    dst[c] = (TO)sum;
  }
}

// The sum over a wave, in lane 63: within rows of 16 lanes by shifts, then over the rows.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr:1
  v = dpp_add<0x112, 0xF>(v);  // row_shr:2
  v = dpp_add<0x114, 0xF>(v);  // row_shr:4
  v = dpp_add<0x118, 0xF>(v);  // row_shr:8
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
}

// The first `pads` blocks zero the padding rows of dy; then one block per token: its
// dy rows and weight gradients, up to eight slots at a time, so that dout and y are read
// once for both. Bound by memory, half reads and half writes: 32768 rows of 4096
// bf16 take 115 us, 5.0 TB/s, where a plain copy reaches 4.85.
template <typename TO, typename TY>
__global__ __launch_bounds__(kThreads) void unpermute_backward_kernel(
    const TO* dout, const TY* y, int32_t rows, int32_t pads, const int32_t* slot_rows, const float* weights,
    const int32_t* sorted, int32_t capacity, const int32_t* ntpp, int32_t n, TY* dy, float* dweights, int32_t topk,
    int32_t H) {
  if ((int32_t)blockIdx.x < pads)
    return zero_padding(dy, sorted, (int32_t)blockIdx.x * kPadRows, capacity, ntpp, n, H);
  __shared__ float part[kThreads / 64][8];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int64_t t = (int32_t)blockIdx.x - pads;
  int32_t row;
  const uint64_t has = token_rows(slot_rows, t, topk, rows, row);
  const bool live = (has >> lane) & 1;
  const float weight = weights && live ? weights[t * topk + lane] : 1.f;
  if (dweights && wave == 0 && lane < topk && !live) dweights[t * topk + lane] = 0.f;
  const TO* d = dout + t * H;
  const int32_t whole = H & ~7;
  in_groups(has, [&](auto width, uint64_t& left) {
    constexpr int K = decltype(width)::value;
    int j[K];
    take<K>(left, j);
    int64_t at[K];
    float wt[K], dot[K] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      at[k] = (int64_t)__builtin_amdgcn_readlane(row, j[k]) * H;
      wt[k] = lane_value(weight, j[k]);
    }
    for (int32_t c = 8 * (int32_t)threadIdx.x; c < whole; c += 8 * kThreads) {
      const Eight<TO> dv = load8(d + c);
      Eight<TY> yv[K];
      if (dweights) {
#pragma unroll
        for (int k = 0; k < K; ++k) yv[k] = load8<kStreamed>(y + at[k] + c);
      }
      if (dy) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Eight<TY> r;
#pragma unroll
          for (int i = 0; i < 8; ++i) r.v[i] = (TY)(wt[k] * (float)dv.v[i]);
          store8<kStreamed>(dy + at[k] + c, r);
        }
      }
      if (dweights) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[k] += (float)dv.v[i] * (float)yv[k].v[i];
      }
    }
    const int32_t c = whole + (int32_t)threadIdx.x;
    if (c < H) {
      const float dv = (float)d[c];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (dweights) dot[k] += dv * (float)y[at[k] + c];
        if (dy) dy[at[k] + c] = (TY)(wt[k] * dv);
      }
    }
    if (!dweights) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float sum = wave_sum(dot[k]);
      if (lane == 63) part[wave][k] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((int)threadIdx.x == k)
        dweights[t * topk + j[k]] = (part[0][k] + part[1][k]) + (part[2][k] + part[3][k]);
    __syncthreads();
  });
}

// Up to this many slots and aligned rows one block writes slot_rows while the others move
// rows, beyond it a token's row is read once for all of its slots. By row against by token,
// bf16 on 48 experts, rows aligned to 128: 2048 slots of hidden 7168 16 against 23 us, 8192
// slots 41 against 49 (hidden 1024: 10 against 15), 16384 slots 73 against 62 (16 against 15).
constexpr int32_t kByRowSlots = 8192, kByRowCapacity = 16384;

int blocks_for(int64_t items, int each) { return (int)((items + each - 1) / each); }

template <typename T>
hipError_t permute(const void* x, int32_t tokens, int32_t topk, int32_t H, const int32_t* sorted, int32_t capacity,
                   const int32_t* ntpp, void* xp, int32_t* slot_rows, hipStream_t stream) {
  const int32_t n = tokens * topk;
  const T* src = static_cast<const T*>(x);
  T* dst = static_cast<T*>(xp);
  if (n <= kByRowSlots && capacity <= kByRowCapacity) {
    hipLaunchKernelGGL((permute_by_row_kernel<T>), dim3(1 + capacity), dim3(kThreads), 0, stream, src, dst, sorted,
                       capacity, ntpp, n, topk, H, slot_rows);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(slot_fill_kernel, dim3(blocks_for(n, kThreads)), dim3(kThreads), 0, stream, slot_rows, n);
  if (capacity > 0) {
    const int32_t pads = blocks_for(capacity, kPadRows);
    hipLaunchKernelGGL(slot_scatter_kernel, dim3(blocks_for(capacity, kThreads)), dim3(kThreads), 0, stream, sorted,
                       capacity, ntpp, n, slot_rows);
    hipLaunchKernelGGL((permute_by_token_kernel<T>), dim3((unsigned)pads + (unsigned)tokens), dim3(kThreads), 0,
                       stream, src, dst, sorted, capacity, ntpp, n, pads, topk, H, slot_rows);
  }
  return hipGetLastError();
}

template <typename TY, typename TO>
hipError_t unpermute(const void* y, int32_t rows, int32_t T, int32_t topk, int32_t H, const int32_t* slot_rows,
                     const float* weights, void* out, hipStream_t stream) {
  // A block's threads make one pass over their columns. Against a block per whole row,
  // hidden 7168, top-8 bf16: 256 tokens 7.4 against 8.8 us, 2048 tokens 48 against 49.
  int32_t cols = 8 * kThreads;
  if ((int64_t)T * ((H + cols - 1) / cols) >= 1 << 23) cols = (H + 7) & ~7;  // a launch has less than 2^32 threads
  const int64_t blocks = (int64_t)T * ((H + cols - 1) / cols);
  hipLaunchKernelGGL((unpermute_kernel<TY, TO>), dim3((unsigned)blocks), dim3(kThreads), 0, stream,
                     static_cast<const TY*>(y), rows, slot_rows, weights, static_cast<TO*>(out), topk, H, cols);
  return hipGetLastError();
}

template <typename TO, typename TY>
hipError_t unpermute_backward(const void* dout, const void* y, int32_t rows, int32_t T, int32_t topk, int32_t H,
                              const int32_t* slot_rows, const float* weights, const int32_t* sorted, int32_t capacity,
                              const int32_t* ntpp, void* dy, float* dweights, hipStream_t stream) {
  const int32_t pads = dy ? blocks_for(capacity, kPadRows) : 0;
  if (T + pads == 0) return hipSuccess;
  hipLaunchKernelGGL((unpermute_backward_kernel<TO, TY>), dim3((unsigned)T + (unsigned)pads), dim3(kThreads), 0,
                     stream, static_cast<const TO*>(dout), static_cast<const TY*>(y), rows, pads, slot_rows, weights,
                     sorted, capacity, ntpp, T * topk, static_cast<TY*>(dy), dweights, topk, H);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_permute(const void* x, int32_t dtype, int32_t T, int32_t topk, int32_t H, const int32_t* sorted,
                          int32_t capacity, const int32_t* ntpp, void* xp, int32_t* slot_rows, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  // rows are only moved: two- and four-byte elements
  if (dtype == kFP32) return permute<float>(x, T, topk, H, sorted, capacity, ntpp, xp, slot_rows, stream);
  return permute<bf16_t>(x, T, topk, H, sorted, capacity, ntpp, xp, slot_rows, stream);
}

hipError_t launch_unpermute(const void* y, int32_t y_dtype, int32_t rows, int32_t T, int32_t topk, int32_t H,
                            const int32_t* slot_rows, const float* weights, void* out, int32_t out_dtype,
                            hipStream_t stream) {
  if (T == 0) return hipSuccess;
  if (y_dtype == kBF16) return unpermute<bf16_t, bf16_t>(y, rows, T, topk, H, slot_rows, weights, out, stream);
  if (y_dtype == kFP16) return unpermute<f16_t, f16_t>(y, rows, T, topk, H, slot_rows, weights, out, stream);
  if (out_dtype == kBF16) return unpermute<float, bf16_t>(y, rows, T, topk, H, slot_rows, weights, out, stream);
  if (out_dtype == kFP16) return unpermute<float, f16_t>(y, rows, T, topk, H, slot_rows, weights, out, stream);
  return unpermute<float, float>(y, rows, T, topk, H, slot_rows, weights, out, stream);
}

hipError_t launch_unpermute_backward(const void* dout, int32_t out_dtype, const void* y, int32_t y_dtype, int32_t rows,
                                     int32_t T, int32_t topk, int32_t H, const int32_t* slot_rows,
                                     const float* weights, const int32_t* sorted, int32_t capacity,
                                     const int32_t* ntpp, void* dy, float* dweights, hipStream_t stream) {
  if (y_dtype == kBF16)
    return unpermute_backward<bf16_t, bf16_t>(dout, y, rows, T, topk, H, slot_rows, weights, sorted, capacity, ntpp,
                                              dy, dweights, stream);
  if (y_dtype == kFP16)
    return unpermute_backward<f16_t, f16_t>(dout, y, rows, T, topk, H, slot_rows, weights, sorted, capacity, ntpp, dy,
                                            dweights, stream);
  if (out_dtype == kBF16)
    return unpermute_backward<bf16_t, float>(dout, y, rows, T, topk, H, slot_rows, weights, sorted, capacity, ntpp,
                                             dy, dweights, stream);
  if (out_dtype == kFP16)
    return unpermute_backward<f16_t, float>(dout, y, rows, T, topk, H, slot_rows, weights, sorted, capacity, ntpp, dy,
                                            dweights, stream);
  return unpermute_backward<float, float>(dout, y, rows, T, topk, H, slot_rows, weights, sorted, capacity, ntpp, dy,
                                          dweights, stream);
}

}  // namespace w4a16
