// Row elements in device code: 8 at a time, for bf16, fp16 and fp32 buffers that
// are aligned to their element type only (gfx950 moves 16 bytes from any such
// address in one instruction).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

// Unaligned vectors of the bits of eight 2-byte or 4-byte elements: their parts of 16 bytes.
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));

template <typename T>
struct Eight {
  typedef T vec __attribute__((ext_vector_type(8)));
  vec v;
};

enum Policy { kCached, kStreamed };  // streamed: will not be read again from this cache

template <Policy P = kCached, typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  constexpr int kParts = sizeof(T) / 2;
  struct {
    uint32_t part[kParts][4];
  } bits;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const u32x4_u* at = reinterpret_cast<const u32x4_u*>(p) + i;
    const u32x4_u x = P == kStreamed ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
    for (int k = 0; k < 4; ++k) bits.part[i][k] = x[k];
  }
  return Eight<T>{__builtin_bit_cast(typename Eight<T>::vec, bits)};
}

template <Policy P = kCached, typename T>
__device__ __forceinline__ void store8(T* p, const Eight<T>& r) {
  constexpr int kParts = sizeof(T) / 2;
  struct Bits {
    uint32_t part[kParts][4];
  };
  const Bits bits = __builtin_bit_cast(Bits, r.v);
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    u32x4_u* at = reinterpret_cast<u32x4_u*>(p) + i;
    const u32x4_u x = {bits.part[i][0], bits.part[i][1], bits.part[i][2], bits.part[i][3]};
    if (P == kStreamed)
      __builtin_nontemporal_store(x, at);
    else
      *at = x;
  }
}

}  // namespace w4a16
