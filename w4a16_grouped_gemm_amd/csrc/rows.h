// Row elements in device code: 8 at a time to and from fp32, for bf16, fp16
// and fp32 buffers that are aligned to their element type only (gfx950 moves 16
// bytes from any such address in one instruction).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

template <typename T>
struct Eight {
  T v[8];
};

template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const Eight<T>& r) {
  __builtin_memcpy(p, &r, sizeof(r));
}

}  // namespace w4a16
