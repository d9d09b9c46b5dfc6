// Tiles of 16-bit products on the matrix cores: C[m, n] = sum_r A[m, r] B[n, r],
// with either operand held in memory along r (a row panel) or along m or n (a
// column panel, whose rows are steps of r).
//
// A workgroup of eight waves computes a tile in stages of 64 steps of r, a
// line of 128 bytes of each row. A stage of both operands is copied from memory straight to LDS
// (global_load_lds_dwordx4) while the stage before it is multiplied. A copy
// writes 64 x 16 bytes side by side in lane order, so where a 16-byte chunk
// lies in LDS is chosen by which lane fetches it: the places are swizzled by
// row so that the fragments' reads hit the banks evenly. What lies outside an
// operand (the end of r, rows without a slot, columns past the last) is copied
// from sixteen zero bytes, in both operands, so that it adds exactly nothing
// whatever the other holds.
//
// The second operand (n) is the instruction's first, so a lane's four
// neighbouring results are four neighbouring columns of one row of C.
#pragma once

#include "rows.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {
namespace tile {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 64;  // steps of r a stage

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <typename T>
using vec8 = typename Eight<T>::vec;

__device__ __forceinline__ floatx16 mfma(vec8<bf16_t> a, vec8<bf16_t> b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mfma(vec8<f16_t> a, vec8<f16_t> b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// What copies from outside an operand read: as long as a row of a tile.
static __device__ __attribute__((aligned(16))) const uint32_t kZeros[128] = {};

// 16 bytes a lane to LDS at `lds` + 16 * lane. Issued from an asm block: the compiler would
// count a builtin's copy as an LDS access and make every later LDS read wait for it. It
// has no register result, the waits are explicit (wait_copies), and the memory clobber
// keeps reads on their side. M0 holds the LDS address, set a wait state before the copy.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

// Until at most N of this wave's copies are on their way.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// This wave's LDS reads have arrived, then all waves meet. Copies stay on their way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)(p);
}

// kOuter rows, each contiguous along r: 128 bytes a row and stage, the chunk c of row i in place
// c ^ (i / 2 % 8), so that sixteen rows' chunks c lie in sixteen places modulo 256.
template <int kOuter>
struct RowPanel {
  static constexpr int kBytes = kOuter * 2 * kStep;
  static constexpr int kUnits = kOuter / 8;  // copies of a stage, 8 rows each
  static constexpr int kMine = (kUnits + kWaves - 1) / kWaves;
  const uint8_t* at[kMine];
  int32_t first[kMine];  // this lane's first step of r in a stage

  // where there are fewer copies than waves, two waves make the same one
  static __device__ __forceinline__ int unit_of(int i, int wave) { return (kMine * wave + i) % kUnits; }
  static __device__ __forceinline__ int row_of(int i, int wave, int lane) { return 8 * unit_of(i, wave) + lane / 8; }
  static __device__ __forceinline__ int swizzle(int row) { return row >> 1 & 7; }

  // row: the start of row row_of(i, ...)
  __device__ __forceinline__ void set(int i, const void* row, int wave, int lane) {
    first[i] = 8 * ((lane & 7) ^ swizzle(row_of(i, wave, lane)));
    at[i] = static_cast<const uint8_t*>(row) + 2 * first[i];
  }
  // copy i of the next stage, of which `left` steps are in the operand
  __device__ __forceinline__ void copy(int i, uint32_t lds, int left, int wave) {
    copy16(left > first[i] ? (const void*)at[i] : (const void*)kZeros, lds + 1024 * unit_of(i, wave));
    at[i] += 2 * kStep;
  }
  // steps 16 k + 8 (lane / 32) + 0..7 of row outer0 + lane % 32; outer0 a multiple of 32
  template <typename T>
  static __device__ __forceinline__ vec8<T> fragment(const uint8_t* panel, int outer0, int k, int lane) {
    const int row = outer0 + (lane & 31);
    return *reinterpret_cast<const vec8<T>*>(panel + row * (2 * kStep) + (((2 * k + (lane >> 5)) ^ swizzle(row)) << 4));
  }
};

// kOuter columns, contiguous at each step of r: kOuter * 2 bytes a step, in parts of 64 bytes,
// the part c of step r in place c ^ (r % 4) (where a step has that many). Four steps' 64 bytes,
// which half a wave reads, then lie in four places modulo 256. kPitch: bytes between steps.
template <int kOuter, int kPitch = kOuter * 2>
struct ColumnPanel {
  static constexpr int kBytes = kOuter * 2 * kStep;
  static constexpr int kUnits = kBytes / 1024;
  static constexpr int kMine = (kUnits + kWaves - 1) / kWaves;
  static constexpr int kLanes = kOuter / 8;  // that copy a step
  static constexpr int kParts = kOuter / 32;
  const uint8_t* at[kMine];
  int32_t first[kMine];
  int64_t stride;  // bytes a stage

  static __device__ __forceinline__ int unit_of(int i, int wave) { return (kMine * wave + i) % kUnits; }
  static __device__ __forceinline__ int swizzle(int step) {
    return kParts >= 4 ? step & 3 : kParts == 2 ? step >> 1 & 1 : 0;
  }
  // base: step 0, column 0 of the panel; steps of ld columns, `columns` of them from `base` on. Columns past
  // those are copies of column 0.
  template <typename T>
  __device__ __forceinline__ void set(const T* base, int64_t ld, int32_t columns, int wave, int lane) {
    stride = ld * kStep * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      first[i] = (64 / kLanes) * unit_of(i, wave) + lane / kLanes;
      const int column = 8 * ((lane % kLanes) ^ (swizzle(first[i]) << 2));
      at[i] = reinterpret_cast<const uint8_t*>(base + first[i] * ld + (column < columns ? column : 0));
    }
  }
  __device__ __forceinline__ void copy(int i, uint32_t lds, int left, int wave) {
    copy16(left > first[i] ? (const void*)at[i] : (const void*)kZeros, lds + 1024 * unit_of(i, wave));
    at[i] += stride;
  }
  // As RowPanel's, by two transposing reads: sixteen lanes read four steps of sixteen columns,
  // lane i the columns 4 (i % 4) + 0..3 of step i / 4, and get column i's four steps.
  template <typename T>
  static __device__ __forceinline__ vec8<T> fragment(const uint8_t* panel, int outer0, int k, int lane) {
    const int i = lane & 15;
    const int part = (outer0 >> 5) ^ swizzle(i >> 2);
    const uint8_t* at = panel + (16 * k + 8 * (lane >> 5) + (i >> 2)) * kPitch + (part << 6) + 32 * (lane >> 4 & 1) + 8 * (i & 3);
    struct {
      shortx4 v[2];
    } r;
    r.v[0] = read_transposed(at);
    r.v[1] = read_transposed(at + 4 * kPitch);
    return __builtin_bit_cast(vec8<T>, r);
  }

 private:
  static __device__ __forceinline__ shortx4 read_transposed(const uint8_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4*)(p));
  }
};

// Bytes of LDS of the loop below: three stages of the panel M, two of N.
template <typename M, typename N>
constexpr int kRingBytes = 3 * M::kBytes + 2 * N::kBytes;

// All stages of a wave's 32 MT rows by 32 NT columns. copy_m(q, LDS address, stage) makes this wave's copy q of a
// stage's panel M (M::kMine of them), copy_n of N. On return the ring is free.
//
// A stage is multiplied in four parts of 16 steps, a part's fragments being read from LDS while the part before
// it is multiplied. Before the last part all waves meet: by then every wave has read all of stage s, and stage s + 1
// has landed. N's slot then takes stage s + 2, copied at once so as to land within a stage; M's slot
// takes stage s + 3, copied in the parts that follow and not waited for until a stage later. So the copies, which at
// 64 bytes a cycle keep the vector cache busy for more than half of the time, are spread over the
// stage, and none is waited for less than three parts after its issue. (Both panels in two slots, all
// copies of a stage in one part: MEASURED.) Copies past the last stage are of zeros. settle() is where the wave
// has no LDS read on its way: scalar loads for the next copies are waited for there.
template <typename T, typename M, typename N, int MT, int NT, typename CopyM, typename CopyN, typename Settle>
__device__ __forceinline__ void loop(uint8_t* ring, int stages, int m0, int n0, int lane, floatx16 (&acc)[MT][NT],
                                     CopyM copy_m, CopyN copy_n, Settle settle) {
  constexpr int kMfmas = MT * NT, kFragments = MT + NT;
  uint8_t* const ring_n = ring + 3 * M::kBytes;
  const uint32_t base_m = lds_address(ring), base_n = base_m + 3 * M::kBytes;
  vec8<T> m[2][MT], n[2][NT];
  auto fetch = [&](int f, const uint8_t* slot_m, const uint8_t* slot_n, int k) {
    if (f < NT)
      n[k & 1][f] = N::template fragment<T>(slot_n, n0 + 32 * f, k, lane);
    else
      m[k & 1][f - NT] = M::template fragment<T>(slot_m, m0 + 32 * (f - NT), k, lane);
  };
  // Part k. Behind its MFMAs, one by one, the next part's fragments and the copies first..last: the matrix
  // cores have work from the first instruction after the barrier on.
  auto part = [&](int k, const uint8_t* slot_m, const uint8_t* slot_n, int to_k, int first, int last, auto copy) {
    int f = 0, q = first;
#pragma unroll
    for (int i = 0; i < kMfmas; ++i) {
      acc[i / NT][i % NT] = mfma(n[k & 1][i % NT], m[k & 1][i / NT], acc[i / NT][i % NT]);
      __builtin_amdgcn_sched_barrier(0);
      for (; f * kMfmas < (i + 1) * kFragments && f < kFragments; ++f) fetch(f, slot_m, slot_n, to_k);
      for (; (q - first) * kMfmas < (i + 1) * (last - first) && q < last; ++q) copy(q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int q = 0; q < M::kMine; ++q) copy_m(q, base_m + s * M::kBytes, s);
#pragma unroll
    for (int q = 0; q < N::kMine; ++q) copy_n(q, base_n + s * N::kBytes, s);
  }
  wait_copies<M::kMine + N::kMine>();
  lds_barrier();
#pragma unroll
  for (int f = 0; f < kFragments; ++f) fetch(f, ring, ring_n, 0);
  int slot = 0;  // M's, in bytes
  for (int s = 0; s < stages; ++s) {
    const int next = slot == 2 * M::kBytes ? 0 : slot + M::kBytes, after = next == 2 * M::kBytes ? 0 : next + M::kBytes;
    const uint8_t *now_m = ring + slot, *now_n = ring_n + (s & 1) * N::kBytes;
    auto far = [&](int q) { copy_m(q, base_m + after, s + 2); };
    constexpr int kThird = (M::kMine + 2) / 3, kTwoThirds = 2 * M::kMine / 3 > kThird ? 2 * M::kMine / 3 : kThird;
    part(0, now_m, now_n, 1, 0, kThird, far);
    part(1, now_m, now_n, 2, kThird, kTwoThirds, far);
    part(2, now_m, now_n, 3, kTwoThirds, M::kMine, far);
    wait_copies<M::kMine>();
    lds_barrier();
    settle();
    part(3, ring + next, ring_n + ((s + 1) & 1) * N::kBytes, 0, 0, N::kMine,
         [&](int q) { copy_n(q, base_n + (s & 1) * N::kBytes, s + 2); });
    slot = next;
  }
  wait_copies<0>();
  lds_barrier();
}

// Sums leave through LDS, 32 rows of a wave's columns at a time, so that a store covers whole
// lines; put(row, column, eight sums) stores those of the tile's row `row`, column `column` on.
template <int MT, int NT, typename Put>
__device__ __forceinline__ void drain(uint8_t* ring, int m0, int n0, int wave, int lane, const floatx16 (&acc)[MT][NT],
                                      Put put) {
  constexpr int kPitch = 32 * NT * 4 + 16;  // 16 bytes between rows: rows begin on other banks
  uint8_t* mine = ring + wave * 32 * kPitch;
  constexpr int kLanes = 4 * NT;  // a row
  constexpr int kRows = 64 / kLanes;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<floatx4*>(mine + (lane & 31) * kPitch + (32 * j + 8 * g + 4 * (lane >> 5)) * 4) =
            floatx4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
#pragma unroll
    for (int r = 0; r < 32 / kRows; ++r) {
      const int row = r * kRows + lane / kLanes, column = 8 * (lane % kLanes);
      const floatx4* at = reinterpret_cast<const floatx4*>(mine + row * kPitch + column * 4);
      const floatx4 lo = at[0], hi = at[1];
      const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      put(m0 + 32 * i + row, n0 + column, v);
    }
  }
}

template <typename O>
__device__ __forceinline__ void store(O* p, const float (&v)[8]) {
  Eight<O> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = (O)v[i];
  store8<kStreamed>(p, r);
}

}  // namespace tile
}  // namespace w4a16
