// Tiles of 16-bit products on the matrix cores: C[m, n] = sum_r A[m, r] B[n, r],
// with either operand held in memory along r (a row panel) or along m or n (a
// column panel, whose rows are steps of r).
//
// A workgroup of eight waves computes a tile in stages of 64 steps of r, a
// line of 128 bytes of each row. A stage of both operands is copied from memory straight to LDS
// (global_load_lds_dwordx4) while the stage before it is multiplied. A copy
// writes 64 x 16 bytes side by side in lane order, so where a 16-byte chunk
// lies in LDS is chosen by which lane fetches it: the places are swizzled by
// row so that the fragments' reads hit the banks evenly. Steps of r that add
// nothing (past the operand's end; in the weights' gradient, rows without a slot)
// are copied from sixteen zero bytes, in both operands, so that they add exactly
// nothing whatever either holds. A row or column of C that is not there (past the
// last; in the product, a row without a slot) is computed from another one's values
// and left out or zeroed where C is stored.
//
// The second operand (n) is the instruction's first, so a lane's four
// neighbouring results are four neighbouring columns of one row of C.
#pragma once

#include "rows.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace w4a16 {
namespace tile {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 64;  // steps of r a stage
constexpr int kXcds = 8;   // workgroups go round-robin to them, each has an L2 of its own

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

// What copies of steps that add nothing read.
static __device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {};

// 16 bytes a lane to LDS at `lds` + 16 * lane. Issued from an asm block: the compiler would
// count a builtin's copy as an LDS access and make every later LDS read wait for it. It
// has no register result, the waits are explicit (wait_copies), and the memory clobber
// keeps reads on their side. M0 holds the LDS address, set a wait state before the copy.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
}
// The same from base + offset (bytes): no vector instruction but the copy. A vector instruction that writes a scalar
// register (a readlane of one that was set aside in a vector register, for instance) must lie five wait states before a
// memory instruction that reads it, and the compiler does not look into the asm. So a scalar instruction of the block
// writes the base anew, as it is: scalar instructions wait by themselves for what they read, and memory instructions for
// what those write. It is M0's wait state too.
__device__ __forceinline__ void copy16(const uint8_t*& base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_mov_b64 %0, %0\n\tglobal_load_lds_dwordx4 %1, %0"
               : "+s"(base)
               : "v"(offset), "s"(lds)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// An address that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const void* p) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  const uint32_t low = __builtin_amdgcn_readfirstlane((uint32_t)at);
  const uint32_t high = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)high << 32 | low);
}

// Until at most N of this wave's copies are on their way.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// This wave's LDS reads have arrived, then all waves meet. Copies stay on their way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Between LDS accesses of one wave by which its lanes exchange values. The hardware keeps their order; this keeps the
// compiler to it, which may otherwise move a lane's access past those of the other lanes that its own address rules out.
__device__ __forceinline__ void lanes_meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)(p);
}

// kOuter rows, each contiguous along r: 2 kSteps bytes a row and stage, a line or two. Sixteen rows' chunks of
// 16 bytes c lie in sixteen places modulo 256: chunk c of row i in place c ^ (i / 2 % 8), with two lines
// c ^ (i % 16).
template <int kOuter, int kSteps = kStep>
struct RowPanel {
  static constexpr int kPitch = 2 * kSteps;
  static constexpr int kBytes = kOuter * kPitch;
  static constexpr int kUnits = kBytes / 1024;  // copies of a stage
  static constexpr int kMine = (kUnits + kWaves - 1) / kWaves;
  static constexpr int kLanes = kPitch / 16;  // that copy a row
  const uint8_t* base;     // of the stage to be copied next
  uint32_t offset[kMine];  // this lane's 16 bytes from there, or `far` the row
  int64_t far;             // bytes a row where 32 bits do not hold the offsets, else 0

  // where there are fewer copies than waves, two waves make the same one
  static __device__ __forceinline__ int unit_of(int i, int wave) { return (kMine * wave + i) % kUnits; }
  static __device__ __forceinline__ int row_of(int i, int wave, int lane) {
    return 64 / kLanes * unit_of(i, wave) + lane / kLanes;
  }
  static __device__ __forceinline__ int swizzle(int row) { return kSteps == 64 ? row >> 1 & 7 : row & 15; }
  // this lane's first step of r in copy i
  static __device__ __forceinline__ int first_of(int i, int wave, int lane) {
    return 8 * (lane % kLanes ^ swizzle(row_of(i, wave, lane)));
  }

  // row `row` of those from base on, of `pitch` bytes, is row_of(i, ...)
  __device__ __forceinline__ void set(int i, uint32_t row, int64_t pitch, int wave, int lane) {
    offset[i] = far ? row : row * (uint32_t)pitch + 2 * first_of(i, wave, lane);
  }
  // to `on` stages on
  __device__ __forceinline__ void go(int on) { base += (int64_t)on * kPitch; }
  // copy i of a stage that lies in the operand as a whole, where nothing is far
  __device__ __forceinline__ void copy(int i, uint32_t lds, int wave) {
    copy16(base, offset[i], lds + 1024 * unit_of(i, wave));
  }
  // copy i of any stage, of which `left` steps are in the operand
  __device__ __forceinline__ void copy(int i, uint32_t lds, int left, int wave, int lane) const {
    const int first = first_of(i, wave, lane);
    const uint8_t* at = base + (far ? (uint64_t)offset[i] * (uint64_t)far + 2 * first : offset[i]);
    copy16(left > first ? (const void*)at : (const void*)kZeros, lds + 1024 * unit_of(i, wave));
  }
  // steps 16 k + 8 (lane / 32) + 0..7 of row outer0 + lane % 32; outer0 a multiple of 32, place that of it
  static __device__ __forceinline__ int place(int outer0, int) { return outer0; }
  template <typename T>
  static __device__ __forceinline__ vec8<T> fragment(const uint8_t* panel, int place, int k, int lane) {
    const int row = place + (lane & 31);
    return *reinterpret_cast<const vec8<T>*>(panel + row * kPitch + (((2 * k + (lane >> 5)) ^ swizzle(row)) << 4));
  }
};

// kOuter columns, contiguous at each step of r: kOuter * 2 bytes a step, in parts of 64 bytes,
// the part c of step r in place c ^ (r % 4) (where a step has that many). Four steps' 64 bytes,
// which half a wave reads, then lie in four places modulo 256.
template <int kOuter, int kSteps = kStep>
struct ColumnPanel {
  static constexpr int kPitch = kOuter * 2;
  static constexpr int kBytes = kPitch * kSteps;
  static constexpr int kUnits = kBytes / 1024;
  static constexpr int kMine = (kUnits + kWaves - 1) / kWaves;
  static constexpr int kLanes = kOuter / 8;  // that copy a step
  static constexpr int kParts = kOuter / 32;
  const uint8_t* base;     // of the stage to be copied next
  uint32_t offset[kMine];  // this lane's 16 bytes from there
  int64_t stride;          // bytes a stage

  static __device__ __forceinline__ int unit_of(int i, int wave) { return (kMine * wave + i) % kUnits; }
  static __device__ __forceinline__ int swizzle(int step) {
    return kParts >= 4 ? step & 3 : kParts == 2 ? step >> 1 & 1 : 0;
  }
  // this lane's step of r in copy i
  static __device__ __forceinline__ int first_of(int i, int wave, int lane) {
    return (64 / kLanes) * unit_of(i, wave) + lane / kLanes;
  }
  // from: step 0, column 0 of the panel; steps of ld columns, `columns` of them from there on. Columns past
  // those are copies of column 0.
  template <typename T>
  __device__ __forceinline__ void set(const T* from, int32_t ld, int32_t columns, int wave, int lane) {
    base = uniform(from);
    stride = (int64_t)ld * kSteps * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int first = first_of(i, wave, lane), column = 8 * ((lane % kLanes) ^ (swizzle(first) << 2));
      offset[i] = (uint32_t)sizeof(T) * ((uint32_t)first * (uint32_t)ld + (uint32_t)(column < columns ? column : 0));
    }
  }
  __device__ __forceinline__ void go(int on) { base += on * stride; }
  __device__ __forceinline__ void copy(int i, uint32_t lds, int wave) {
    copy16(base, offset[i], lds + 1024 * unit_of(i, wave));
  }
  __device__ __forceinline__ void copy(int i, uint32_t lds, int left, int wave, int lane) const {
    const bool inside = left > first_of(i, wave, lane);
    copy16(inside ? (const void*)(base + offset[i]) : (const void*)kZeros, lds + 1024 * unit_of(i, wave));
  }
  // As RowPanel's, by two transposing reads: sixteen lanes read four steps of sixteen columns,
  // lane i the columns 4 (i % 4) + 0..3 of step i / 4, and get column i's four steps.
  static __device__ __forceinline__ int place(int outer0, int lane) {
    const int i = lane & 15;
    const int part = (outer0 >> 5) ^ swizzle(i >> 2);
    int at = (8 * (lane >> 5) + (i >> 2)) * kPitch + (part << 6) + 32 * (lane >> 4 & 1) + 8 * (i & 3);
    asm volatile("" : "+v"(at));  // as it is, not in its terms at every read
    return at;
  }
  template <typename T>
  static __device__ __forceinline__ vec8<T> fragment(const uint8_t* panel, int place, int k, int) {
    const uint8_t* at = panel + place + 16 * k * kPitch;
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

// Bytes of LDS of the loop below.
template <typename M, typename N, int kAhead>
constexpr int kRingBytes = (kAhead + 1) * M::kBytes + kAhead * N::kBytes;

// The first kAhead stages' copies, next(stage) before those of each but the first and behind them. The slot of M
// after them stays as it is.
template <typename M, typename N, int kAhead, int kBytesM, typename CopyM, typename CopyN, typename Next>
__device__ __forceinline__ void prologue(const uint8_t* ring, CopyM copy_m, CopyN copy_n, Next next) {
  const uint32_t base_m = lds_address(ring), base_n = base_m + (kAhead + 1) * kBytesM;
#pragma unroll
  for (int s = 0; s < kAhead; ++s) {
#pragma unroll
    for (int q = 0; q < M::kMine; ++q) copy_m(q, base_m + s * kBytesM, s, std::false_type());
#pragma unroll
    for (int q = 0; q < N::kMine; ++q) copy_n(q, base_n + s * N::kBytes, s, std::false_type());
    next(s + 1);
  }
}

// All stages of a wave's 32 MT rows by 32 NT columns. copy_m(q, LDS address, stage, kind) makes this wave's copy q of a
// stage's panel M (M::kMine of them), copy_n of N. ring: kAhead + 1 stages of at most
// kBytesM of M, kAhead of N; prologue has been called for them. All waves are past it on return.
// kind is true in the first `whole` stages, as long as real() says so before each: copies that need no look at what
// lies outside the operand, and no vector instruction beside them. (With two compares and a 64-bit address for
// every copy: 1720 instead of 1670 us for the case below, transposed 1770 instead of 1650.)
//
// A stage is multiplied in four parts of 16 steps, a part's fragments being read from LDS while the part before
// it is multiplied. Before the last part all waves meet: by then every wave has read all of stage s, and stage s + 1
// has landed. N's slot then takes stage s + kAhead, copied at once so as to land in time; M's slot takes stage
// s + kAhead + 1, copied in the parts that follow. So the copies, which at 64 bytes a cycle keep the vector cache busy
// for more than half of a 256 x 256 tile's time, are spread over the stage, and none is waited for less than three
// parts after its issue. (32768 rows, 16 experts, 4096 x 7168, kAhead 2, on one card: 1618 us; both panels in two slots
// with the copies in one part 1805, in two parts 1732, in all four 1904.) Copies past the last stage are of zeros.
// ahead(stage) comes before the first part and turn() after the last, for scalar loads that the copies of the
// next stage need: while one is on its way every wait for LDS is for all reads and for it, and here that is one
// wait, a part after its issue (issued where the copies need them, twice a stage, the weights' gradient of
// 32768 rows, 16 experts, 4096 x 7168 took 1894 instead of 1800 us).
template <typename T, typename M, typename N, int kAhead, int kBytesM, int MT, int NT, typename CopyM, typename CopyN,
          typename Real, typename Ahead, typename Turn>
__device__ __forceinline__ void loop(uint8_t* ring, int whole, int stages, int m0, int n0, int lane,
                                     floatx16 (&acc)[MT][NT], CopyM copy_m, CopyN copy_n, Real real, Ahead ahead, Turn turn) {
  static_assert(kAhead >= 2, "a stage is read while the next one lands");
  constexpr int kMfmas = MT * NT, kFragments = MT + NT;
  uint8_t* const ring_n = ring + (kAhead + 1) * kBytesM;
  const uint32_t base_m = lds_address(ring), base_n = base_m + (kAhead + 1) * kBytesM;
  vec8<T> m[2][MT], n[2][NT];
  int place_m[MT], place_n[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) place_m[i] = M::place(m0 + 32 * i, lane);
#pragma unroll
  for (int j = 0; j < NT; ++j) place_n[j] = N::place(n0 + 32 * j, lane);
  auto fetch = [&](int f, const uint8_t* slot_m, const uint8_t* slot_n, int k) {
    if (f < NT)
      n[k & 1][f] = N::template fragment<T>(slot_n, place_n[f], k, lane);
    else
      m[k & 1][f - NT] = M::template fragment<T>(slot_m, place_m[f - NT], k, lane);
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
  wait_copies<0>();  // and for the stores of a tile before, whose order among the copies is not known
  lds_barrier();
#pragma unroll
  for (int f = 0; f < kFragments; ++f) fetch(f, ring, ring_n, 0);
  int s = 0, at_m = 0, at_n = 0;  // the slots of stage s, in bytes
  auto multiply = [&](auto kind) {
    const int next_m = at_m == kAhead * kBytesM ? 0 : at_m + kBytesM;
    const int next_n = at_n == (kAhead - 1) * N::kBytes ? 0 : at_n + N::kBytes;
    const uint8_t *slot_m = ring + at_m, *slot_n = ring_n + at_n;
    const uint32_t free_m = base_m + (at_m == 0 ? kAhead * kBytesM : at_m - kBytesM);  // of stage s - 1
    auto far = [&](int q) { copy_m(q, free_m, s + kAhead, kind); };
    constexpr int kThird = (M::kMine + 2) / 3, kTwoThirds = 2 * M::kMine / 3 > kThird ? 2 * M::kMine / 3 : kThird;
    ahead(s + kAhead + 1);
    part(0, slot_m, slot_n, 1, 0, kThird, far);
    part(1, slot_m, slot_n, 2, kThird, kTwoThirds, far);
    part(2, slot_m, slot_n, 3, kTwoThirds, M::kMine, far);
    // a wave's copies land in order: younger than stage s + 1's are M's of kAhead - 1 stages and N's of kAhead - 2
    wait_copies<(kAhead - 1) * M::kMine + (kAhead - 2) * N::kMine>();
    lds_barrier();
    part(3, ring + next_m, ring_n + next_n, 0, 0, N::kMine, [&](int q) { copy_n(q, base_n + at_n, s + kAhead, kind); });
    turn();
    at_m = next_m;
    at_n = next_n;
  };
  // two loops: with the choice inside of one the compiler moves all the sums about
  for (; s < whole && real(); ++s) multiply(std::true_type());
  for (; s < stages; ++s) multiply(std::false_type());
  wait_copies<0>();
  lds_barrier();
}

// All stages of a tile of 32 MT rows by 32 NT columns that the eight waves share along r: of each stage of 128
// steps wave w multiplies 16, so that a stage costs one barrier and one wait for LDS, where a wave's share of a
// small tile would wait for LDS in every part. kAhead stages in LDS (copy makes both panels' copies of one, of the
// whole kind as above in the first `whole` stages where kSome). acc: each wave's share of the sums.
template <typename T, typename M, typename N, int kAhead, bool kSome, int MT, int NT, typename Copy>
__device__ __forceinline__ void shared_loop(uint8_t* ring, int whole, int stages, int wave, int lane,
                                            floatx16 (&acc)[MT][NT], Copy copy) {
  constexpr int kBytes = M::kBytes + N::kBytes, kCopies = M::kMine + N::kMine;
  const uint32_t base = lds_address(ring);
#pragma unroll
  for (int s = 0; s < kAhead - 1; ++s) copy(base + s * kBytes, s, std::false_type());
  int place_m[MT], place_n[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) place_m[i] = M::place(32 * i, lane);
#pragma unroll
  for (int j = 0; j < NT; ++j) place_n[j] = N::place(32 * j, lane);
  int s = 0, slot = 0, free = (kAhead - 1) * kBytes;
  auto stretch = [&](int to, auto kind) {
    for (; s < to; ++s) {
      wait_copies<(kAhead - 2) * kCopies>();
      lds_barrier();  // stage s has landed, stage s - 1 has been read
      vec8<T> m[MT], n[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) n[j] = N::template fragment<T>(ring + slot + M::kBytes, place_n[j], wave, lane);
#pragma unroll
      for (int i = 0; i < MT; ++i) m[i] = M::template fragment<T>(ring + slot, place_m[i], wave, lane);
      copy(base + free, s + kAhead - 1, kind);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma(n[j], m[i], acc[i][j]);
      free = slot;
      slot = slot == (kAhead - 1) * kBytes ? 0 : slot + kBytes;
    }
  };
  if constexpr (kSome) stretch(whole, std::true_type());
  stretch(stages, std::false_type());
  wait_copies<0>();
  lds_barrier();
}

// The waves' shares, added in wave order; put(row, column, sums) gets four columns. ring: kSumsBytes of LDS.
template <int MT, int NT>
constexpr int kSumsBytes = kWaves * 32 * MT * 32 * NT * (int)sizeof(float);
template <int MT, int NT, typename Put>
__device__ __forceinline__ void shared_drain(uint8_t* ring, int wave, int lane, const floatx16 (&acc)[MT][NT], Put put) {
  constexpr int kRows = 32 * MT, kQuads = 8 * NT;
  floatx4* sums = reinterpret_cast<floatx4*>(ring);  // [wave][row][quad], a quad's place swizzled by row
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int row = 32 * i + (lane & 31), quad = 8 * j + 2 * g + (lane >> 5);
        sums[(wave * kRows + row) * kQuads + (quad ^ (row & 7))] =
            floatx4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
      }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < kRows * kQuads; i += kThreads) {
    const int row = i / kQuads, quad = i % kQuads;
    floatx4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += sums[(k * kRows + row) * kQuads + (quad ^ (row & 7))];
    put(row, 4 * quad, v);
  }
}

// A wave's sums leave through kDrainBytes / kWaves of LDS of its own, so that a store covers whole lines (16 bytes a lane,
// eight lanes a line; 32 bytes side by side straight from the registers took 1650 instead of 1577 us, streamed 1707):
// put(row, column, line) gets 16 bytes of O, columns of one row. A lane holds four columns of a row and lane + 32 the
// next four; 16-bit values of two such groups are exchanged between the two lanes, so that LDS is written by 16 bytes
// too. The 16-byte chunk c of row i lies in place c ^ (i % 8).
constexpr int kDrainBytes = kWaves * 32 * 128;
template <typename O, int MT, int NT, typename Put>
__device__ __forceinline__ void drain(uint8_t* scratch, int m0, int n0, int wave, int lane,
                                      const floatx16 (&acc)[MT][NT], Put put) {
  typedef O four __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  constexpr int kEach = 16 / (int)sizeof(O);
  constexpr int kLine = 8 * kEach;                       // columns of a line
  constexpr int kSide = kLine / 32 < NT ? kLine / 32 : NT;  // fragments side by side in a line (or as many as there are)
  constexpr int kLanes = 32 * kSide / kEach;             // that store a row
  uint8_t* const mine = scratch + wave * 32 * 128;
  const int row = lane & 31, half = lane >> 5;
  auto write = [&](int chunk, u32x4 v) {
    *reinterpret_cast<u32x4*>(mine + row * 128 + ((chunk ^ (row & 7)) << 4)) = v;
  };
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j0 = 0; j0 < NT; j0 += kSide) {
#pragma unroll
      for (int side = 0; side < kSide; ++side) {
        const floatx16& sums = acc[i][j0 + side];
        if constexpr (sizeof(O) == 4) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            write(2 * g + half, __builtin_bit_cast(u32x4, floatx4{sums[4 * g], sums[4 * g + 1], sums[4 * g + 2],
                                                                  sums[4 * g + 3]}));
        } else {
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            four x, y;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = (O)sums[4 * g + k];
              y[k] = (O)sums[4 * g + 4 + k];
            }
            const u32x2 a = __builtin_bit_cast(u32x2, x), b = __builtin_bit_cast(u32x2, y);
            // lanes 32-63 of the first change places with lanes 0-31 of the second
            const auto p = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
            const auto q = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
            write(4 * side + g + half, u32x4{p[0], q[0], p[1], q[1]});
          }
        }
      }
      lanes_meet();
#pragma unroll
      for (int r = 0; r < 32; r += 64 / kLanes) {
        const int at = r + lane / kLanes, chunk = lane % kLanes;
        put(m0 + 32 * i + at, n0 + 32 * j0 + kEach * chunk,
            *reinterpret_cast<const u32x4*>(mine + at * 128 + ((chunk ^ (at & 7)) << 4)));
      }
      lanes_meet();  // before the next fragments overwrite what other lanes read
    }
}

// 16 bytes of O, to and from an aligned place.
template <typename O>
struct Line {
  static constexpr int kEach = 16 / (int)sizeof(O);
  static __device__ __forceinline__ void store(O* p, u32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  }
};

// Four values to and from an aligned place.
template <typename O>
struct Four {
  typedef O vec __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ void store(O* p, floatx4 v) {
    vec r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (O)v[i];
    *reinterpret_cast<vec*>(p) = r;
  }
  static __device__ __forceinline__ floatx4 load(const O* p) {
    const vec r = *reinterpret_cast<const vec*>(p);
    return floatx4{(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
  }
};

}  // namespace tile
}  // namespace w4a16
