// Building blocks of the operators' kernels (gfx950): matrix operand and
// accumulator types, waits, the workgroup barrier without a wait of its own, the
// conversion of two values at a time, a wave's sum.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace rs {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) char lds_char;

// Waits for all but VM of the wave's loads (and LDS reads, with LGKM). The
// builtin, unlike assembly text, tells the compiler what has arrived.
template <int VM, bool LGKM>
__device__ __forceinline__ void wait() {
  static_assert(VM < 64, "a six-bit counter");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (VM >> 4) << 14 | 0x70 | (LGKM ? 0 : 0xf00));
}

// Workgroup barrier without a wait of its own; no memory access moves across.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The thread's number, as a value that the compiler cannot see through: what
// is computed from it is computed anew for each tile instead of being kept in
// registers through the multiplication, which needs all of them.
__device__ __forceinline__ int fresh_thread() {
  int t = static_cast<int>(threadIdx.x);
  asm volatile("" : "+v"(t));
  return t;
}

// Two values rounded to nearest-even bf16 by one instruction.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, b2));
}

// Sums by additions of neighbours' values, which cost an instruction each
// instead of a trip through LDS: of a row of 16 lanes, in its last one, and of
// the wave, in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_lane(float x) {
  return x + __uint_as_float(static_cast<uint32_t>(
                 __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(x)), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ float row_sum_last(float x) {   // the lanes 1, 2, 4, 8 ahead
  return add_lane<0x118, 0xf>(add_lane<0x114, 0xf>(add_lane<0x112, 0xf>(add_lane<0x111, 0xf>(x))));
}
__device__ __forceinline__ float from_lane(float x, int lane) {
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(x)), lane)));
}
__device__ __forceinline__ float wave_sum(float x) {   // and the last lanes of the row and of the half ahead
  return from_lane(add_lane<0x143, 0xc>(add_lane<0x142, 0xa>(row_sum_last(x))), 63);
}

}  // namespace
}  // namespace rs
