// Building blocks of the matrix-core kernels (gfx950): operand and accumulator
// types, waits, the workgroup barrier without a wait of its own.
#pragma once

#include <hip/hip_runtime.h>

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

}  // namespace
}  // namespace rs
