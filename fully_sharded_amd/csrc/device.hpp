// Device code shared by the files of kernels with matrix products: vector
// types, bf16 conversions, loads that go straight to LDS, and their waits.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace fsdp {

using u16 = uint16_t;
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint32_t f32_to_bf16(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// 16 bytes per lane from global memory to LDS at a wave-uniform address, lane
// after lane.  An asm statement (its only register is M0): of the builtin the
// compiler waits for all loads under way before every transposing LDS read,
// which it cannot tell from a read of the bytes being loaded.  M0 as an
// operand that the compiler sets, apart from the load, took 0.4-0.6% longer.
// Waited for by wait_and_meet.
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               : "=&{m0}"(m0)
               : "v"(from), "s"(__builtin_amdgcn_readfirstlane(to))
               : "memory");
}

// Wait until all of this wave's LDS reads are done (the builtin, not an asm
// statement: the compiler counts on from it).
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
}
// Wait until at most N of this wave's global accesses are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// Wait for all of this wave's LDS accesses, then for the other waves; global
// loads into registers stay under way.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// Wait for all but N global accesses and all LDS reads, then for the others.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N < 64);
  // products stay on their side: those before it hide the loads waited for
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace fsdp
