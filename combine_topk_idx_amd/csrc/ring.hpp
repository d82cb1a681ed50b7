#pragma once

// Loads issued before this point stay before it: without it the optimizer
// moves the loads of a software ring from the end of one iteration to the
// start of the next, right before their use.
__device__ __forceinline__ void keep_loads() { asm volatile("" ::: "memory"); }

// LDS written by some lanes of a wave is read by others: its accesses
// complete in order, the compiler must not move them across.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
