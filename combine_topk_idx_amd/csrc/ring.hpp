#pragma once

// Loads issued before this point stay before it: without it the optimizer
// moves the loads of a software ring from the end of one iteration to the
// start of the next, right before their use.
__device__ __forceinline__ void keep_loads() { asm volatile("" ::: "memory"); }
