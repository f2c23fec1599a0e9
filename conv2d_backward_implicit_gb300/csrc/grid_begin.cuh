// grid_begin.cuh -- the start of a kernel launched with programmatic stream
// serialisation: everything before it touches only the block's own shared and tensor
// memory.
#pragma once

// Waits for the grids before this one in the stream, then lets the next one begin its
// own preamble.  In this order no grid runs beside the one two before it, so that what
// this one reads is not being written by anything; it is read with ordinary loads all the
// same, not the read-only path, which asks for memory that nothing writes from the launch
// on -- and the launch comes before the wait.
__device__ __forceinline__ void grid_begin() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
