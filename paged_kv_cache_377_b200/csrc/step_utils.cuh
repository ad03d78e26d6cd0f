// step_utils.cuh -- what the kernels over a step's ragged batch share: launches
// that overlap, and each sequence's rows.
#pragma once

#include <stdint.h>

namespace pkv {

// A kernel launched by launch_overlapped may start while the one before it in the stream ends: nothing in global
// memory is touched before depend_wait(), which returns once that kernel is done and its writes are visible.
// depend_release() lets the next such kernel start.
__device__ __forceinline__ void depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void depend_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The rows q0 .. q0 + n - 1 that sequence s brings to a step of num_tokens rows. False, and n = 0, where its starts fall or
// leave the step; they are compared before they are subtracted, since the difference of any two words may not fit one.
__device__ __forceinline__ bool query_rows(const int32_t *query_start, int s, int num_tokens, int &q0, int &n) {
    q0 = query_start[s];
    const int q1 = query_start[s + 1];
    const bool good = q0 >= 0 && q0 <= q1 && q1 <= num_tokens;
    n = good ? q1 - q0 : 0;
    return good;
}

}  // namespace pkv
