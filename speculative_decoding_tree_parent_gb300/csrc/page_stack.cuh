// The free stack's check, shared by the two page-table kernels.
#pragma once

namespace specv {

// Whether a stack of n0 free pages that `back` pages (>= 0) return to stays within [0, num_pages]. Any
// n0 may come from the caller's buffer, so no sum is formed before it is known to fit.
__host__ __device__ __forceinline__ bool page_stack_holds(int n0, int back, int num_pages) {
  return n0 >= 0 && n0 <= num_pages && back <= num_pages - n0;
}

}  // namespace specv
