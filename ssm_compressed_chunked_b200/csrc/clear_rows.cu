// Zeros in the token rows that no sequence owns.
//
// The operators of the SSM block leave such rows of their outputs as they are.  What a later product makes of them
// is added to a residual stream, so a composed block sets the last of them to zero first: the product of a
// zero row is zero, and the stream's row stays what it was.
//
// A block takes every gridDim.x-th row; the rows to clear are few (a batch's padding), so the time is a launch's:
// 1.1 to 1.3 us in a stream of kernels (1 to 256 rows of 2048 bf16 channels), 0.8 to 1.8 us of a composed block's
// 52 (one row) to 650 us (16384 rows).  A memset of the whole buffer would write 67 MB for the 16384 rows.
#include "common.cuh"
#include "launch.h"

namespace attamba {

namespace {
constexpr int kThreads = 128;

// rows of `vecs` 16-byte pieces, `ld` pieces apart: those from *end on, or those with a negative slot
__global__ void __launch_bounds__(kThreads) clear_rows_kernel(uint4* y, int64_t ld, int vecs, int64_t rows, const int32_t* end,
                                                              const int32_t* slots) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t first = end ? min((int64_t)max(0, *end), rows) : 0;
  for (int64_t row = first + blockIdx.x; row < rows; row += gridDim.x) {
    if (slots && __ldg(slots + row) >= 0) continue;
    for (int v = threadIdx.x; v < vecs; v += kThreads) y[row * ld + v] = make_uint4(0, 0, 0, 0);
  }
}
}  // namespace

cudaError_t launch_clear_rows(void* y, int64_t ld_bytes, int32_t row_bytes, int64_t rows, const int32_t* end,
                              const int32_t* slots, cudaStream_t s) {
  const int blocks = (int)(rows < 592 ? rows : 592);   // four on each of 148 SMs
  return launch_dependent(clear_rows_kernel, dim3(blocks), kThreads, s, static_cast<uint4*>(y), ld_bytes / 16, row_bytes / 16,
                          rows, end, slots);
}

}  // namespace attamba
