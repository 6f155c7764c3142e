// norm.h -- host-side launchers of the norms around a block (norm.hip): pointers
// and sizes are checked by norm_api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdr {

// Operands of gdr_block_norm and its gradient (gdr.h); unused ones are NULL.
struct BlockNorm {
  const void *x, *w_after, *gate, *residual, *w_before;
  void *h, *y;
  const void *dh, *dy;
  void *dx, *dgate, *dresidual;
  float *part_after, *part_before;  // [block_norm_backward_blocks][D]
  int64_t rows;
  int D, act, in_dtype, w_dtype, out_dtype;
  float scale, eps;
};

// Workgroups of the gradient kernel, and so rows of its partial sums.
int block_norm_backward_blocks(int64_t rows, int D);

hipError_t launch_block_norm(const BlockNorm& p, hipStream_t stream);
hipError_t launch_block_norm_backward(const BlockNorm& p, float* dw_after, float* dw_before,
                                      hipStream_t stream);

}  // namespace gdr
