// product.h -- host-side launcher of the product in 8 bits (product.hip): pointers and
// sizes are checked by product_api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdr {

// Operands of gdr_product8 (gdr.h).
struct Product8 {
  const uint8_t *a, *w;
  const float *a_scale, *w_scale;
  void* out;
  int M, N, K, out_dtype;
};

hipError_t launch_product8(const Product8& p, hipStream_t stream);

}  // namespace gdr
