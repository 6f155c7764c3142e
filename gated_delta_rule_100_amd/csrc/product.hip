// product.hip -- the product in 8 bits with a scale for each block of 128 (gdr_product8
// in gdr.h) on gfx950, one thread an output.
#include "gdr_device.h"
#include "product.h"

namespace gdr {
namespace {

template <Dt OUT>
__global__ void product8_kernel(Product8 p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(p.M) * p.N) return;
  const int64_t m = i / p.N, n = i % p.N, kb = (p.K + 127) / 128;
  const uint32_t* a = reinterpret_cast<const uint32_t*>(p.a + m * p.K);
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p.w + n * p.K);
  float sum = 0.f;
  for (int64_t b = 0; b < kb; ++b) {
    float part = 0.f;
    for (int k = static_cast<int>(b) * 32; k < min(p.K / 4, static_cast<int>(b) * 32 + 32); ++k) {
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a[k], 0), __builtin_amdgcn_cvt_f32_fp8(w[k], 0), part);
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a[k], 1), __builtin_amdgcn_cvt_f32_fp8(w[k], 1), part);
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a[k], 2), __builtin_amdgcn_cvt_f32_fp8(w[k], 2), part);
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a[k], 3), __builtin_amdgcn_cvt_f32_fp8(w[k], 3), part);
    }
    sum = fmaf(p.a_scale[m * kb + b] * p.w_scale[n / 128 * kb + b], part, sum);
  }
  store_scalar<OUT>(p.out, i, sum);
}

}  // namespace

hipError_t launch_product8(const Product8& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.M) * p.N + 255) / 256));
  if (p.out_dtype == 0) hipLaunchKernelGGL(product8_kernel<Dt::BF16>, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(product8_kernel<Dt::F32>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace gdr
