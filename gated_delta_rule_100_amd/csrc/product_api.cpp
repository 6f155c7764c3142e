// product_api.cpp -- the C ABI of the product in 8 bits: host-side validation and
// dispatch (conventions as in api.cpp).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gdr.h"
#include "api_internal.h"
#include "product.h"

namespace {

using gdr::fail;

// (a tile's rows are addressed by 32 bits)
constexpr int kMaxSize = 1 << 24, kMaxDepth = 1 << 22;
constexpr int64_t kResults = int64_t{1} << 36;  // fewer than these

int max_rows(int N) {
  if (N <= 0 || N > kMaxSize) return 0;
  const int64_t most = (kResults - 1) / N;
  return most < kMaxSize ? static_cast<int>(most) : kMaxSize;
}

}  // namespace

extern "C" {

int gdr_product8_max_rows(int N) { return max_rows(N); }

gdr_status gdr_product8(const void* a, const float* a_scale, const void* w, const float* w_scale,
                        void* out, int M, int N, int K, gdr_dtype out_dtype, gdr_stream_t stream) {
  const char* who = "gdr_product8";
  if (M < 0 || N <= 0 || K <= 0 || N > kMaxSize || K > kMaxDepth || M > max_rows(N))
    return fail(GDR_ERR_INVALID_ARG, "%s: M=%d N=%d K=%d", who, M, N, K);
  if (K % 16 != 0) return fail(GDR_ERR_UNSUPPORTED, "%s: K=%d is not a multiple of 16", who, K);
  if (out_dtype != GDR_BF16 && out_dtype != GDR_FP32)
    return fail(GDR_ERR_UNSUPPORTED, "%s: dtype codes must be GDR_BF16 or GDR_FP32", who);
  if (M > 0 && (!a || !a_scale || !w || !w_scale || !out))
    return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  for (const void* q : {a, static_cast<const void*>(a_scale), w, static_cast<const void*>(w_scale),
                        static_cast<const void*>(out)})
    if ((reinterpret_cast<uintptr_t>(q) & 15u) != 0)
      return fail(GDR_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  if (M == 0) return gdr::ok();
  const gdr_status s = gdr::check_device();
  if (s != GDR_OK) return s;
  gdr::Product8 p{};
  p.a = static_cast<const uint8_t*>(a); p.w = static_cast<const uint8_t*>(w);
  p.a_scale = a_scale; p.w_scale = w_scale; p.out = out;
  p.M = M; p.N = N; p.K = K; p.out_dtype = out_dtype;
  return gdr::hip_status(gdr::launch_product8(p, static_cast<hipStream_t>(stream)),
                         "gdr_product8 launch");
}

}  // extern "C"
