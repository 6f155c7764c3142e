// norm_api.cpp -- the C ABI of the norms around a block: host-side validation
// and dispatch (conventions as in api.cpp).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gdr.h"
#include "api_internal.h"
#include "norm.h"

namespace {

using gdr::BlockNorm;
using gdr::check_device;
using gdr::fail;
using gdr::hip_status;
using gdr::ok;

constexpr int kMaxWidth = 16384;
// A launch has fewer than 2^32 threads, at most max(8, D / 4) a row.
constexpr int64_t kMaxRows = int64_t{1} << 28, kMaxElements = int64_t{1} << 33;

bool valid_dtype(int d) { return d == GDR_BF16 || d == GDR_FP32; }

bool valid_rows(int64_t rows, int D) { return rows >= 0 && rows <= kMaxRows && rows * D < kMaxElements; }

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t partial_bytes(int64_t rows, int D) {
  return align_up(sizeof(float) * static_cast<size_t>(gdr::block_norm_backward_blocks(rows, D)) * D);
}

gdr_status check_common(const char* who, const BlockNorm& p) {
  if (p.D < 1 || p.D > kMaxWidth)
    return fail(GDR_ERR_UNSUPPORTED, "%s: D=%d not in [1, %d]", who, p.D, kMaxWidth);
  if (!valid_rows(p.rows, p.D))
    return fail(GDR_ERR_INVALID_ARG, "%s: rows=%lld", who, static_cast<long long>(p.rows));
  if (!valid_dtype(p.in_dtype) || !valid_dtype(p.w_dtype) || !valid_dtype(p.out_dtype))
    return fail(GDR_ERR_UNSUPPORTED, "%s: dtype codes must be GDR_BF16 or GDR_FP32", who);
  if (p.gate && p.act != GDR_GATE_SILU && p.act != GDR_GATE_SIGMOID)
    return fail(GDR_ERR_INVALID_ARG, "%s: act must be GDR_GATE_SILU or GDR_GATE_SIGMOID", who);
  if (!(p.eps >= 0.f)) return fail(GDR_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  const void* ptrs[] = {p.x, p.w_after, p.gate, p.residual, p.w_before, p.h, p.y, p.dh, p.dy,
                        p.dx, p.dgate, p.dresidual};
  for (const void* q : ptrs)
    if (q && (reinterpret_cast<uintptr_t>(q) & 15u) != 0)
      return fail(GDR_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  return GDR_OK;
}

}  // namespace

extern "C" {

gdr_status gdr_block_norm(const void* x, const void* w_after, const void* gate,
                          const void* residual, const void* w_before, void* h, void* y,
                          int64_t rows, int D, float scale, float eps, gdr_gate act,
                          gdr_dtype in_dtype, gdr_dtype w_dtype, gdr_dtype out_dtype,
                          gdr_stream_t stream) {
  const char* who = "gdr_block_norm";
  BlockNorm p{};
  p.x = x; p.w_after = w_after; p.gate = gate; p.residual = residual; p.w_before = w_before;
  p.h = h; p.y = y;
  p.rows = rows; p.D = D; p.act = act;
  p.in_dtype = in_dtype; p.w_dtype = w_dtype; p.out_dtype = out_dtype;
  p.scale = scale; p.eps = eps;
  if (rows > 0 && (!x || (!h && !y))) return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  if (rows > 0 && (y != nullptr) != (w_before != nullptr))
    return fail(GDR_ERR_INVALID_ARG, "%s: y is given exactly when w_before is", who);
  if (h && h == y) return fail(GDR_ERR_INVALID_ARG, "%s: h and y must not be one buffer", who);
  if (in_dtype != out_dtype)
    for (const void* q : {x, gate, residual})
      if (q && (q == h || q == y))
        return fail(GDR_ERR_INVALID_ARG, "%s: in place needs one dtype", who);
  gdr_status s = check_common(who, p);
  if (s != GDR_OK) return s;
  if (rows == 0) return ok();
  s = check_device();
  if (s != GDR_OK) return s;
  return hip_status(gdr::launch_block_norm(p, static_cast<hipStream_t>(stream)),
                    "gdr_block_norm launch");
}

gdr_status gdr_block_norm8(const void* x, const void* w_after, const void* gate,
                           const void* residual, const void* w_before, void* h, void* y8,
                           float* y_scale, int64_t rows, int D, float scale, float eps,
                           gdr_gate act, gdr_dtype in_dtype, gdr_dtype w_dtype,
                           gdr_dtype out_dtype, gdr_stream_t stream) {
  const char* who = "gdr_block_norm8";
  BlockNorm p{};
  p.x = x; p.w_after = w_after; p.gate = gate; p.residual = residual; p.w_before = w_before;
  p.h = h; p.y8 = y8; p.y_scale = y_scale;
  p.rows = rows; p.D = D; p.act = act;
  p.in_dtype = in_dtype; p.w_dtype = w_dtype; p.out_dtype = out_dtype;
  p.scale = scale; p.eps = eps;
  if (rows > 0 && (!x || !y8 || !y_scale)) return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  for (const void* q : {x, gate, residual, static_cast<const void*>(h), static_cast<const void*>(y_scale)})
    if (q && q == y8) return fail(GDR_ERR_INVALID_ARG, "%s: y8 must have a buffer of its own", who);
  if (h && in_dtype != out_dtype)
    for (const void* q : {x, gate, residual})
      if (q == h) return fail(GDR_ERR_INVALID_ARG, "%s: in place needs one dtype", who);
  gdr_status s = check_common(who, p);
  if (s != GDR_OK) return s;
  if (D % 16 != 0) return fail(GDR_ERR_UNSUPPORTED, "%s: D=%d is not a multiple of 16", who, D);
  for (const void* q : {static_cast<const void*>(y8), static_cast<const void*>(y_scale)})
    if ((reinterpret_cast<uintptr_t>(q) & 15u) != 0)
      return fail(GDR_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  if (rows == 0) return ok();
  s = check_device();
  if (s != GDR_OK) return s;
  return hip_status(gdr::launch_block_norm8(p, static_cast<hipStream_t>(stream)),
                    "gdr_block_norm8 launch");
}

size_t gdr_block_norm_backward_workspace_bytes(int64_t rows, int D) {
  if (D < 1 || D > kMaxWidth || !valid_rows(rows, D)) return 0;
  return 2 * partial_bytes(rows, D);
}

gdr_status gdr_block_norm_backward(const void* x, const void* w_after, const void* gate,
                                   const void* residual, const void* w_before, const void* dh,
                                   const void* dy, void* dx, void* dgate, void* dresidual,
                                   float* dw_after, float* dw_before, int64_t rows, int D,
                                   float scale, float eps, gdr_gate act, gdr_dtype in_dtype,
                                   gdr_dtype w_dtype, gdr_dtype out_dtype, void* workspace,
                                   size_t workspace_bytes, gdr_stream_t stream) {
  const char* who = "gdr_block_norm_backward";
  BlockNorm p{};
  p.x = x; p.w_after = w_after; p.gate = gate; p.residual = residual; p.w_before = w_before;
  p.dh = dh; p.dy = dy; p.dx = dx; p.dgate = dgate; p.dresidual = dresidual;
  p.rows = rows; p.D = D; p.act = act;
  p.in_dtype = in_dtype; p.w_dtype = w_dtype; p.out_dtype = out_dtype;
  p.scale = scale; p.eps = eps;
  if (rows > 0 && (!x || !dx || (!dh && !dy)))
    return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  if (rows > 0 && (dy != nullptr) != (w_before != nullptr))
    return fail(GDR_ERR_INVALID_ARG, "%s: dy is given exactly when w_before is", who);
  if ((dgate && !gate) || (dw_after && !w_after) || (dw_before && !w_before))
    return fail(GDR_ERR_INVALID_ARG, "%s: gradient of an operand that is not given", who);
  gdr_status s = check_common(who, p);
  if (s != GDR_OK) return s;
  if (dw_after || dw_before) {
    const size_t one = partial_bytes(rows, D), need = 2 * one;
    if (workspace_bytes < need || (!workspace && need > 0))
      return fail(GDR_ERR_INVALID_ARG, "%s: workspace of %zu bytes, need %zu", who, workspace_bytes, need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
      return fail(GDR_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
    float* part = static_cast<float*>(workspace);
    if (dw_after) p.part_after = part;
    if (dw_before) p.part_before = part + one / sizeof(float);
  }
  s = check_device();
  if (s != GDR_OK) return s;
  return hip_status(gdr::launch_block_norm_backward(p, dw_after, dw_before,
                                                    static_cast<hipStream_t>(stream)),
                    "gdr_block_norm_backward launch");
}

}  // extern "C"
