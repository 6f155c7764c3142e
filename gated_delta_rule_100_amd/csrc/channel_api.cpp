// channel_api.cpp -- the C ABI of the recurrence with a decay for each channel:
// host-side validation and dispatch (conventions as in api.cpp).
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "../../include/gdr.h"
#include "api_internal.h"
#include "channel.h"

namespace {

using gdr::Channel;
using gdr::check_device;
using gdr::fail;
using gdr::hip_status;
using gdr::ok;

constexpr int kMaxWidth = 1 << 20, kMaxSeqs = 1 << 20;

bool valid_dtype(int d) { return d == GDR_BF16 || d == GDR_FP32; }

// Workgroups hold 64 tokens by 64 channels at least, 256 threads each, and a launch has
// fewer than 2^32 threads.
bool fits(int T, int D) {
  return (static_cast<int64_t>(T) / 64 + 1) * (D / 64 + 1) < (int64_t{1} << 24);
}

// Checks shared by the entry points; resolves strides of 0.  rows: T, or N of a step.
gdr_status check_common(const char* who, int rows, Channel* p, std::initializer_list<const void*> ptrs) {
  if (rows < 0 || p->N <= 0 || p->N > kMaxSeqs)
    return fail(GDR_ERR_INVALID_ARG, "%s: tokens=%d N=%d", who, rows, p->N);
  if (p->D < 1 || p->D > kMaxWidth)
    return fail(GDR_ERR_UNSUPPORTED, "%s: D=%d not in [1, %d]", who, p->D, kMaxWidth);
  if (static_cast<int64_t>(p->N) * p->D > INT32_MAX)
    return fail(GDR_ERR_INVALID_ARG, "%s: N*D too large", who);
  if (!fits(rows, p->D))
    return fail(GDR_ERR_INVALID_ARG, "%s: %d tokens of %d channels are more than a launch holds", who,
                rows, p->D);
  if (!valid_dtype(p->io_dtype) || !valid_dtype(p->g_dtype))
    return fail(GDR_ERR_UNSUPPORTED, "%s: dtype codes must be GDR_BF16 or GDR_FP32", who);
  if (p->gate != GDR_CHANNEL_LOG && p->gate != GDR_CHANNEL_LOGIT)
    return fail(GDR_ERR_INVALID_ARG, "%s: gate must be GDR_CHANNEL_LOG or GDR_CHANNEL_LOGIT", who);
  if (p->complement != 0 && p->complement != 1)
    return fail(GDR_ERR_INVALID_ARG, "%s: complement must be 0 or 1", who);
  struct { int64_t* s; const char* name; } strides[] = {{&p->x_stride, "x_stride"},
                                                        {&p->g_stride, "g_stride"}};
  for (auto& r : strides) {
    if (*r.s == 0) *r.s = p->D;
    if (*r.s < p->D || *r.s > (int64_t{1} << 24))
      return fail(GDR_ERR_INVALID_ARG, "%s: %s=%lld must be 0 or from %d to 2^24", who, r.name,
                  static_cast<long long>(*r.s), p->D);
  }
  for (const void* q : ptrs)
    if (q && (reinterpret_cast<uintptr_t>(q) & 15u) != 0)
      return fail(GDR_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  return GDR_OK;
}

gdr_status check_workspace(const char* who, const void* workspace, size_t bytes, size_t need) {
  if (bytes < need || (!workspace && need > 0))
    return fail(GDR_ERR_INVALID_ARG, "%s: workspace of %zu bytes, need %zu", who, bytes, need);
  return GDR_OK;
}

size_t workspace_bytes_of(int T, int D) {
  if (T < 0 || D < 1 || D > kMaxWidth || !fits(T, D)) return 0;
  return gdr::channel_workspace_bytes(T, D);
}

}  // namespace

extern "C" {

gdr_status gdr_channel_decode(const void* x, const void* g, float* state, void* h, int N, int D,
                              int64_t x_stride, int64_t g_stride, gdr_channel_gate gate,
                              int complement, gdr_dtype io_dtype, gdr_dtype g_dtype,
                              gdr_stream_t stream) {
  const char* who = "gdr_channel_decode";
  if (!x || !g || !state || !h) return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  Channel p{};
  p.x = x; p.g = g; p.state_in = state; p.state_out = state; p.h = h;
  p.T = N; p.N = N; p.D = D; p.x_stride = x_stride; p.g_stride = g_stride;
  p.gate = gate; p.complement = complement; p.io_dtype = io_dtype; p.g_dtype = g_dtype;
  gdr_status s = check_common(who, N, &p, {x, g, state, h});
  if (s == GDR_OK && h == x && p.x_stride != D)
    s = fail(GDR_ERR_INVALID_ARG, "%s: in place needs a dense x", who);
  if (s == GDR_OK) s = check_device();
  if (s != GDR_OK) return s;
  return hip_status(gdr::launch_channel_decode(p, static_cast<hipStream_t>(stream)),
                    "gdr_channel_decode launch");
}

size_t gdr_channel_prefill_workspace_bytes(int T_total, int D) { return workspace_bytes_of(T_total, D); }

size_t gdr_channel_backward_workspace_bytes(int T_total, int D) { return workspace_bytes_of(T_total, D); }

gdr_status gdr_channel_prefill(const void* x, const void* g, const int32_t* cu_seqlens, int N,
                               const float* state_in, float* state_out, void* h, int T_total,
                               int D, int64_t x_stride, int64_t g_stride, gdr_channel_gate gate,
                               int complement, gdr_dtype io_dtype, gdr_dtype g_dtype,
                               void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  const char* who = "gdr_channel_prefill";
  if (!cu_seqlens || (T_total > 0 && (!x || !g || !h)))
    return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  Channel p{};
  p.x = x; p.g = g; p.cu = cu_seqlens; p.state_in = state_in; p.state_out = state_out; p.h = h;
  p.T = T_total; p.N = N; p.D = D; p.x_stride = x_stride; p.g_stride = g_stride;
  p.gate = gate; p.complement = complement; p.io_dtype = io_dtype; p.g_dtype = g_dtype;
  gdr_status s = check_common(who, T_total, &p, {x, g, cu_seqlens, state_in, state_out, h, workspace});
  if (s == GDR_OK && T_total > 0 && h == x && p.x_stride != D)
    s = fail(GDR_ERR_INVALID_ARG, "%s: in place needs a dense x", who);
  if (s == GDR_OK) s = check_workspace(who, workspace, workspace_bytes, workspace_bytes_of(T_total, D));
  if (s == GDR_OK) s = check_device();
  if (s != GDR_OK) return s;
  return hip_status(gdr::launch_channel_prefill(p, workspace, static_cast<hipStream_t>(stream)),
                    "gdr_channel_prefill launch");
}

gdr_status gdr_channel_backward(const void* x, const void* g, const void* h,
                                const int32_t* cu_seqlens, int N, const float* state_in,
                                const void* dh, const float* dstate_out, void* dx, void* dg,
                                float* dstate_in, int T_total, int D, int64_t x_stride,
                                int64_t g_stride, gdr_channel_gate gate, int complement,
                                gdr_dtype io_dtype, gdr_dtype g_dtype, void* workspace,
                                size_t workspace_bytes, gdr_stream_t stream) {
  const char* who = "gdr_channel_backward";
  if (!cu_seqlens || (T_total > 0 && (!g || !h || !dh || !dx || !dg || (complement && !x))))
    return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  Channel p{};
  p.x = x; p.g = g; p.cu = cu_seqlens; p.state_in = state_in; p.h = const_cast<void*>(h);
  p.dh = dh; p.dstate_out = dstate_out; p.dx = dx; p.dg = dg; p.dstate_in = dstate_in;
  p.T = T_total; p.N = N; p.D = D; p.x_stride = x ? x_stride : 0; p.g_stride = g_stride;
  p.gate = gate; p.complement = complement; p.io_dtype = io_dtype; p.g_dtype = g_dtype;
  gdr_status s = check_common(who, T_total, &p, {x, g, h, cu_seqlens, state_in, dh, dstate_out, dx, dg,
                                                 dstate_in, workspace});
  if (s == GDR_OK) s = check_workspace(who, workspace, workspace_bytes, workspace_bytes_of(T_total, D));
  if (s == GDR_OK) s = check_device();
  if (s != GDR_OK) return s;
  return hip_status(gdr::launch_channel_backward(p, workspace, static_cast<hipStream_t>(stream)),
                    "gdr_channel_backward launch");
}

}  // extern "C"
