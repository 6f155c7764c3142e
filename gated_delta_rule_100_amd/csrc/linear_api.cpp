// linear_api.cpp -- the C ABI of linear attention with a decay for each head:
// host-side validation and dispatch (conventions as in api.cpp).
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "../../include/gdr.h"
#include "api_internal.h"
#include "launch.h"

namespace {

using gdr::check_device;
using gdr::fail;
using gdr::hip_status;
using gdr::LinearBatch;
using gdr::LinearGates;
using gdr::LinearPass;
using gdr::LinearRows;
using gdr::ok;

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool valid_dtype(int d) { return d == GDR_BF16 || d == GDR_FP32; }

bool valid_dim(int d) { return d == 64 || d == 128; }

size_t elem_size(int dtype) { return dtype == GDR_BF16 ? 2 : 4; }

// Checks shared by the three entry points; resolves strides of 0 to dense.
// tokens: T_total, or N of a decode step.
gdr_status check_common(const char* who, int tokens, int N, int H, int Hk, int dk, int dv,
                        int64_t* qs, int64_t* ks, int64_t* vs, int decay, int in_dtype,
                        int out_dtype, std::initializer_list<const void*> ptrs) {
  if (tokens < 0 || N <= 0 || H <= 0 || Hk <= 0)
    return fail(GDR_ERR_INVALID_ARG, "%s: tokens=%d N=%d H=%d Hk=%d", who, tokens, N, H, Hk);
  if (H % Hk != 0) return fail(GDR_ERR_INVALID_ARG, "%s: H=%d is not a multiple of Hk=%d", who, H, Hk);
  if (N > 65536 || H > 65535) return fail(GDR_ERR_INVALID_ARG, "%s: N or H too large", who);
  if (!valid_dim(dk) || !valid_dim(dv))
    return fail(GDR_ERR_UNSUPPORTED, "%s: (dk, dv) = (%d, %d) not in {64, 128} x {64, 128}", who, dk, dv);
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
    return fail(GDR_ERR_UNSUPPORTED, "%s: dtype codes must be GDR_BF16 or GDR_FP32", who);
  if (decay != GDR_DECAY_TOKEN && decay != GDR_DECAY_HEAD)
    return fail(GDR_ERR_INVALID_ARG, "%s: decay must be GDR_DECAY_TOKEN or GDR_DECAY_HEAD", who);
  // grids count one workgroup for every 16 state rows
  if (static_cast<int64_t>(tokens) * H > INT32_MAX || static_cast<int64_t>(N) * H > INT32_MAX / 8)
    return fail(GDR_ERR_INVALID_ARG, "%s: tokens*H or N*H too large", who);
  const int64_t per16 = 16 / static_cast<int64_t>(elem_size(in_dtype));
  struct { int64_t* s; int64_t width; const char* name; } rows[] = {
      {qs, static_cast<int64_t>(Hk) * dk, "q_stride"},
      {ks, static_cast<int64_t>(Hk) * dk, "k_stride"},
      {vs, static_cast<int64_t>(H) * dv, "v_stride"}};
  for (auto& r : rows) {
    if (*r.s == 0) *r.s = r.width;
    if (*r.s < r.width || *r.s % per16 != 0 || *r.s > (int64_t{1} << 24))
      return fail(GDR_ERR_INVALID_ARG,
                  "%s: %s=%lld must be 0 or from %lld to 2^24 and a multiple of %lld", who, r.name, static_cast<long long>(*r.s), static_cast<long long>(r.width),
                  static_cast<long long>(per16));
  }
  for (const void* p : ptrs)
    if (p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0)
      return fail(GDR_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  return GDR_OK;
}

gdr_status hip_fail(hipError_t e, const char* who, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(GDR_ERR_HIP, "%s: %s: %s", who, what, hipGetErrorString(e));
}

// Workspace of the gradient: fp32 dq and dk of every value head when heads are
// shared, the partial sums of dg, and dg of every token for one decay a head.
struct BackwardSizes {
  size_t part_q = 0, part_k = 0, row = 0, col = 0, end = 0, dgt = 0;
  size_t total() const { return part_q + part_k + row + col + end + dgt; }
};

BackwardSizes backward_sizes(int T_total, int N, int H, int Hk, int dk, int dv) {
  BackwardSizes z;
  const size_t th = static_cast<size_t>(T_total) * H * sizeof(float);
  if (H != Hk) z.part_q = z.part_k = align_up(th * dk);
  z.row = align_up(th * (dk / 16));
  z.col = align_up(th * (dv / 16));
  z.end = align_up(static_cast<size_t>(N) * H * (dk / 16) * sizeof(float));
  z.dgt = align_up(th);
  return z;
}

}  // namespace

extern "C" {

gdr_status gdr_linear_decode(const void* q, const void* k, const void* v, const float* g,
                             float* state, void* o, int N, int H, int Hk, int dk, int dv,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                             gdr_decay decay, gdr_dtype in_dtype, gdr_dtype out_dtype,
                             gdr_stream_t stream) {
  const char* who = "gdr_linear_decode";
  if (!q || !k || !v || !g || !state || !o) return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  gdr_status s = check_common(who, N, N, H, Hk, dk, dv, &q_stride, &k_stride, &v_stride, decay,
                              in_dtype, out_dtype, {q, k, v, g, state, o});
  if (s == GDR_OK) s = check_device();
  if (s != GDR_OK) return s;
  return hip_status(gdr::launch_linear_decode(q, k, v, {g, decay == GDR_DECAY_TOKEN}, state, o, N,
                                              H, Hk, dk, dv, q_stride, k_stride, v_stride, scale,
                                              in_dtype, out_dtype, static_cast<hipStream_t>(stream)),
                    "gdr_linear_decode launch");
}

size_t gdr_linear_prefill_workspace_bytes(int T_total, int N, int H, int dk, int dv,
                                          gdr_dtype in_dtype) {
  (void)T_total; (void)N; (void)H; (void)dk; (void)dv; (void)in_dtype;
  return 0;
}

gdr_status gdr_linear_prefill(const void* q, const void* k, const void* v, const float* g,
                              const int32_t* cu_seqlens, int N, const float* state_in,
                              float* state_out, void* o, int T_total, int H, int Hk, int dk,
                              int dv, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              float scale, gdr_decay decay, gdr_dtype in_dtype,
                              gdr_dtype out_dtype, void* workspace, size_t workspace_bytes,
                              gdr_stream_t stream) {
  const char* who = "gdr_linear_prefill";
  if (!cu_seqlens) return fail(GDR_ERR_INVALID_ARG, "%s: NULL cu_seqlens", who);
  if (T_total > 0 && (!q || !k || !v || !g || !o)) return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  gdr_status s = check_common(who, T_total, N, H, Hk, dk, dv, &q_stride, &k_stride, &v_stride,
                              decay, in_dtype, out_dtype,
                              {q, k, v, g, state_in, state_out, o, workspace});
  if (s != GDR_OK) return s;
  const size_t need = gdr_linear_prefill_workspace_bytes(T_total, N, H, dk, dv, in_dtype);
  if (workspace_bytes < need || (!workspace && need > 0))
    return fail(GDR_ERR_INVALID_ARG, "%s: workspace of %zu bytes, need %zu", who, workspace_bytes, need);
  s = check_device();
  if (s != GDR_OK) return s;
  const LinearBatch b{cu_seqlens, N, H, T_total, in_dtype, {g, decay == GDR_DECAY_TOKEN}};
  LinearPass p{};
  p.x = {q, q_stride, H / Hk};
  p.y = {k, k_stride, H / Hk};
  p.w = {v, v_stride, 1};
  p.out = o;
  p.start = state_in;
  p.end = state_out;
  p.row = dk;
  p.col = 1;
  p.us = 1.f;
  p.os = scale;
  p.od = dv;
  p.kd = dk;
  p.out_dtype = out_dtype;
  return hip_fail(gdr::launch_linear_pass(b, p, static_cast<hipStream_t>(stream)), who, "scan");
}

size_t gdr_linear_backward_workspace_bytes(int T_total, int N, int H, int Hk, int dk, int dv,
                                           gdr_dtype in_dtype) {
  if (T_total < 0 || N <= 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || !valid_dim(dk) ||
      !valid_dim(dv) || !valid_dtype(in_dtype))
    return 0;
  return backward_sizes(T_total, N, H, Hk, dk, dv).total();
}

gdr_status gdr_linear_backward(const void* q, const void* k, const void* v, const float* g,
                               const int32_t* cu_seqlens, int N, const float* state_in,
                               const void* d_o, const float* dstate_out, void* dq, void* dk_out,
                               void* dv_out, float* dg, float* dstate_in, int T_total, int H,
                               int Hk, int dk, int dv, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, float scale, gdr_decay decay,
                               gdr_dtype in_dtype, gdr_dtype grad_dtype, void* workspace,
                               size_t workspace_bytes, gdr_stream_t stream) {
  const char* who = "gdr_linear_backward";
  if (!cu_seqlens) return fail(GDR_ERR_INVALID_ARG, "%s: NULL cu_seqlens", who);
  if (T_total > 0 && (!q || !k || !v || !g || !d_o || !dq || !dk_out || !dv_out))
    return fail(GDR_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  if (dstate_in && dstate_in == dstate_out)
    return fail(GDR_ERR_INVALID_ARG, "%s: dstate_in must not be dstate_out", who);
  gdr_status s = check_common(who, T_total, N, H, Hk, dk, dv, &q_stride, &k_stride, &v_stride,
                              decay, in_dtype, grad_dtype,
                              {q, k, v, g, state_in, d_o, dstate_out, dq, dk_out, dv_out, dg,
                               dstate_in, workspace});
  if (s != GDR_OK) return s;
  const BackwardSizes z = backward_sizes(T_total, N, H, Hk, dk, dv);
  if (workspace_bytes < z.total() || (!workspace && z.total() > 0))
    return fail(GDR_ERR_INVALID_ARG, "%s: workspace of %zu bytes, need %zu", who, workspace_bytes, z.total());
  s = check_device();
  if (s != GDR_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const LinearBatch b{cu_seqlens, N, H, T_total, in_dtype, {g, decay == GDR_DECAY_TOKEN}};
  char* ws = static_cast<char*>(workspace);
  auto take = [&](size_t bytes) {
    float* f = reinterpret_cast<float*>(ws);
    ws += bytes;
    return f;
  };
  const int group = H / Hk;
  float* part_q = take(z.part_q);
  float* part_k = take(z.part_k);
  float* row = take(z.row);
  float* col = take(z.col);
  float* end = take(z.end);
  float* dgt = take(z.dgt);
  const LinearRows rq{q, q_stride, group}, rk{k, k_stride, group}, rv{v, v_stride, 1},
      rd{d_o, static_cast<int64_t>(H) * dv, 1};
  LinearPass pq{}, pv{}, pk{};
  pq.x = rd; pq.y = rv; pq.w = rk; pq.e = rq;
  pq.out = group > 1 ? static_cast<void*>(part_q) : dq;
  pq.out_dtype = group > 1 ? GDR_FP32 : grad_dtype;
  pq.start = state_in;
  pq.row = 1; pq.col = dk; pq.od = dk; pq.kd = dv;
  pq.us = 1.f; pq.os = scale;
  if (dg) {
    pq.dot = row;
    pq.end_with = dstate_out;
    pq.end_dot = end;
  }
  pv.x = rk; pv.y = rq; pv.w = rd; pv.e = rv;
  pv.out = dv_out; pv.out_dtype = grad_dtype;
  pv.dot = dg ? col : nullptr;
  pv.start = dstate_out;
  pv.end = dstate_in;
  pv.row = dk; pv.col = 1; pv.od = dv; pv.kd = dk;
  pv.us = scale; pv.os = 1.f; pv.backward = 1;
  pk.x = rv; pk.y = rd; pk.w = rq;
  pk.out = group > 1 ? static_cast<void*>(part_k) : dk_out;
  pk.out_dtype = group > 1 ? GDR_FP32 : grad_dtype;
  pk.start = dstate_out;
  pk.row = 1; pk.col = dk; pk.od = dk; pk.kd = dv;
  pk.us = scale; pk.os = 1.f; pk.backward = 1;
  hipError_t e = gdr::launch_linear_pass(b, pq, st);
  if (e == hipSuccess) e = gdr::launch_linear_pass(b, pv, st);
  if (e == hipSuccess) e = gdr::launch_linear_pass(b, pk, st);
  if (e != hipSuccess) return hip_fail(e, who, "scan");
  if (group > 1 && T_total > 0) {
    e = gdr::launch_linear_group_sum(b, part_q, group, dk, dq, grad_dtype, st);
    if (e == hipSuccess) e = gdr::launch_linear_group_sum(b, part_k, group, dk, dk_out, grad_dtype, st);
    if (e != hipSuccess) return hip_fail(e, who, "shared heads");
  }
  if (dg) {
    float* to = decay == GDR_DECAY_TOKEN ? dg : dgt;
    e = gdr::launch_linear_dg(b, row, dk / 16, col, dv / 16, dstate_out ? end : nullptr, dk / 16,
                              to, st);
    if (e == hipSuccess && decay == GDR_DECAY_HEAD) e = gdr::launch_linear_dg_heads(b, dgt, dg, st);
    if (e != hipSuccess) return hip_fail(e, who, "gate gradient");
  }
  return ok();
}

}  // extern "C"
