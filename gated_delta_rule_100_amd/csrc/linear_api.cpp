// linear_api.cpp -- the C ABI of linear attention with a decay for each head:
// host-side validation and dispatch (conventions as in api.cpp).
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "../../include/gdr.h"
#include "api_internal.h"
#include "launch.h"
#include "linear.h"

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
  // a launch has fewer than 2^32 threads, 1024 at most for a (sequence, head)
  if (static_cast<int64_t>(tokens) * H > INT32_MAX || static_cast<int64_t>(N) * H > 4000000)
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
                  "%s: %s=%lld must be 0 or from %lld to 2^24 and a multiple of %lld", who, r.name,
                  static_cast<long long>(*r.s), static_cast<long long>(r.width),
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

// Tokens of a segment, or 0 to walk whole sequences.  A scan workgroup takes a
// compute unit for one (unit, head), about 4.3 us a chunk of 64 tokens (bf16, 128 x
// 128) with all of them at work, so segments are as long as 256 workgroups allow:
// fewer states to form and pass on (4 x 4096 tokens, 16 heads, two sets of inputs in
// turn: 134 us of scan, segment states and chain at 1024 tokens, 154 at 512 and 176 at
// 2048; 131072 tokens, 4 heads: 235 at 2048, 259 at 1024, 327 at 4096).  The states
// cost two launches, so a sequence has to be some chunks longer than a segment before
// that pays (gradient of one sequence, 128 x 128, bf16 / fp32: 800 tokens, 4 heads 43 /
// 53 us in segments, 62 / 152 without; 800 tokens, 16 heads 74 / 102 and 64 / 156).
//
// The host knows only the average length, and takes four times it for the longest
// one.  Many sequences of one length are right to be walked whole (32 of 1024 tokens,
// 32 heads: 340 us, 385 in segments), but so are then those beside a much longer one,
// whose walk takes its whole length: one of 16384 tokens beside 31 of 528, 32 heads,
// 857 us (471 in segments); 131072 tokens beside 255 single ones, 4 heads, 6.7 ms
// (0.29).  Such a sequence is faster in a call of its own.
int segment_tokens(int T_total, int N, int H, bool gradient) {
  const int64_t th = static_cast<int64_t>(T_total) * H;
  const int64_t seg = (th + 256 * 64 - 1) / (256 * 64) * 64;
  const int64_t longest = 4 * ((static_cast<int64_t>(T_total) + N - 1) / N);
  const int64_t most = longest < T_total ? longest : T_total;
  return most >= seg + (gradient ? 256 : 512) ? static_cast<int>(seg) : 0;
}

// Segment tables and states of `kinds` directions.
struct SegmentSizes {
  int seg = 0, units = 0;
  size_t offs = 0, idx = 0, states = 0, decays = 0;
  int kinds = 0;
  size_t total() const { return offs + idx + kinds * (states + decays); }
};

SegmentSizes segment_sizes(int T_total, int N, int H, int dk, int dv, int kinds) {
  SegmentSizes z;
  z.seg = segment_tokens(T_total, N, H, kinds > 1);
  z.units = z.seg ? T_total / z.seg + N : N;
  if (!z.seg) return z;
  z.kinds = kinds;
  const size_t pairs = static_cast<size_t>(z.units) * H;
  if (N > gdr::kInlineSeqs) {
    z.offs = align_up(sizeof(int32_t) * (static_cast<size_t>(N) + 1));
    z.idx = align_up(sizeof(int32_t) * 2 * static_cast<size_t>(z.units));
  }
  z.states = align_up(sizeof(float) * pairs * dk * dv);
  z.decays = align_up(sizeof(float) * pairs);
  return z;
}

// Workspace of the gradient: segments, fp32 dq and dk of every value head when
// heads are shared, the partial sums of dg, and its sums over units for one
// decay a head.
struct BackwardSizes {
  SegmentSizes seg;
  size_t part_q = 0, part_k = 0, row = 0, col = 0, start = 0, end = 0, sums = 0;
  size_t total() const { return seg.total() + part_q + part_k + row + col + start + end + sums; }
};

BackwardSizes backward_sizes(int T_total, int N, int H, int Hk, int dk, int dv) {
  BackwardSizes z;
  z.seg = segment_sizes(T_total, N, H, dk, dv, 2);
  const size_t th = static_cast<size_t>(T_total) * H * sizeof(float);
  const size_t pairs = static_cast<size_t>(z.seg.units) * H;
  if (H != Hk) z.part_q = z.part_k = align_up(th * dk);
  z.row = z.col = align_up(th);
  z.start = align_up(pairs * (dv / 16) * sizeof(float));
  z.end = align_up(pairs * (dk / 16) * sizeof(float));
  z.sums = align_up(pairs * sizeof(double));
  return z;
}

// Workspace pieces in order.
struct Carver {
  char* at;
  template <class T>
  T* take(size_t bytes) {
    T* p = reinterpret_cast<T*>(at);
    at += bytes;
    return p;
  }
};

// Lays out the segments of a batch in the workspace.
hipError_t make_segments(LinearBatch* b, const SegmentSizes& z, Carver* ws, hipStream_t st) {
  b->seg = z.seg;
  b->units = z.units;
  if (!z.seg || !z.offs) return hipSuccess;
  int32_t* offs = ws->take<int32_t>(z.offs);
  int32_t* idx = ws->take<int32_t>(z.idx);
  b->seg_offs = offs;
  b->seg_idx = idx;
  return gdr::launch_layout(b->cu, b->N, z.seg, offs, idx, z.units, st);
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
  if (T_total < 0 || N <= 0 || H <= 0 || !valid_dim(dk) || !valid_dim(dv) || !valid_dtype(in_dtype))
    return 0;
  return segment_sizes(T_total, N, H, dk, dv, 1).total();
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
  hipStream_t st = static_cast<hipStream_t>(stream);
  LinearBatch b{cu_seqlens, N, H, T_total, in_dtype, {g, decay == GDR_DECAY_TOKEN}};
  const SegmentSizes z = segment_sizes(T_total, N, H, dk, dv, 1);
  Carver ws{static_cast<char*>(workspace)};
  hipError_t e = make_segments(&b, z, &ws, st);
  if (e != hipSuccess) return hip_fail(e, who, "segments");
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
  if (z.seg) {
    float* states = ws.take<float>(z.states);
    float* decays = ws.take<float>(z.decays);
    e = gdr::launch_linear_starts(b, dv, dk, {p.y, p.w, 1.f, state_in, states, decays, state_out},
                                  nullptr, st);
    if (e != hipSuccess) return hip_fail(e, who, "segment states");
    p.start = states;
  }
  return hip_fail(gdr::launch_linear_prompt(b, p, st), who, "scan");
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
  // the sums over shared heads: one launch of a thread for four values
  if (H != Hk && static_cast<int64_t>(T_total) * Hk * dk > (int64_t{1} << 34) - 1024)
    return fail(GDR_ERR_INVALID_ARG, "%s: tokens*Hk*dk too large for shared heads", who);
  const BackwardSizes z = backward_sizes(T_total, N, H, Hk, dk, dv);
  if (workspace_bytes < z.total() || (!workspace && z.total() > 0))
    return fail(GDR_ERR_INVALID_ARG, "%s: workspace of %zu bytes, need %zu", who, workspace_bytes, z.total());
  s = check_device();
  if (s != GDR_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  LinearBatch b{cu_seqlens, N, H, T_total, in_dtype, {g, decay == GDR_DECAY_TOKEN}};
  Carver ws{static_cast<char*>(workspace)};
  hipError_t e = make_segments(&b, z.seg, &ws, st);
  if (e != hipSuccess) return hip_fail(e, who, "segments");
  float *starts = nullptr, *ends = nullptr, *decays = nullptr, *decays_back = nullptr;
  if (z.seg.seg) {
    starts = ws.take<float>(z.seg.states);
    ends = ws.take<float>(z.seg.states);
    decays = ws.take<float>(z.seg.decays);
    decays_back = ws.take<float>(z.seg.decays);
  }
  const int group = H / Hk;
  float* part_q = ws.take<float>(z.part_q);
  float* part_k = ws.take<float>(z.part_k);
  float* row = ws.take<float>(z.row);
  float* col = ws.take<float>(z.col);
  float* start = ws.take<float>(z.start);
  float* end = ws.take<float>(z.end);
  double* sums = ws.take<double>(z.sums);
  const LinearRows rq{q, q_stride, group}, rk{k, k_stride, group}, rv{v, v_stride, 1},
      rd{d_o, static_cast<int64_t>(H) * dv, 1};
  // states in front of every unit's walk: S forwards, R backwards
  const float *from = state_in, *behind = dstate_out;
  if (z.seg.seg) {
    const gdr::LinearStates back{rq, rd, scale, dstate_out, ends, decays_back, dstate_in};
    e = gdr::launch_linear_starts(b, dv, dk, {rk, rv, 1.f, state_in, starts, decays, nullptr}, &back,
                                  st);
    if (e != hipSuccess) return hip_fail(e, who, "segment states");
    from = starts;
    behind = ends;
  }
  LinearPass pq{}, pv{}, pk{};
  pq.x = rd; pq.y = rv; pq.w = rk; pq.e = rq;
  pq.out = group > 1 ? static_cast<void*>(part_q) : dq;
  pq.out_dtype = group > 1 ? GDR_FP32 : grad_dtype;
  pq.start = from;
  pq.row = 1; pq.col = dk; pq.od = dk; pq.kd = dv;
  pq.us = 1.f; pq.os = scale;
  if (dg) {
    pq.dot = row;
    pq.end_with = behind;
    pq.end_dot = end;
  }
  pv.x = rk; pv.y = rq; pv.w = rd; pv.e = rv;
  pv.out = dv_out; pv.out_dtype = grad_dtype;
  if (dg) {
    pv.dot = col;
    pv.end_with = from;
    pv.end_dot = start;
  }
  pv.start = behind;
  pv.end = dstate_in;
  pv.row = dk; pv.col = 1; pv.od = dv; pv.kd = dk;
  pv.us = scale; pv.os = 1.f; pv.backward = 1;
  pk.x = rv; pk.y = rd; pk.w = rq;
  pk.out = group > 1 ? static_cast<void*>(part_k) : dk_out;
  pk.out_dtype = group > 1 ? GDR_FP32 : grad_dtype;
  pk.start = behind;
  pk.row = 1; pk.col = dk; pk.od = dk; pk.kd = dv;
  pk.us = scale; pk.os = 1.f; pk.backward = 1;
  e = gdr::launch_linear_grads(b, pq, pv, pk, st);
  if (e != hipSuccess) return hip_fail(e, who, "scan");
  if (group > 1 && T_total > 0) {
    e = gdr::launch_linear_group_sum(b, part_q, part_k, group, dk, dq, dk_out, grad_dtype, st);
    if (e != hipSuccess) return hip_fail(e, who, "shared heads");
  }
  if (dg) {
    const bool heads = decay == GDR_DECAY_HEAD;
    e = gdr::launch_linear_dg(b, row, col, from ? start : nullptr, dv / 16,
                              behind ? end : nullptr, dk / 16, heads ? nullptr : dg,
                              heads ? sums : nullptr, st);
    if (e == hipSuccess && heads) e = gdr::launch_linear_dg_heads(b, sums, dg, st);
    if (e != hipSuccess) return hip_fail(e, who, "gate gradient");
  }
  return ok();
}

}  // extern "C"
