// linear.hip -- linear attention with a decay for each head on gfx950.
//
// One kernel computes a pass of the recurrence (launch.h, LinearPass) token by
// token: a 256-thread workgroup holds 16 state rows of one (sequence, head),
// 16 lanes to a row, and walks the sequence's tokens.
#include "gdr_device.h"
#include "launch.h"

namespace gdr {
namespace {

constexpr float kMinGate = -110.f;  // e^-110 is zero in fp32: stands for every smaller g

__device__ __forceinline__ float load_gate(const LinearGates& g, size_t t, int h, int H) {
  const float x = g.per_token ? g.g[t * H + h] : g.g[h];
  return x < kMinGate ? kMinGate : x;
}

template <Dt IN>
__global__ __launch_bounds__(256) void linear_walk_kernel(LinearBatch b, LinearPass p) {
  const int blocks = p.od / 16;
  const int rb = blockIdx.x % blocks, nh = blockIdx.x / blocks;
  const int n = nh / b.H, h = nh % b.H;
  const int lane16 = threadIdx.x & 15, rr = threadIdx.x >> 4, row = 16 * rb + rr;
  const int cpl = p.kd / 16;  // 4 or 8 columns a lane
  int tb = b.cu[n], te = b.cu[n + 1];
  tb = tb < 0 ? 0 : (tb > b.T_total ? b.T_total : tb);
  te = te < tb ? tb : (te > b.T_total ? b.T_total : te);
  const size_t sbase = static_cast<size_t>(nh) * p.od * p.kd + row * p.row;
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    z[i] = i < cpl && p.start ? p.start[sbase + (lane16 + 16 * i) * p.col] : 0.f;
  __shared__ float part[16];
  for (int s = 0; s < te - tb; ++s) {
    const size_t t = p.backward ? te - 1 - s : tb + s;
    const size_t xi = t * p.x.stride + static_cast<size_t>(h / p.x.group) * p.kd + lane16;
    const size_t yi = t * p.y.stride + static_cast<size_t>(h / p.y.group) * p.kd + lane16;
    const float w = load_scalar<IN>(p.w.p, t * p.w.stride +
                                               static_cast<size_t>(h / p.w.group) * p.od + row);
    const float alpha = expf(load_gate(b.gates, t, h, b.H));
    float before = 0.f, own = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= cpl) continue;
      const float xv = load_scalar<IN>(p.x.p, xi + 16 * i);
      const float yv = load_scalar<IN>(p.y.p, yi + 16 * i);
      if (!p.backward) z[i] *= alpha;
      before = fmaf(z[i], xv, before);
      const float add = p.us * w * yv;
      own = fmaf(add, xv, own);
      z[i] += add;
      if (p.backward) z[i] *= alpha;
    }
    before = row16_sum(before) * p.os;
    own = row16_sum(own) * p.os;
    const size_t oi = (t * b.H + h) * p.od + row;
    if (lane16 == 0) {
      if (p.out_dtype == 0) store_scalar<Dt::BF16>(p.out, oi, before + own);
      else store_scalar<Dt::F32>(p.out, oi, before + own);
    }
    if (p.dot) {
      if (lane16 == 0)
        part[rr] = before * load_scalar<IN>(p.e.p, t * p.e.stride +
                                                       static_cast<size_t>(h / p.e.group) * p.od + row);
      __syncthreads();
      if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int i = 0; i < 16; ++i) sum += part[i];
        p.dot[static_cast<size_t>(rb) * b.T_total * b.H + t * b.H + h] = sum;
      }
      __syncthreads();
    }
  }
  float ed = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= cpl) continue;
    if (p.end) p.end[sbase + (lane16 + 16 * i) * p.col] = z[i];
    if (p.end_with) ed = fmaf(z[i], p.end_with[sbase + (lane16 + 16 * i) * p.col], ed);
  }
  if (p.end_with) {
    ed = row16_sum(ed);
    if (lane16 == 0) part[rr] = ed;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.f;
      for (int i = 0; i < 16; ++i) sum += part[i];
      p.end_dot[static_cast<size_t>(rb) * b.N * b.H + nh] = sum;
    }
  }
}

__global__ __launch_bounds__(64) void linear_dg_kernel(LinearBatch b, const float* row,
                                                       int row_parts, const float* col,
                                                       int col_parts, const float* end_dot,
                                                       int end_parts, float* dg) {
  const int nh = blockIdx.x * 64 + threadIdx.x;
  if (nh >= b.N * b.H) return;
  const int n = nh / b.H, h = nh % b.H;
  int tb = b.cu[n], te = b.cu[n + 1];
  tb = tb < 0 ? 0 : (tb > b.T_total ? b.T_total : tb);
  te = te < tb ? tb : (te > b.T_total ? b.T_total : te);
  const size_t th = static_cast<size_t>(b.T_total) * b.H;
  float acc = 0.f;
  if (end_dot)
    for (int i = 0; i < end_parts; ++i) acc += end_dot[static_cast<size_t>(i) * b.N * b.H + nh];
  for (int t = te - 1; t >= tb; --t) {
    const size_t at = static_cast<size_t>(t) * b.H + h;
    float r = 0.f, c = 0.f;
    for (int i = 0; i < row_parts; ++i) r += row[i * th + at];
    for (int i = 0; i < col_parts; ++i) c += col[i * th + at];
    acc += r - c;
    dg[at] = acc;
  }
}

__global__ __launch_bounds__(256) void linear_dg_heads_kernel(LinearBatch b, const float* dg_t,
                                                              float* dg) {
  const int h = blockIdx.x;
  int te = b.cu[b.N];
  te = te < 0 ? 0 : (te > b.T_total ? b.T_total : te);
  double acc = 0;
  for (int t = threadIdx.x; t < te; t += 256) acc += dg_t[static_cast<size_t>(t) * b.H + h];
  __shared__ double part[256];
  part[threadIdx.x] = acc;
  __syncthreads();
  for (int s = 128; s > 0; s >>= 1) {
    if (threadIdx.x < s) part[threadIdx.x] += part[threadIdx.x + s];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[h] = static_cast<float>(part[0]);
}

__global__ __launch_bounds__(256) void linear_group_sum_kernel(LinearBatch b, const float* part,
                                                               int group, int d, void* out,
                                                               int out_dtype) {
  int te = b.cu[b.N];
  te = te < 0 ? 0 : (te > b.T_total ? b.T_total : te);
  const int hk = b.H / group;
  const size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= static_cast<size_t>(te) * hk * d) return;
  const size_t th = i / d;
  const int col = i % d;
  const size_t t = th / hk;
  const int hh = th % hk;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < group; ++j)
    acc += *reinterpret_cast<const floatx4*>(part + (t * b.H + hh * group + j) * d + col);
  for (int e = 0; e < 4; ++e) {
    if (out_dtype == 0) store_scalar<Dt::BF16>(out, i + e, acc[e]);
    else store_scalar<Dt::F32>(out, i + e, acc[e]);
  }
}

// One token: row i of a state becomes alpha s_i + v_i k, its output scale s_i . q.
template <Dt IN, Dt OUT>
__global__ __launch_bounds__(256) void linear_decode_kernel(
    const void* q, const void* k, const void* v, LinearGates g, float* state, void* o, int H,
    int group, int dk, int dv, int64_t qs, int64_t ks, int64_t vs, float scale) {
  const int blocks = dv / 16;
  const int rb = blockIdx.x % blocks, nh = blockIdx.x / blocks;
  const int n = nh / H, h = nh % H;
  const int lane16 = threadIdx.x & 15, row = 16 * rb + (threadIdx.x >> 4);
  const float alpha = expf(load_gate(g, n, h, H));
  const float vv = load_scalar<IN>(v, n * vs + static_cast<size_t>(h) * dv + row);
  float* s = state + (static_cast<size_t>(nh) * dv + row) * dk + lane16;
  float acc = 0.f;
  for (int i = 0; i < dk / 16; ++i) {
    const size_t at = static_cast<size_t>(h / group) * dk + lane16 + 16 * i;
    const float x = fmaf(vv, load_scalar<IN>(k, n * ks + at), alpha * s[16 * i]);
    s[16 * i] = x;
    acc = fmaf(x, load_scalar<IN>(q, n * qs + at), acc);
  }
  acc = row16_sum(acc);
  if (lane16 == 0) store_scalar<OUT>(o, static_cast<size_t>(nh) * dv + row, scale * acc);
}

}  // namespace

hipError_t launch_linear_decode(const void* q, const void* k, const void* v,
                                const LinearGates& g, float* state, void* o, int N, int H, int Hk,
                                int dk, int dv, int64_t qs, int64_t ks, int64_t vs, float scale,
                                int in_dtype, int out_dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(N) * H * (dv / 16));
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, stream, q, k, v, g, state, o, H, H / Hk, dk, dv,
                       qs, ks, vs, scale);
    return hipGetLastError();
  };
  if (in_dtype == 0)
    return out_dtype == 0 ? go(linear_decode_kernel<Dt::BF16, Dt::BF16>)
                          : go(linear_decode_kernel<Dt::BF16, Dt::F32>);
  return out_dtype == 0 ? go(linear_decode_kernel<Dt::F32, Dt::BF16>)
                        : go(linear_decode_kernel<Dt::F32, Dt::F32>);
}

hipError_t launch_linear_pass(const LinearBatch& b, const LinearPass& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(b.N) * b.H * (p.od / 16));
  if (b.in_dtype == 0)
    hipLaunchKernelGGL(linear_walk_kernel<Dt::BF16>, grid, dim3(256), 0, stream, b, p);
  else
    hipLaunchKernelGGL(linear_walk_kernel<Dt::F32>, grid, dim3(256), 0, stream, b, p);
  return hipGetLastError();
}

hipError_t launch_linear_dg(const LinearBatch& b, const float* row, int row_parts,
                            const float* col, int col_parts, const float* end_dot, int end_parts,
                            float* dg, hipStream_t stream) {
  hipLaunchKernelGGL(linear_dg_kernel, dim3((b.N * b.H + 63) / 64), dim3(64), 0, stream, b, row,
                     row_parts, col, col_parts, end_dot, end_parts, dg);
  return hipGetLastError();
}

hipError_t launch_linear_dg_heads(const LinearBatch& b, const float* dg_t, float* dg,
                                  hipStream_t stream) {
  hipLaunchKernelGGL(linear_dg_heads_kernel, dim3(b.H), dim3(256), 0, stream, b, dg_t, dg);
  return hipGetLastError();
}

hipError_t launch_linear_group_sum(const LinearBatch& b, const float* part, int group, int d,
                                   void* out, int out_dtype, hipStream_t stream) {
  const size_t n = static_cast<size_t>(b.T_total) * (b.H / group) * d / 4;
  hipLaunchKernelGGL(linear_group_sum_kernel, dim3((n + 255) / 256), dim3(256), 0, stream, b, part,
                     group, d, out, out_dtype);
  return hipGetLastError();
}

}  // namespace gdr
