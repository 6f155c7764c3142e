// channel.hip -- the recurrence with a decay for each channel (gdr_channel_* in
// gdr.h) and its gradient on gfx950, one thread a sequence and channel.
#include <type_traits>

#include "channel.h"
#include "gdr_device.h"

namespace gdr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Decay a and its complement 1 - a.
struct Decay {
  float a, rest;
};

// 1 - e^g without cancellation: for g above -1/2 the series to g^9 (its next term is
// 2.7e-10 of the result), below it 1 - a, which loses at most one bit and a half.
__device__ __forceinline__ float rest_of_log(float g, float a) {
  float p = 1.f / 362880.f;
  p = fmaf(p, g, 1.f / 40320.f);
  p = fmaf(p, g, 1.f / 5040.f);
  p = fmaf(p, g, 1.f / 720.f);
  p = fmaf(p, g, 1.f / 120.f);
  p = fmaf(p, g, 1.f / 24.f);
  p = fmaf(p, g, 1.f / 6.f);
  p = fmaf(p, g, 0.5f);
  p = fmaf(p, g, 1.f);
  return fabsf(g) < 0.5f ? -g * p : 1.f - a;
}

// By the hardware's base-2 exponential and reciprocal (one unit in the last place
// each).  A logit's two halves both come from e^-|z|, so neither is a difference.
template <bool LOGIT, bool REST>
__device__ __forceinline__ Decay decay_of(float g) {
  if constexpr (LOGIT) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(g));
    const float r = __builtin_amdgcn_rcpf(1.f + e), s = e * r;
    return g < 0.f ? Decay{s, r} : Decay{r, s};
  } else {
    const float a = __builtin_amdgcn_exp2f(kLog2e * g);
    return {a, REST ? rest_of_log(g, a) : 0.f};
  }
}

template <Dt IO, Dt G, bool LOGIT, bool COMP>
__global__ void channel_decode_kernel(Channel p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<int64_t>(p.N) * p.D) return;
  const int64_t n = i / p.D, c = i % p.D;
  const float x = load_scalar<IO>(p.x, n * p.x_stride + c);
  const Decay d = decay_of<LOGIT, COMP>(load_scalar<G>(p.g, n * p.g_stride + c));
  const float s = fmaf(d.a, p.state_in[i], COMP ? d.rest * x : x);
  p.state_out[i] = s;
  store_scalar<IO>(p.h, i, s);
}

template <Dt IO, Dt G, bool LOGIT, bool COMP>
__global__ void channel_prefill_kernel(Channel p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<int64_t>(p.N) * p.D) return;
  const int64_t n = i / p.D, c = i % p.D;
  const int lo = min(max(p.cu[n], 0), p.T), hi = min(max(p.cu[n + 1], 0), p.T);
  float s = p.state_in ? p.state_in[i] : 0.f;
  for (int64_t t = lo; t < hi; ++t) {
    const float x = load_scalar<IO>(p.x, t * p.x_stride + c);
    const Decay d = decay_of<LOGIT, COMP>(load_scalar<G>(p.g, t * p.g_stride + c));
    s = fmaf(d.a, s, COMP ? d.rest * x : x);
    store_scalar<IO>(p.h, t * p.D + c, s);
  }
  if (p.state_out) p.state_out[i] = s;
}

template <Dt IO, Dt G, bool LOGIT, bool COMP>
__global__ void channel_backward_kernel(Channel p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<int64_t>(p.N) * p.D) return;
  const int64_t n = i / p.D, c = i % p.D;
  const int lo = min(max(p.cu[n], 0), p.T), hi = min(max(p.cu[n + 1], 0), p.T);
  float carry = p.dstate_out ? p.dstate_out[i] : 0.f;
  for (int64_t t = hi - 1; t >= lo; --t) {
    const Decay d = decay_of<LOGIT, COMP || LOGIT>(load_scalar<G>(p.g, t * p.g_stride + c));
    const float r = carry + load_scalar<IO>(p.dh, t * p.D + c);
    float prev = t > lo ? load_scalar<IO>(p.h, (t - 1) * p.D + c) : p.state_in ? p.state_in[i] : 0.f;
    if (COMP) prev -= load_scalar<IO>(p.x, t * p.x_stride + c);
    carry = d.a * r;
    store_scalar<IO>(p.dx, t * p.D + c, COMP ? d.rest * r : r);
    store_scalar<G>(p.dg, t * p.D + c, carry * prev * (LOGIT ? d.rest : 1.f));
  }
  if (p.dstate_in) p.dstate_in[i] = carry;
}

// Calls go(IO, G, LOGIT, COMP) for an operand's types and form.
template <class F>
hipError_t by_form(const Channel& p, F&& go) {
  using std::bool_constant;
  auto form = [&](auto io, auto g) {
    if (p.gate == 0)
      return p.complement ? go(io, g, bool_constant<false>(), bool_constant<true>())
                          : go(io, g, bool_constant<false>(), bool_constant<false>());
    return p.complement ? go(io, g, bool_constant<true>(), bool_constant<true>())
                        : go(io, g, bool_constant<true>(), bool_constant<false>());
  };
  const std::integral_constant<Dt, Dt::BF16> bf16;
  const std::integral_constant<Dt, Dt::F32> f32;
  if (p.io_dtype == 0) return p.g_dtype == 0 ? form(bf16, bf16) : form(bf16, f32);
  return p.g_dtype == 0 ? form(f32, bf16) : form(f32, f32);
}

dim3 grid(const Channel& p) {
  return dim3(static_cast<unsigned>((static_cast<int64_t>(p.N) * p.D + 255) / 256));
}

}  // namespace

size_t channel_workspace_bytes(int, int) { return 0; }

hipError_t launch_channel_decode(const Channel& p, hipStream_t stream) {
  return by_form(p, [&](auto io, auto g, auto logit, auto comp) {
    hipLaunchKernelGGL((channel_decode_kernel<io.value, g.value, logit.value, comp.value>), grid(p),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
  });
}

hipError_t launch_channel_prefill(const Channel& p, void*, hipStream_t stream) {
  return by_form(p, [&](auto io, auto g, auto logit, auto comp) {
    hipLaunchKernelGGL((channel_prefill_kernel<io.value, g.value, logit.value, comp.value>), grid(p),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
  });
}

hipError_t launch_channel_backward(const Channel& p, void*, hipStream_t stream) {
  return by_form(p, [&](auto io, auto g, auto logit, auto comp) {
    hipLaunchKernelGGL((channel_backward_kernel<io.value, g.value, logit.value, comp.value>), grid(p),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
  });
}

}  // namespace gdr
