// channel.h -- host-side launchers of the recurrence with a decay for each channel
// (channel.hip): pointers and sizes are checked by channel_api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace gdr {

// Operands of gdr_channel_* (gdr.h); unused ones are NULL, strides are resolved.
struct Channel {
  const void *x, *g;
  const int32_t* cu;
  const float* state_in;  // decode: the state, read and written through state_out
  float* state_out;
  void* h;                // written by prefill and decode, read by the gradient
  const void* dh;
  const float* dstate_out;
  void *dx, *dg;
  float* dstate_in;
  int T, N, D;
  int64_t x_stride, g_stride;
  int gate, complement, io_dtype, g_dtype;
};

// Bytes that a pass over T tokens of D channels needs at most.
size_t channel_workspace_bytes(int T, int D);

hipError_t launch_channel_decode(const Channel& p, hipStream_t stream);
hipError_t launch_channel_prefill(const Channel& p, void* workspace, hipStream_t stream);
hipError_t launch_channel_backward(const Channel& p, void* workspace, hipStream_t stream);

}  // namespace gdr
