// linear.h -- host-side launchers of linear attention with a decay for each head
// (linear.hip): pointers and sizes are checked by linear_api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdr {

// Decays: one value for each token and head ([T, H]) or for each head ([H]).
struct LinearGates {
  const float* g;
  int per_token;
};

// A packed batch, and the units its passes walk: the sequences (seg == 0,
// units = N), or segments of seg tokens of them (launch_layout with seg as its
// chunk: seg_offs [N + 1], seg_idx [units][2], slots past the real count -1;
// NULL for at most kInlineSeqs sequences, where the kernels form the table).
constexpr int kInlineSeqs = 64;
struct LinearBatch {
  const int32_t* cu;
  int N, H, T_total, in_dtype;
  LinearGates gates;
  int seg, units;
  const int32_t *seg_offs, *seg_idx;
};

// One pass of the recurrence over every unit, in either direction.  With a
// state Z [od, kd] per (unit, head), rows x, y of kd and w of od values:
//   forward:   Z_t = alpha_t Z_{t-1} + us w_t y_t^T,  out_t = os Z_t x_t
//   backward:  Z_t = alpha_{t+1} Z_{t+1} + us w_t y_t^T,  out_t = os Z_t x_t
// The prompt pass is (x, y, w) = (q, k, v) forward; the gradients are
// dq: (do, v, k) forward, dv: (k, q, do) backward, dk: (v, do, q) backward.
// Head h reads head h / group of a tensor; a token's row starts at
// token * stride + head * width elements.
struct LinearRows {
  const void* p;
  int64_t stride;
  int group;
};

struct LinearPass {
  LinearRows x, y, w;
  LinearRows e;        // rows of od values to dot with the outputs (dot != NULL)
  void* out;           // [T, H, od]
  float* dot;          // [H][T] e_t . out_t without the token's own term, or NULL
  const float* start;  // [units * H] states the walks start from, NULL for zero
  float* end;          // [N * H] states where the last walk of a sequence ends,
                       // NULL: not written; not written for sequences without units
  const float* end_with;  // [units * H] states to dot with those at a walk's end, or NULL
  float* end_dot;         // [od / 16][units * H] partial sums of that dot product
  int64_t row, col;    // element strides of a state row and column, in start,
                       // end and end_with (od * kd elements a state)
  float us, os;
  int od, kd, backward, out_dtype;
};

hipError_t launch_linear_decode(const void* q, const void* k, const void* v,
                                const LinearGates& g, float* state, void* o, int N, int H, int Hk,
                                int dk, int dv, int64_t qs, int64_t ks, int64_t vs, float scale,
                                int in_dtype, int out_dtype, hipStream_t stream);

// A forward pass without dot products.
hipError_t launch_linear_prompt(const LinearBatch& b, const LinearPass& p, hipStream_t stream);

// The passes of a gradient: dq forwards, dv and dk backwards; dot products in both
// of the first two or in none.
hipError_t launch_linear_grads(const LinearBatch& b, const LinearPass& pq, const LinearPass& pv,
                               const LinearPass& pk, hipStream_t stream);

// States at the start of every segment's walk, [units * H] of od rows and kd
// columns: the segments' own states from zero (y, w, us as in a pass) and their
// decays [units * H], then the chain over each sequence's segments from `from`
// ([N * H], NULL for zero).  last ([N * H] or NULL) gets `from` where a sequence
// has no tokens.  One job forwards and, when given, one backwards.
struct LinearStates {
  LinearRows y, w;
  float us;
  const float* from;
  float *states, *decays, *last;
};
hipError_t launch_linear_starts(const LinearBatch& b, int od, int kd, const LinearStates& forward,
                                const LinearStates* backward, hipStream_t stream);

// dg_t = dg_{t+1} + row_t - col_t over every unit, from its end's dot product and
// back to its start's (NULL: zero); row and col are [H][T], start_dot and end_dot
// partial sums [parts][units * H].  dg_t goes to dg ([T, H]), or its sum
// over the unit's tokens to unit_sum ([units * H]).
hipError_t launch_linear_dg(const LinearBatch& b, const float* row, const float* col,
                            const float* start_dot, int start_parts, const float* end_dot,
                            int end_parts, float* dg, double* unit_sum, hipStream_t stream);

// dg[h] = sum over units of unit_sum.
hipError_t launch_linear_dg_heads(const LinearBatch& b, const double* unit_sum, float* dg,
                                  hipStream_t stream);

// Sums of two [T, H, d] fp32 tensors over groups of heads to [T, H / group, d] of
// out_dtype, for the tokens of the batch's sequences.
hipError_t launch_linear_group_sum(const LinearBatch& b, const float* part_q, const float* part_k,
                                   int group, int d, void* dq, void* dk, int out_dtype,
                                   hipStream_t stream);

}  // namespace gdr
