// norm.hip -- the norms around a block with its gate and scaled residual
// (gdr_block_norm in gdr.h), and their gradient, on gfx950.
//
// Both are streams: every operand is read once and every result written once,
// and a row stays in the registers of its threads between the sums.  TPR
// threads hold a row, E elements each; rows of up to 1024 values are summed
// inside a wave, longer ones across the waves of a workgroup.  The gradient
// runs a fixed number of workgroups over the rows, so that each thread keeps
// the weight gradients of its columns in registers; one workgroup's sums go to
// the workspace and a second kernel adds them in order.
//
// TPR and E: eight consecutive elements a thread (16-byte accesses of bf16) as
// long as a row then fits 64 threads, sixteen up to 1024 values, so that its sums
// need no barrier; longer rows take 256 threads up to 4096 values and 1024 beyond,
// where a wave's registers would not hold the row.
#include <type_traits>

#include "gdr_device.h"
#include "norm.h"

namespace gdr {
namespace {

// Row layout: D % 8 == 0 gives each thread pieces of 8 consecutive elements
// (16-byte accesses), other D single elements TPR apart.
template <int TPR>
__device__ __forceinline__ int element(int i, int t, bool vec) {
  return vec ? ((i >> 3) * TPR + t) * 8 + (i & 7) : i * TPR + t;
}

template <Dt IN, int TPR, int E>
__device__ __forceinline__ void load_row(const void* base, size_t row, int D, int t, bool vec,
                                         float (&out)[E]) {
  const size_t at = row * D;
  if (vec) {
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const int c = (j * TPR + t) * 8;
      float x[8];
      if (c < D) {
        load_vec<IN, 8>(base, at + c, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) out[8 * j + e] = x[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = i * TPR + t;
      out[i] = c < D ? load_scalar<IN>(base, at + c) : 0.f;
    }
  }
}

template <int TPR, int E>
__device__ __forceinline__ void load_weight(const void* w, int dtype, int D, int t, bool vec,
                                            float (&out)[E]) {
  if (dtype == 0) load_row<Dt::BF16, TPR, E>(w, 0, D, t, vec, out);
  else load_row<Dt::F32, TPR, E>(w, 0, D, t, vec, out);
}

template <bool STREAM, class V>
__device__ __forceinline__ void put(V* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// STREAM: past the caches (vectors only).
template <int TPR, int E, bool STREAM = false>
__device__ __forceinline__ void store_row(void* base, int dtype, size_t row, int D, int t, bool vec,
                                          const float (&x)[E]) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const size_t at = row * D;
  if (vec) {
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const int c = (j * TPR + t) * 8;
      if (c >= D) continue;
      if (dtype == 0) {
        f32x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x[8 * j + e];
        put<STREAM>(reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at + c),
                    __builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8)));
      } else {
        floatx4* p = reinterpret_cast<floatx4*>(static_cast<float*>(base) + at + c);
        put<STREAM>(p, floatx4{x[8 * j], x[8 * j + 1], x[8 * j + 2], x[8 * j + 3]});
        put<STREAM>(p + 1, floatx4{x[8 * j + 4], x[8 * j + 5], x[8 * j + 6], x[8 * j + 7]});
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = i * TPR + t;
      if (c >= D) continue;
      if (dtype == 0) store_scalar<Dt::BF16>(base, at + c, x[i]);
      else store_scalar<Dt::F32>(base, at + c, x[i]);
    }
  }
}

// Sum of x over the TPR threads of a row, the same bits in each of them.  Rows
// of several waves go through LDS; two slots alternate, so that one barrier a
// sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float (*lds)[16], int& slot) {
  constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int s = 1; s < W; s <<= 1) x += __shfl_xor(x, s);
  if constexpr (TPR > 64) {
    slot ^= 1;
    if ((threadIdx.x & 63) == 0) lds[slot][threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) x += lds[slot][i];
  }
  return x;
}

// 1 / (1 + e^-z) by the hardware's base-2 exponential and reciprocal (one unit in
// the last place each; e^-z may overflow to infinity: 0).
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// s = sigmoid(z) and 1 - s = sigmoid(-z), both from e^-|z|: 1 - s of a rounded s
// loses the slope of open gates (6% of it at z = 16, all from 17.4 on).
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid_and_rest(float z) {
  const float a = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(z));
  const float r = __builtin_amdgcn_rcpf(1.f + a), b = a * r;
  return z < 0.f ? Sigmoid{b, r} : Sigmoid{r, b};
}

// A row's operands as loaded, for 16-byte accesses: the next row's are read while
// one is computed.
template <Dt IN, int E>
struct RawRow {
  static constexpr int N = E / 8 * (IN == Dt::BF16 ? 1 : 2);
  uint4 v[N];
};
template <Dt IN, int TPR, int E>
__device__ __forceinline__ void load_raw(const void* base, size_t row, int D, int t, RawRow<IN, E>& r) {
  constexpr int PER = IN == Dt::BF16 ? 1 : 2;
  const char* p = static_cast<const char*>(base) + row * D * (IN == Dt::BF16 ? 2 : 4);
#pragma unroll
  for (int j = 0; j < E / 8; ++j) {
    const int c = (j * TPR + t) * 8;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      r.v[PER * j + i] = c < D ? reinterpret_cast<const uint4*>(p + c * (PER == 1 ? 2 : 4))[i]
                               : make_uint4(0, 0, 0, 0);
  }
}
template <Dt IN, int E>
__device__ __forceinline__ void widen(const RawRow<IN, E>& r, float (&x)[E]) {
#pragma unroll
  for (int j = 0; j < RawRow<IN, E>::N; ++j) {
    const uint32_t w[4] = {r.v[j].x, r.v[j].y, r.v[j].z, r.v[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (IN == Dt::BF16) {
        x[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
        x[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        x[4 * j + i] = __uint_as_float(w[i]);
      }
    }
  }
}

// Largest of x over the 16 (8 with HALF) consecutive lanes that share a scale, in each
// of them: partners as in row16_sum.
template <bool HALF>
__device__ __forceinline__ float block_max(float x) {
  auto with = [&](auto ctrl) {
    x = fmaxf(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                     0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, true)));
  };
  with(std::integral_constant<int, 0xB1>());
  with(std::integral_constant<int, 0x4E>());
  with(std::integral_constant<int, 0x141>());
  if constexpr (!HALF) with(std::integral_constant<int, 0x128>());
  return x;
}

// A row as e4m3 with one scale for each 128 values: 16 threads' pieces of 8 (rows of up
// to 64 values: all 8 threads of the row).  The quotient is a product with 448 / max,
// which the conversion rounds once more: a value within 2^-23 of the middle between two
// e4m3 numbers may take the other one.  The largest becomes 448 (1 + 2^-23) at most and
// rounds to 448, so nothing needs a clamp, which would lose a NaN.  Residual and norm of 16384
// x 2048 bf16: 45.8 us, 5.1 TB/s, the rate of a copy; what a row is written as costs nothing.
template <int TPR, int E>
__device__ __forceinline__ void store_row8(void* y8, float* y_scale, size_t row, int D, int t,
                                           const float (&x)[E]) {
  const size_t blocks = static_cast<size_t>(D + 127) / 128;
#pragma unroll
  for (int j = 0; j < E / 8; ++j) {
    const int c = (j * TPR + t) * 8;
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[8 * j + e]));
    top = block_max<TPR == 8>(top);
    const bool some = !(top < 0x1p-100f);
    const float f = some ? 448.f / top : 0.f;
    if (c >= D) continue;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* v = x + 8 * j + 4 * i;
      int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * f, v[1] * f, 0, false);
      w[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * f, v[3] * f, q, true));
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(y8) + row * D + c) = make_uint2(w[0], w[1]);
    if (c % 128 == 0) y_scale[row * blocks + c / 128] = some ? top / 448.f : 0.f;
  }
}

// 262144 rows of 128, bf16, gate: 39.3 us, 5.1 TB/s, the rate of a copy of this size
// (two rows a thread, loaded together: 43.7); 64 rows of 2048 with both norms: 9 us,
// a launch.
template <Dt IN, int TPR, int E, bool vec, bool Q8>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_kernel(BlockNorm p) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, RPB = THREADS / TPR;
  __shared__ float lds[2][16];
  int slot = 0;
  const int t = threadIdx.x % TPR;
  const float inv_d = 1.f / static_cast<float>(p.D);
  const size_t row = static_cast<size_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  // (rows of several waves have a workgroup each: no barrier is missed)
  if (row >= static_cast<size_t>(p.rows)) return;
  float x[E], z[E], r[E], wa[E], wb[E];
  load_row<IN, TPR, E>(p.x, row, p.D, t, vec, x);
  if (p.gate) load_row<IN, TPR, E>(p.gate, row, p.D, t, vec, z);
  if (p.residual) load_row<IN, TPR, E>(p.residual, row, p.D, t, vec, r);
  if (p.w_after) load_weight<TPR, E>(p.w_after, p.w_dtype, p.D, t, vec, wa);
  if (p.w_before) load_weight<TPR, E>(p.w_before, p.w_dtype, p.D, t, vec, wb);
  if (p.w_after) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
    const float inv = rsqrtf(row_sum<TPR>(ss, lds, slot) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = x[i] * inv * wa[i];
  }
  if (p.gate) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] *= sigmoid(z[i]) * (p.act == 0 ? z[i] : 1.f);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = p.residual ? fmaf(p.scale, x[i], r[i]) : p.scale * x[i];
  if (p.w_before) {
    float y[E];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
    const float inv = rsqrtf(row_sum<TPR>(ss, lds, slot) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = x[i] * inv * wb[i];
    if constexpr (Q8) store_row8<TPR, E>(p.y8, p.y_scale, row, p.D, t, y);
    else store_row<TPR, E>(p.y, p.out_dtype, row, p.D, t, vec, y);
  } else if constexpr (Q8) {
    store_row8<TPR, E>(p.y8, p.y_scale, row, p.D, t, x);
  }
  if (p.h) store_row<TPR, E>(p.h, p.out_dtype, row, p.D, t, vec, x);
}

// Eight streams of rows (x, gate, residual, dh, dy; dx, dgate, dresidual): 16384
// rows of 2048, bf16, 112 us with the sum of the weights' gradients, 4.8 TB/s.  The
// next row's reads are in flight while one is computed (205 us without), and stores go
// past the caches, whose lines the reads want (114 through them, 76 against 72 at
// 262144 x 128; fp32 rows of 2048 are the exception, 215 through them and 235 past them.
// The forward kernel, one pass and one or two stores, is 2% faster through them).
//
// Every optional operand is a run-time branch, so that all of them have registers at
// once.  bf16 rows of up to 512 values are asked to fit four waves a SIMD all the same
// and spill 58 registers, most of them of operands that a call does not have: 262144
// rows of 128 with norm and gate take 74 us, 83 without the request; 131072 rows with
// all operands 66 us with it and without.  Rows of 256 threads are not asked to: they
// would spill 23 (16384 rows of 2048, norm and gate: 95 us, 87 without).  Rows of more
// than 8192 values, whose 1024 threads have 128 registers at most, spill 256 to 275:
// right, but slower.
template <Dt IN, int TPR, int E, bool vec>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256,
                             IN == Dt::BF16 && TPR <= 64 && E == 8 ? 4 : 1)
void block_norm_backward_kernel(BlockNorm p) {
  constexpr int THREADS = TPR > 256 ? TPR : 256, RPB = THREADS / TPR;
  __shared__ float lds[2][16];
  int slot = 0;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv_d = 1.f / static_cast<float>(p.D);
  float wa[E], wb[E], ga[E], gb[E];
#pragma unroll
  for (int i = 0; i < E; ++i) wa[i] = wb[i] = ga[i] = gb[i] = 0.f;
  if (p.w_after) load_weight<TPR, E>(p.w_after, p.w_dtype, p.D, t, vec, wa);
  if (p.w_before) load_weight<TPR, E>(p.w_before, p.w_dtype, p.D, t, vec, wb);
  const size_t rows = static_cast<size_t>(p.rows), step = static_cast<size_t>(gridDim.x) * RPB;
  size_t row = static_cast<size_t>(blockIdx.x) * RPB + sub;
  // (rows of 1024 threads have no registers left for it)
  constexpr bool AHEAD = vec && TPR <= 256;
  RawRow<IN, E> nx, nz, nd, nr, ny;
  auto read = [&](size_t at) {
    if (!AHEAD || at >= rows) return;
    load_raw<IN, TPR, E>(p.x, at, p.D, t, nx);
    if (p.gate) load_raw<IN, TPR, E>(p.gate, at, p.D, t, nz);
    if (p.dh) load_raw<IN, TPR, E>(p.dh, at, p.D, t, nd);
    if (p.w_before) load_raw<IN, TPR, E>(p.dy, at, p.D, t, ny);
    if (p.w_before && p.residual) load_raw<IN, TPR, E>(p.residual, at, p.D, t, nr);
  };
  read(row);
  for (; row < rows; row += step) {
    float x[E], z[E], d[E], h[E], dy[E];
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = h[i] = 0.f;
    if constexpr (AHEAD) {
      widen<IN, E>(nx, x);
      if (p.gate) widen<IN, E>(nz, z);
      if (p.dh) widen<IN, E>(nd, d);
      if (p.w_before) widen<IN, E>(ny, dy);
      if (p.w_before && p.residual) widen<IN, E>(nr, h);
      read(row + step);
    } else {
      load_row<IN, TPR, E>(p.x, row, p.D, t, vec, x);
      if (p.gate) load_row<IN, TPR, E>(p.gate, row, p.D, t, vec, z);
      if (p.dh) load_row<IN, TPR, E>(p.dh, row, p.D, t, vec, d);
      if (p.w_before) load_row<IN, TPR, E>(p.dy, row, p.D, t, vec, dy);
      if (p.w_before && p.residual) load_row<IN, TPR, E>(p.residual, row, p.D, t, vec, h);
    }
    float ix = 1.f;
    if (p.w_after) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
      ix = rsqrtf(row_sum<TPR>(ss, lds, slot) * inv_d + p.eps);
    }
    if (p.w_before) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        float u = p.w_after ? x[i] * ix * wa[i] : x[i];
        if (p.gate) u *= sigmoid(z[i]) * (p.act == 0 ? z[i] : 1.f);
        h[i] = fmaf(p.scale, u, h[i]);
        ss = fmaf(h[i], h[i], ss);
      }
      const float ih = rsqrtf(row_sum<TPR>(ss, lds, slot) * inv_d + p.eps);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        h[i] *= ih;
        gb[i] = fmaf(dy[i], h[i], gb[i]);
        dy[i] *= wb[i];
        dot = fmaf(dy[i], h[i], dot);
      }
      dot = row_sum<TPR>(dot, lds, slot) * inv_d;
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = fmaf(ih, fmaf(-h[i], dot, dy[i]), d[i]);
    }
    if (p.dresidual) store_row<TPR, E, true>(p.dresidual, p.out_dtype, row, p.D, t, vec, d);
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] *= p.scale;
    if (p.gate) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float n = p.w_after ? x[i] * ix * wa[i] : x[i];
        const Sigmoid g = sigmoid_and_rest(z[i]);
        const float slope = g.s * (p.act == 0 ? fmaf(z[i], g.rest, 1.f) : g.rest);
        const float a = p.act == 0 ? g.s * z[i] : g.s;
        z[i] = d[i] * n * slope;
        d[i] *= a;
      }
      if (p.dgate) store_row<TPR, E, true>(p.dgate, p.out_dtype, row, p.D, t, vec, z);
    }
    if (p.w_after) {
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        x[i] *= ix;
        ga[i] = fmaf(d[i], x[i], ga[i]);
        d[i] *= wa[i];
        dot = fmaf(d[i], x[i], dot);
      }
      dot = row_sum<TPR>(dot, lds, slot) * inv_d;
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = ix * fmaf(-x[i], dot, d[i]);
    }
    store_row<TPR, E, true>(p.dx, p.out_dtype, row, p.D, t, vec, d);
  }
  // this workgroup's weight gradients: rows of one column added in order
  __shared__ float cols[RPB > 1 ? THREADS * E : 1];
  auto partial = [&](const float (&g)[E], float* to) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) cols[(sub * TPR + t) * E + i] = g[i];
      __syncthreads();
      for (int i = threadIdx.x; i < TPR * E; i += THREADS) {
        float sum = 0.f;
        for (int s = 0; s < RPB; ++s) sum += cols[s * TPR * E + i];
        const int c = element<TPR>(i % E, i / E, vec);
        if (c < p.D) to[static_cast<size_t>(blockIdx.x) * p.D + c] = sum;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = element<TPR>(i, t, vec);
        if (c < p.D) to[static_cast<size_t>(blockIdx.x) * p.D + c] = g[i];
      }
    }
  };
  if (p.part_after) partial(ga, p.part_after);
  if (p.part_before) partial(gb, p.part_before);
}

// dw[c] = sum over the workgroups' rows of part[., c]: 16 columns a workgroup, 64
// threads to a column with 16 loads each in flight, so that 1024 rows are one round.
// 1024 x 2048 twice: 7.0 us (12.2 with 32 columns a workgroup and four loads in
// flight); a launch and one read of memory.
constexpr int kColumns = 16;
__global__ __launch_bounds__(1024) void block_norm_weights_kernel(const float* pa, const float* pb,
                                                                  float* dwa, float* dwb, int parts,
                                                                  int D) {
  const float* part = blockIdx.y == 0 ? pa : pb;
  float* dw = blockIdx.y == 0 ? dwa : dwb;
  if (!dw) return;
  __shared__ float lds[16][kColumns];
  const int cc = threadIdx.x % kColumns, rr = threadIdx.x / kColumns, c = blockIdx.x * kColumns + cc;
  float sum = 0.f;
  if (c < D)
    for (int i0 = rr; i0 < parts; i0 += 1024) {
      float x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int i = i0 + 64 * j;
        x[j] = i < parts ? part[static_cast<size_t>(i) * D + c] : 0.f;
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1)
#pragma unroll
        for (int j = 0; j < d; ++j) x[j] += x[j + d];
      sum += x[0];
    }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if ((threadIdx.x & 63) < kColumns) lds[threadIdx.x >> 6][cc] = sum;
  __syncthreads();
  if (rr == 0 && c < D) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) all += lds[i][cc];
    dw[c] = all;
  }
}

// Calls go(TPR, E) for a row of D values.
template <class F>
hipError_t by_width(int D, F&& go) {
  using std::integral_constant;
#define GDR_WIDTH(most, tpr, e) \
  if (D <= most) return go(integral_constant<int, tpr>(), integral_constant<int, e>())
  GDR_WIDTH(64, 8, 8);
  GDR_WIDTH(128, 16, 8);
  GDR_WIDTH(256, 32, 8);
  GDR_WIDTH(512, 64, 8);
  GDR_WIDTH(1024, 64, 16);
  GDR_WIDTH(2048, 256, 8);
  GDR_WIDTH(4096, 256, 16);
  GDR_WIDTH(8192, 1024, 8);
  return go(integral_constant<int, 1024>(), integral_constant<int, 16>());
#undef GDR_WIDTH
}

// Rows held at once by a workgroup of by_width's shape.
int rows_per_block(int D) { return D <= 64 ? 32 : D <= 128 ? 16 : D <= 256 ? 8 : D <= 1024 ? 4 : 1; }

}  // namespace

// Workgroups of the gradient: as many as a compute unit's registers hold at once, four
// of rows inside a wave (up to 1024 values), two of rows of 256 threads and one of rows
// of 1024 threads.  262144 rows of 128, bf16, norm and gate: 72 us with 1024 workgroups,
// 78 with 512, 74 with 2048.  All operands: 16384 rows of 2048 112 us with 512, 116 with
// 768, 138 with 1024, 128 with 2048; 8192 rows of 4096 119 with 512, 132 with 768, 131
// with 1024; 4096 rows of 8192 159 with 256, 205 with 1024.
int block_norm_backward_blocks(int64_t rows, int D) {
  const int64_t rpb = rows_per_block(D), n = (rows + rpb - 1) / rpb;
  const int64_t most = D <= 1024 ? 1024 : D <= 4096 ? 512 : 256;
  return static_cast<int>(n < most ? n : most);
}

hipError_t launch_block_norm(const BlockNorm& p, hipStream_t stream) {
  const int64_t rpb = rows_per_block(p.D);
  return by_width(p.D, [&](auto tpr, auto el) {
    constexpr int T = decltype(tpr)::value, E = decltype(el)::value;
    auto go = [&](auto in, auto vec) {
      hipLaunchKernelGGL((block_norm_kernel<decltype(in)::value, T, E, decltype(vec)::value, false>),
                         dim3(static_cast<unsigned>((p.rows + rpb - 1) / rpb)), dim3(T > 256 ? T : 256),
                         0, stream, p);
      return hipGetLastError();
    };
    const std::integral_constant<Dt, Dt::BF16> bf16;
    const std::integral_constant<Dt, Dt::F32> f32;
    if (p.D % 8 == 0) return p.in_dtype == 0 ? go(bf16, std::true_type()) : go(f32, std::true_type());
    return p.in_dtype == 0 ? go(bf16, std::false_type()) : go(f32, std::false_type());
  });
}

hipError_t launch_block_norm8(const BlockNorm& p, hipStream_t stream) {
  const int64_t rpb = rows_per_block(p.D);
  return by_width(p.D, [&](auto tpr, auto el) {
    constexpr int T = decltype(tpr)::value, E = decltype(el)::value;
    auto go = [&](auto in) {
      hipLaunchKernelGGL((block_norm_kernel<decltype(in)::value, T, E, true, true>),
                         dim3(static_cast<unsigned>((p.rows + rpb - 1) / rpb)), dim3(T > 256 ? T : 256),
                         0, stream, p);
      return hipGetLastError();
    };
    return p.in_dtype == 0 ? go(std::integral_constant<Dt, Dt::BF16>())
                           : go(std::integral_constant<Dt, Dt::F32>());
  });
}

hipError_t launch_block_norm_backward(const BlockNorm& p, float* dw_after, float* dw_before,
                                      hipStream_t stream) {
  const int blocks = block_norm_backward_blocks(p.rows, p.D);
  if (blocks > 0) {
    const hipError_t e = by_width(p.D, [&](auto tpr, auto el) {
      constexpr int T = decltype(tpr)::value, E = decltype(el)::value;
      auto go = [&](auto in, auto vec) {
        hipLaunchKernelGGL((block_norm_backward_kernel<decltype(in)::value, T, E, decltype(vec)::value>),
                           dim3(blocks), dim3(T > 256 ? T : 256), 0, stream, p);
        return hipGetLastError();
      };
      const std::integral_constant<Dt, Dt::BF16> bf16;
      const std::integral_constant<Dt, Dt::F32> f32;
      if (p.D % 8 == 0) return p.in_dtype == 0 ? go(bf16, std::true_type()) : go(f32, std::true_type());
      return p.in_dtype == 0 ? go(bf16, std::false_type()) : go(f32, std::false_type());
    });
    if (e != hipSuccess) return e;
  }
  if (!dw_after && !dw_before) return hipSuccess;
  hipLaunchKernelGGL(block_norm_weights_kernel, dim3((p.D + kColumns - 1) / kColumns, 2),
                     dim3(1024), 0, stream, p.part_after, p.part_before, dw_after, dw_before,
                     blocks, p.D);
  return hipGetLastError();
}

}  // namespace gdr
