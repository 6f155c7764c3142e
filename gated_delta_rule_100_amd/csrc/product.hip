// product.hip -- the product in 8 bits with a scale for each block of 128 (gdr_product8
// in gdr.h) on gfx950.
//
// out[m][n] = sum_b (sa[m][b] sw[n/128][b]) sum_{k in b} a[m][k] w[n][k].  The inner sum of
// a 16 x 16 tile is one matrix instruction (16x16x128) from zero, so a block's scales meet
// its sum in fp32 outside: four multiply-adds a lane for each instruction, which other
// waves' matrix instructions cover.  w takes the instruction's rows and a its columns, so
// that a lane has one row m, whose scale is one number, and four consecutive n.
//
// Lane (c = lane % 16, q = lane / 16) gives 16 bytes at k = 16 q and 16 at k = 64 + 16 q of
// its row of w and of a: any order of k is right that both have.
#include <type_traits>

#include "gdr_device.h"
#include "product.h"

namespace gdr {
namespace {

typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;

// A lane's 32 values of a row, as the matrix instructions take them.
template <Dt OUT>
struct Frag;

// bf16 results: the 8-bit instruction.  It adds the products of 8 consecutive k aligned to
// the largest of them, in multiples of 2^-13 of its power of two, and everything else in
// fp32: 1.5e-5 of normal data's sums, a hundredth of what rounding to bf16 takes.
template <>
struct Frag<Dt::BF16> {
  intx8 x;
  __device__ __forceinline__ void set(intx8 v) { x = v; }
};
__device__ __forceinline__ floatx4 block_sum(const Frag<Dt::BF16>& w, const Frag<Dt::BF16>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.x, a.x, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                          0, 0, 0);
}

// fp32 results: the same values as fp16 numbers, which hold them, and fp32 sums throughout,
// at half the rate.
template <>
struct Frag<Dt::F32> {
  halfx8 x[4];
  __device__ __forceinline__ void set(intx8 v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const halfx2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[i], 1.f, false);
      const halfx2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[i], 1.f, true);
      x[i / 2][4 * (i & 1) + 0] = lo[0];
      x[i / 2][4 * (i & 1) + 1] = lo[1];
      x[i / 2][4 * (i & 1) + 2] = hi[0];
      x[i / 2][4 * (i & 1) + 3] = hi[1];
    }
  }
};
__device__ __forceinline__ floatx4 block_sum(const Frag<Dt::F32>& w, const Frag<Dt::F32>& a) {
  floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.x[i], a.x[i], s, 0, 0, 0);
  return s;
}

__device__ __forceinline__ intx8 join(intx4 lo, intx4 hi) {
  return intx8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// Four consecutive outputs of a row, of which `some` exist.
template <Dt OUT>
__device__ __forceinline__ void store4(void* out, size_t at, int some, bool vec, floatx4 x) {
  if (vec && some >= 4) {
    if constexpr (OUT == Dt::F32) {
      *reinterpret_cast<floatx4*>(static_cast<float*>(out) + at) = x;
    } else {
      const uint32_t lo = f32_to_bf16_bits(x[0]) | static_cast<uint32_t>(f32_to_bf16_bits(x[1])) << 16;
      const uint32_t hi = f32_to_bf16_bits(x[2]) | static_cast<uint32_t>(f32_to_bf16_bits(x[3])) << 16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(lo, hi);
    }
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < some) store_scalar<OUT>(out, at + r, x[r]);
  }
}

// 16 or 4 bytes a lane from memory to consecutive LDS.
__device__ __forceinline__ void copy16(const void* src, void* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src),
                                   (__attribute__((address_space(3))) void*)(lds), 16, 0, 0);
}
__device__ __forceinline__ void copy4(const void* src, void* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src),
                                   (__attribute__((address_space(3))) void*)(lds), 4, 0, 0);
}

// Tile (im, in) of the grid's tm x tn for workgroup `id`: workgroups go round the 8 XCDs,
// so each XCD gets a run of tiles of its own, which walks groups of 8 rows of tiles, and
// the tiles of one moment share rows of a and w in its L2.
__device__ __forceinline__ void tile_of(int id, int tm, int tn, int* im, int* in) {
  const int total = tm * tn, each = total / 8, more = total % 8, x = id % 8;
  const int at = x * each + (x < more ? x : more) + id / 8;
  const int group = at / (8 * tn), rows = min(8, tm - group * 8), rest = at - group * 8 * tn;
  *im = group * 8 + rest % rows;
  *in = rest / rows;
}

// A BM x BN tile by WM x WN waves.  Blocks of 128 k of both operands go through LDS,
// straight from memory, one while the one before it is multiplied.  A row of a block is
// 8 pieces of 16 bytes, piece c at c ^ (row / 2 % 8): the 16 rows that lanes read at once
// then fall on all banks.
template <Dt OUT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 2) void product8_tile_kernel(Product8 p, int tm, int tn) {
  constexpr int WAVES = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  static_assert(kBlock % (BN / WN) == 0, "a wave's columns share a scale");
  constexpr int COPIES = (BM + BN) / 8 / WAVES;  // of 8 rows, a wave
  static_assert(COPIES * WAVES * 8 == BM + BN && BM % 8 == 0, "copies");
  struct Stage {
    uint8_t rows[BN + BM][kBlock];  // w, then a
    float sa[BM < 64 ? 64 : BM];
  };
  __shared__ Stage stage[2];
  int im, in;
  tile_of(blockIdx.x, tm, tn, &im, &in);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, c16 = lane & 15, q = lane >> 4;
  const int m0 = im * BM, n0 = in * BN, kb = (p.K + kBlock - 1) / kBlock;
  const uint8_t* a0 = p.a + static_cast<size_t>(m0) * p.K;
  const uint8_t* w0 = p.w + static_cast<size_t>(n0) * p.K;
  // bytes from a tile's first row to what this lane copies; rows past the end are the last
  uint32_t from[COPIES];
  int piece[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    const int g = i * WAVES + wave, r = g * 8 + (lane >> 3);
    piece[i] = (lane & 7) ^ (r >> 1 & 7);
    const int row = g < BN / 8 ? min(r, p.N - 1 - n0) : min(r - BN, p.M - 1 - m0);
    from[i] = static_cast<uint32_t>(row) * p.K + piece[i] * 16;
  }
  const int sm = min(wave * 64 + lane, min(BM - 1, p.M - 1 - m0));
  const float* sa0 = p.a_scale + static_cast<size_t>(m0 + sm) * kb;
  const float* sw0 = p.w_scale + static_cast<size_t>(min(n0 + wn * (BN / WN), p.N - 1) / kBlock) * kb;
  const auto issue = [&](int b) {
    Stage& s = stage[b & 1];
    const bool whole = (b + 1) * kBlock <= p.K;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int g = i * WAVES + wave;
      const uint8_t* src = (g < BN / 8 ? w0 : a0) + static_cast<size_t>(b) * kBlock;
      if (whole) {
        copy16(src + from[i], s.rows[g * 8]);
      } else {  // the last block: zeros behind the rows' end
        intx4 x = {0, 0, 0, 0};
        if (b * kBlock + piece[i] * 16 < p.K) x = *reinterpret_cast<const intx4*>(src + from[i]);
        *reinterpret_cast<intx4*>(&s.rows[g * 8][0] + lane * 16) = x;
      }
    }
    if (wave * 64 < BM) copy4(sa0 + b, s.sa + wave * 64);
  };
  floatx4 acc[MT][NT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int near = c16 * kBlock + ((q ^ (c16 >> 1)) * 16), far = near ^ 64;
  issue(0);
  float next_sw = sw0[0];
  for (int b = 0; b < kb; ++b) {
    const float sw = next_sw;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (b + 1 < kb) {
      next_sw = sw0[b + 1];
      issue(b + 1);
    }
    const Stage& s = stage[b & 1];
    const uint8_t* wr = s.rows[wn * (BN / WN)];
    const uint8_t* ar = s.rows[BN + wm * (BM / WM)];
    const auto read = [&](const uint8_t* rows, int t) {
      return join(*reinterpret_cast<const intx4*>(rows + t * 16 * kBlock + near),
                  *reinterpret_cast<const intx4*>(rows + t * 16 * kBlock + far));
    };
    Frag<OUT> wf[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wf[i].set(read(wr, i));
    float scale[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) scale[j] = s.sa[wm * (BM / WM) + j * 16 + c16] * sw;
    floatx4 part[2][NT];
#pragma unroll
    for (int j = 0; j <= MT; ++j) {
      if (j < MT) {
        Frag<OUT> af;
        af.set(read(ar, j));
#pragma unroll
        for (int i = 0; i < NT; ++i) part[j & 1][i] = block_sum(wf[i], af);
      }
      if (j > 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[j - 1][i][r] = fmaf(scale[j - 1], part[(j - 1) & 1][i][r], acc[j - 1][i][r]);
      }
    }
  }
  const bool vec = p.N % 4 == 0;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = m0 + wm * (BM / WM) + j * 16 + c16;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int n = n0 + wn * (BN / WN) + i * 16 + 4 * q;
      if (n < p.N) store4<OUT>(p.out, static_cast<size_t>(m) * p.N + n, p.N - n, vec, acc[j][i]);
    }
  }
}

// Few rows: up to 16 MT of a against 16 NT of w, whose bytes come straight from memory to
// the matrix instructions' registers.  The waves take every kWaves-th block of k and add up
// in LDS at the end.
constexpr int kWaves = 8;
template <Dt OUT, int MT, int NT>
__global__ __launch_bounds__(kWaves * 64) void product8_rows_kernel(Product8 p) {
  __shared__ floatx4 sums[kWaves][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * MT * 16, n0 = blockIdx.x * NT * 16, kb = (p.K + kBlock - 1) / kBlock;
  const uint8_t *ar[MT], *wr[NT];
  const float* sa[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = min(m0 + j * 16 + c16, p.M - 1);
    ar[j] = p.a + static_cast<size_t>(m) * p.K + q * 16;
    sa[j] = p.a_scale + static_cast<size_t>(m) * kb;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) wr[i] = p.w + static_cast<size_t>(min(n0 + i * 16 + c16, p.N - 1)) * p.K + q * 16;
  const float* sw = p.w_scale + static_cast<size_t>(n0 / kBlock) * kb;
  struct Block {
    intx8 w[NT], a[MT];
    float scale[MT];
  };
  const auto read = [&](int b, Block& x) {
    const int64_t k = static_cast<int64_t>(b) * kBlock;
    const bool lo = k + q * 16 < p.K, hi = k + 64 + q * 16 < p.K;
    const auto row = [&](const uint8_t* r) {
      const intx4 zero = {0, 0, 0, 0};
      return join(lo ? *reinterpret_cast<const intx4*>(r + k) : zero,
                  hi ? *reinterpret_cast<const intx4*>(r + k + 64) : zero);
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) x.w[i] = row(wr[i]);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      x.a[j] = row(ar[j]);
      x.scale[j] = sa[j][b] * sw[b];
    }
  };
  floatx4 acc[MT][NT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  Block x, y;
  if (wave < kb) read(wave, x);
  for (int b = wave; b < kb; b += kWaves) {
    const bool more = b + kWaves < kb;
    if (more) read(b + kWaves, y);
    Frag<OUT> wf[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wf[i].set(x.w[i]);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      Frag<OUT> af;
      af.set(x.a[j]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const floatx4 part = block_sum(wf[i], af);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][i][r] = fmaf(x.scale[j], part[r], acc[j][i][r]);
      }
    }
    if (more) x = y;
  }
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NT; ++i) sums[wave][j * NT + i][lane] = acc[j][i];
  __syncthreads();
  const bool vec = p.N % 4 == 0;
  for (int t = wave; t < MT * NT; t += kWaves) {
    floatx4 x4 = sums[0][t][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v)
#pragma unroll
      for (int r = 0; r < 4; ++r) x4[r] += sums[v][t][lane][r];
    const int m = m0 + t / NT * 16 + c16, n = n0 + t % NT * 16 + 4 * q;
    if (m < p.M && n < p.N) store4<OUT>(p.out, static_cast<size_t>(m) * p.N + n, p.N - n, vec, x4);
  }
}

template <Dt OUT, int BM, int BN, int WM, int WN>
hipError_t launch_tiles(const Product8& p, hipStream_t stream) {
  const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  hipLaunchKernelGGL((product8_tile_kernel<OUT, BM, BN, WM, WN>), dim3(static_cast<unsigned>(tm) * tn),
                     dim3(WM * WN * 64), 0, stream, p, tm, tn);
  return hipGetLastError();
}

template <Dt OUT, int MT, int NT>
hipError_t launch_rows(const Product8& p, hipStream_t stream) {
  hipLaunchKernelGGL((product8_rows_kernel<OUT, MT, NT>),
                     dim3((p.N + NT * 16 - 1) / (NT * 16), (p.M + MT * 16 - 1) / (MT * 16)),
                     dim3(kWaves * 64), 0, stream, p);
  return hipGetLastError();
}

template <Dt OUT>
hipError_t launch(const Product8& p, hipStream_t stream) {
  const int64_t big = static_cast<int64_t>((p.M + 255) / 256) * ((p.N + 255) / 256);
  if (p.M <= 16) return p.N >= 8192 ? launch_rows<OUT, 1, 2>(p, stream) : launch_rows<OUT, 1, 1>(p, stream);
  if (p.M <= 32) return p.N >= 8192 ? launch_rows<OUT, 2, 2>(p, stream) : launch_rows<OUT, 2, 1>(p, stream);
  if (p.M <= 64) return p.N >= 8192 ? launch_rows<OUT, 4, 2>(p, stream) : launch_rows<OUT, 4, 1>(p, stream);
  // (fp32 results: the larger tile would spill registers)
  if constexpr (OUT == Dt::BF16)
    if (big >= 192) return launch_tiles<OUT, 256, 256, 2, 4>(p, stream);
  return launch_tiles<OUT, 128, 128, 2, 2>(p, stream);
}

}  // namespace

hipError_t launch_product8(const Product8& p, hipStream_t stream) {
  return p.out_dtype == 0 ? launch<Dt::BF16>(p, stream) : launch<Dt::F32>(p, stream);
}

}  // namespace gdr
