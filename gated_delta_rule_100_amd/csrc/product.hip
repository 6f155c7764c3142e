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
#include "product_lanes.h"

namespace gdr {
namespace {

typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

// f(0), f(1), ... with their arguments as constants (the loop is too long for the compiler
// to unroll).
template <int N, int I = 0, class F>
__device__ __forceinline__ void steps(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    steps<N, I + 1>(f);
  }
}

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

// Two tiles side by side (n = 4 q + r of each at lane q) as bf16, eight consecutive n of both
// together a lane: lane q has n = 8 q to 8 q + 7.  Halves of the wave change places, then its
// rows of 16 lanes; the lanes of one row m go the same way, so all of them are to be there.
__device__ __forceinline__ uintx4 pair_of_tiles(floatx4 a, floatx4 b) {
  const auto two = [](float lo, float hi) {
    typedef float floatx2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{lo, hi}), bf16x2));
  };
  const uint32_t x[2] = {two(a[0], a[1]), two(a[2], a[3])}, y[2] = {two(b[0], b[1]), two(b[2], b[3])};
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto h = __builtin_amdgcn_permlane32_swap(x[i], y[i], false, false);
    const auto r = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
    lo[i] = r[0];
    hi[i] = r[1];
  }
  return uintx4{lo[0], lo[1], hi[0], hi[1]};
}

// Four tiles side by side as bf16, a row's 128 bytes in eight lanes, rows 0 to 7 in `first` and
// 8 to 15 in `second`: lane c of 16 has row c % 8, and the second 64 bytes from c = 8 on.
// Stores of whole lines: 16384 x 8192 x 2048 takes 264 us with them, 277 with halves of lines
// that follow each other and 300 where the other columns' stores are between the halves.
__device__ __forceinline__ void lines_of_tiles(bool low, const floatx4* x, uintx4* first, uintx4* second) {
  const uintx4 left = pair_of_tiles(x[0], x[1]), right = pair_of_tiles(x[2], x[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t other = __builtin_amdgcn_update_dpp(0, low ? right[i] : left[i], 0x128, 0xf, 0xf, false);  // from lane c ^ 8
    (*first)[i] = low ? left[i] : other;
    (*second)[i] = low ? other : right[i];
  }
}

// 16 or 4 bytes a lane from memory, `off` behind a scalar base, to consecutive LDS.  The
// compiler would wait for the builtin's copy before every later read of LDS, of the other
// buffer too; written out, the copy has no register that it returns, and arrive() below is
// what waits for it.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)(p)));
}
template <int AT>
__device__ __forceinline__ void copy16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base),
               "i"(AT) : "m0", "scc");
}
__device__ __forceinline__ void copy4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base) : "m0");
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

// Tiles of BM x BN by WM x WN waves, in KG groups of them that take every KG-th block of 128 k
// and add up at a tile's end; a workgroup stays for every gridDim.x-th tile and takes the
// blocks of all of them as one sequence.  Blocks of both operands go through NB buffers of LDS
// a group, straight from memory.  A wave holds a block's rows of a in registers and passes
// over its rows of w; during the last pass it reads the next block's rows of a in the places
// of those that it has used, so the one barrier of a block stands before that pass, in the
// middle of products whose operands are there:
//   - behind the barrier the next block has landed, and nobody reads this one's buffer any
//     more: its copies for NB blocks on start;
//   - no product waits for LDS, and a tile's first products not for the stores of the tile
//     before it.
// A row of a block is 8 pieces of 16 bytes, piece c at c ^ (row / 2 % 8): the 16 rows that
// lanes read at once then fall on all banks.  The scales of a come 8 blocks at a time, since
// a row's are 32 bytes of one line then (a third of all L2 requests were for them, one by one).
//
// 256 x 256, bf16 results, 16384 x 8192 x 2048: 268 us, 2050 TFLOP/s; 8192 x 8192 x 8192: 450
// us, 2440 TFLOP/s.  What bounds it: a SIMD's two waves hardly issue more than their matrix
// instructions' time holds (4 multiply-adds behind each, the copies: the first 177 us become
// 214 with the copies, of 4 bytes as of 16 each), and at K = 2048 the results' 268 MB take 54
// us more, as if nothing ran beside them.  (348 us with the barrier between blocks, 280 with
// addresses formed for each copy.)
constexpr int kScales = 8;
template <Dt OUT, int BM, int BN, int WM, int WN, int KG, int NB>
__global__ __launch_bounds__(WM * WN * KG * 64, 2) void product8_tile_kernel(Product8 p, int tm, int tn) {
  constexpr int WAVES = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16, STEPS = MT * NT;
  static_assert(kBlock % (BN / WN) == 0, "a wave's columns share a scale");
  constexpr int COPIES = (BM + BN) / 8 / WAVES;  // of 8 rows, a wave
  constexpr int SCALES = BM * kScales / 64 / WAVES;
  static_assert(COPIES * WAVES * 8 == BM + BN && BN / 8 % WAVES == 0, "copies");
  static_assert(COPIES % 2 == 0, "copies in halves");
  static_assert(SCALES * WAVES * 64 == BM * kScales, "scales");
  static_assert(WAVES % 2 == 0, "a lane's piece");
  static_assert(KG == 1 || WAVES * 64 >= BM, "a lane's row of scales");
  static_assert(NT % 2 == 0, "rows of w in two places");
  __shared__ uint8_t all_rows[KG][NB][BN + BM][kBlock];  // of w, then of a
  __shared__ float all_scales[KG][NB][BM][kScales];
  __shared__ floatx4 sums[KG > 1 ? KG - 1 : 1][KG > 1 ? WAVES : 1][KG > 1 ? STEPS : 1][64];
  const int lane = threadIdx.x & 63, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = any_wave / WAVES, wave = any_wave % WAVES;
  const int wm = wave / WN, wn = wave % WN, c16 = lane & 15, q = lane >> 4;
  const int kb = (p.K + kBlock - 1) / kBlock, turns = (kb + KG - 1) / KG, tiles = tm * tn;
  auto& rows = all_rows[kg];
  auto& scales = all_scales[kg];
  // The lane for addresses that are needed once in a while: formed from it each time, they
  // take no registers in between.
  const auto anew = [&] {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };
  // A place in the sequence of blocks: tile and turn, and in LDS the offset of its buffer of
  // rows and of its scales.  Past the last tile the numbers stay those of the last.  What a
  // block does with scalars is kept to few instructions: two waves of a SIMD have no others
  // beside them, and each instruction takes as long from a wave as a multiply-add.
  constexpr uint32_t kRows = (BN + BM) * kBlock, kScale = BM * kScales * 4;
  struct Place {
    int tile, m0, n0, turn;
    uint32_t rows, scales;
  };
  const auto block = [&](const Place& c) { return c.turn * KG + kg; };
  const auto enter = [&](Place& c) {
    if (c.tile >= tiles) return;
    int im, in;
    tile_of(c.tile, tm, tn, &im, &in);
    c.m0 = im * BM;
    c.n0 = in * BN;
  };
  const bool ragged = p.K % (kBlock * KG) != 0;
  // Calls `turned` in a tile's next turn, `entered` in the first of another tile.
  const auto advance = [&](Place& c, auto turned, auto entered) {
    c.rows = c.rows + kRows == NB * kRows ? 0 : c.rows + kRows;
    c.scales += 4;
    if (++c.turn == turns) {
      c.turn = 0;
      c.tile += gridDim.x;
      enter(c);
      entered();
    } else {
      turned();
    }
    if (c.turn % kScales == 0) {  // a row's scales in the next buffer
      c.scales = (c.scales - 4) / kScale * kScale + kScale;
      if (c.scales == NB * kScale) c.scales = 0;
    }
  };
  // A lane copies the same piece of each row; rows past the end are the last.  Where a last
  // block has no such piece, it takes the row's first bytes of the block, and writes zeros
  // over them before they are read.  `to` is what is copied, from these addresses.
  const uint32_t piece = ((lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7)) * 16;
  const auto missing = [&](int b) { return b * kBlock + static_cast<int>(piece) >= p.K; };
  Place to{static_cast<int>(blockIdx.x), 0, 0, 0, 0, 0};
  const uint8_t *from_w, *from_a;
  uint32_t from[COPIES];
  constexpr int WCOPIES = BN / 8 / WAVES;
  // A tile's last block may be short, or not there at all.  (The lane's difference is formed
  // here: as a branch of the lane's own it would make the numbers of a Place the lane's.)
  const uint32_t lost = missing((turns - 1) * KG + kg) ? piece : 0;
  const auto last_turn = [&] {
    if (!ragged || to.turn != turns - 1) return;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) from[i] -= lost;
  };
  const auto aim = [&] {
    const int first = min(kg, kb - 1) * kBlock;
    from_w = p.w + static_cast<size_t>(to.n0) * p.K + first;
    from_a = p.a + static_cast<size_t>(to.m0) * p.K + first;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int r = (i * WAVES + wave) * 8 + (anew() >> 3);
      const int row = i < WCOPIES ? min(r, p.N - 1 - to.n0) : min(r - BN, p.M - 1 - to.m0);
      from[i] = static_cast<uint32_t>(row) * p.K + piece;
    }
    last_turn();
  };
  const auto advance_to = [&] {
    advance(to, [&] {
      if (block(to) < kb) {
        from_w += KG * kBlock;
        from_a += KG * kBlock;
      }
      last_turn();
    }, aim);
  };
  const uint32_t rows_lds = lds_address(rows[0][wave * 8]);
  const auto copy_rows = [&](auto copy) {
    constexpr int i = decltype(copy)::value;
    copy16<i * WAVES * 8 * kBlock>(i < WCOPIES ? from_w : from_a, from[i], rows_lds + to.rows);
  };
  const auto copy_scales = [&] {
    if (to.turn % kScales != 0) return;
#pragma unroll
    for (int i = 0; i < SCALES; ++i) {
      const int r = (i * WAVES + wave) * (64 / kScales), l = anew();
      const int m = min(r + l / kScales, p.M - 1 - to.m0), b = min(block(to) + l % kScales * KG, kb - 1);
      copy4(p.a_scale + static_cast<size_t>(to.m0) * kb, (static_cast<uint32_t>(m) * kb + b) * 4,
            lds_address(scales[0][r]) + to.scales);
    }
  };
  // Waits for this wave's LDS accesses and for all its memory accesses but the copies of the
  // NB - 2 blocks behind the next (scales among them only make it wait for more) and, where
  // they came last, a whole tile's stores; then for the other waves.
  constexpr int STORES = OUT == Dt::BF16 ? STEPS / 2 : STEPS, LATER = (NB - 2) * COPIES;
  static_assert(LATER + STORES < 64, "vmcnt");
  const auto arrive = [&](bool stores) {
    constexpr int all = LATER + STORES;
    asm volatile("" ::: "memory");
    if (stores) __builtin_amdgcn_s_waitcnt(0x0070 | (all & 15) | (all >> 4) << 14);
    else __builtin_amdgcn_s_waitcnt(0x0070 | (LATER & 15) | (LATER >> 4) << 14);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int near = c16 * kBlock + ((q ^ (c16 >> 1)) * 16), far = near ^ 64;
  const auto read = [&](const uint8_t* at, int t) {
    return join(*reinterpret_cast<const intx4*>(at + t * 16 * kBlock + near),
                *reinterpret_cast<const intx4*>(at + t * 16 * kBlock + far));
  };
  const uint8_t* const rows_of_w = rows[0][wn * (BN / WN)];
  const uint8_t* const rows_of_a = rows[0][BN + wm * (BM / WM)];
  const auto zero_missing = [&](uint32_t buffer) {
    const int l = anew();
#pragma unroll
    for (int i = 0; i < COPIES; ++i)
      *reinterpret_cast<intx4*>(&rows[0][(i * WAVES + wave) * 8][0] + buffer + l * 16) = intx4{0, 0, 0, 0};
  };
  // A group without a block in a tile's last turn has zeros for it, and the scales of the last
  // block that is there: they become zeros too, since an infinite one would make NaN of them.
  const auto without = [&](const Place& c) { return KG > 1 && block(c) >= kb; };
  const auto zero_scales = [&](const Place& c, float* scale_of_w) {
    const int r = wave * 64 + anew();
    if (r < BM) *reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(scales[0][r]) + c.scales) = 0.f;
    *scale_of_w = 0.f;
  };
  // A block's scales of this lane's rows of a, and the wave's scale of w.
  const uint8_t* const scales_of_a = reinterpret_cast<const uint8_t*>(scales[0][wm * (BM / WM) + c16]);
  const auto scale_of_a = [&](const Place& c, int j) {
    return *reinterpret_cast<const float*>(scales_of_a + c.scales + j * 16 * kScales * 4);
  };
  Place now = to, next = to;
  const float* scale_of_w;  // of `next`'s tile
  const auto aim_scale = [&] {
    scale_of_w = p.w_scale + static_cast<size_t>(min(next.n0 + wn * (BN / WN), p.N - 1) / kBlock) * kb;
  };
  const auto next_scale_of_w = [&] {  // (constant address space: a scalar load)
    return ((const __attribute__((address_space(4))) float*)(scale_of_w))[min(block(next), kb - 1)];
  };
  const auto advance_next = [&] { advance(next, [] {}, aim_scale); };

  // `to` is what is copied, `next` what is read, `now` what is multiplied
  constexpr int HALF = COPIES / 2;
  enter(to);
  aim();
  now = next = to;
  aim_scale();
  float sw = next_scale_of_w();
  advance_next();
#pragma unroll
  for (int d = 0; d < NB - 1; ++d) {
    copy_scales();
    steps<COPIES>(copy_rows);
    advance_to();
  }
  arrive(false);
  if (ragged && turns == 1) {
    if (missing(kg)) zero_missing(0);
    if (without(now)) zero_scales(now, &sw);
    arrive(false);
  }
  copy_scales();
  steps<HALF>(copy_rows);
  intx8 ar[MT], wr[2];
  float sa[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    ar[j] = read(rows_of_a, j);
    sa[j] = scale_of_a(now, j);
  }
  wr[0] = read(rows_of_w, 0);
  bool copied = false, stores = false;  // all of `to` is on its way; stores came after it
  while (now.tile < tiles) {
    floatx4 acc[MT][NT];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int m_at = now.m0, n_at = now.n0;
    int left = turns;
    do {
    float next_sw = 0.f;
    Frag<OUT> af[MT], wf;
    floatx4 part[4];
    float scale[MT];
    steps<STEPS + 3>([&](auto step) {
      constexpr int t = decltype(step)::value, i = t / MT, j = t % MT;
      if constexpr (t < STEPS) {
        if constexpr (j == 0) {
          // (in time for the wait behind it: while it is on its way, waits for LDS are waits
          // for everything)
          if constexpr (i == (NT > 2 ? 1 : 0)) next_sw = next_scale_of_w();
          if constexpr (i == NT - 1) {  // the next block has landed
            arrive(stores);
            if (ragged && next.turn == turns - 1) {
              if (missing(block(next))) zero_missing(next.rows);
              if (without(next)) zero_scales(next, &next_sw);
              lds_barrier();
            }
            advance_to();
            copy_scales();
          }
          wf.set(wr[i & 1]);
          wr[(i + 1) & 1] = i < NT - 1 ? read(rows_of_w + now.rows, i + 1) : read(rows_of_w + next.rows, 0);
        }
        if constexpr (i == 0) {
          af[j].set(ar[j]);
          scale[j] = sa[j] * sw;
        }
        part[t & 3] = block_sum(wf, af[j]);
        if constexpr (i == NT - 1) {
          ar[j] = read(rows_of_a + next.rows, j);
          sa[j] = scale_of_a(next, j);
        }
        // half of the copies in this pass, half in the next block's first
        steps<(j + 1) * HALF / MT - j * HALF / MT>([&](auto c) {
          constexpr int at = j * HALF / MT + decltype(c)::value;
          if constexpr (i == NT - 1) copy_rows(std::integral_constant<int, at>());
          if constexpr (i == 0)
            if (!copied) copy_rows(std::integral_constant<int, HALF + at>());
        });
      }
      // a block sum meets the scales three products later
      if constexpr (t >= 3) {
        constexpr int u = t - 3;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[u % MT][u / MT][r] = fmaf(scale[u % MT], part[u & 3][r], acc[u % MT][u / MT][r]);
        // (here: the compiler would put it off past the branches of a block's middle, with
        // every block sum in registers until then)
        asm volatile("" : "+v"(acc[u % MT][u / MT]));
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    sw = next_sw;
    now = next;
    advance_next();
    copied = stores = false;
    } while (--left > 0);
    steps<COPIES - HALF>([&](auto c) { copy_rows(std::integral_constant<int, HALF + decltype(c)::value>()); });
    copied = true;
    if constexpr (KG > 1) {
      if (kg > 0) steps<STEPS>([&](auto t) { sums[kg - 1][wave][decltype(t)::value][lane] = acc[decltype(t)::value / NT][decltype(t)::value % NT]; });
      lds_barrier();
      if (kg > 0) continue;
      steps<STEPS>([&](auto t) {
#pragma unroll
        for (int g = 0; g < KG - 1; ++g) acc[decltype(t)::value / NT][decltype(t)::value % NT] += sums[g][wave][decltype(t)::value][lane];
      });
    }
    stores = m_at + BM <= p.M && n_at + BN <= p.N && p.N % 8 == 0;
    asm volatile("" ::: "memory");
    const bool vec = p.N % 4 == 0;
    if (OUT == Dt::BF16 && NT % 4 == 0 && stores) {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
#pragma unroll
        for (int i = 0; i < NT; i += 4) {
          const int l = anew();
          const bool low = (l & 8) == 0;
          uintx4 first, second;
          lines_of_tiles(low, &acc[j][i], &first, &second);
          const size_t at = static_cast<size_t>(m_at + wm * (BM / WM) + j * 16) * p.N + n_at + wn * (BN / WN) + i * 16;
          uint8_t* const out = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.out) + at);
          const uint32_t off = (static_cast<uint32_t>(l & 7) * p.N + (l >> 4) * 8 + (low ? 0 : 32)) * 2;
          *reinterpret_cast<uintx4*>(out + off) = first;
          *reinterpret_cast<uintx4*>(out + static_cast<size_t>(p.N) * 16 + off) = second;
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      asm volatile("" ::: "memory");
      continue;
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int l = anew(), m = m_at + wm * (BM / WM) + j * 16 + (l & 15);
      const int n0 = n_at + wn * (BN / WN);
      if (m >= p.M) continue;
      const size_t at = static_cast<size_t>(m) * p.N;
      if (OUT == Dt::BF16 && p.N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          const int n = n0 + i * 16 + (l >> 4) * 8;
          const uintx4 x = pair_of_tiles(acc[j][i], acc[j][i + 1]);
          if (n < p.N) *reinterpret_cast<uintx4*>(static_cast<uint16_t*>(p.out) + at + n) = x;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int n = n0 + i * 16 + 4 * (l >> 4);
          if (n < p.N) store4<OUT>(p.out, at + n, p.N - n, vec, acc[j][i]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("" ::: "memory");
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // no copy outlives the workgroup's LDS
}

// Few outputs: 16 MT rows of a against 16 NT of w, whose bytes come straight from memory to
// the matrix instructions' registers.  The waves take every kWaves-th block of k, without a
// barrier, and add up in LDS at the end.  1 x 2048 x 2048: 3.8 us, 16 x 8192 x 4096: 10.0 us,
// 3.4 TB/s (a launch and one read of memory each).
constexpr int kWaves = 8;
template <Dt OUT, int MT, int NT, int AHEAD>
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
    ar[j] = p.a + static_cast<size_t>(m) * p.K;
    sa[j] = p.a_scale + static_cast<size_t>(m) * kb;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) wr[i] = p.w + static_cast<size_t>(min(n0 + i * 16 + c16, p.N - 1)) * p.K;
  const float* sw = p.w_scale + static_cast<size_t>(n0 / kBlock) * kb;
  // A block as loaded.  Lanes behind the rows' end load the rows' first bytes, without a
  // branch (lane_offset), and have them taken for zeros when they are used.
  struct Block {
    intx4 w[NT][2], a[MT][2];
    float sa[MT], sw;
  };
  const auto read = [&](int b, Block& x) {
    const int lo = lane_offset(p.K, b, q, 0), hi = lane_offset(p.K, b, q, 1);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      x.w[i][0] = *reinterpret_cast<const intx4*>(wr[i] + lo);
      x.w[i][1] = *reinterpret_cast<const intx4*>(wr[i] + hi);
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      x.a[j][0] = *reinterpret_cast<const intx4*>(ar[j] + lo);
      x.a[j][1] = *reinterpret_cast<const intx4*>(ar[j] + hi);
      x.sa[j] = sa[j][b];
    }
    x.sw = sw[b];
  };
  floatx4 acc[MT][NT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const auto multiply = [&](int b, Block& x) {
    if ((b + 1) * kBlock > p.K) {
      const intx4 zero = {0, 0, 0, 0};
      const bool lo = lane_has(p.K, b, q, 0), hi = lane_has(p.K, b, q, 1);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        x.w[i][0] = lo ? x.w[i][0] : zero;
        x.w[i][1] = hi ? x.w[i][1] : zero;
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        x.a[j][0] = lo ? x.a[j][0] : zero;
        x.a[j][1] = hi ? x.a[j][1] : zero;
      }
    }
    Frag<OUT> wf[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wf[i].set(join(x.w[i][0], x.w[i][1]));
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      Frag<OUT> af;
      af.set(join(x.a[j][0], x.a[j][1]));
      const float scale = x.sa[j] * x.sw;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const floatx4 part = block_sum(wf[i], af);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][i][r] = fmaf(scale, part[r], acc[j][i][r]);
      }
    }
  };
  // `mine` blocks, AHEAD of them on their way: the loop's reads are unconditional, so that a
  // block is waited for without those behind it.
  const int mine = wave < kb ? (kb - wave + kWaves - 1) / kWaves : 0;
  const auto block = [&](int s) { return wave + s * kWaves; };
  Block ring[AHEAD];
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
    if (d < mine) read(block(d), ring[d]);
  int s = 0;
  for (; s + 2 * AHEAD <= mine; s += AHEAD)
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      multiply(block(s + d), ring[d]);
      read(block(s + AHEAD + d), ring[d]);
    }
#pragma unroll
  for (int d = 0; d < 2 * AHEAD - 1; ++d)
    if (s + d < mine) {
      multiply(block(s + d), ring[d % AHEAD]);
      if (d < AHEAD - 1 && s + AHEAD + d < mine) read(block(s + AHEAD + d), ring[d % AHEAD]);
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

template <Dt OUT, int BM, int BN, int WM, int WN, int KG, int NB>
hipError_t launch_tiles(const Product8& p, hipStream_t stream) {
  const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  const int64_t tiles = static_cast<int64_t>(tm) * tn, most = WM * WN * KG > 4 ? 256 : 512;
  hipLaunchKernelGGL((product8_tile_kernel<OUT, BM, BN, WM, WN, KG, NB>), dim3(static_cast<unsigned>(tiles < most ? tiles : most)),
                     dim3(WM * WN * KG * 64), 0, stream, p, tm, tn);
  return hipGetLastError();
}

template <Dt OUT, int MT, int NT, int AHEAD>
hipError_t launch_rows(const Product8& p, hipStream_t stream) {
  hipLaunchKernelGGL((product8_rows_kernel<OUT, MT, NT, AHEAD>),
                     dim3((p.N + NT * 16 - 1) / (NT * 16), (p.M + MT * 16 - 1) / (MT * 16)),
                     dim3(kWaves * 64), 0, stream, p);
  return hipGetLastError();
}

// By how many workgroups a shape gives, one or two a compute unit being what hides latency.
// Measured with bf16 results (us, replayed graph, weights from memory; rows of 16 x 16 and
// 16 x 32, tiles of 32, of 64, of 64 x 128, of 128, of 256):
//      16 x 2048 x 2048    4.9   5.9   5.9   8.0  11.0  15.7  24.9
//      64 x 2048 x 2048    7.2   5.9   6.0   8.2  11.4  16.3  25.7
//     128 x 2048 x 2048   11.8   9.6   6.2   8.1  11.3  16.8  26.6
//      64 x 8192 x 4096   38.1  31.0  14.2  14.0  19.8  33.9  48.3
//     512 x 2048 x 2048   38.3  31.4  15.2   9.0  11.7  16.8  28.3
//    1024 x 2048 x 2048   72.9  60.5  26.4  14.4  12.2  17.2  28.1
//     512 x 8192 x 4096    282   227  82.5  44.7  30.4  36.5  51.7
//    1024 x 8192 x 4096    560   451   158  82.5  54.8  43.0  56.1
//    4096 x 4096 x 4096   1112   893   296   163   105  83.1  65.3
// and with fp32 results, for which the rule takes the fastest too but for 64 x 8192 x 4096, by 2%:
//      16 x 2048 x 2048    4.9   5.8   6.7  10.2  15.8  21.0
//      64 x 2048 x 2048    7.2   5.8   6.8  10.4  16.5  21.6
//     128 x 2048 x 2048   12.0   9.7   6.9  10.4  16.4  22.5
//      64 x 8192 x 4096   38.7  31.9  16.5  16.8  28.8  40.1
//     512 x 2048 x 2048   38.8  32.4  18.1  11.1  16.7  23.2
//    1024 x 2048 x 2048   73.7  62.0  32.5  18.7  17.4  23.6
//     512 x 8192 x 4096    282   236   101  59.6  45.5  48.8
//    1024 x 8192 x 4096    559   465   197   113  85.4  69.9
//    4096 x 4096 x 4096   1114   923   391   218   161   136
// Up to 16 rows every workgroup reads a alone, and what counts is w's stream: 16 x 8192 x 4096
// 12.3 and 10.1 with 16 and 32 columns.
template <Dt OUT>
hipError_t launch(const Product8& p, hipStream_t stream) {
  const auto tiles = [&](int bm, int bn) {
    return static_cast<int64_t>((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn);
  };
  if (p.M <= 16 ? p.N <= 4096 : tiles(16, 16) <= 256) return launch_rows<OUT, 1, 1, 4>(p, stream);
  if (p.M <= 16 || tiles(16, 32) <= 256) return launch_rows<OUT, 1, 2, 4>(p, stream);
  if (tiles(32, 32) <= 256) return launch_tiles<OUT, 32, 32, 2, 1, 4, 3>(p, stream);
  if (tiles(64, 64) <= 256) return launch_tiles<OUT, 64, 64, 2, 2, 2, 3>(p, stream);
  if (tiles(64, 128) <= 512) return launch_tiles<OUT, 64, 128, 2, 2, 1, 3>(p, stream);
  // (fp32 results: the larger tile would spill registers)
  if constexpr (OUT == Dt::BF16)
    if (tiles(256, 256) >= 192) return launch_tiles<OUT, 256, 256, 4, 2, 1, 2>(p, stream);
  return launch_tiles<OUT, 128, 128, 2, 2, 1, 2>(p, stream);
}

}  // namespace

hipError_t launch_product8(const Product8& p, hipStream_t stream) {
  return p.out_dtype == 0 ? launch<Dt::BF16>(p, stream) : launch<Dt::F32>(p, stream);
}

}  // namespace gdr
