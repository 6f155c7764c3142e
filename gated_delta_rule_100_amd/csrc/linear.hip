// linear.hip -- linear attention with a decay for each head on gfx950: prompts
// and gradients in chunks of tokens on the matrix cores, single tokens as a
// stream.
//
// A pass of the recurrence (linear.h, LinearPass) over one chunk, with G_t the
// prefix sums of the chunk's gates, C its last token and Z the state before it:
//   out_t = os ( sum_{s <= t} e^{G_t - G_s} us (x_t . y_s) w_s + e^{G_t} Z x_t )
//   Z    <- e^{G_C} Z + us sum_s e^{G_C - G_s} w_s y_s^T
// and walking backwards, with Z the state behind the chunk,
//   out_t = os ( sum_{s >= t} e^{G_s - G_t} us (x_t . y_s) w_s + e^{G_C - G_t} Z x_t )
//   Z    <- e^{G_C} Z + us sum_s e^{G_s} w_s y_s^T.
// All exponents are <= 0 for g <= 0.
#include <type_traits>

#include "linear.h"
#include "mfma_planes.h"

namespace gdr {
namespace {

constexpr float kMinGate = -110.f;  // e^-110 is zero in fp32: stands for every smaller g

__device__ __forceinline__ float clamp_gate(float g) { return g < kMinGate ? kMinGate : g; }

__device__ __forceinline__ void token_range(const LinearBatch& b, int n, int& tb, int& te) {
  tb = b.cu[n];
  te = b.cu[n + 1];
  tb = tb < 0 ? 0 : (tb > b.T_total ? b.T_total : tb);
  te = te < tb ? tb : (te > b.T_total ? b.T_total : te);
}

// Sequence and tokens [tb, te) of a unit, and whether it is the first and the
// last of its sequence.
struct Unit {
  int n, tb, te;
  bool first, last;
};

// The units of a sequence: its first `count - tail` segments are units from,
// from + 1, ..; with tail, its last one (shorter than the others) is unit tail_at.
struct SequenceUnits {
  int from, count, tail, tail_at;
  __device__ __forceinline__ int at(int j) const { return j < count - tail ? from + j : tail_at; }
};

// The segment table of at most kInlineSeqs sequences, formed by every wave for
// itself with one sequence a lane (a launch and a dependent read less than a
// table in memory).  All whole segments come first, then the sequences' shorter
// last ones by falling length: the hardware starts workgroups in order, so the
// long walks start first (32768 tokens in 8 sequences, 32 heads: 440 us with the last
// ones in the order of the sequences, 409 this way).
struct SegmentTable {
  int whole;      // inclusive prefix sum of whole segments, lane n for sequence n
  int tail;       // tokens of the shorter last segment, 0 for none
  int rank;       // its place among them
  int all_whole;
};
__device__ __forceinline__ SegmentTable segment_table(const LinearBatch& b, int lane) {
  int tb = 0, te = 0;
  if (lane < b.N) token_range(b, lane, tb, te);
  SegmentTable p;
  p.whole = (te - tb) / b.seg;
  p.tail = (te - tb) % b.seg;
  p.rank = 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int w = __shfl_up(p.whole, d);
    if (lane >= d) p.whole += w;
  }
  for (int m = 0; m < b.N; ++m) {
    const int t = __builtin_amdgcn_readlane(p.tail, m);
    p.rank += t > p.tail || (t == p.tail && m < lane);
  }
  p.all_whole = __builtin_amdgcn_readlane(p.whole, 63);
  return p;
}

__device__ __forceinline__ SequenceUnits sequence_units(const LinearBatch& b, int n) {
  SequenceUnits r;
  if (b.seg_offs) {
    int u0 = b.seg_offs[n], u1 = b.seg_offs[n + 1];
    u0 = u0 < 0 ? 0 : (u0 > b.units ? b.units : u0);
    u1 = u1 < u0 ? u0 : (u1 > b.units ? b.units : u1);
    r = {u0, u1 - u0, 0, 0};
  } else {
    const SegmentTable p = segment_table(b, threadIdx.x & 63);
    const int w1 = __builtin_amdgcn_readlane(p.whole, n);
    const int w0 = n > 0 ? __builtin_amdgcn_readlane(p.whole, n - 1) : 0;
    const int tail = __builtin_amdgcn_readlane(p.tail, n) > 0;
    r = {w0, w1 - w0 + tail, tail, p.all_whole + __builtin_amdgcn_readlane(p.rank, n)};
    // (offsets that go back or past the tokens could name more units than there are)
    if (r.from + r.count - r.tail > b.units || (r.tail && r.tail_at >= b.units)) r.count = r.tail = 0;
  }
  return r;
}

// False for a slot without a segment.
__device__ __forceinline__ bool unit_at(const LinearBatch& b, int u, Unit& r) {
  if (b.seg == 0) {
    r.n = u;
    r.first = r.last = true;
    token_range(b, u, r.tb, r.te);
    return true;
  }
  int j;
  if (b.seg_idx) {
    r.n = b.seg_idx[2 * u];
    j = b.seg_idx[2 * u + 1];
    if (r.n < 0 || r.n >= b.N || j < 0) return false;
  } else {
    const int lane = threadIdx.x & 63;
    const SegmentTable p = segment_table(b, lane);
    const bool whole = u < p.all_whole;
    const uint64_t found = __ballot(lane < b.N && (whole ? u < p.whole
                                                         : p.tail > 0 && p.rank == u - p.all_whole));
    if (found == 0) return false;
    r.n = __builtin_ctzll(found);
    const int before = r.n > 0 ? __builtin_amdgcn_readlane(p.whole, r.n - 1) : 0;
    j = whole ? u - before : __builtin_amdgcn_readlane(p.whole, r.n) - before;
  }
  int tb, te;
  token_range(b, r.n, tb, te);
  const int64_t from = tb + static_cast<int64_t>(j) * b.seg;
  if (from >= te) return false;
  r.tb = static_cast<int>(from);
  r.te = te - r.tb < b.seg ? te : r.tb + b.seg;
  r.first = j == 0;
  r.last = r.te == te;
  return true;
}

// ---- operands
//
// A fragment is eight elements of the contraction index for one row or column
// (lane (c, g) = (lane % 16, lane / 16)): one bf16x8 for bf16 inputs, eight
// floats for fp32 ones, multiplied by one 16x16x32 bf16 product or eight
// 16x16x4 fp32 products.  fp32 values beside bf16 inputs (P, the state, the
// decayed w) are three bf16 planes.
constexpr int kPlanes = 3;
struct F32x8 {
  float v[8];
};
template <Dt IN>
struct FragOf { using type = bf16x8; };
template <>
struct FragOf<Dt::F32> { using type = F32x8; };
template <Dt IN>
using Frag = typename FragOf<IN>::type;

template <Dt IN>
struct Planes {
  static constexpr int N = IN == Dt::F32 ? 1 : kPlanes;
  Frag<IN> p[N];
};

__device__ __forceinline__ floatx4 mma(const bf16x8& a, const bf16x8& b, floatx4 acc) {
  return mfma16x16x32(a, b, acc);
}
__device__ __forceinline__ floatx4 mma(const F32x8& a, const F32x8& b, floatx4 acc) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], acc, 0, 0, 0);
  return acc;
}
template <Dt IN>
__device__ __forceinline__ Planes<IN> to_planes(const float (&x)[8]) {
  Planes<IN> r;
  if constexpr (IN == Dt::F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.p[0].v[i] = x[i];
  } else {
    split8<kPlanes>(x, r.p);
  }
  return r;
}

// ---- tiles in LDS
//
// Rows of CH 16-byte pieces; piece i of row r lies at i ^ perm(r).  perm gives
// the 16 rows of a row fragment distinct 16-byte banks, and the four rows of a
// transposing read distinct groups of four pieces.
template <int CH>
__device__ __forceinline__ int perm(int r) {
  if constexpr (CH >= 16) return ((r & 3) << 2) | ((r >> 2) & 3);
  else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// Byte offset of a lane's part of a row fragment (elements 32 kb + 8 g .. + 7 of
// row c) and of a transposing read (rows 4 g + c / 4, columns 32 jb + 8 (c % 4)).
// perm has period 16 in the row, so other rows are a constant further on.
template <int CH>
__device__ __forceinline__ int row_lane(int c, int g, int kb) {
  return c * CH * 16 + 16 * ((4 * kb + g) ^ perm<CH>(c));
}
template <int CH>
__device__ __forceinline__ int col_lane(int c, int g, int jb) {
  const int r = 4 * g + (c >> 2);
  return r * CH * 16 + 16 * ((4 * jb + (c & 3)) ^ perm<CH>(r));
}

// Row fragment: elements 32 kb + 8 g .. + 7 of row r0 + c (r0 a multiple of 16;
// lane: row_lane of kb, used for bf16).
template <Dt IN, int CH>
__device__ __forceinline__ Frag<IN> row_frag(const unsigned char* tile, int r0, int kb, int c, int g,
                                             int lane) {
  if constexpr (IN == Dt::BF16) {
    return *reinterpret_cast<const bf16x8*>(tile + lane + r0 * CH * 16);
  } else {
    const unsigned char* row = tile + (r0 + c) * CH * 16;
    const int i = 8 * kb + 2 * g;
    const floatx4 a = *reinterpret_cast<const floatx4*>(row + 16 * (i ^ perm<CH>(c)));
    const floatx4 b = *reinterpret_cast<const floatx4*>(row + 16 * ((i + 1) ^ perm<CH>(c)));
    return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
}

// Two transposing reads, 16 rows apart (ds_read_b64_tr_b16: element e of lane c
// comes from input lane 4 e + c / 4, element c % 4).
template <int CH>
__device__ __forceinline__ bf16x8 read_tr_pair(const unsigned char* p) {
  const shortx4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4*)p);
  const shortx4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) shortx4*)(p + 16 * CH * 16));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int CH>
__device__ __forceinline__ F32x8 read_columns(const unsigned char* tile, int r0, int col, int g) {
  F32x8 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * (i >> 2) + 4 * g + (i & 3);
    f.v[i] = *reinterpret_cast<const float*>(tile + r * CH * 16 + 16 * ((col >> 2) ^ perm<CH>(r)) +
                                             4 * (col & 3));
  }
  return f;
}

// Column fragments of the 32 rows r0 ..: rows r0 + 4g + e in slots e and r0 +
// 16 + 4g + e in slots 4 + e (the order in which two stacked output tiles
// present their rows).  wide: of column 32 jb + 8 (c / 4) + c % 4 + 4 half (lane:
// col_lane of jb); narrow: of column col + c.
template <Dt IN, int CH>
__device__ __forceinline__ Frag<IN> col_frag_wide(const unsigned char* tile, int r0, int jb, int half,
                                                  int c, int g, int lane) {
  if constexpr (IN == Dt::BF16) return read_tr_pair<CH>(tile + lane + r0 * CH * 16 + 8 * half);
  else return read_columns<CH>(tile, r0, 32 * jb + 4 * half + 8 * (c >> 2) + (c & 3), g);
}
template <Dt IN, int CH>
__device__ __forceinline__ Frag<IN> col_frag_narrow(const unsigned char* tile, int r0, int col, int c,
                                                    int g) {
  if constexpr (IN == Dt::BF16) {
    const int r = 4 * g + (c >> 2), at = col + 4 * (c & 3);
    return read_tr_pair<CH>(tile + (r0 + r) * CH * 16 + 16 * ((at >> 3) ^ perm<CH>(r)) + 2 * (at & 7));
  } else {
    return read_columns<CH>(tile, r0, col + c, g);
  }
}

// Four elements col .. col + 3 of row r, widened (col a multiple of 4).
template <Dt IN, int CH>
__device__ __forceinline__ floatx4 row4(const unsigned char* tile, int r, int col) {
  const unsigned char* row = tile + r * CH * 16;
  if constexpr (IN == Dt::BF16) {
    const uint2 u = *reinterpret_cast<const uint2*>(row + 16 * ((col >> 3) ^ perm<CH>(r)) + 2 * (col & 7));
    return floatx4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                   __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)};
  } else {
    return *reinterpret_cast<const floatx4*>(row + 16 * ((col >> 2) ^ perm<CH>(r)));
  }
}

__device__ __forceinline__ float frag_value(const bf16x8& f, int i) { return static_cast<float>(f[i]); }
__device__ __forceinline__ float frag_value(const F32x8& f, int i) { return f.v[i]; }

// Workgroup barriers.  The copy waves wait for their own loads; the compute
// waves wait for their LDS accesses only (their global stores stay in flight).
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ void copy16(const void* src, void* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src),
                                   (__attribute__((address_space(3))) void*)(lds), 16, 0, 0);
}

// Gate factors of a chunk, one token a lane: G in log2 units as hi + lo, e^G,
// e^{G_C - G} and e^{G_C}.  Prefix sums in fp64, so that the error of a decay
// does not grow with |G|.
struct Gates {
  float hi, lo, from_start, to_end, all;
};
template <int C>
__device__ __forceinline__ Gates chunk_gates(float gate, bool per_token, int lane, int len) {
  double G;
  if (per_token) {
    G = lane < len ? static_cast<double>(clamp_gate(gate)) : 0.0;
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
      const double up = __shfl_up(G, d);
      if (lane >= d) G += up;
    }
  } else {
    G = static_cast<double>(clamp_gate(gate)) * (lane < len ? lane + 1 : len);
  }
  G *= 1.4426950408889634;
  const double end = __shfl(G, C - 1);
  Gates r;
  r.hi = static_cast<float>(G);
  r.lo = static_cast<float>(G - r.hi);
  r.from_start = exp2f(r.hi) * fmaf(r.lo, 0.69314718f, 1.f);
  r.to_end = exp2f(static_cast<float>(end - G));
  const float eh = static_cast<float>(end), el = static_cast<float>(end - eh);
  r.all = exp2f(eh) * fmaf(el, 0.69314718f, 1.f);
  return r;
}

// ---- the chunk scan
//
// One workgroup for a (unit, head): a unit is a sequence, or a segment of one.
// It holds the whole state of od = 16 W rows, so that x, y and the scores are read
// and formed once.  Its waves have three roles:
//   - W compute waves hold 16 state rows each for the whole walk, as output
//     tiles of the state update: lane (c, g) holds Z[c][32 j + 8 g + 0..7],
//     which is also the fragment of Z in the product with x.  In step s they
//     form out = Z x + P w and the update of Z for chunk s;
//   - SW score waves form the scores x.y of chunk s + 1, with their decays, in
//     registers: they do not depend on the state, and their arithmetic fills
//     the issue slots that the compute waves' chain leaves;
//   - CW copy waves copy the x and y rows of chunk s + 2 and the w rows of chunk
//     s + 1 to LDS (global-to-LDS loads) and form the gate factors of s + 2.
//     They are waves of their own because a wave's LDS reads wait for all its
//     global-to-LDS loads in flight (copies by the score waves: 5.05 us a chunk of
//     64 tokens, 128 x 128, by waves of their own 3.0, at two planes of Z and P).
// Two barriers a chunk: one behind its last reads, and one behind the score
// waves' writing P^T for the next chunk (right after the former, while the
// compute waves form Z x).
//
// Numerics beside bf16 inputs: the state stays fp32 in registers; Z, P and the
// decayed w enter the products as three bf16 planes, their full 24 bits, whatever
// the outputs' type and whether dg is wanted.  (Two planes of Z and P leave an
// error of 2.5e-6, three 1.9e-7, fp32's own, which the sums of dg and of shared
// heads and fp32 outputs need.  Two take 4% less of 4 x 4096 tokens, 115 against 120
// us, and 10% less of 32768 packed tokens, 361 against 403.)
// fp32 inputs run on fp32 matrix instructions throughout.
//
// What bounds it is the chain of a step, read, multiply, barrier, read, multiply,
// with two compute waves a SIMD to hide it: no unit is full (matrix instructions 40%
// of a step, vector ones 53%, LDS 42%, memory 3.9 TB/s of q, k, v and o while the steps
// run).  4 x 4096 tokens, 16 heads, bf16: 81 us for 16 chunks a workgroup, 4.3 us a
// chunk beside 12 us of start and end, and 120 us with the segments' states and their
// chain (2.3 TB/s of q, k, v and o once).  Tried and not kept, against 115 us and a
// gradient of 343, at two planes of Z and P in prompts: four compute waves of 32
// rows each, which halve the LDS reads (119; 381); y reads without their two-way bank
// conflicts, at twice the x reads (118; 350); matrix and vector instructions
// interleaved by scheduling groups (123; 374-398); wave priorities (115; 345-354).
template <Dt IN, int KD, int W, bool DOT, int SW>
struct ScanCfg {
  static constexpr int ES = IN == Dt::BF16 ? 2 : 4;
  static constexpr int C = IN == Dt::BF16 ? 64 : 32;  // tokens a chunk (fp32: half, for LDS)
  static constexpr int NT = C / 16, NB = C / 32;
  static constexpr int KB = KD / 32;          // 32-deep blocks over kd
  static constexpr int OD = 16 * W;           // columns of w
  static constexpr int CHK = KD * ES / 16, CHV = OD * ES / 16;
  static constexpr int CW = SW == 3 ? 1 : 4;  // copy waves
  static constexpr int THREADS = 64 * (W + SW + CW);
  // three buffers of x and y rows, two of w rows
  static constexpr int X_BYTES = C * KD * ES, W_BYTES = C * OD * ES;
  static constexpr int OFF_W = 3 * 2 * X_BYTES;
  // three of gate factors: G in log2 units as a sum of two floats, the factors
  // of Z x_t and of the update, e^{G_C}
  static constexpr int GATE_BYTES = (4 * C + 4) * 4;
  static constexpr int OFF_G = OFF_W + 2 * W_BYTES;
  // P^T fragments (row tile, 32-deep block) on the walked side of the diagonal,
  // PL planes each, and the scores of a token with itself
  static constexpr int PL = Planes<IN>::N;
  static constexpr int FRAG = IN == Dt::BF16 ? 1024 : 2048;
  static constexpr int FRAGS = NB == 2 ? 6 : 2;
  static constexpr int P_BYTES = FRAGS * PL * FRAG;
  static constexpr int OFF_P = OFF_G + 3 * GATE_BYTES;
  static constexpr int OFF_DIAG = OFF_P + P_BYTES;
  // two of the compute waves' parts of the dot products
  static constexpr int OFF_DOT = OFF_DIAG + C * 4;
  static constexpr int BYTES = OFF_DOT + (DOT ? 2 * W * C * 4 : 0);
  static_assert(BYTES <= 160 * 1024, "LDS");
};

// Index of the P^T fragment of row tile tt and block sb.
template <int NB, bool BACK>
__device__ __forceinline__ int p_frag(int tt, int sb) {
  if constexpr (NB == 1) return tt;
  else if constexpr (BACK) return tt < 2 ? 2 * tt + sb : tt + 2;
  else return tt < 2 ? tt : 2 * tt - 2 + sb;
}

// Four consecutive columns of a state row, col elements apart.
__device__ __forceinline__ floatx4 load_state4(const float* p, int64_t col) {
  if (col == 1) return *reinterpret_cast<const floatx4*>(p);
  return floatx4{p[0], p[col], p[2 * col], p[3 * col]};
}
__device__ __forceinline__ void store_state4(float* p, int64_t col, const floatx4& z) {
  if (col == 1) {
    *reinterpret_cast<floatx4*>(p) = z;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e * col] = z[e];
  }
}

template <Dt IN, int KD, int W, bool DOT, bool BACK, int SW>
__device__ __forceinline__ void scan_pass(const LinearBatch& b, const LinearPass& p,
                                          unsigned char* lds) {
  using Cfg = ScanCfg<IN, KD, W, DOT, SW>;
  constexpr int CW = Cfg::CW;
  constexpr int C = Cfg::C, NT = Cfg::NT, NB = Cfg::NB, KB = Cfg::KB, ES = Cfg::ES, PL = Cfg::PL;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = blockIdx.x, h = pair % b.H;
  Unit unit;
  if (!unit_at(b, pair / b.H, unit)) return;
  const int tb = unit.tb, te = unit.te;
  const int chunks = (te - tb + C - 1) / C;
  // token range of the s-th chunk of the walk
  auto chunk_at = [&](int s, int& tok) {
    tok = tb + (BACK ? chunks - 1 - s : s) * C;
    return te - tok < C ? te - tok : C;
  };
  // buffer i of x and y rows and of gate factors (chunk s uses buffer s % 3)
  auto x_tile = [&](int i) { return lds + i * 2 * Cfg::X_BYTES; };
  auto gate_row = [&](int i) {
    return reinterpret_cast<float*>(lds + Cfg::OFF_G + i * Cfg::GATE_BYTES);
  };
  auto next = [](int i) { return i == 2 ? 0 : i + 1; };

  if (wave >= W + SW) {  // ---- copy waves
    if (chunks == 0) return;
    const int cw = wave - W - SW;
    auto rows = [&](const LinearRows& r, int width) {
      return static_cast<const char*>(r.p) + static_cast<size_t>(h / r.group) * width * ES;
    };
    const char* xs = rows(p.x, KD);
    const char* ys = rows(p.y, KD);
    const char* ws = rows(p.w, Cfg::OD);
    const size_t xst = p.x.stride * ES, yst = p.y.stride * ES, wst = p.w.stride * ES;
    // Byte offsets of this lane's 16-byte pieces inside a chunk: 64 rows apart
    // they stay below 2^32 (strides are at most 2^24 elements).  In a chunk
    // shorter than C the rows past its end repeat its last token: nothing
    // outside the sequence is read, and their factors are zero.
    constexpr int NX = C * Cfg::CHK / 64 / CW, NW = C * Cfg::CHV / 64 / CW;
    uint32_t xo[NX], yo[NX], wo[NW];
    auto piece = [&](int i, auto ch, int len, size_t stride) {
      constexpr int CH = decltype(ch)::value;
      const int q = 64 * (cw + CW * i) + lane, r = q / CH, pc = q % CH;
      return static_cast<uint32_t>((r < len ? r : len - 1) * stride + 16 * (pc ^ perm<CH>(r)));
    };
    const std::integral_constant<int, Cfg::CHK> chk;
    const std::integral_constant<int, Cfg::CHV> chv;
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      xo[i] = piece(i, chk, C, xst);
      yo[i] = piece(i, chk, C, yst);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) wo[i] = piece(i, chv, C, wst);
    auto copy_rows = [&](int s, const char* src, size_t stride, const uint32_t (&full)[NX],
                         unsigned char* to) {
      int tok;
      const int len = chunk_at(s, tok);
      const char* base = src + static_cast<size_t>(tok) * stride;
      if (len == C) {
#pragma unroll
        for (int i = 0; i < NX; ++i) copy16(base + full[i], to + 1024 * (cw + CW * i));
      } else {
#pragma unroll
        for (int i = 0; i < NX; ++i) copy16(base + piece(i, chk, len, stride), to + 1024 * (cw + CW * i));
      }
    };
    auto copy_x = [&](int s, int buf) { copy_rows(s, xs, xst, xo, x_tile(buf)); };
    auto copy_y = [&](int s, int buf) { copy_rows(s, ys, yst, yo, x_tile(buf) + Cfg::X_BYTES); };
    auto copy_w = [&](int s) {
      int tok;
      const int len = chunk_at(s, tok);
      const char* wb = ws + static_cast<size_t>(tok) * wst;
      unsigned char* to = lds + Cfg::OFF_W + (s & 1) * Cfg::W_BYTES + 1024 * cw;
      if (len == C) {
#pragma unroll
        for (int i = 0; i < NW; ++i) copy16(wb + wo[i], to + 1024 * CW * i);
      } else {
#pragma unroll
        for (int i = 0; i < NW; ++i) copy16(wb + piece(i, chv, len, wst), to + 1024 * CW * i);
      }
    };
    auto load_gate = [&](int s) {
      if (cw != 0) return 0.f;
      int tok;
      const int len = chunk_at(s, tok);
      if (!b.gates.per_token) return b.gates.g[h];
      return lane < len ? b.gates.g[static_cast<size_t>(tok + lane) * b.H + h] : 0.f;
    };
    auto put_gates = [&](int s, int buf, float gate) {
      if (cw != 0) return;
      int tok;
      const int len = chunk_at(s, tok);
      float* f = gate_row(buf);
      const Gates v = chunk_gates<C>(gate, b.gates.per_token, lane, len);
      if (lane < C) {
        f[lane] = v.hi;
        f[C + lane] = v.lo;
        f[2 * C + lane] = p.os * (BACK ? v.to_end : v.from_start);
        f[3 * C + lane] = lane < len ? p.us * (BACK ? v.from_start : v.to_end) : 0.f;
        if (lane == 0) f[4 * C] = v.all;
      }
    };
    const float g0 = load_gate(0), g1 = chunks > 1 ? load_gate(1) : 0.f;
    copy_x(0, 0);
    copy_y(0, 0);
    copy_w(0);
    if (chunks > 1) {
      copy_x(1, 1);
      copy_y(1, 1);
    }
    put_gates(0, 0, g0);
    if (chunks > 1) put_gates(1, 1, g1);
    __builtin_amdgcn_s_waitcnt(0);
    bare_barrier();
    // the dot products of chunk s, one token a lane
    auto store_dots = [&](int s) {
      if (!DOT || cw != CW - 1) return;
      int tok;
      const int len = chunk_at(s, tok);
      const float* part = reinterpret_cast<const float*>(lds + Cfg::OFF_DOT) + (s & 1) * W * C;
      float sum = 0.f;
      if (lane < C) {
#pragma unroll
        for (int i = 0; i < W; ++i) sum += part[i * C + lane];
      }
      if (lane < len)
        p.dot[static_cast<size_t>(h) * b.T_total + tok + lane] = sum;
    };
    for (int s = 0, buf = 2; s < chunks; ++s, buf = next(buf)) {
      float gate = 0.f;
      if (s > 0) store_dots(s - 1);
      if (s + 2 < chunks) gate = load_gate(s + 2);
      if (s + 1 < chunks) copy_w(s + 1);
      if (s + 2 < chunks) copy_x(s + 2, buf);
      bare_barrier();
      if (s + 2 < chunks) {
        copy_y(s + 2, buf);
        put_gates(s + 2, buf, gate);
      }
      __builtin_amdgcn_s_waitcnt(0);
      bare_barrier();
    }
    store_dots(chunks - 1);
    return;
  }

  if (wave >= W) {  // ---- score waves
    if (chunks == 0) return;
    const int sw = wave - W;
    // Tiles (row tile, column tile) of this wave, of the ten (fp32: three) on the
    // walked side of the diagonal; tiles 2 i and 2 i + 1 have one row tile.  Some
    // are formed twice (the same values).
    constexpr int PER = NB == 1 ? 1 : SW == 4 ? 3 : 4;
    int tts[PER], sts[PER];
    if constexpr (NB == 1) {
      tts[0] = sw == 0 ? 0 : 1;
      sts[0] = sw < 2 ? 0 : 1;
    } else if constexpr (SW == 4) {
      tts[0] = tts[1] = 3 - sw;
      sts[0] = 0;
      sts[1] = sw < 3 ? 1 : 0;
      tts[2] = sw == 1 ? 2 : 3;
      sts[2] = sw < 2 ? 2 : 3;
    } else {  // a row tile each, the last wave the two shortest
      tts[0] = tts[1] = 3 - sw;
      tts[2] = tts[3] = sw == 2 ? 0 : 3 - sw;
      sts[0] = 0;
      sts[1] = 1;
      sts[2] = sw == 2 ? 0 : 2;
      sts[3] = sw == 2 ? 0 : 3 - sw;
    }
    if (BACK)
      for (int i = 0; i < PER; ++i) {
        tts[i] = NT - 1 - tts[i];
        sts[i] = NT - 1 - sts[i];
      }
    const float ps = p.us * p.os;
    int kl[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) kl[kb] = row_lane<Cfg::CHK>(c, g, kb);
    float v[PER][4], own[PER];
    auto scores = [&](int s, int buf) {
      int tok;
      const int len = chunk_at(s, tok);
      const unsigned char *X = x_tile(buf), *Y = X + Cfg::X_BYTES;
      const float* gate = gate_row(buf);
      floatx4 acc[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        Frag<IN> xf;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (i % 2 == 0) xf = row_frag<IN, Cfg::CHK>(X, 16 * tts[i], kb, c, g, kl[kb]);
          acc[i] = mma(row_frag<IN, Cfg::CHK>(Y, 16 * sts[i], kb, c, g, kl[kb]), xf, acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int t = 16 * tts[i] + c, s4 = 16 * sts[i] + 4 * g;
        const float gh = gate[t], gl = gate[C + t];
        const floatx4 sh = *reinterpret_cast<const floatx4*>(gate + s4);
        const floatx4 sl = *reinterpret_cast<const floatx4*>(gate + C + s4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = (gh - sh[e]) + (gl - sl[e]);
          // (the scale as a factor: as log2 of it in the exponent it would be off by up
          // to |log2 scale| 2^-24 in every score)
          const float x = acc[i][e] * (ps * __builtin_amdgcn_exp2f(BACK ? -d : d));
          const int sc = s4 + e;
          if (DOT && sc == t) own[i] = x;
          const bool in = BACK ? (DOT ? sc > t : sc >= t) && sc < len : (DOT ? sc < t : sc <= t);
          v[i][e] = in ? x : 0.f;
        }
      }
    };
    auto put_scores = [&]() {
      float* diag = reinterpret_cast<float*>(lds + Cfg::OFF_DIAG);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (DOT && sts[i] == tts[i] && (c >> 2) == g) diag[16 * tts[i] + c] = own[i];
        const int half = sts[i] & 1;
        unsigned char* to = lds + Cfg::OFF_P + p_frag<NB, BACK>(tts[i], sts[i] >> 1) * PL * Cfg::FRAG;
        if constexpr (IN == Dt::F32) {
          *reinterpret_cast<floatx4*>(to + lane * 32 + 16 * half) =
              floatx4{v[i][0], v[i][1], v[i][2], v[i][3]};
        } else {
          uint32_t lo[PL], hi[PL];
          split2<PL>(v[i][0], v[i][1], lo);
          split2<PL>(v[i][2], v[i][3], hi);
#pragma unroll
          for (int q = 0; q < PL; ++q)
            *reinterpret_cast<uint2*>(to + q * Cfg::FRAG + lane * 16 + 8 * half) = make_uint2(lo[q], hi[q]);
        }
      }
    };
    bare_barrier();  // the first chunks are there
    scores(0, 0);
    for (int s = 0, buf = 1; s < chunks; ++s, buf = next(buf)) {
      put_scores();
      lds_barrier();  // P of chunk s is there
      if (s + 1 < chunks) scores(s + 1, buf);
      lds_barrier();  // chunk s is done
    }
    return;
  }

  // ---- compute waves
  constexpr int OD = Cfg::OD;
  const int od = 16 * wave;  // this wave's columns of w
  const size_t zbase = static_cast<size_t>(pair) * OD * KD + (od + c) * p.row;
  floatx4 z[KD / 16];  // z[2 j + i][e] = Z[od + c][32 j + 8 g + 4 i + e]
#pragma unroll
  for (int j = 0; j < KD / 16; ++j) {
    const int k = 32 * (j >> 1) + 8 * g + 4 * (j & 1);
    z[j] = p.start ? load_state4(p.start + zbase + k * p.col, p.col) : floatx4{0.f, 0.f, 0.f, 0.f};
  }
  if (chunks > 0) {
    // the halves of P^T fragments beyond the diagonal stay zero
    for (int i = threadIdx.x; i < Cfg::P_BYTES / 16; i += 64 * W)
      *reinterpret_cast<uint4*>(lds + Cfg::OFF_P + 16 * i) = make_uint4(0, 0, 0, 0);
    lds_barrier();
  }
  const size_t out_es = p.out_dtype == 0 ? 2 : 4;
  const uint32_t out_row = static_cast<uint32_t>(b.H * OD * out_es);
  const uint32_t out_lane = c * out_row + static_cast<uint32_t>(4 * g * out_es);
  const size_t e_col = DOT ? static_cast<size_t>(h / p.e.group) * OD + od + 4 * g : 0;
  int kl[KB], jl[KD / 32];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    kl[kb] = row_lane<Cfg::CHK>(c, g, kb);
    jl[kb] = col_lane<Cfg::CHK>(c, g, kb);
  }
  for (int s = 0, buf = 0; s < chunks; ++s, buf = next(buf)) {
    int tok;
    const int len = chunk_at(s, tok);
    const unsigned char *X = x_tile(buf), *Y = X + Cfg::X_BYTES;
    const unsigned char* Wt = lds + Cfg::OFF_W + (s & 1) * Cfg::W_BYTES;
    const unsigned char* P = lds + Cfg::OFF_P;
    const float* gate = gate_row(buf);
    const float* diag = reinterpret_cast<const float*>(lds + Cfg::OFF_DIAG);

    // the rows to dot with the outputs: loaded first, used last
    float ev[DOT ? NT : 1][4];
    if constexpr (DOT) {
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        const int t = 16 * tt + c, row = tok + (t < len ? t : len - 1);
        load_vec<IN, 4>(p.e.p, static_cast<size_t>(row) * p.e.stride + e_col, ev[tt]);
      }
    }

    // out^T = Z x^T, rows od, columns t: the x fragments of a block are read
    // while the block before it is multiplied, and the row tiles' chains alternate
    floatx4 o[NT];
#pragma unroll
    for (int tt = 0; tt < NT; ++tt) o[tt] = floatx4{0.f, 0.f, 0.f, 0.f};
    Frag<IN> xf[2][NT];
#pragma unroll
    for (int tt = 0; tt < NT; ++tt) xf[0][tt] = row_frag<IN, Cfg::CHK>(X, 16 * tt, 0, c, g, kl[0]);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (kb + 1 < KB) {
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
          xf[(kb + 1) & 1][tt] = row_frag<IN, Cfg::CHK>(X, 16 * tt, kb + 1, c, g, kl[kb + 1]);
      }
      const float zz[8] = {z[2 * kb][0], z[2 * kb][1], z[2 * kb][2], z[2 * kb][3],
                           z[2 * kb + 1][0], z[2 * kb + 1][1], z[2 * kb + 1][2], z[2 * kb + 1][3]};
      const Planes<IN> zp = to_planes<IN>(zz);
#pragma unroll
      for (int q = PL - 1; q >= 0; --q)
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) o[tt] = mma(zp.p[q], xf[kb & 1][tt], o[tt]);
    }
    Frag<IN> wf[NB];
#pragma unroll
    for (int sb = 0; sb < NB; ++sb)
      wf[sb] = col_frag_narrow<IN, Cfg::CHV>(Wt, 32 * sb, 16 * wave, c, g);
#pragma unroll
    for (int tt = 0; tt < NT; ++tt) o[tt] *= gate[2 * C + 16 * tt + c];
    bare_barrier();  // P of chunk s is there

    // + w^T P^T
#pragma unroll
    for (int sb = 0; sb < NB; ++sb) {
      Planes<IN> pf[NT];
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        if (BACK ? sb < (tt >> 1) : sb > (tt >> 1)) continue;
        const unsigned char* from = P + p_frag<NB, BACK>(tt, sb) * PL * Cfg::FRAG;
        if constexpr (IN == Dt::F32) {
          const floatx4 a = *reinterpret_cast<const floatx4*>(from + lane * 32);
          const floatx4 d = *reinterpret_cast<const floatx4*>(from + lane * 32 + 16);
          pf[tt].p[0] = {{a[0], a[1], a[2], a[3], d[0], d[1], d[2], d[3]}};
        } else {
#pragma unroll
          for (int q = 0; q < PL; ++q)
            pf[tt].p[q] = *reinterpret_cast<const bf16x8*>(from + q * Cfg::FRAG + lane * 16);
        }
      }
#pragma unroll
      for (int q = PL - 1; q >= 0; --q)
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) {
          if (BACK ? sb < (tt >> 1) : sb > (tt >> 1)) continue;
          o[tt] = mma(wf[sb], pf[tt].p[q], o[tt]);
        }
    }

    // Z <- e^{G_C} Z + (update factors . w)^T y, two tiles' y fragments at a time
    const float gc = gate[4 * C];
#pragma unroll
    for (int j = 0; j < KD / 16; ++j) z[j] *= gc;
#pragma unroll
    for (int sb = 0; sb < NB; ++sb) {
      const floatx4 f0 = *reinterpret_cast<const floatx4*>(gate + 3 * C + 32 * sb + 4 * g);
      const floatx4 f1 = *reinterpret_cast<const floatx4*>(gate + 3 * C + 32 * sb + 16 + 4 * g);
      Frag<IN> yf[2][2];
      auto read_y = [&](int jb, Frag<IN> (&f)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          f[i] = col_frag_wide<IN, Cfg::CHK>(Y, 32 * sb, jb, i, c, g, jl[jb]);
      };
      read_y(0, yf[0]);
      float u[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = frag_value(wf[sb], e) * f0[e];
        u[4 + e] = frag_value(wf[sb], 4 + e) * f1[e];
      }
      const Planes<IN> up = to_planes<IN>(u);
#pragma unroll
      for (int jb = 0; jb < KD / 32; ++jb) {
        if (jb + 1 < KD / 32) read_y(jb + 1, yf[(jb + 1) & 1]);
#pragma unroll
        for (int q = Planes<IN>::N - 1; q >= 0; --q)
#pragma unroll
          for (int i = 0; i < 2; ++i) z[2 * jb + i] = mma(yf[jb & 1][i], up.p[q], z[2 * jb + i]);
      }
    }

    // outputs
    if constexpr (DOT) {
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        const int t = 16 * tt + c;
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = fmaf(ev[tt][e], o[tt][e], dot);
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        if (g == 0)
          (reinterpret_cast<float*>(lds + Cfg::OFF_DOT) + ((s & 1) * W + wave) * C)[t] = dot;
        o[tt] += diag[t] * row4<IN, Cfg::CHV>(Wt, t, 16 * wave + 4 * g);
      }
    }
    char* out = static_cast<char*>(p.out) +
                ((static_cast<size_t>(tok) * b.H + h) * OD + od) * out_es;
    auto store = [&](int tt) {
      const uint32_t at = out_lane + 16 * tt * out_row;
      if (p.out_dtype == 0) {
        uint32_t lo[1], hi[1];
        split2<1>(o[tt][0], o[tt][1], lo);
        split2<1>(o[tt][2], o[tt][3], hi);
        *reinterpret_cast<uint2*>(out + at) = make_uint2(lo[0], hi[0]);
      } else {
        *reinterpret_cast<floatx4*>(out + at) = o[tt];
      }
    };
    if (len == C) {
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) store(tt);
    } else {
#pragma unroll
      for (int tt = 0; tt < NT; ++tt)
        if (16 * tt + c < len) store(tt);
    }
    lds_barrier();  // chunk s is done
  }

  float ed = 0.f;
  const bool ends = p.end && (BACK ? unit.first : unit.last);
  const size_t ebase = (static_cast<size_t>(unit.n) * b.H + h) * OD * KD + (od + c) * p.row;
#pragma unroll
  for (int j = 0; j < KD / 16; ++j) {
    const size_t at = (32 * (j >> 1) + 8 * g + 4 * (j & 1)) * p.col;
    if (p.end_with) {
      const floatx4 r = load_state4(p.end_with + zbase + at, p.col);
#pragma unroll
      for (int e = 0; e < 4; ++e) ed = fmaf(z[j][e], r[e], ed);
    }
    if (ends) store_state4(p.end + ebase + at, p.col, z[j]);
  }
  if (p.end_with) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) ed += __shfl_xor(ed, d);
    if (lane == 0) p.end_dot[static_cast<size_t>(od / 16) * b.units * b.H + pair] = ed;
  }
}

// Score waves of a workgroup: with eight compute waves three and one copy wave
// (168 registers a wave; with 128 the fp32 and the dot passes spill), with four
// compute waves four and four copy waves.
template <int W>
constexpr int score_waves() { return W == 8 ? 3 : 4; }

template <Dt IN, int KD, int OD, bool DOT>
using ScanCfgOf = ScanCfg<IN, KD, OD / 16, DOT, score_waves<OD / 16>()>;

template <Dt IN, int KD, int OD>
__global__ __launch_bounds__((ScanCfgOf<IN, KD, OD, false>::THREADS))
void linear_scan_kernel(LinearBatch b, LinearPass p) {
  __shared__ __align__(1024) unsigned char lds[ScanCfgOf<IN, KD, OD, false>::BYTES];
  scan_pass<IN, KD, OD / 16, false, false, score_waves<OD / 16>()>(b, p, lds);
}

// The three passes of a gradient (dq, dv, dk) in one launch: their workgroups follow
// each other without the gaps of launches, and run side by side where one pass does
// not fill the GPU (6 fp32 sequences of up to 777 tokens, 8 heads, 64 x 128: 85 us
// in three launches, 73 in one).  One pass after the other: the three of a unit side
// by side, to share their rows in the caches, take 2% longer.
template <Dt IN, int DK, int DV, bool DOT>
struct GradCfg {
  using K = ScanCfgOf<IN, DV, DK, DOT>;  // dq and dk
  using V = ScanCfgOf<IN, DK, DV, DOT>;  // dv
  static constexpr int THREADS = K::THREADS, BYTES = K::BYTES > V::BYTES ? K::BYTES : V::BYTES;
  static_assert(V::THREADS == THREADS, "one launch");
};
template <Dt IN, int DK, int DV, bool DOT>
__global__ __launch_bounds__((GradCfg<IN, DK, DV, DOT>::THREADS))
void linear_grad_kernel(LinearBatch b, LinearPass pq, LinearPass pv, LinearPass pk) {
  __shared__ __align__(1024) unsigned char lds[GradCfg<IN, DK, DV, DOT>::BYTES];
  constexpr int WK = DK / 16, WV = DV / 16, SK = score_waves<WK>(), SV = score_waves<WV>();
  if (blockIdx.y == 0) scan_pass<IN, DV, WK, DOT, false, SK>(b, pq, lds);
  else if (blockIdx.y == 1) scan_pass<IN, DK, WV, DOT, true, SV>(b, pv, lds);
  else scan_pass<IN, DV, WK, false, true, SK>(b, pk, lds);
}

// ---- states at the starts of segments
//
// A segment's own state, from zero: the update of the scan alone.  It is a
// stream of y and w rows, so the copy waves run three chunks ahead (four buffers,
// one barrier a chunk); one wave forms the gate factors.  4 x 4096 tokens, 16 heads,
// bf16: 37 us, 3.6 TB/s; bound by the copies and 10 us of start and end.
template <Dt IN, int KD, int W>
struct LocalCfg {
  static constexpr int ES = IN == Dt::BF16 ? 2 : 4;
  static constexpr int C = IN == Dt::BF16 ? 64 : 32;
  static constexpr int NB = C / 32;
  static constexpr int OD = 16 * W;
  static constexpr int CHK = KD * ES / 16, CHV = OD * ES / 16;
  // copy waves: with four the fp32 form has 128 registers a wave and spills (4 x 2048
  // tokens, 16 heads: prompt 175 us, with two 158); bf16 prompts take as long with both
  static constexpr int CW = 2;
  static constexpr int THREADS = 64 * (W + CW + 1);
  static constexpr int STAGES = 4;
  static constexpr int Y_BYTES = C * KD * ES, W_BYTES = C * OD * ES;
  static constexpr int BUF = Y_BYTES + W_BYTES;
  static constexpr int GATE_BYTES = (C + 4) * 4;  // update factors, e^{G_C}
  static constexpr int OFF_G = STAGES * BUF;
  static constexpr int BYTES = OFF_G + 2 * GATE_BYTES;
  // copies of a chunk by one copy wave
  static constexpr int NY = C * CHK / 64 / CW, NW = C * CHV / 64 / CW;
  static_assert(BYTES <= 160 * 1024, "LDS");
  static_assert(2 * (NY + NW) < 64, "copies in flight");
};

// Waits until at most n of this wave's loads and stores are in flight.
template <int N>
__device__ __forceinline__ void wait_vmem() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

template <Dt IN, int KD, int W, bool BACK>
__device__ __forceinline__ void local_states(const LinearBatch& b, const LinearStates& job,
                                             unsigned char* lds) {
  using Cfg = LocalCfg<IN, KD, W>;
  constexpr int C = Cfg::C, NB = Cfg::NB, ES = Cfg::ES, NY = Cfg::NY, NW = Cfg::NW, CW = Cfg::CW;
  const LinearRows &y = job.y, &w = job.w;
  const float us = job.us;
  float *states = job.states, *decays = job.decays;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = blockIdx.x, h = pair % b.H;
  Unit unit;
  if (!unit_at(b, pair / b.H, unit)) return;
  if (BACK ? unit.first : unit.last) return;  // nothing starts from its end
  const int tb = unit.tb, te = unit.te, chunks = (te - tb + C - 1) / C;
  auto chunk_at = [&](int s, int& tok) {
    tok = tb + (BACK ? chunks - 1 - s : s) * C;
    return te - tok < C ? te - tok : C;
  };
  if (wave == W + CW) {  // ---- gate wave
    auto load = [&](int s) {
      int tok;
      const int len = chunk_at(s, tok);
      if (!b.gates.per_token) return b.gates.g[h];
      return lane < len ? b.gates.g[static_cast<size_t>(tok + lane) * b.H + h] : 0.f;
    };
    auto put = [&](int s, float gate) {
      int tok;
      const int len = chunk_at(s, tok);
      const Gates v = chunk_gates<C>(gate, b.gates.per_token, lane, len);
      float* f = reinterpret_cast<float*>(lds + Cfg::OFF_G + (s & 1) * Cfg::GATE_BYTES);
      if (lane < C) f[lane] = lane < len ? us * (BACK ? v.from_start : v.to_end) : 0.f;
      if (lane == 0) f[C] = v.all;
    };
    float ahead = chunks > 1 ? load(1) : 0.f;
    put(0, load(0));
    lds_barrier();
    for (int s = 0; s < chunks; ++s) {
      const float gate = ahead;
      if (s + 2 < chunks) ahead = load(s + 2);
      if (s + 1 < chunks) put(s + 1, gate);
      lds_barrier();
    }
    return;
  }
  if (wave >= W) {  // ---- copy waves
    const int cw = wave - W;
    const char* ys = static_cast<const char*>(y.p) + static_cast<size_t>(h / y.group) * KD * ES;
    const char* ws = static_cast<const char*>(w.p) +
                     static_cast<size_t>(h / w.group) * Cfg::OD * ES;
    const size_t yst = y.stride * ES, wst = w.stride * ES;
    auto piece = [&](int i, auto ch, int len, size_t stride) {
      constexpr int CH = decltype(ch)::value;
      const int q = 64 * (cw + CW * i) + lane, r = q / CH, pc = q % CH;
      return static_cast<uint32_t>((r < len ? r : len - 1) * stride + 16 * (pc ^ perm<CH>(r)));
    };
    const std::integral_constant<int, Cfg::CHK> chk;
    const std::integral_constant<int, Cfg::CHV> chv;
    uint32_t yo[NY], wo[NW];
#pragma unroll
    for (int i = 0; i < NY; ++i) yo[i] = piece(i, chk, C, yst);
#pragma unroll
    for (int i = 0; i < NW; ++i) wo[i] = piece(i, chv, C, wst);
    auto bring = [&](int s) {  // NY + NW copies
      int tok;
      const int len = chunk_at(s, tok);
      const char* yb = ys + static_cast<size_t>(tok) * yst;
      const char* wb = ws + static_cast<size_t>(tok) * wst;
      unsigned char* to = lds + (s % Cfg::STAGES) * Cfg::BUF + 1024 * cw;
      if (len == C) {
#pragma unroll
        for (int i = 0; i < NY; ++i) copy16(yb + yo[i], to + 1024 * CW * i);
#pragma unroll
        for (int i = 0; i < NW; ++i) copy16(wb + wo[i], to + Cfg::Y_BYTES + 1024 * CW * i);
      } else {
#pragma unroll
        for (int i = 0; i < NY; ++i) copy16(yb + piece(i, chk, len, yst), to + 1024 * CW * i);
#pragma unroll
        for (int i = 0; i < NW; ++i)
          copy16(wb + piece(i, chv, len, wst), to + Cfg::Y_BYTES + 1024 * CW * i);
      }
    };
    // chunk s + 1 is there when the copies of the (at most two) chunks behind it
    // are all that is in flight
    auto wait_for = [&](int behind) {
      if (behind >= 2) wait_vmem<2 * (NY + NW)>();
      else if (behind == 1) wait_vmem<NY + NW>();
      else wait_vmem<0>();
    };
    const int lead = chunks < 3 ? chunks : 3;
    for (int s = 0; s < lead; ++s) bring(s);
    wait_for(lead - 1);
    bare_barrier();
    for (int s = 0; s < chunks; ++s) {
      if (s + 3 < chunks) bring(s + 3);
      const int left = chunks - 2 - s;  // chunks behind s + 1
      wait_for(left < 2 ? left : 2);
      bare_barrier();
    }
    return;
  }
  // ---- compute waves
  const int od = 16 * wave;
  floatx4 z[KD / 16];
#pragma unroll
  for (int j = 0; j < KD / 16; ++j) z[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  float decay = 1.f;
  int jl[KD / 32];
#pragma unroll
  for (int j = 0; j < KD / 32; ++j) jl[j] = col_lane<Cfg::CHK>(c, g, j);
  bare_barrier();
  for (int s = 0; s < chunks; ++s) {
    const unsigned char* Y = lds + (s % Cfg::STAGES) * Cfg::BUF;
    const float* f = reinterpret_cast<const float*>(lds + Cfg::OFF_G + (s & 1) * Cfg::GATE_BYTES);
    const float gc = f[C];
    decay *= gc;
#pragma unroll
    for (int j = 0; j < KD / 16; ++j) z[j] *= gc;
#pragma unroll
    for (int sb = 0; sb < NB; ++sb) {
      const Frag<IN> wf = col_frag_narrow<IN, Cfg::CHV>(Y + Cfg::Y_BYTES, 32 * sb, 16 * wave, c, g);
      const floatx4 f0 = *reinterpret_cast<const floatx4*>(f + 32 * sb + 4 * g);
      const floatx4 f1 = *reinterpret_cast<const floatx4*>(f + 32 * sb + 16 + 4 * g);
      float u[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = frag_value(wf, e) * f0[e];
        u[4 + e] = frag_value(wf, 4 + e) * f1[e];
      }
      const Planes<IN> up = to_planes<IN>(u);
#pragma unroll
      for (int j0 = 0; j0 < KD / 16; j0 += 4) {
        Frag<IN> yf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          yf[j] = col_frag_wide<IN, Cfg::CHK>(Y, 32 * sb, (j0 + j) >> 1, j & 1, c, g, jl[(j0 + j) >> 1]);
#pragma unroll
        for (int q = Planes<IN>::N - 1; q >= 0; --q)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[j0 + j] = mma(yf[j], up.p[q], z[j0 + j]);
      }
    }
    lds_barrier();
  }
  float* to = states + (static_cast<size_t>(pair) * Cfg::OD + od + c) * KD;
#pragma unroll
  for (int j = 0; j < KD / 16; ++j)
    *reinterpret_cast<floatx4*>(to + 32 * (j >> 1) + 8 * g + 4 * (j & 1)) = z[j];
  if (od == 0 && lane == 0) decays[pair] = decay;
}

// One job forwards (blockIdx.y = 0), one backwards (1).
template <Dt IN, int KD, int W>
__global__ __launch_bounds__((LocalCfg<IN, KD, W>::THREADS)) void linear_local_kernel(
    LinearBatch b, LinearStates forward, LinearStates backward) {
  __shared__ __align__(1024) unsigned char lds[LocalCfg<IN, KD, W>::BYTES];
  if (blockIdx.y == 0) local_states<IN, KD, W, false>(b, forward, lds);
  else local_states<IN, KD, W, true>(b, backward, lds);
}

// The chain over a sequence's segments, elementwise: states[u] becomes the state
// in front of segment u's walk.  One thread has four elements; kAhead segments
// are read before the first is needed (4 sequences of 4 segments, 16 heads: 8 us;
// bound by its launch and two dependent reads).
constexpr int kAhead = 8;
__global__ __launch_bounds__(256) void linear_starts_kernel(LinearBatch b, int per,
                                                            LinearStates forward,
                                                            LinearStates backward) {
  const bool BACK = blockIdx.y == 1;
  const LinearStates& job = BACK ? backward : forward;
  const float *from = job.from, *decays = job.decays;
  float *states = job.states, *last = job.last;
  const int blocks = per / 1024, nh = blockIdx.x / blocks;
  const int n = nh / b.H, h = nh % b.H;
  const size_t at = (blockIdx.x % blocks) * 1024 + 4 * threadIdx.x;
  const SequenceUnits units = sequence_units(b, n);
  const int count = units.count;
  floatx4 z = {0.f, 0.f, 0.f, 0.f};
  if (from) z = *reinterpret_cast<const floatx4*>(from + static_cast<size_t>(nh) * per + at);
  if (count == 0) {
    if (last) *reinterpret_cast<floatx4*>(last + static_cast<size_t>(nh) * per + at) = z;
    return;
  }
  for (int i0 = 0; i0 < count; i0 += kAhead) {
    floatx4 own[kAhead];
    float d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= count - 1) continue;  // the last walk's own state is not needed
      const int u = units.at(BACK ? count - 1 - (i0 + i) : i0 + i);
      const size_t pair = static_cast<size_t>(u) * b.H + h;
      own[i] = *reinterpret_cast<const floatx4*>(states + pair * per + at);
      d[i] = decays[pair];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= count) continue;
      const int u = units.at(BACK ? count - 1 - (i0 + i) : i0 + i);
      *reinterpret_cast<floatx4*>(states + (static_cast<size_t>(u) * b.H + h) * per + at) = z;
      if (i0 + i < count - 1) z = d[i] * z + own[i];
    }
  }
}

// ---- gate gradient
//
// One workgroup a (unit, head): suffix sums of row - col from the unit's end, 1024
// tokens at a time (four a thread, 256 apart, whose scans run side by side), in
// fp64.  The roundings of row and col add up like a random walk over the unit, but
// its value at both ends is known as a product of two states (start_dot, end_dot),
// so what the sums miss at the start is spread evenly over the unit's tokens (1024
// tokens, 16 heads: relative error of dg, fp32 inputs, 1.6e-6 without this and 9.4e-7
// with it at gates of -0.8 a token, 4.4e-7 and 2.9e-7 at -0.016).
__global__ __launch_bounds__(256) void linear_dg_kernel(LinearBatch b, const float* row,
                                                        const float* col, const float* start_dot,
                                                        int start_parts, const float* end_dot,
                                                        int end_parts, float* dg, double* unit_sum) {
  constexpr int B = 4, SPAN = 256 * B;
  __shared__ double wave_sum[2][B][4], whole[4];
  const int pair = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = pair % b.H;
  Unit unit;
  double total = 0.0;
  if (unit_at(b, pair / b.H, unit) && unit.te > unit.tb) {
    const size_t units = static_cast<size_t>(b.units) * b.H;
    double acc = 0.0, start = 0.0;
    if (end_dot)
      for (int i = 0; i < end_parts; ++i) acc += end_dot[i * units + pair];
    if (start_dot)
      for (int i = 0; i < start_parts; ++i) start += start_dot[i * units + pair];
    auto load = [&](int t) {
      double v = 0.0;
      if (t >= unit.tb) {
        const size_t at = static_cast<size_t>(h) * b.T_total + t;
        v = static_cast<double>(row[at]) - col[at];
      }
      return v;
    };
    const double to_start = start - acc;
    const int len = unit.te - unit.tb;
    double all = 0.0;  // the sum over the unit (of one span: from its scan)
    if (len > SPAN) {
      for (int t = unit.te - 1 - tid; t >= unit.tb; t -= 256) all += load(t);
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) all += __shfl_xor(all, d);
      if (lane == 0) whole[wave] = all;
      __syncthreads();
      all = whole[0] + whole[1] + whole[2] + whole[3];
    }
    for (int hi = unit.te, slot = 0; hi > unit.tb; hi -= SPAN, slot ^= 1) {
      double v[B];  // thread 0 has the latest token of each block
#pragma unroll
      for (int e = 0; e < B; ++e) v[e] = load(hi - 1 - tid - 256 * e);
#pragma unroll
      for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int e = 0; e < B; ++e) {
          const double up = __shfl_up(v[e], d);
          if (lane >= d) v[e] += up;
        }
#pragma unroll
      for (int e = 0; e < B; ++e)
        if (lane == 63) wave_sum[slot][e][wave] = v[e];
      __syncthreads();
      double sum = 0.0;
#pragma unroll
      for (int e = 0; e < B; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i == wave) v[e] += acc + sum;
          sum += wave_sum[slot][e][i];
        }
      acc += sum;
      if (len <= SPAN) all = sum;
      const double miss = (to_start - all) / len;  // a token
#pragma unroll
      for (int e = 0; e < B; ++e) {
        const int t = hi - 1 - tid - 256 * e;
        if (t < unit.tb) continue;
        double r = v[e] + miss * (unit.te - t);
        if ((b.gates.per_token ? b.gates.g[static_cast<size_t>(t) * b.H + h] : b.gates.g[h]) < kMinGate)
          r = 0.0;  // a decay of zero
        total += r;
        if (dg) dg[static_cast<size_t>(t) * b.H + h] = static_cast<float>(r);
      }
    }
  }
  if (unit_sum) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
    __syncthreads();
    if (lane == 0) whole[wave] = total;
    __syncthreads();
    if (tid == 0) unit_sum[pair] = whole[0] + whole[1] + whole[2] + whole[3];
  }
}

__global__ __launch_bounds__(64) void linear_dg_heads_kernel(LinearBatch b, const double* unit_sum,
                                                             float* dg) {
  const int h = blockIdx.x, lane = threadIdx.x;
  double acc = 0.0;
  for (int u = lane; u < b.units; u += 64) acc += unit_sum[static_cast<size_t>(u) * b.H + h];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) acc += __shfl_xor(acc, d);
  if (lane == 0) dg[h] = static_cast<float>(acc);
}

// Sums over the value heads that share a head: dq (blockIdx.y = 0) and dk (1).
__global__ __launch_bounds__(256) void linear_group_sum_kernel(LinearBatch b, const float* part_q,
                                                               const float* part_k, int group, int d,
                                                               void* dq, void* dk, int out_dtype) {
  const float* part = blockIdx.y == 0 ? part_q : part_k;
  void* out = blockIdx.y == 0 ? dq : dk;
  int te = b.cu[b.N];
  te = te < 0 ? 0 : (te > b.T_total ? b.T_total : te);
  const int hk = b.H / group;
  const size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= static_cast<size_t>(te) * hk * d) return;
  // rows of a token's shared head are `group` rows of its value heads
  const float* from = part + i / d * group * d + i % d;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < group; ++j) acc += *reinterpret_cast<const floatx4*>(from + static_cast<size_t>(j) * d);
  if (out_dtype == 0) {
    uint32_t lo[1], hi[1];
    split2<1>(acc[0], acc[1], lo);
    split2<1>(acc[2], acc[3], hi);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) = make_uint2(lo[0], hi[0]);
  } else {
    *reinterpret_cast<floatx4*>(static_cast<float*>(out) + i) = acc;
  }
}

// One token: row i of a state becomes alpha s_i + v_i k, its output scale s_i . q.
// The state is read once and written once, and that stream is the whole cost:
// 16 lanes to a row with 16-byte non-temporal accesses, ROWS rows of one head a
// workgroup, every load issued before any arithmetic, no LDS.  64 sequences, 32
// heads, 128 x 128: 43.3 us, 6.2 TB/s of state; 3 sequences, 16 heads: 7.9 us, a
// launch.
constexpr int kDecodeThreads = 256;

template <int DK, int DV, Dt IN, Dt OUT, int ROWS>
__global__ __launch_bounds__(kDecodeThreads) void linear_decode_kernel(
    const void* __restrict__ q, const void* __restrict__ k, const void* __restrict__ v,
    LinearGates gates, float* __restrict__ state, void* __restrict__ o, int H, int group,
    int64_t qs, int64_t ks, int64_t vs, float scale) {
  constexpr int RG = kDecodeThreads / 16, RPT = ROWS / RG, VEC = DK / 64, WPP = DV / ROWS;
  const int pair = blockIdx.x / WPP, r0 = (blockIdx.x % WPP) * ROWS;
  const int n = pair / H, h = pair % H, hk = h / group;
  const int lane16 = threadIdx.x & 15, rg = threadIdx.x >> 4;
  floatx4* S = reinterpret_cast<floatx4*>(state + static_cast<size_t>(pair) * DV * DK);
  floatx4 st[RPT][VEC];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      st[i][j] = __builtin_nontemporal_load(&S[((r0 + rg + RG * i) * DK + 4 * lane16 + 64 * j) / 4]);
  float kk[VEC][4], qq[VEC][4], vv[RPT];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const size_t at = static_cast<size_t>(hk) * DK + 4 * lane16 + 64 * j;
    load_vec<IN, 4>(k, n * ks + at, kk[j]);
    load_vec<IN, 4>(q, n * qs + at, qq[j]);
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    vv[i] = load_scalar<IN>(v, n * vs + static_cast<size_t>(h) * DV + r0 + rg + RG * i);
  const float alpha = expf(clamp_gate(gates.per_token ? gates.g[pair] : gates.g[h]));
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = fmaf(vv[i], kk[j][e], alpha * st[i][j][e]);
        st[i][j][e] = x;
        acc = fmaf(x, qq[j][e], acc);
      }
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      __builtin_nontemporal_store(st[i][j], &S[((r0 + rg + RG * i) * DK + 4 * lane16 + 64 * j) / 4]);
    acc = row16_sum(acc);
    if (lane16 == i)
      store_scalar<OUT>(o, static_cast<size_t>(pair) * DV + r0 + rg + RG * i, scale * acc);
  }
}

}  // namespace

hipError_t launch_linear_decode(const void* q, const void* k, const void* v,
                                const LinearGates& g, float* state, void* o, int N, int H, int Hk,
                                int dk, int dv, int64_t qs, int64_t ks, int64_t vs, float scale,
                                int in_dtype, int out_dtype, hipStream_t stream) {
  constexpr int ROWS = 32;
  const dim3 grid(static_cast<unsigned>(N) * H * (dv / ROWS));
  const LinearGates gates = g;
  auto by_out = [&](auto dkc, auto dvc, auto in) {
    constexpr int DK = decltype(dkc)::value, DV = decltype(dvc)::value;
    constexpr Dt IN = decltype(in)::value;
    if (out_dtype == 0)
      hipLaunchKernelGGL((linear_decode_kernel<DK, DV, IN, Dt::BF16, ROWS>), grid, dim3(kDecodeThreads),
                         0, stream, q, k, v, gates, state, o, H, H / Hk, qs, ks, vs, scale);
    else
      hipLaunchKernelGGL((linear_decode_kernel<DK, DV, IN, Dt::F32, ROWS>), grid, dim3(kDecodeThreads),
                         0, stream, q, k, v, gates, state, o, H, H / Hk, qs, ks, vs, scale);
    return hipGetLastError();
  };
  const std::integral_constant<int, 64> d64;
  const std::integral_constant<int, 128> d128;
  auto by_dims = [&](auto in) {
    if (dk == 64) return dv == 64 ? by_out(d64, d64, in) : by_out(d64, d128, in);
    return dv == 64 ? by_out(d128, d64, in) : by_out(d128, d128, in);
  };
  return in_dtype == 0 ? by_dims(std::integral_constant<Dt, Dt::BF16>())
                       : by_dims(std::integral_constant<Dt, Dt::F32>());
}

namespace {

// Calls go(IN, KD, OD) with the types of a pass.
template <class F>
hipError_t by_type(int in_dtype, int kd, int od, F&& go) {
  const std::integral_constant<int, 64> d64;
  const std::integral_constant<int, 128> d128;
  auto with = [&](auto in) {
    if (kd == 64) return od == 64 ? go(in, d64, d64) : go(in, d64, d128);
    return od == 64 ? go(in, d128, d64) : go(in, d128, d128);
  };
  return in_dtype == 0 ? with(std::integral_constant<Dt, Dt::BF16>())
                       : with(std::integral_constant<Dt, Dt::F32>());
}

unsigned scan_grid(const LinearBatch& b) { return static_cast<unsigned>(b.units * b.H); }

}  // namespace

hipError_t launch_linear_prompt(const LinearBatch& b, const LinearPass& p, hipStream_t stream) {
  return by_type(b.in_dtype, p.kd, p.od, [&](auto in, auto kd, auto od) {
    constexpr Dt IN = decltype(in)::value;
    constexpr int KD = decltype(kd)::value, OD = decltype(od)::value;
    hipLaunchKernelGGL((linear_scan_kernel<IN, KD, OD>), dim3(scan_grid(b)),
                       dim3(ScanCfgOf<IN, KD, OD, false>::THREADS), 0, stream, b, p);
    return hipGetLastError();
  });
}

hipError_t launch_linear_grads(const LinearBatch& b, const LinearPass& pq, const LinearPass& pv,
                               const LinearPass& pk, hipStream_t stream) {
  return by_type(b.in_dtype, pv.kd, pv.od, [&](auto in, auto dk, auto dv) {
    constexpr Dt IN = decltype(in)::value;
    constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
    const dim3 grid(scan_grid(b), 3);
    if (pq.dot)
      hipLaunchKernelGGL((linear_grad_kernel<IN, DK, DV, true>), grid,
                         dim3(GradCfg<IN, DK, DV, true>::THREADS), 0, stream, b, pq, pv, pk);
    else
      hipLaunchKernelGGL((linear_grad_kernel<IN, DK, DV, false>), grid,
                         dim3(GradCfg<IN, DK, DV, false>::THREADS), 0, stream, b, pq, pv, pk);
    return hipGetLastError();
  });
}

hipError_t launch_linear_starts(const LinearBatch& b, int od, int kd, const LinearStates& forward,
                                const LinearStates* backward, hipStream_t stream) {
  const int ways = backward ? 2 : 1;
  const LinearStates& back = backward ? *backward : forward;
  const hipError_t e = by_type(b.in_dtype, kd, od, [&](auto in, auto kdim, auto odim) {
    constexpr Dt IN = decltype(in)::value;
    constexpr int KD = decltype(kdim)::value, W = decltype(odim)::value / 16;
    hipLaunchKernelGGL((linear_local_kernel<IN, KD, W>), dim3(scan_grid(b), ways),
                       dim3(LocalCfg<IN, KD, W>::THREADS), 0, stream, b, forward, back);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  const int per = od * kd;
  hipLaunchKernelGGL(linear_starts_kernel, dim3(static_cast<unsigned>(b.N) * b.H * (per / 1024), ways),
                     dim3(256), 0, stream, b, per, forward, back);
  return hipGetLastError();
}

hipError_t launch_linear_dg(const LinearBatch& b, const float* row, const float* col,
                            const float* start_dot, int start_parts, const float* end_dot,
                            int end_parts, float* dg, double* unit_sum, hipStream_t stream) {
  hipLaunchKernelGGL(linear_dg_kernel, dim3(b.units * b.H), dim3(256), 0, stream, b, row, col, start_dot,
                     start_parts, end_dot, end_parts, dg, unit_sum);
  return hipGetLastError();
}

hipError_t launch_linear_dg_heads(const LinearBatch& b, const double* unit_sum, float* dg,
                                  hipStream_t stream) {
  hipLaunchKernelGGL(linear_dg_heads_kernel, dim3(b.H), dim3(64), 0, stream, b, unit_sum, dg);
  return hipGetLastError();
}

hipError_t launch_linear_group_sum(const LinearBatch& b, const float* part_q, const float* part_k,
                                   int group, int d, void* dq, void* dk, int out_dtype,
                                   hipStream_t stream) {
  const size_t n = static_cast<size_t>(b.T_total) * (b.H / group) * d / 4;
  hipLaunchKernelGGL(linear_group_sum_kernel, dim3((n + 255) / 256, 2), dim3(256), 0, stream, b,
                     part_q, part_k, group, d, dq, dk, out_dtype);
  return hipGetLastError();
}

}  // namespace gdr
