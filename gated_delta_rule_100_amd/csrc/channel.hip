// channel.hip -- the recurrence with a decay for each channel (gdr_channel_* in
// gdr.h) and its gradient on gfx950.
//
// A token maps a channel's state s to a s + b.  Such maps join, (A', B') after (A, B)
// being (A' A, A' B + B'), so a long sequence is cut up in time and every input is
// still read once:
//   - a thread holds L tokens of V channels in its registers and joins their maps;
//   - the GROUPS threads of a channel in a workgroup meet in LDS: a tile of TT tokens;
//   - tiles of one channel meet in memory: a workgroup publishes its tile's map, reads
//     those of the tiles before it and so has the state that its tile starts from,
//     while its rows wait in registers; then every thread walks its tokens and stores.
// The packed batch is one time axis: the first token of a sequence has a map that
// forgets what was before (kForget in A's place, its own initial state in B), so that ragged
// batches make no difference.  The gradient is the same scan from the last token to the first,
// of c_t = a_t (dh_t + c_{t+1}), whose r_t = dh_t + c_{t+1} gives dx and dg.
//
// Order.  Every join happens in one fixed order, so results do not depend on which
// workgroup is first: tiles of a span (kSpan of them) are folded from the span's first
// on, spans from any span whose state is known, each by the same operation as the one
// that published it.
//
// Waiting.  A workgroup takes its tile by a ticket (an atomic counter) and waits for
// tiles of lower tickets only, which run already, so every wait ends whatever the order
// of dispatch.  What is published is one word, written and read at once (map: two
// floats in 8 bytes, state: 4 bytes), so no fence orders anything; all ones stand for
// "not yet", which a fill kernel writes before each pass.  A wait is bounded all the
// same (kPatience) and a ticket checked, for a workspace that two calls share against the
// rules: their results are wrong, but they end and stay inside their operands.
//
// What bounds it: memory.  2048 channels, 4 sequences of 4096 tokens, bf16 logits and
// complement: 55.5 us, 3.6 TB/s of the bytes that have to move (1 GiB copied: 5.1 TB/s); 8
// ragged sequences, 32768 tokens of 4096 channels, fp32 decays: 225 us, 4.8 TB/s; one of
// 131072 tokens, 512 channels: 102 us, 4.0 TB/s; gradient of the first: 95 us, 4.2 TB/s.
// What is left is a fill kernel (5 us with its launch), the first's vector instructions for
// two exponentials and two reciprocals an element, and tiles that wait for those before.
#include <type_traits>

#include "channel.h"
#include "channel_order.h"
#include "gdr_device.h"

namespace gdr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Tiles of a span, and spans looked back at together.  Measured (prompts and the document of
// above, when they took 59 and 104 us): spans of 16 tiles 64 and 110, of 4 tiles 59 and 114; 8 spans 64 and
// 112, 2 spans 59 and 109, 1 span 59 and 134.
constexpr int kSpan = 8;
constexpr int kBack = 4;
constexpr int kPatience = 1 << 22;
constexpr uint32_t kNone = 0xFFFFFFFFu;

// What workgroups of one pass tell each other, for `width` channels (whole columns).
struct Links {
  uint32_t* ticket;              // [cols] counters, kTicketStep apart
  unsigned long long* tile_map;  // [tiles][width]
  unsigned long long* span_map;  // [spans][width]
  uint32_t* span_end;            // [spans][width] state behind a span
  int tiles, cols;
  size_t width;
};

// Decay a, its complement 1 - a, and log2 a of a GDR_CHANNEL_LOG gate.
struct Decay {
  float a, rest, log2;
};

// 1 - e^g without cancellation: for g above -1/2 the series to g^9 (its next term is below
// 7e-10 of the result), below it 1 - a, which loses at most one bit and a half.
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

// By the hardware's base-2 exponential and reciprocal (one unit in the last place each).  Of a
// logit the smaller of a and 1 - a is q = e^-|z| / (1 + e^-|z|) and the other 1 - q with one
// rounding, no difference that cancels; NaN passes.  Errors of decays close to 1 add up over
// the 1 / (1 - a) tokens that a state remembers: with 1 / (1 + e^-z) for a, bf16 logits of
// sequences of 3000 and 500 tokens left states off by 3e-6, and by 3.6e-7 so, for 2 us of the
// prompts.
template <bool LOGIT, bool REST>
__device__ __forceinline__ Decay decay_of(float g) {
  if constexpr (LOGIT) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(g));
    const float r = __builtin_amdgcn_rcpf(1.f + e), q = e * r, m = fmaf(-e, r, 1.f);
    const bool neg = g < 0.f;
    return {neg ? q : m, neg ? m : q, 0.f};
  } else {
    const float l = kLog2e * g, a = __builtin_amdgcn_exp2f(l);
    return {a, REST ? rest_of_log(g, a) : 0.f, l};
  }
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// V consecutive values of a row as loaded, and some < V of them at a row's end.
template <Dt D, int V>
struct Raw {
  static constexpr int N = D == Dt::BF16 ? V / 2 : V;
  uint32_t w[N];
  __device__ __forceinline__ void load(const void* base, size_t at) {
    const char* p = static_cast<const char*>(base) + at * (D == Dt::BF16 ? 2 : 4);
    if constexpr (N == 2) {
      const uint2 t = *reinterpret_cast<const uint2*>(p);
      w[0] = t.x; w[1] = t.y;
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const u32x4 t = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p) + i);
        w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
      }
    }
  }
  // wherever a row of values starts
  __device__ __forceinline__ void load_any(const void* base, size_t at, int some) {
    if (some >= V) {
      __builtin_memcpy(w, static_cast<const char*>(base) + at * (D == Dt::BF16 ? 2 : 4), sizeof w);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < some) {
          if constexpr (D == Dt::BF16)
            w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at + i]) << i % 2 * 16;
          else w[i] = static_cast<const uint32_t*>(base)[at + i];
        }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (D == Dt::F32) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

template <Dt D, int V>
__device__ __forceinline__ void store_vec(void* base, size_t at, const float (&x)[V]) {
  if constexpr (D == Dt::F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      w[i] = f32_to_bf16_bits(x[2 * i]) | static_cast<uint32_t>(f32_to_bf16_bits(x[2 * i + 1])) << 16;
    char* p = static_cast<char*>(base) + at * 2;
    if constexpr (V == 4) __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2*>(p));
    else __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4*>(p));
  }
}
template <Dt D, int V>
__device__ __forceinline__ void store_any(void* base, size_t at, int some, const float (&x)[V]) {
  if (some >= V) {
    if constexpr (D == Dt::F32) {
      __builtin_memcpy(static_cast<float*>(base) + at, x, sizeof x);
    } else {
      uint32_t w[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        w[i] = f32_to_bf16_bits(x[2 * i]) | static_cast<uint32_t>(f32_to_bf16_bits(x[2 * i + 1])) << 16;
      __builtin_memcpy(static_cast<uint16_t*>(base) + at, w, sizeof w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < some) store_scalar<D>(base, at + i, x[i]);
  }
}

// The V channels from c on of rows: all there and on 16 bytes with ALIGNED, otherwise
// `some` of them wherever they are.
template <int V, bool ALIGNED>
struct Columns {
  int some;
  __device__ __forceinline__ Columns(int D, int c) : some(D - c) {}
  template <Dt D>
  __device__ __forceinline__ void load(Raw<D, V>& r, const void* base, size_t at) const {
    if constexpr (ALIGNED) r.load(base, at);
    else r.load_any(base, at, some);
  }
  template <Dt D>
  __device__ __forceinline__ void store(void* base, size_t at, const float (&x)[V]) const {
    if constexpr (ALIGNED) store_vec<D, V>(base, at, x);
    else store_any<D, V>(base, at, some, x);
  }
  __device__ __forceinline__ void load_state(const float* base, size_t at, float (&x)[V]) const {
    if (!base) {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = 0.f;
    } else {
      Raw<Dt::F32, V> r;
      load(r, base, at);
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = r[v];
    }
  }
};

// A map that starts a sequence has -0 for its A, which no product of decays is: it forgets the
// state before, whatever that is (infinities and NaN do not reach another sequence), and a
// product of decays that is 0 does not (0 times them is NaN: they do not get lost in their own).
constexpr float kForget = -0.f;
__device__ __forceinline__ bool forgets(float A) { return __float_as_uint(A) == 0x80000000u; }
// State behind a map (A, B) from state s, and the A of two maps, A's first.
__device__ __forceinline__ float through(float A, float B, float s) { return forgets(A) ? B : fmaf(A, s, B); }
__device__ __forceinline__ float joined(float A, float then) {
  return forgets(A) || forgets(then) ? kForget : A * then;
}

// Words that workgroups exchange: all ones is "not yet" (a NaN of these bits is
// replaced by another).
__device__ __forceinline__ uint32_t word(float x) {
  const uint32_t w = __float_as_uint(x);
  return w == kNone ? 0x7FC00000u : w;
}
__device__ __forceinline__ void tell(unsigned long long* at, float A, float B) {
  __hip_atomic_store(at, static_cast<unsigned long long>(word(A)) << 32 | word(B), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void tell(uint32_t* at, float x) {
  __hip_atomic_store(at, word(x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T ask(const T* at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
struct Map {
  unsigned long long w;
  __device__ __forceinline__ bool known() const { return static_cast<uint32_t>(w >> 32) != kNone; }
  __device__ __forceinline__ float A() const { return __uint_as_float(static_cast<uint32_t>(w >> 32)); }
  __device__ __forceinline__ float B() const { return __uint_as_float(static_cast<uint32_t>(w)); }
};
constexpr unsigned long long kNoMap = ~0ull;
// A column's counter has 128 bytes to itself.
constexpr int kTicketStep = 32;

// State behind span `span` - 1 of channel ch: from the nearest span whose end state is
// known, or that forgets what was before it, through the maps of those after it.
__device__ __forceinline__ float span_start(const Links& k, int span, size_t ch) {
  for (int tries = 0; tries < kPatience; ++tries) {
    uint32_t end[kBack];
    Map map[kBack];
#pragma unroll
    for (int i = 0; i < kBack; ++i) {
      const int j = span - 1 - i;
      end[i] = kNone;
      map[i].w = kNoMap;
      if (j >= 0) {
        end[i] = ask(k.span_end + j * k.width + ch);
        map[i].w = ask(k.span_map + j * k.width + ch);
      }
    }
    int from = -1;
    bool open = true;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kBack; ++i) {
      if (!open) continue;
      if (end[i] != kNone) {
        s = __uint_as_float(end[i]);
        from = i;
        open = false;
      } else if (!map[i].known()) {
        open = false;
      } else if (forgets(map[i].A())) {
        s = map[i].B();
        from = i;
        open = false;
      }
    }
    if (from >= 0) {
#pragma unroll
      for (int i = kBack - 2; i >= 0; --i)
        if (i < from) s = through(map[i].A(), map[i].B(), s);
      return s;
    }
    __builtin_amdgcn_s_sleep(2);
  }
  return __uint_as_float(0x7FC00000u);
}

// Publishes the map (A, B) of tile `i` (in the order of the pass) for channel ch and
// returns the state that the tile starts from.
__device__ __forceinline__ float tile_start(const Links& k, int i, size_t ch, float A, float B) {
  tell(k.tile_map + i * k.width + ch, A, B);
  const int span = i / kSpan, at = i % kSpan;
  const unsigned long long* first = k.tile_map + static_cast<size_t>(span) * kSpan * k.width + ch;
  Map map[kSpan - 1];
  uint32_t before = kNone;  // the end of the span before, mostly known by now
  if (span > 0) before = ask(k.span_end + (span - 1) * k.width + ch);
#pragma unroll
  for (int j = 0; j < kSpan - 1; ++j) {
    map[j].w = kNoMap;
    if (j < at) map[j].w = ask(first + j * k.width);
  }
  for (int tries = 0; tries < kPatience; ++tries) {
    bool all = true;
#pragma unroll
    for (int j = 0; j < kSpan - 1; ++j)
      if (j < at && !map[j].known()) all = false;
    if (all) break;
    __builtin_amdgcn_s_sleep(1);
#pragma unroll
    for (int j = 0; j < kSpan - 1; ++j)
      if (j < at && !map[j].known()) map[j].w = ask(first + j * k.width);
  }
  // the maps before this tile, joined
  float pa = 1.f, pb = 0.f;
#pragma unroll
  for (int j = 0; j < kSpan - 1; ++j)
    if (j < at) {
      pb = through(map[j].A(), map[j].B(), pb);
      pa = joined(pa, map[j].A());
    }
  const bool last = at == kSpan - 1;
  const float sa = joined(pa, A), sb = through(A, B, pb);
  if (last) tell(k.span_map + span * k.width + ch, sa, sb);
  float s = 0.f;
  if (span > 0 && !forgets(pa)) s = before != kNone ? __uint_as_float(before) : span_start(k, span, ch);
  if (last) tell(k.span_end + span * k.width + ch, through(sa, sb, s));
  return through(pa, pb, s);
}

__global__ void channel_clear_kernel(uint32_t* words, size_t tickets, size_t n) {
  const size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const uint32_t w = i < tickets ? 0 : kNone;
  if (i < n) reinterpret_cast<uint4*>(words)[i] = make_uint4(w, w, w, w);
}

// First m in [0, N] with cu[m] >= t (N + 1 if none), by 64 probes of a wave at a time.
__device__ __forceinline__ int first_at(const int32_t* cu, int N, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = N + 1;  // the answer is in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 63) / 64, i = lo + lane * step;
    const bool below = i < lo + len && cu[i] < t;
    const int c = __popcll(__ballot(below));
    if (step == 1) return lo + c;
    if (c == 0) return lo;
    lo += (c - 1) * step + 1;
    const int rest = N + 1 - lo;
    len = step - 1 < rest ? step - 1 : rest;
  }
  return lo;
}

// Token t of a pass over TT tokens by L per thread, V channels a thread.
template <int V, int L, int THREADS>
struct Shape {
  static constexpr int CC = 128, LANES = CC / V, GROUPS = THREADS / LANES, TT = GROUPS * L;
};

// BACK: the gradient, from the last token to the first.
// Rows wait in registers as loaded and the walk forms its decays anew: decays or maps kept
// in fp32 take 64 registers more, and with fewer waves a compute unit everything is slower.
// Three (bf16 rows with fp32 gates, half as many registers again) or four waves a SIMD are
// what the rows allow without spills.
template <Dt IO, Dt G, bool LOGIT, bool COMP, bool ALIGNED, int V, int L, int THREADS, bool BACK>
__global__ __launch_bounds__(THREADS, BACK ? 1 : IO == Dt::BF16 && G == Dt::F32 ? 3 : 4)
void channel_scan_kernel(Channel p, Links k) {
  using S = Shape<V, L, THREADS>;
  constexpr int CC = S::CC, TT = S::TT, GROUPS = S::GROUPS;
  constexpr bool REST = COMP || (BACK && LOGIT);
  __shared__ uint32_t ticket;
  __shared__ int first_of[TT], last_of[TT];  // sequence that starts, or ends, at a token
  __shared__ int offsets[64];
  __shared__ float map_a[GROUPS][CC], map_b[GROUPS][CC];
  const int tid = threadIdx.x, lane = tid % S::LANES, group = tid / S::LANES;
  const int col = blockIdx.x % k.cols;
  // Offsets of up to 63 sequences: asked for before the rows, which they would wait for
  // (prompts 55.6 us, 59.3 with offsets behind the rows; gradient 94 and 96; but 4096 + 4096
  // tokens of 2048 channels in fp32 50 and 47.7: there they come behind).
  const bool few = (BACK || IO == Dt::BF16) && p.N < 64;
  const int offset = few ? p.cu[min(tid & 63, p.N)] : 0;
  int order = 0;
  if (k.tiles > 1) {
    if (tid == 0) ticket = atomicAdd(k.ticket + col * kTicketStep, 1u);
    lds_barrier();
    if (!has_tile(ticket, k.tiles)) return;
    order = static_cast<int>(ticket);
  }
  const int tile = tile_of_ticket(order, k.tiles, BACK);
  const int t0 = tile * TT, tg = t0 + group * L;
  const int c = col * CC + lane * V;
  const bool mine = c < p.D;
  const Columns<V, ALIGNED> at_c(p.D, c);
  // rows: u is x, or dh of the gradient
  Raw<IO, V> u[L], x[COMP && BACK ? L : 1], prev[BACK ? L : 1];
  Raw<G, V> g[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int t = tg + i;
    if (mine && t < p.T) {
      const size_t row = static_cast<size_t>(t);
      at_c.load(g[i], p.g, row * p.g_stride + c);
      if constexpr (BACK) {
        at_c.load(u[i], p.dh, row * p.D + c);
        if (t > 0) at_c.load(prev[i], p.h, (row - 1) * p.D + c);
        else prev[i] = {};
        if constexpr (COMP) at_c.load(x[i], p.x, row * p.x_stride + c);
      } else {
        at_c.load(u[i], p.x, row * p.x_stride + c);
      }
    }
  }
  // where sequences start and end among the tile's tokens
  for (int i = tid; i < TT; i += THREADS) first_of[i] = last_of[i] = -1;
  const auto inside = [&](int at) { return min(max(at, 0), p.T); };
  int valid, m0;
  if (few) {
    if (tid < 64) offsets[tid] = inside(offset);
    valid = inside(__builtin_amdgcn_readlane(offset, p.N));
    m0 = __popcll(__ballot((tid & 63) <= p.N && offset < t0));
  } else {
    valid = inside(p.cu[p.N]);
    m0 = first_at(p.cu, p.N, t0);
  }
  lds_barrier();
  const auto cu = [&](int m) { return few ? offsets[m] : inside(p.cu[m]); };
  const int until = tile == k.tiles - 1 ? p.T : t0 + TT - 1;  // empty sequences are this tile's up to here
  for (int m = m0 + tid; m <= p.N; m += THREADS) {
    const int at = cu(m);
    if (at > t0 + TT) break;
    if (at < t0) continue;
    if (m < p.N && at < t0 + TT && cu(m + 1) > at) first_of[at - t0] = m;
    if (m > 0 && at > t0 && cu(m - 1) < at) last_of[at - 1 - t0] = m - 1;
  }
  // empty sequences pass their state on
  const float* from = BACK ? p.dstate_out : p.state_in;
  float* to = BACK ? p.dstate_in : p.state_out;
  if (to && mine)
    for (int m = m0 + group; m < p.N; m += GROUPS) {
      const int at = cu(m);
      if (at > until) break;
      if (cu(m + 1) > at) continue;
      float s[V];
      at_c.load_state(from, static_cast<size_t>(m) * p.D + c, s);
      at_c.template store<Dt::F32>(to, static_cast<size_t>(m) * p.D + c, s);
    }
  lds_barrier();
  // the maps of this thread's tokens, joined.  `enter`: sequences whose first token of
  // the pass is here; the state of the latest is kept, for its buffer may be written
  // by the thread that holds the sequence's end (in place) before the walk below.
  const int* enter = BACK ? last_of : first_of;
  float A[V], B[V], kept[V];
  int kept_at = -1;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = LOGIT ? 1.f : 0.f;
    B[v] = 0.f;
  }
  bool forget = false;
  if (mine) {
#pragma unroll
    for (int ii = 0; ii < L; ++ii) {
      const int i = BACK ? L - 1 - ii : ii;
      if (tg + i >= valid) continue;
      const int n = enter[group * L + i];
      if (n >= 0) {
        at_c.load_state(from, static_cast<size_t>(n) * p.D + c, kept);
        kept_at = i;
        forget = true;
#pragma unroll
        for (int v = 0; v < V; ++v) B[v] = kept[v];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Decay d = decay_of<LOGIT, COMP && !BACK>(g[i][v]);
        if constexpr (BACK) {
          B[v] = d.a * (u[i][v] + B[v]);
        } else {
          B[v] = fmaf(d.a, B[v], COMP ? d.rest * u[i][v] : u[i][v]);
        }
        if constexpr (LOGIT) A[v] *= d.a;
        else A[v] += d.log2;  // one exponential of the sum below: one rounding for L decays
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (!LOGIT) A[v] = __builtin_amdgcn_exp2f(A[v]);
      if (forget) A[v] = kForget;
    }
    store_vec<Dt::F32, V>(&map_a[group][0], lane * V, A);
    store_vec<Dt::F32, V>(&map_b[group][0], lane * V, B);
  }
  lds_barrier();
  // one thread a channel: the tile's map, the state it starts from, and each group's
  if (tid < CC && col * CC + tid < p.D) {
    float s = 0.f;
    if (k.tiles > 1) {
      float ta = 1.f, tb = 0.f;
#pragma unroll
      for (int j = 0; j < GROUPS; ++j) {
        const int at = BACK ? GROUPS - 1 - j : j;
        const float ga = map_a[at][tid];
        tb = through(ga, map_b[at][tid], tb);
        ta = joined(ta, ga);
      }
      s = tile_start(k, order, static_cast<size_t>(col) * CC + tid, ta, tb);
    }
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      const int at = BACK ? GROUPS - 1 - j : j;
      const float ga = map_a[at][tid], gb = map_b[at][tid];
      map_b[at][tid] = s;
      s = through(ga, gb, s);
    }
  }
  lds_barrier();
  if (!mine) return;
  float s[V];
  {
    Raw<Dt::F32, V> r;
    r.load(&map_b[group][0], lane * V);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = r[v];
  }
  // the walk
#pragma unroll
  for (int ii = 0; ii < L; ++ii) {
    const int i = BACK ? L - 1 - ii : ii, t = tg + i;
    if (t >= valid) continue;
    const size_t at = static_cast<size_t>(t) * p.D + c;
    const int first = first_of[group * L + i], last = last_of[group * L + i];
    const int in = BACK ? last : first, out = BACK ? first : last;
    if (in >= 0) {
      if (i == kept_at) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = kept[v];
      } else {
        at_c.load_state(from, static_cast<size_t>(in) * p.D + c, s);
      }
    }
    if constexpr (BACK) {
      float before[V], dx[V], dg[V];
      if (first >= 0) {
        at_c.load_state(p.state_in, static_cast<size_t>(first) * p.D + c, before);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) before[v] = prev[i][v];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Decay d = decay_of<LOGIT, REST>(g[i][v]);
        const float r = u[i][v] + s[v];
        s[v] = d.a * r;
        dx[v] = COMP ? d.rest * r : r;
        if constexpr (COMP) before[v] -= x[i][v];
        dg[v] = s[v] * before[v];
        if constexpr (LOGIT) dg[v] *= d.rest;
      }
      at_c.template store<IO>(p.dx, at, dx);
      at_c.template store<G>(p.dg, at, dg);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Decay d = decay_of<LOGIT, REST>(g[i][v]);
        s[v] = fmaf(d.a, s[v], COMP ? d.rest * u[i][v] : u[i][v]);
      }
      at_c.template store<IO>(p.h, at, s);
    }
    if (out >= 0 && to) at_c.template store<Dt::F32>(to, static_cast<size_t>(out) * p.D + c, s);
  }
}

// One token: a thread holds V channels of a sequence.  64 sequences, 4096 channels: 3.1 us,
// a launch.
constexpr int kDecodeThreads = 256;
template <Dt IO, Dt G, bool LOGIT, bool COMP, bool ALIGNED, int V>
__global__ __launch_bounds__(kDecodeThreads) void channel_decode_kernel(Channel p, int pieces) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kDecodeThreads + threadIdx.x;
  if (i >= static_cast<int64_t>(p.N) * pieces) return;
  const int64_t n = i / pieces;
  const int c = static_cast<int>(i % pieces) * V;
  const Columns<V, ALIGNED> at_c(p.D, c);
  Raw<IO, V> x;
  Raw<G, V> g;
  float s[V];
  at_c.load(x, p.x, n * p.x_stride + c);
  at_c.load(g, p.g, n * p.g_stride + c);
  at_c.load_state(p.state_in, n * p.D + c, s);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Decay d = decay_of<LOGIT, COMP>(g[v]);
    s[v] = fmaf(d.a, s[v], COMP ? d.rest * x[v] : x[v]);
  }
  at_c.template store<Dt::F32>(p.state_out, n * p.D + c, s);
  at_c.template store<IO>(p.h, n * p.D + c, s);
}

// Calls go(IO, G, LOGIT, COMP, ALIGNED) for an operand's types and form; ALIGNED where the 8
// (fp32: 4) channels of a thread are on 16 bytes in every row and all there.
template <Dt IO>
constexpr int kChannels = IO == Dt::BF16 ? 8 : 4;
template <class F>
hipError_t by_form(const Channel& p, F&& go) {
  using std::bool_constant;
  using std::integral_constant;
  const int64_t by = p.D | p.x_stride | p.g_stride;
  auto form = [&](auto io, auto g, auto aligned) {
    if (p.gate == 0)
      return p.complement ? go(io, g, bool_constant<false>(), bool_constant<true>(), aligned)
                          : go(io, g, bool_constant<false>(), bool_constant<false>(), aligned);
    return p.complement ? go(io, g, bool_constant<true>(), bool_constant<true>(), aligned)
                        : go(io, g, bool_constant<true>(), bool_constant<false>(), aligned);
  };
  auto width = [&](auto io, auto g) {
    constexpr int V = kChannels<io.value>;
    if (by % V == 0) return form(io, g, bool_constant<true>());
    return form(io, g, bool_constant<false>());
  };
  const integral_constant<Dt, Dt::BF16> bf16;
  const integral_constant<Dt, Dt::F32> f32;
  if (p.io_dtype == 0) return p.g_dtype == 0 ? width(bf16, bf16) : width(bf16, f32);
  return p.g_dtype == 0 ? width(f32, bf16) : width(f32, f32);
}

// Tokens of a tile are 64 at least, and columns have 128 channels.
constexpr int kLeastTile = 64, kColumn = 128;

size_t ticket_bytes(size_t cols) { return cols * kTicketStep * sizeof(uint32_t); }

size_t links_bytes(size_t tiles, size_t cols, size_t width) {
  const size_t spans = (tiles + kSpan - 1) / kSpan;
  return tiles > 1 ? ticket_bytes(cols) + width * (8 * tiles + 12 * spans) : 0;
}

// 8 tokens a thread: with 4, prompts took 65 us (59), the packed batch 256 (232), the document
// 132 (104) and the gradient 94 (96); 16 spill.  Rows that are not on 16
// bytes, 8192 tokens of 2047 channels in bf16: 51 us (76 element by element; 25 at 2048): a lane's
// 16 bytes are then more than one access of the cache, 3 times as many in all, and rows' lines
// are asked for from both sides, 1.4 times as many requests to L2 and 1.5 times the bytes read.
template <bool BACK>
hipError_t launch_scan(const Channel& p, void* workspace, hipStream_t stream) {
  return by_form(p, [&](auto io, auto g, auto logit, auto comp, auto aligned) {
    constexpr int V = kChannels<decltype(io)::value>, L = 8, THREADS = 256;
    using S = Shape<V, L, THREADS>;
    static_assert(S::TT >= kLeastTile && S::CC == kColumn, "workspace sizes");
    Links k{};
    k.tiles = p.T > 0 ? (p.T + S::TT - 1) / S::TT : 1;
    k.cols = (p.D + S::CC - 1) / S::CC;
    k.width = static_cast<size_t>(k.cols) * S::CC;
    if (k.tiles > 1) {
      const size_t spans = (k.tiles + kSpan - 1) / kSpan;
      char* at = static_cast<char*>(workspace);
      k.ticket = reinterpret_cast<uint32_t*>(at);
      k.tile_map = reinterpret_cast<unsigned long long*>(at + ticket_bytes(k.cols));
      k.span_map = k.tile_map + k.tiles * k.width;
      k.span_end = reinterpret_cast<uint32_t*>(k.span_map + spans * k.width);
      const size_t n = links_bytes(k.tiles, k.cols, k.width) / 16;
      hipLaunchKernelGGL(channel_clear_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256),
                         0, stream, k.ticket, ticket_bytes(k.cols) / 16, n);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((channel_scan_kernel<io.value, g.value, logit.value, comp.value, aligned.value, V, L, THREADS, BACK>),
                       dim3(static_cast<unsigned>(k.tiles) * k.cols), dim3(THREADS), 0, stream, p, k);
    return hipGetLastError();
  });
}

}  // namespace

size_t channel_workspace_bytes(int T, int D) {
  const size_t tiles = (static_cast<size_t>(T) + kLeastTile - 1) / kLeastTile;
  const size_t cols = (static_cast<size_t>(D) + kColumn - 1) / kColumn;
  return links_bytes(tiles, cols, cols * kColumn);
}

hipError_t launch_channel_decode(const Channel& p, hipStream_t stream) {
  return by_form(p, [&](auto io, auto g, auto logit, auto comp, auto aligned) {
    constexpr int V = kChannels<decltype(io)::value>;
    const int pieces = (p.D + V - 1) / V;
    const int64_t threads = static_cast<int64_t>(p.N) * pieces;
    hipLaunchKernelGGL((channel_decode_kernel<io.value, g.value, logit.value, comp.value, aligned.value, V>),
                       dim3(static_cast<unsigned>((threads + kDecodeThreads - 1) / kDecodeThreads)), dim3(kDecodeThreads),
                       0, stream, p, pieces);
    return hipGetLastError();
  });
}

hipError_t launch_channel_prefill(const Channel& p, void* workspace, hipStream_t stream) {
  return launch_scan<false>(p, workspace, stream);
}

hipError_t launch_channel_backward(const Channel& p, void* workspace, hipStream_t stream) {
  return launch_scan<true>(p, workspace, stream);
}

}  // namespace gdr
