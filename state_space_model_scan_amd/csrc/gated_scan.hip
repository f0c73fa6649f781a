// gated_scan.hip -- the gated linear recurrence over packed tokens
// (gated_scan_varlen_fwd), its gradient (gated_scan_varlen_bwd) and its
// single-token step (gated_scan_update).
//
// All three stream: the forward reads three io elements and writes one, the
// gradient reads four and writes three.  What keeps a scan from streaming is
// its order, so the packed tokens are cut into tiles without regard to the
// sequences, each tile is read once and held in registers, and what a tile does
// to the state entering it, h -> P h + H, is formed before that state is known.
// A workgroup takes a tile of 64 NV channels; its waves take its tokens.
//
//   1. a wave folds its tokens to (P, H); the pairs meet in LDS;
//   2. the tile's own pair is published, and the state entering the tile is put
//      together from what the tiles before it have published;
//   3. every wave runs the recurrence from its own entering state and stores.
//
// Tiles come in groups.  A tile joins the state that left the group before with
// the pairs of its group's tiles in order, and a group's last tile publishes the
// state that leaves the group: so the chain of waits has a link per group, and
// the order of every sum is fixed.  The gradient's adjoint goes the same way
// from the last tile to the first; the states it needs come from the forward's
// kept ones, so nothing waits for them.
//
// Measured on bf16 (us; bytes over time): 16384 x 2560 forward 78 (4.4 TB/s, a
// copy makes 5.1), gradient 163 (3.6), 65536 x 2560 forward 255 to 262 (5.2); a
// sequence a thread of every channel took 1973, 2961 and 33887.  What bounds them is
// HBM in the forward of many tokens, in the gradient memory and the vector units in
// turn (78 instructions an element, 64% of the time busy), and below some 10^7 elements
// the workgroups' own length: loads, the pairs' way through LDS, stores.  The step of
// 256 x 5120 takes 5.5 (3.8), that of one request 2.6: latency.
//
// A published pair is one 64-bit store, its own flag: the words are filled with
// ones by a launch before, and P is never that NaN.  A tile waits only for tiles
// of smaller tickets, and a ticket is drawn when its workgroup runs: what is
// waited for is always running or done.  The wait is bounded all the same; at
// its end the state is NaN.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "column_sum.h"
#include "gated_util.h"
#include "host_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

// Shapes: T tokens a wave, W waves a workgroup, G tiles a group.  `Fill` is the
// waves a SIMD that the registers are to allow.
template <int T_, int W_, int G_, int Fill_>
struct Shape {
  static constexpr int T = T_, W = W_, G = G_, Fill = Fill_, Tile = T_ * W_;
};
using Fwd = Shape<16, 8, 8, 4>;
using FwdSmall = Shape<8, 8, 8, 8>;
using BwdMany = Shape<16, 4, 8, 3>;
using BwdLong = Shape<8, 16, 16, 4>;
using BwdSmall = Shape<8, 8, 8, 4>;
static_assert(GATED_CHUNK % Fwd::T == 0 && GATED_CHUNK % FwdSmall::T == 0, "a state is kept by the wave whose first token it enters");
static_assert(BwdMany::Tile % GATED_CHUNK == 0 && BwdLong::Tile % GATED_CHUNK == 0 && BwdSmall::Tile % GATED_CHUNK == 0,
              "a tile of the gradient starts from a kept state");
constexpr int kMaxPolls = 1 << 20;     // of a microsecond or more each

struct GatedParams {
  const void *x, *r, *i, *dout;
  void *out, *dx, *dr, *di;
  const float *A, *rb, *ib, *h0, *dfin;
  float *state, *ckpt, *part, *dinit;
  const int32_t *cu, *seen, *slots;
  unsigned long long *pairs, *ends;    // (tiles, channels) and (groups, channels): what tiles publish
  unsigned *ticket;                    // NULL: one tile of tokens, nothing to wait for
  int64_t total, nseq, channels, nslots, xs, rs, is, os, dos, dxs, drs, dis;
  int tiles, strips;
};

// A wave's tokens of a tensor, as a buffer: an address is the buffer's base, a
// scalar offset (the token's) and a lane's offset (the channels'), which costs a
// load no vector instruction.  The offsets stay below the buffer's 2^31 bytes, as
// validate.cpp refuses strides above 2^24 elements; a lane without channels has
// an offset behind them, where loads give 0 and stores do nothing, so that no
// load or store is in a branch.
template <int IO>
constexpr int kSize = IO == 0 ? 4 : 2;
constexpr uint32_t kBytes = 0x80000000u;

template <int IO>
struct Rows {
  __amdgpu_buffer_rsrc_t at;
  uint32_t step;   // bytes from a token to the next
  __device__ __forceinline__ Rows(const void *p, int64_t stride, int64_t t0, int64_t strip)
      : at(__builtin_amdgcn_make_buffer_rsrc(static_cast<char *>(const_cast<void *>(p)) + (t0 * stride + strip) * kSize<IO>, 0,
                                             kBytes, 0x00027000)),
        step(static_cast<uint32_t>(stride) * kSize<IO>) {}
};
// What a lane reads of token q: 32 bits (two 16-bit elements or one of 32), or a
// single 16-bit element where rows are odd or not aligned.
template <int IO, int NV>
__device__ __forceinline__ uint32_t take(const Rows<IO> &r, uint32_t lane, int q) {
  static_assert(IO ? NV <= 2 : NV == 1, "at most 32 bits");
  if constexpr (IO != 0 && NV == 1) return __builtin_amdgcn_raw_buffer_load_b16(r.at, lane, q * r.step, 0);
  else return __builtin_amdgcn_raw_buffer_load_b32(r.at, lane, q * r.step, 0);
}
template <int IO, int NV>
__device__ __forceinline__ void put(const Rows<IO> &r, uint32_t lane, int q, const float (&v)[NV]) {
  if constexpr (IO == 0)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r.at, lane, q * r.step, 0);
  else if constexpr (NV == 1)
    __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(float_to_half_bits<IO>(v[0])), r.at, lane, q * r.step, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b32(float_to_half_bits<IO>(v[0]) | (float_to_half_bits<IO>(v[1]) << 16), r.at, lane, q * r.step, 0);
}
template <int IO>
__device__ __forceinline__ float part(uint32_t w, int k) {
  if constexpr (IO == 0) return __uint_as_float(w);
  else if constexpr (IO == 1) return __uint_as_float(k ? w & 0xffff0000u : w << 16);
  else return half_bits_to_float<IO>(k ? w >> 16 : w & 0xffffu);
}
// The token that is read for token q of a wave's: behind the last one (and where
// the wave has none) its words come again, so that no load is in a branch.
// Nothing that a token's result depends on lies there.
template <int T>
struct Reads {
  int64_t first;   // the token that is read for token t0
  int last;        // and how many more there are, at most T - 1
  __device__ __forceinline__ Reads(int64_t t0, int64_t total)
      : first(t0 < total ? t0 : total - 1), last(t0 + T <= total ? T - 1 : t0 < total ? static_cast<int>(total - 1 - t0) : 0) {}
  __device__ __forceinline__ int of(int q) const { return q < last ? q : last; }
};

// Which of the tokens t0 .. t0 + T - 1 are the first and the last of their
// sequence, and which belong to one (bit k: token t0 + k).  Uniform.
struct Marks {
  uint32_t first, last, live;
};
// An edge for every lane, asked for before anything else; of 64 and more
// sequences, marks_of looks for those that matter.
__device__ __forceinline__ int32_t edges_of(const GatedParams &p) {
  const int lane = threadIdx.x & 63;
  return p.nseq < 64 ? p.cu[lane < p.nseq ? lane : p.nseq] : 0;
}
template <int T>
__device__ __forceinline__ Marks marks_of(const GatedParams &p, int64_t t0, int32_t edge) {
  static_assert(T <= 16, "two halves of a word");
  const int lane = threadIdx.x & 63;
  uint32_t bits = 0;
  // edge k, d tokens behind t0
  auto add = [&](int64_t k, int64_t d) {
    uint32_t mine = 0;
    if (k < p.nseq && d >= 0 && d < T) mine |= 1u << d;
    if (k > 0 && k <= p.nseq && d > 0 && d <= T) mine |= 0x10000u << (d - 1);
    for (uint64_t b = __ballot(mine != 0); b; b &= b - 1)
      bits |= static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(mine), __builtin_ctzll(b)));
  };
  int64_t from, to;
  if (p.nseq < 64) {
    add(lane, edge - t0);
    from = __builtin_amdgcn_readlane(edge, 0);
    to = __builtin_amdgcn_readlane(edge, static_cast<int>(p.nseq));
  } else {
    int64_t base = wave_search(p.nseq, [&](int64_t s) { return p.cu[s] <= t0; });
    bool more = true;
    while (more) {
      const int64_t k = base + lane, d = (k <= p.nseq ? static_cast<int64_t>(p.cu[k]) : t0 + T + 1) - t0;
      add(k, d);
      more = __ballot(d <= T) == ~0ull;   // all 64 edges are here or before: there may be others
      base += 64;
    }
    from = p.cu[0];
    to = p.cu[p.nseq];
  }
  from -= t0;
  to = (to < p.total ? to : p.total) - t0;
  uint32_t live = to <= 0 ? 0u : to >= T ? (1u << T) - 1 : (1u << to) - 1;
  if (from > 0) live &= from >= T ? 0u : ~((1u << from) - 1);
  return {bits & 0xffffu & live, (bits >> 16) & live, live};
}
// The parameters of channels c .. c + NV - 1.  (Without a bias A is read in its
// place, and not used.)
template <int NV>
__device__ __forceinline__ void channels_of(const GatedParams &p, int64_t c, Channel (&ch)[NV]) {
  const float *rb = p.rb ? p.rb : p.A, *ib = p.ib ? p.ib : p.A;
  float A[NV], r[NV], i[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    A[n] = p.A[c + n];
    r[n] = rb[c + n];
    i[n] = ib[c + n];
  }
#pragma unroll
  for (int n = 0; n < NV; ++n) ch[n] = channel_of(A[n], p.rb ? r[n] : 0.0f, p.ib ? i[n] : 0.0f);
}
// The sequence of token t (every lane has to be there).
__device__ __forceinline__ int64_t sequence_of(const GatedParams &p, int64_t t) {
  return wave_search(p.nseq, [&](int64_t s) { return p.cu[s] <= t; });
}

// ---------------------------------------------------------------------------
// what tiles publish
// ---------------------------------------------------------------------------

constexpr uint32_t kNothing = 0xffffffffu;
constexpr float kFresh = -1.0f;   // P of tokens with a sequence's start among them: nothing that entered is left

// (h -> P h + H) of a state.  Of no state nothing is left, though P be inf, as it
// is over a tile where A > 0: token by token that stays 0.
__device__ __forceinline__ float through(float P, float H, float h) { return P < 0.0f || h == 0.0f ? H : fmaf(P, h, H); }
// P of tokens behind others
__device__ __forceinline__ float joined(float first, float then) { return then < 0.0f || first < 0.0f ? kFresh : first * then; }

__device__ __forceinline__ void publish(unsigned long long *at, float P, float H) {
  const uint32_t flag = P != P ? 0x7fc00000u : __float_as_uint(P);
  __hip_atomic_store(at, flag | static_cast<unsigned long long>(__float_as_uint(H)) << 32, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long look(const unsigned long long *at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool there(unsigned long long v) { return static_cast<uint32_t>(v) != kNothing; }

// The tile of this workgroup: in the order of the tickets, strip by strip.  (There
// are as many tickets as tiles, unless another call draws from the same workspace
// at the same time, which it must not: a ticket beyond the tiles then does nothing.)
__device__ __forceinline__ int draw_ticket(const GatedParams &p) {
  if (!p.ticket) return blockIdx.x;
  __shared__ int drawn;
  if (threadIdx.x == 0) drawn = static_cast<int>(__hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(drawn);
}

__global__ void __launch_bounds__(256) gated_clear_kernel(uint4 *words, int64_t n, unsigned *ticket) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (k < n) words[k] = make_uint4(kNothing, kNothing, kNothing, kNothing);
  if (k == 0) *ticket = 0;
}

// What a workgroup's waves tell each other: their pairs, what the tile has to
// join (place 0 the group before, then the tiles before), and the states that
// enter the waves.
template <int NV, typename Sh>
struct Meeting {
  static constexpr int S = 64 * NV;
  float2 pair[Sh::W][S];
  float2 came[Sh::G][S];
  float enter[Sh::W][S];
  int fresh;   // nothing that enters the tile is used: a sequence starts (in the scan's direction) with it

  __device__ __forceinline__ void tell(int wave, int lane, const float (&p)[NV], const float (&h)[NV]) {
#pragma unroll
    for (int n = 0; n < NV; ++n) pair[wave][lane * NV + n] = make_float2(p[n], h[n]);
  }
  __device__ __forceinline__ void hear(int wave, int lane, float (&h)[NV]) const {
#pragma unroll
    for (int n = 0; n < NV; ++n) h[n] = enter[wave][lane * NV + n];
  }
};

// Publishes the tile's pair, joins what it waits for, and leaves in `enter` the
// states that enter the waves.  k: the tile, counted in the scan's direction
// (BACK: from the last).  Every thread has to be there.  (The loops over pairs
// are unrolled by four: in full they held 32 and more registers at the one place
// where every token's values are held too.)
template <int NV, typename Sh, bool BACK>
__device__ __forceinline__ void link_tile(const GatedParams &p, Meeting<NV, Sh> &m, int k, int64_t strip) {
  constexpr int S = 64 * NV, W = Sh::W, G = Sh::G, kParts = 64 * W / S, kEach = G / kParts;
  static_assert(G % kParts == 0, "every thread looks at as many places");
  const int ch = threadIdx.x % S, part = threadIdx.x / S, j = k % G;
  const int64_t c = strip + ch;
  const bool on = c < p.channels, next = k + 1 < p.tiles, closes = j == G - 1;
  if (p.ticket) {
    const bool looks = k > 0 && !m.fresh;
    if (part == 0 && next && !closes) {
      float P = 1.0f, H = 0.0f;
#pragma unroll 4
      for (int q = 0; q < W; ++q) {
        const float2 v = m.pair[BACK ? W - 1 - q : q][ch];
        H = through(v.x, v.y, H);
        P = joined(P, v.x);
      }
      if (on) publish(p.pairs + static_cast<int64_t>(k) * p.channels + c, P, H);
    }
    unsigned long long got[kEach];
    const unsigned long long *at[kEach];
    bool wait = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int q = part + e * kParts;   // place 0: the group before; place q: the group's tile q - 1
      const bool wants = looks && on && (q == 0 ? k >= G : q <= j);
      at[e] = q == 0 ? p.ends + (static_cast<int64_t>(k / G) - 1) * p.channels + c
                     : p.pairs + (static_cast<int64_t>(k - j) + q - 1) * p.channels + c;
      got[e] = wants ? kNothing : 0ull;
      wait = wait || wants;
    }
    for (int polls = 0; __ballot(wait); ++polls) {
      wait = false;
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (!there(got[e])) {
          got[e] = polls < kMaxPolls ? look(at[e]) : 0x7fc00000bf800000ull;   // (kFresh, NaN)
          wait = wait || !there(got[e]);
        }
      if (__ballot(wait)) __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      m.came[part + e * kParts][ch] =
          make_float2(__uint_as_float(static_cast<uint32_t>(got[e])), __uint_as_float(static_cast<uint32_t>(got[e] >> 32)));
    __syncthreads();
  }
  if (part == 0) {
    float h = 0.0f;
    if (p.ticket) {
      h = m.came[0][ch].y;
#pragma unroll 4
      for (int q = 1; q <= j; ++q) h = through(m.came[q][ch].x, m.came[q][ch].y, h);
    }
#pragma unroll 4
    for (int q = 0; q < W; ++q) {
      const int w = BACK ? W - 1 - q : q;
      m.enter[w][ch] = h;
      h = through(m.pair[w][ch].x, m.pair[w][ch].y, h);
    }
    if (p.ticket && next && closes && on) publish(p.ends + static_cast<int64_t>(k / G) * p.channels + c, 0.0f, h);
  }
  __syncthreads();
}

// A value for each token of `bits` (0 for the others): of[s][c], s the token's
// sequence.  One search at a time: unrolled for every token, the searches were
// most of the kernel's code.
template <int NV, int T>
__device__ __forceinline__ void of_sequences(const GatedParams &p, const float *of, uint32_t bits, int64_t t0, int64_t c, bool on,
                                             float (&v)[T][NV]) {
#pragma unroll
  for (int q = 0; q < T; ++q)
#pragma unroll
    for (int n = 0; n < NV; ++n) v[q][n] = 0.0f;
  if (!of) return;
  for (; bits; bits &= bits - 1) {
    const int at = __builtin_ctz(bits);
    const int64_t s = sequence_of(p, t0 + at);
    float w[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) w[n] = on ? of[s * p.channels + c + n] : 0.0f;
#pragma unroll
    for (int q = 0; q < T; ++q)
#pragma unroll
      for (int n = 0; n < NV; ++n) v[q][n] = q == at ? w[n] : v[q][n];
  }
}
// The cached state of the sequence that starts at token t (0 for a new request).
template <int NV>
__device__ __forceinline__ void cached_state(const GatedParams &p, int64_t t, int64_t c, bool on, float (&h)[NV]) {
#pragma unroll
  for (int n = 0; n < NV; ++n) h[n] = 0.0f;
  if (!p.state || !p.seen) return;
  const int64_t s = sequence_of(p, t), slot = p.slots ? p.slots[s] : s;
  if (slot < 0 || slot >= p.nslots || p.seen[s] <= 0 || !on) return;
#pragma unroll
  for (int n = 0; n < NV; ++n) h[n] = p.state[slot * p.channels + c + n];
}
// The value of token `at` (uniform) of T.
template <int NV, int T>
__device__ __forceinline__ void of_token(const float (&v)[T][NV], int at, float (&w)[NV]) {
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    w[n] = v[0][n];
#pragma unroll
    for (int q = 1; q < T; ++q) w[n] = q == at ? v[q][n] : w[n];
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <int IO, int NV, typename Sh>
__global__ void __launch_bounds__(64 * Sh::W, Sh::Fill) gated_fwd_kernel(const GatedParams p) {
  constexpr int T = Sh::T;
  __shared__ Meeting<NV, Sh> meet;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t edge = edges_of(p);
  const int drawn = draw_ticket(p);
  const int k = drawn / p.strips;
  if (k >= p.tiles) return;
  const int strip = (drawn - k * p.strips) * 64 * NV, c = strip + lane * NV;   // (channels fit 24 bits, as strides do)
  const int64_t t0 = static_cast<int64_t>(k) * Sh::Tile + wave * T;
  const bool on = c < p.channels;
  const uint32_t at = on ? lane * NV * kSize<IO> : kBytes;

  Channel ch[NV];
  channels_of<NV>(p, on ? c : strip, ch);
  uint32_t rw[T], iw[T], xw[T];
  {
    const Reads<T> read(t0, p.total);
    const int64_t t = read.first;
    const Rows<IO> r(p.r, p.rs, t, strip), i(p.i, p.is, t, strip), x(p.x, p.xs, t, strip);
#pragma unroll
    for (int q = 0; q < T; ++q) {   // token by token: the first can be worked on while the others are on their way
      const int k = read.of(q);
      rw[q] = take<IO, NV>(r, at, k);
      iw[q] = take<IO, NV>(i, at, k);
      xw[q] = take<IO, NV>(x, at, k);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const Marks marks = marks_of<T>(p, t0, edge);
  const bool plain = marks.first == 0 && marks.last == 0 && marks.live == (1u << T) - 1;

  float a[T][NV], b[T][NV];
#pragma unroll
  for (int q = 0; q < T; ++q) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const Gates g = gates_of(part<IO>(rw[q], n), part<IO>(iw[q], n), ch[n]);
      a[q][n] = g.a;
      b[q][n] = __builtin_amdgcn_sqrtf(g.m2) * (g.iota * part<IO>(xw[q], n));
    }
    if (q & 1) __builtin_amdgcn_sched_barrier(0);   // (the tokens' temporaries apart)
  }
  // the state before the wave's first token, for the gradient
  const bool keeps = p.ckpt && t0 % GATED_CHUNK == 0 && t0 < p.total;
  auto keep = [&](const float (&v)[NV]) {
    if (on)
#pragma unroll
      for (int n = 0; n < NV; ++n) p.ckpt[t0 / GATED_CHUNK * p.channels + c + n] = v[n];
  };
  float P[NV], H[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    H[n] = 0.0f;
    P[n] = 1.0f;
  }
  if (marks.first == 0) {
#pragma unroll
    for (int q = 0; q < T; ++q)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        H[n] = fmaf(a[q][n], H[n], b[q][n]);
        P[n] *= a[q][n];
      }
  } else {
    for (uint32_t left = marks.first; left; left &= left - 1) {   // a start's cached state enters with its token's input
      const int from = __builtin_ctz(left);
      float h[NV];
      cached_state<NV>(p, t0 + from, c, on, h);   // (now: once the pair is published, the sequence's end may be written)
      if (from == 0 && keeps) keep(h);
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int q = 0; q < T; ++q) b[q][n] = q == from ? fmaf(a[q][n], h[n], b[q][n]) : b[q][n];
    }
#pragma unroll
    for (int q = 0; q < T; ++q)
#pragma unroll
      for (int n = 0; n < NV; ++n) H[n] = marks.first >> q & 1 ? b[q][n] : fmaf(a[q][n], H[n], b[q][n]);
#pragma unroll
    for (int n = 0; n < NV; ++n) P[n] = kFresh;
  }
  meet.tell(wave, lane, P, H);
  if (wave == 0) meet.fresh = marks.first & 1;
  __syncthreads();
  link_tile<NV, Sh, false>(p, meet, k, strip);

  float h[NV];
  meet.hear(wave, lane, h);
  if (keeps && !(marks.first & 1)) {
    float v[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) v[n] = marks.live & 1 ? h[n] : 0.0f;
    keep(v);
  }
  const Rows<IO> out(p.out, p.os, t0, strip);
  if (plain) {
#pragma unroll
    for (int q = 0; q < T; ++q) {
#pragma unroll
      for (int n = 0; n < NV; ++n) h[n] = fmaf(a[q][n], h[n], b[q][n]);
      put<IO, NV>(out, at, q, h);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < T; ++q) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      h[n] = marks.first >> q & 1 ? b[q][n] : fmaf(a[q][n], h[n], b[q][n]);
      b[q][n] = h[n];
    }
    if (marks.live >> q & 1) put<IO, NV>(out, at, q, h);
  }
  if (!p.state) return;
  for (uint32_t left = marks.last; left; left &= left - 1) {
    const int to = __builtin_ctz(left);
    const int64_t s = sequence_of(p, t0 + to), slot = p.slots ? p.slots[s] : s;
    if (slot < 0 || slot >= p.nslots) continue;
    of_token<NV, T>(b, to, h);
    if (on)
#pragma unroll
      for (int n = 0; n < NV; ++n) p.state[slot * p.channels + c + n] = h[n];
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

// Of an element's values the gradient needs after the waves have met: a, and
//   e = m iota     (dx = G e, di = dx x (1 - iota); the input's part of the state is e x)
//   u = a iota / m (q = G rho a (h_{t-1} - u x), dr = A (1 - rho) q)
//   1 - iota, and rho with 1 - rho in one register (in two they did not fit: 202 us
//   for 16384 x 2560 instead of 164; as differences they would lose their bits: 162)
template <int IO, int NV, typename Sh>
__global__ void __launch_bounds__(64 * Sh::W, Sh::Fill) gated_bwd_kernel(const GatedParams p) {
  constexpr int T = Sh::T, W = Sh::W, S = 64 * NV;
  __shared__ Meeting<NV, Sh> meet;   // the adjoint's pairs
  __shared__ float2 fore[W][S];      // the states' pairs; then a wave's sums of q and dr
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t edge = edges_of(p);
  const int drawn = draw_ticket(p);
  const int back = drawn / p.strips, k = p.tiles - 1 - back;   // the last tile first
  if (k < 0) return;
  const int strip = (drawn - back * p.strips) * S, c = strip + lane * NV;
  const int64_t t0 = static_cast<int64_t>(k) * Sh::Tile + wave * T;
  const bool on = c < p.channels;
  const uint32_t at = on ? lane * NV * kSize<IO> : kBytes;

  Channel ch[NV];
  channels_of<NV>(p, on ? c : strip, ch);
  float h[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n)
    h[n] = p.ckpt[static_cast<int64_t>(k) * (Sh::Tile / GATED_CHUNK) * p.channels + (on ? c : strip) + n];
  uint32_t rw[T], iw[T], xw[T], gw[T];
  {
    const Reads<T> read(t0, p.total);
    const int64_t t = read.first;
    const Rows<IO> r(p.r, p.rs, t, strip), i(p.i, p.is, t, strip), x(p.x, p.xs, t, strip), g(p.dout, p.dos, t, strip);
#pragma unroll
    for (int q = 0; q < T; ++q) {
      const int k = read.of(q);
      rw[q] = take<IO, NV>(r, at, k);
      iw[q] = take<IO, NV>(i, at, k);
      xw[q] = take<IO, NV>(x, at, k);
      gw[q] = take<IO, NV>(g, at, k);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const Marks marks = marks_of<T>(p, t0, edge);
  const bool plain = marks.first == 0 && marks.last == 0 && marks.live == (1u << T) - 1;

  // x and dout stay as they were loaded, two 16-bit elements a register, and are
  // unpacked where they are used (the empty assembly keeps the unpacked ones from
  // being kept); the scheduling fences keep the tokens' temporaries apart.
  constexpr bool kPairs = IO != 0 && NV == 1;
  constexpr int kHeld = kPairs ? T / 2 : T;
  uint32_t xh[kHeld], gh[kHeld];
  auto held = [&](const uint32_t (&w)[kHeld], int q, int n) {
    return kPairs ? part<IO>(w[q / 2], q & 1) : part<IO>(w[kPairs ? 0 : q], n);
  };
  auto apart = [&]() {
#pragma unroll
    for (int q = 0; q < kHeld; ++q) asm("" : "+v"(xh[q]), "+v"(gh[q]));
  };
  float a[T][NV], e[T][NV], u[T][NV], gate[T][NV], shut_i[T][NV];
#pragma unroll
  for (int q = 0; q < T; ++q) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const Gates g = gates_of(part<IO>(rw[q], n), part<IO>(iw[q], n), ch[n]);
      const float inv_m = g.m2 > 1e-37f ? __builtin_amdgcn_rsqf(g.m2) : 0.0f;
      a[q][n] = g.a;
      e[q][n] = g.m2 * inv_m * g.iota;
      u[q][n] = g.a * inv_m * g.iota;
      gate[q][n] = fold_gate(g.w_r, g.rho);
      shut_i[q][n] = shut(g.w_i, g.iota);
      // (formed here: put off, what they are formed from took the registers, 171 us for 16384 x 2560 instead of 164)
      asm("" : "+v"(a[q][n]), "+v"(e[q][n]), "+v"(u[q][n]), "+v"(gate[q][n]), "+v"(shut_i[q][n]));
    }
    if constexpr (kPairs) {
      if (q & 1) {
        xh[q / 2] = xw[q - 1] | xw[q] << 16;
        gh[q / 2] = gw[q - 1] | gw[q] << 16;
        asm("" : "+v"(xh[q / 2]), "+v"(gh[q / 2]));
      }
    } else {
      xh[q] = xw[q];
      gh[q] = gw[q];
    }
    if (q & 1) __builtin_amdgcn_sched_barrier(0);
  }
  {
    float P[NV], H[NV], Pb[NV], Hb[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      P[n] = 1.0f;
      H[n] = Hb[n] = 0.0f;
    }
    auto fold = [&](auto inside) {
      constexpr bool kInside = decltype(inside)::value;
      apart();
      float at_edge[kInside ? 1 : T][NV];
      if constexpr (!kInside) of_sequences<NV, T>(p, p.h0, marks.first, t0, c, on, at_edge);
#pragma unroll
      for (int q = 0; q < T; ++q)
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const float from = !kInside && (marks.first >> q & 1) ? at_edge[kInside ? 0 : q][n] : H[n];
          H[n] = fmaf(a[q][n], from, e[q][n] * held(xh, q, n));
          P[n] *= a[q][n];
        }
      if constexpr (!kInside) of_sequences<NV, T>(p, p.dfin, marks.last, t0, c, on, at_edge);
#pragma unroll
      for (int q = T - 1; q >= 0; --q)
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const float from = !kInside && (marks.last >> q & 1) ? at_edge[kInside ? 0 : q][n] : Hb[n];
          Hb[n] = a[q][n] * (held(gh, q, n) + from);
        }
    };
    if (plain) fold(std::true_type{});
    else fold(std::false_type{});
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      Pb[n] = marks.last ? kFresh : P[n];
      P[n] = marks.first ? kFresh : P[n];
      fore[wave][lane * NV + n] = make_float2(P[n], H[n]);
    }
    meet.tell(wave, lane, Pb, Hb);
    if (wave == W - 1) meet.fresh = marks.last >> (T - 1) & 1;
  }
  __syncthreads();
  link_tile<NV, Sh, true>(p, meet, back, strip);

  // The states before this wave's tokens (u becomes what q's other factors act
  // on), then the adjoint; without tests where no sequence starts or ends.
#pragma unroll 4
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const float2 v = fore[w][lane * NV + n];
      h[n] = through(v.x, v.y, h[n]);
    }
  float come[NV], sum[3][NV];
  meet.hear(wave, lane, come);
#pragma unroll
  for (int n = 0; n < NV; ++n) sum[0][n] = sum[1][n] = sum[2][n] = 0.0f;
  const Rows<IO> to_x(p.dx, p.dxs, t0, strip), to_r(p.dr, p.drs, t0, strip), to_i(p.di, p.dis, t0, strip);
  auto walk = [&](auto inside) {
    constexpr bool kInside = decltype(inside)::value;
    apart();
    float at_edge[kInside ? 1 : T][NV];
    if constexpr (!kInside) of_sequences<NV, T>(p, p.h0, marks.first, t0, c, on, at_edge);
#pragma unroll
    for (int q = 0; q < T; ++q) {
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (!kInside && (marks.first >> q & 1)) h[n] = at_edge[kInside ? 0 : q][n];
        const float x = held(xh, q, n);
        u[q][n] = fmaf(-u[q][n], x, h[n]);
        h[n] = fmaf(a[q][n], h[n], e[q][n] * x);
      }
    }
    apart();
    if constexpr (!kInside) of_sequences<NV, T>(p, p.dfin, marks.last, t0, c, on, at_edge);
#pragma unroll
    for (int q = T - 1; q >= 0; --q) {
      float dx[NV], dr[NV], di[NV];
      const bool live = kInside || (marks.live >> q & 1);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (!kInside && (marks.last >> q & 1)) come[n] = at_edge[kInside ? 0 : q][n];
        const float x = held(xh, q, n), adj = held(gh, q, n) + come[n];
        come[n] = a[q][n] * adj;
        float rho, shut_r;
        unfold_gate(gate[q][n], rho, shut_r);
        const float w = come[n] * rho * u[q][n];
        dx[n] = adj * e[q][n];
        dr[n] = ch[n].A * shut_r * w;
        di[n] = dx[n] * shut_i[q][n] * x;
        if (!live) dx[n] = dr[n] = di[n] = 0.0f;
        sum[0][n] += live ? w : 0.0f;
        sum[1][n] += dr[n];
        sum[2][n] += di[n];
        if constexpr (!kInside) u[q][n] = come[n];
      }
      if (kInside || t0 + q < p.total) {
        put<IO, NV>(to_x, at, q, dx);
        put<IO, NV>(to_r, at, q, dr);
        put<IO, NV>(to_i, at, q, di);
      }
      __builtin_amdgcn_sched_barrier(0);   // (the sums at once, not behind the last token from registers)
    }
    if (kInside || !p.dinit) return;
    for (uint32_t left = marks.first; left; left &= left - 1) {
      const int from = __builtin_ctz(left);
      const int64_t s = sequence_of(p, t0 + from);
      float v[NV];
      of_token<NV, T>(u, from, v);
      if (on)
#pragma unroll
        for (int n = 0; n < NV; ++n) p.dinit[s * p.channels + c + n] = v[n];
    }
  };
  if (plain) walk(std::true_type{});
  else walk(std::false_type{});
  // the tile's sums over its tokens, the waves in order
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    fore[wave][lane * NV + n] = make_float2(sum[0][n], sum[1][n]);
    meet.enter[wave][lane * NV + n] = sum[2][n];
  }
  __syncthreads();
  if (wave < 3 && on) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      float v = 0.0f;
#pragma unroll 4
      for (int w = 0; w < W; ++w)
        v += wave == 0 ? fore[w][lane * NV + n].x : wave == 1 ? fore[w][lane * NV + n].y : meet.enter[w][lane * NV + n];
      p.part[(static_cast<int64_t>(k) * 3 + wave) * p.channels + c + n] = v;
    }
  }
}

// The tiles' sums, added; and, by the workgroups behind those, what empty
// sequences pass on.
struct SumParams {
  const float *part, *dfin;
  float *to[3], *dinit;
  const int32_t *cu;
  int64_t tiles, channels, total;
  int sum_blocks;
};
__global__ void __launch_bounds__(kSumThreads) gated_sum_kernel(const SumParams p) {
  if (static_cast<int>(blockIdx.x) >= p.sum_blocks) {
    const int64_t s = blockIdx.x - p.sum_blocks;
    int64_t lo = p.cu[s], hi = p.cu[s + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.total ? p.total : hi;
    if (hi > lo) return;
    for (int64_t c = threadIdx.x; c < p.channels; c += kSumThreads)
      p.dinit[s * p.channels + c] = p.dfin ? p.dfin[s * p.channels + c] : 0.0f;
    return;
  }
  const int64_t cols = 3 * p.channels, col = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const double v = column_sum(p.part, p.tiles, cols, col);
  if (threadIdx.x >= 32 || col >= cols) return;
  const int64_t j = col / p.channels;
  if (p.to[j]) p.to[j][col - j * p.channels] = static_cast<float>(v);
}

// V neighbouring elements (V = 1: at any address)
template <int IO, int V>
struct Vec {
  RawV<IO, V> r;
  __device__ __forceinline__ void load(const void *p, int64_t i) { r.load_vec(p, i); }
  __device__ __forceinline__ float get(int k) const { return r.get(k); }
};
template <int IO>
struct Vec<IO, 1> {
  float v;
  __device__ __forceinline__ void load(const void *p, int64_t i) { v = load_io<IO>(p, i); }
  __device__ __forceinline__ float get(int) const { return v; }
};

struct UpdateParams {
  const void *x, *r, *i;
  void *out;
  const float *A, *rb, *ib;
  float *state;
  const int32_t *seen, *slots;
  int64_t channels, nslots, xs, rs, is, os;
};

// V neighbouring channels a lane: every access of a request's row is 8 to 16
// bytes a lane where the rows allow it.
template <int IO, int V>
__global__ void __launch_bounds__(256) gated_update_kernel(const UpdateParams p) {
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * V;
  if (c >= p.channels) return;
  const int64_t b = blockIdx.x;
  const int64_t slot = p.slots ? p.slots[b] : b;
  const bool cached = slot >= 0 && slot < p.nslots, known = cached && p.seen && p.seen[b] > 0;
  float *state = p.state + (cached ? slot : 0) * p.channels + c;
  const float *rb = p.rb ? p.rb : p.A, *ib = p.ib ? p.ib : p.A;   // (read in the place of biases that are not there)
  Vec<IO, V> x, r, i;
  Vec<0, V> A, rv, iv, h;
  x.load(p.x, b * p.xs + c);
  r.load(p.r, b * p.rs + c);
  i.load(p.i, b * p.is + c);
  h.load(state, 0);
  A.load(p.A, c);
  rv.load(rb, c);
  iv.load(ib, c);
  float out[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const Gates g = gates_of(r.get(k), i.get(k), channel_of(A.get(k), p.rb ? rv.get(k) : 0.0f, p.ib ? iv.get(k) : 0.0f));
    out[k] = fmaf(g.a, known ? h.get(k) : 0.0f, __builtin_amdgcn_sqrtf(g.m2) * (g.iota * x.get(k)));
  }
  if constexpr (V == 1) store_one<IO>(p.out, b * p.os + c, out[0]);
  else store_n<IO, V>(p.out, b * p.os + c, out, V, true);
  if (!cached) return;
  if constexpr (V == 1) state[0] = out[0];
  else store_n<0, V>(state, 0, out, V, true);
}

GatedParams gated_params(const gated_scan_varlen_args_t &a) {
  GatedParams p{};
  p.x = a.x; p.xs = a.x_stride;
  p.r = a.r; p.rs = a.r_stride;
  p.i = a.i; p.is = a.i_stride;
  p.A = a.A; p.rb = a.r_bias; p.ib = a.i_bias; p.cu = a.cu_seqlens;
  p.total = a.total; p.nseq = a.nseq; p.channels = a.channels;
  p.ckpt = a.checkpoints;
  return p;
}

// Rows of 16-bit elements of which two neighbours can be read at once.
bool pairs_of(int32_t io, const void *p, int64_t stride) {
  return io != SSM_F32 && stride % 2 == 0 && (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

// The tiles of a call, and what they publish: pairs (tiles, channels), the
// groups' ends, and the tickets' counter; nothing for a single tile of tokens.
struct Tiling {
  int64_t tiles, words;   // words: of 16 bytes, without the counter's
  size_t bytes;
  int threads;
};
template <typename Sh>
Tiling tiling(int64_t total, int64_t channels) {
  Tiling t{};
  t.tiles = (total + Sh::Tile - 1) / Sh::Tile;
  t.threads = 64 * Sh::W;
  if (t.tiles > 1) {
    t.words = ((t.tiles + (t.tiles + Sh::G - 1) / Sh::G) * channels + 1) / 2;
    t.bytes = static_cast<size_t>(t.words + 1) * 16;
  }
  return t;
}
// Points p at the workspace and enqueues its clearing.  The grid of a launch.
int lay_out(GatedParams &p, const Tiling &t, void *workspace, int nv, hipStream_t stream, unsigned &grid) {
  const int64_t strips = (p.channels + 64 * nv - 1) / (64 * nv);
  if (t.tiles > 0x7fffffffLL / strips || !grid_fits(t.tiles * strips, t.threads)) return SSM_ERR_SHAPE;
  p.tiles = static_cast<int>(t.tiles);
  p.strips = static_cast<int>(strips);
  grid = static_cast<unsigned>(t.tiles * strips);
  if (t.tiles == 1) return SSM_OK;
  p.pairs = static_cast<unsigned long long *>(workspace);
  p.ends = p.pairs + t.tiles * p.channels;
  p.ticket = reinterpret_cast<unsigned *>(static_cast<uint4 *>(workspace) + t.words);
  hipLaunchKernelGGL(gated_clear_kernel, dim3(static_cast<unsigned>((t.words + 255) / 256)), dim3(256), 0, stream,
                     static_cast<uint4 *>(workspace), t.words, p.ticket);
  return SSM_OK;
}

template <typename F>
int by_io(int32_t io, F &&launch) {
  using std::integral_constant;
  if (io == SSM_BF16) launch(integral_constant<int, SSM_BF16>{});
  else if (io == SSM_F16) launch(integral_constant<int, SSM_F16>{});
  else launch(integral_constant<int, SSM_F32>{});
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

namespace {

int64_t parts_of(int64_t n, int64_t size) { return (n + size - 1) / size; }

// How a forward is cut.  Where there are fewer workgroups than compute units, a
// workgroup's own work is what counts, so it is made smaller: single channels a
// lane, then fewer tokens.  Measured on bf16, two channels / one / FwdSmall (us),
// with W the workgroups of two channels a lane:
//   1000 x 2560 (W 160)  13.4 / 14.6 / 17.3     2000 x 512 (W 64)   12.9 / 10.9 / 12.3
//   500 x 2560 (80)      11.5 / 10.3 / 12.2     1000 x 512 (32)     11.3 / 9.6 / 8.9
//   256 x 2560 (40)      11.2 / 9.3 / 8.9       64 x 2560 (20)      7.8 / 5.8 / 4.7
// Up to Fwd's one tile of tokens nothing has to be cleared and waited for, which
// FwdSmall's two have: 128 x 2560 8.3 / 6.3 / 7.7.
bool fwd_small(int64_t total, int64_t channels) {
  if (total > FwdSmall::Tile && total <= Fwd::Tile) return false;
  return 4 * parts_of(total, FwdSmall::Tile) * parts_of(channels, 64) <= 3 * static_cast<int64_t>(cu_count_cached());
}
bool fwd_single(int64_t total, int64_t channels) {
  return 2 * parts_of(total, Fwd::Tile) * parts_of(channels, 128) <= cu_count_cached();
}
Tiling fwd_tiling(const gated_scan_varlen_args_t &a) {
  return fwd_small(a.total, a.channels) ? tiling<FwdSmall>(a.total, a.channels) : tiling<Fwd>(a.total, a.channels);
}

}  // namespace

extern "C" int gated_scan_varlen_fwd_workspace_size(const gated_scan_varlen_args_t *a, size_t *bytes) {
  const int st = gated_scan_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = fwd_tiling(*a).bytes;
  return SSM_OK;
}

extern "C" int gated_scan_varlen_fwd(const gated_scan_varlen_args_t *a, void *stream_ptr) {
  const int st = gated_scan_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  const Tiling t = fwd_tiling(*a);
  if (t.bytes && (!a->workspace || a->workspace_bytes < t.bytes)) return SSM_ERR_WORKSPACE;
  if (t.bytes && !aligned16(a->workspace)) return SSM_ERR_UNSUPPORTED;
  GatedParams p = gated_params(*a);
  p.out = a->out; p.os = a->out_stride;
  p.state = a->state; p.nslots = a->state_slots; p.seen = a->cache_seqlens; p.slots = a->slots;
  const int32_t io = a->io_dtype;
  const bool small = fwd_small(a->total, a->channels);
  const bool two = !small && !fwd_single(a->total, a->channels) && a->channels % 2 == 0 && pairs_of(io, a->x, a->x_stride) &&
                   pairs_of(io, a->r, a->r_stride) && pairs_of(io, a->i, a->i_stride) && pairs_of(io, a->out, a->out_stride);
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  unsigned grid = 0;
  const int laid = lay_out(p, t, a->workspace, two ? 2 : 1, stream, grid);
  if (laid != SSM_OK) return laid;
  return by_io(io, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    if (small) hipLaunchKernelGGL((gated_fwd_kernel<IO, 1, FwdSmall>), dim3(grid), dim3(t.threads), 0, stream, p);
    else if (two) hipLaunchKernelGGL((gated_fwd_kernel<IO, IO ? 2 : 1, Fwd>), dim3(grid), dim3(t.threads), 0, stream, p);
    else hipLaunchKernelGGL((gated_fwd_kernel<IO, 1, Fwd>), dim3(grid), dim3(t.threads), 0, stream, p);
  });
}

namespace {

// How a gradient is cut.  Many small workgroups of many tokens a lane keep the
// memory busiest; where they are few, workgroups of fewer tokens a lane; and where
// a few strips have long chains to wait for, large ones, which have half as many
// links.  Measured on bf16, BwdMany / BwdLong / BwdSmall (us), with the tiles of 64
// tokens and the strips of 64 channels:
//   16384 x 2560 (256 x 40) 162 / 209 / 182     4000 x 512 (63 x 8)  29 / 21 / 28
//   8000 x 2560 (125 x 40)  94 / 112 / 100      2000 x 512 (32 x 8)  20 / 17.7 / 18.3
//   4000 x 2560 (63 x 40)   58 / 61 / 57        1000 x 512 (16 x 8)  17 / 16.9 / 15.2
//   2000 x 2560 (32 x 40)   40 / 38 / 36        256 x 2560 (4 x 40)  17 / 16.2 / 14.5
//   500 x 2560 (8 x 40)     21 / 17.8 / 18.5
//   128 x 2560 (2 x 40: one tile, nothing to wait for)  16 / 12.3 / 13.0
// fp32's inputs take twice the registers, with which BwdMany's 16 tokens do not fit:
//   8192 x 2560 fp32 175 / 138 / 125
enum Cut { kMany, kLong, kSmall };
Cut bwd_cut(const gated_scan_varlen_args_t &f) {
  const int64_t tiles = parts_of(f.total, GATED_CHUNK), all = tiles * parts_of(f.channels, 64), cus = cu_count_cached();
  if (all > 12 * cus) return f.io_dtype == SSM_F32 ? kSmall : kMany;
  return tiles == 2 || (tiles >= 24 && all <= 4 * cus) ? kLong : kSmall;
}
Tiling bwd_tiling(const gated_scan_varlen_args_t &f) {
  const Cut cut = bwd_cut(f);
  return cut == kMany ? tiling<BwdMany>(f.total, f.channels) : cut == kLong ? tiling<BwdLong>(f.total, f.channels)
                                                                            : tiling<BwdSmall>(f.total, f.channels);
}

}  // namespace

extern "C" int gated_scan_varlen_bwd_workspace_size(const gated_scan_varlen_bwd_args_t *a, size_t *bytes) {
  const int st = gated_scan_varlen_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  const Tiling t = bwd_tiling(a->fwd);
  *bytes = t.bytes + static_cast<size_t>(t.tiles) * 3 * a->fwd.channels * sizeof(float);
  return SSM_OK;
}

extern "C" int gated_scan_varlen_bwd(const gated_scan_varlen_bwd_args_t *a, void *stream_ptr) {
  size_t need = 0;
  const int st = gated_scan_varlen_bwd_workspace_size(a, &need);
  if (st != SSM_OK) return st;
  if (!a->workspace || a->workspace_bytes < need) return SSM_ERR_WORKSPACE;
  if (!aligned16(a->workspace)) return SSM_ERR_UNSUPPORTED;
  const gated_scan_varlen_args_t &f = a->fwd;
  const Tiling t = bwd_tiling(f);
  GatedParams p = gated_params(f);
  p.dout = a->dout; p.dos = a->dout_stride;
  p.dx = a->dx; p.dxs = a->dx_stride;
  p.dr = a->dr; p.drs = a->dr_stride;
  p.di = a->di; p.dis = a->di_stride;
  p.h0 = a->initial_states; p.dfin = a->dfinal_states; p.dinit = a->dinitial_states;
  p.part = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + t.bytes);
  SumParams s{};
  s.part = p.part; s.dfin = p.dfin; s.dinit = p.dinit; s.cu = p.cu;
  s.to[0] = a->dA; s.to[1] = a->dr_bias; s.to[2] = a->di_bias;
  s.tiles = t.tiles; s.channels = p.channels; s.total = p.total;
  const int64_t sums = (3 * p.channels + 31) / 32, blocks = sums + (p.dinit ? p.nseq : 0);
  if (!grid_fits(blocks, kSumThreads)) return SSM_ERR_SHAPE;
  s.sum_blocks = static_cast<int>(sums);
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  unsigned grid = 0;
  const int laid = lay_out(p, t, a->workspace, 1, stream, grid);
  if (laid != SSM_OK) return laid;
  const Cut cut = bwd_cut(f);
  return by_io(f.io_dtype, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    auto go = [&](auto shape) {
      hipLaunchKernelGGL((gated_bwd_kernel<IO, 1, decltype(shape)>), dim3(grid), dim3(t.threads), 0, stream, p);
    };
    if (cut == kLong) go(BwdLong{});
    else if (cut == kSmall) go(BwdSmall{});
    else if constexpr (IO != SSM_F32) go(BwdMany{});
    hipLaunchKernelGGL(gated_sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kSumThreads), 0, stream, s);
  });
}

extern "C" int gated_scan_update(const gated_scan_update_args_t *a, void *stream_ptr) {
  const int st = gated_scan_update_validate(a);
  if (st != SSM_OK) return st;
  const int32_t io = a->io_dtype;
  auto wide = [&](const void *p, int64_t stride) {
    return stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (io == SSM_F32 ? 15u : 7u)) == 0;
  };
  const bool four = a->channels % 4 == 0 && wide(a->x, a->x_stride) && wide(a->r, a->r_stride) && wide(a->i, a->i_stride) &&
                    wide(a->out, a->out_stride) && aligned16(a->state) && aligned16(a->A) && aligned16(a->r_bias) &&
                    aligned16(a->i_bias);
  const int64_t gy = (a->channels + (four ? 1023 : 255)) / (four ? 1024 : 256);
  if (gy > 65535 || !grid_fits(a->batch, 256)) return SSM_ERR_SHAPE;
  UpdateParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.r = a->r; p.rs = a->r_stride;
  p.i = a->i; p.is = a->i_stride;
  p.out = a->out; p.os = a->out_stride;
  p.A = a->A; p.rb = a->r_bias; p.ib = a->i_bias;
  p.state = a->state; p.nslots = a->state_slots; p.seen = a->cache_seqlens; p.slots = a->slots;
  p.channels = a->channels;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const dim3 grid(static_cast<unsigned>(a->batch), static_cast<unsigned>(gy));
  return by_io(io, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    if (four) hipLaunchKernelGGL((gated_update_kernel<IO, 4>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((gated_update_kernel<IO, 1>), grid, dim3(256), 0, stream, p);
  });
}
