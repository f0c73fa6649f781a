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
// A published pair is one 64-bit store, its own flag: the words are filled with
// ones by a launch before, and P is never that NaN.  A tile waits only for tiles
// of smaller tickets, and a ticket is drawn when its workgroup runs: what is
// waited for is always running or done.  The wait is bounded all the same; at
// its end the state is NaN.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gated_util.h"
#include "host_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kGroup = 8;              // tiles of a group
constexpr int kFwdTok = 16;            // tokens of a wave, forward
constexpr int kBwdTok = 8;             // and in the gradient
constexpr int kWaves = 8;              // waves of a workgroup
constexpr int kFwdTile = kFwdTok * kWaves;
constexpr int kBwdTile = kBwdTok * kWaves;
static_assert(kBwdTile == GATED_CHUNK && GATED_CHUNK % kFwdTok == 0, "a tile of the gradient starts from a kept state");
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

// What a lane reads of a token: 32 bits (two 16-bit elements or one of 32), or
// a single 16-bit element where rows are odd or not aligned.
// Addresses are a uniform row and a lane's 32-bit offset.
template <int IO>
struct Elem {
  using type = std::conditional_t<IO == 0, uint32_t, uint16_t>;
};
template <int IO>
__device__ __forceinline__ const void *row_at(const void *p, int64_t i) {
  return static_cast<const typename Elem<IO>::type *>(p) + i;
}
template <int IO>
__device__ __forceinline__ void *row_at(void *p, int64_t i) {
  return static_cast<typename Elem<IO>::type *>(p) + i;
}
template <int IO, int NV>
__device__ __forceinline__ uint32_t take(const void *row, uint32_t bytes) {
  static_assert(IO ? NV <= 2 : NV == 1, "at most 32 bits");
  const char *at = static_cast<const char *>(row) + bytes;
  if constexpr (IO != 0 && NV == 1) return *reinterpret_cast<const uint16_t *>(at);
  else return *reinterpret_cast<const uint32_t *>(at);
}
template <int IO>
__device__ __forceinline__ float part(uint32_t w, int k) {
  if constexpr (IO == 0) return __uint_as_float(w);
  else if constexpr (IO == 1) return __uint_as_float(k ? w & 0xffff0000u : w << 16);
  else return half_bits_to_float<IO>(k ? w >> 16 : w & 0xffffu);
}
template <int IO, int NV>
__device__ __forceinline__ void put(void *row, uint32_t bytes, const float (&v)[NV]) {
  char *at = static_cast<char *>(row) + bytes;
  if constexpr (NV == 1) store_one<IO>(at, 0, v[0]);
  else *reinterpret_cast<uint32_t *>(at) = float_to_half_bits<IO>(v[0]) | (float_to_half_bits<IO>(v[1]) << 16);
}
// The words of T tokens from t0 on (0 behind the last token); at: the lane's offset in a row.
template <int IO, int NV, int T>
__device__ __forceinline__ void take_all(uint32_t (&w)[T], const void *p, int64_t stride, int64_t t0, int64_t strip, int64_t total,
                                         uint32_t at) {
  const int64_t first = t0 * stride + strip;
  if (t0 + T <= total) {
#pragma unroll
    for (int q = 0; q < T; ++q) w[q] = take<IO, NV>(row_at<IO>(p, first + q * stride), at);
  } else {
#pragma unroll
    for (int q = 0; q < T; ++q) w[q] = t0 + q < total ? take<IO, NV>(row_at<IO>(p, first + q * stride), at) : 0u;
  }
}

// Which of the tokens t0 .. t0 + T - 1 are the first and the last of their
// sequence, and which belong to one (bit k: token t0 + k).  Uniform.
struct Marks {
  uint32_t first, last, live;
};
template <int T>
__device__ __forceinline__ Marks marks_of(const GatedParams &p, int64_t t0) {
  static_assert(T <= 16, "two halves of a word");
  const int lane = threadIdx.x & 63;
  uint32_t bits = 0;
  int64_t base = p.nseq < 64 ? 0 : wave_search(p.nseq, [&](int64_t s) { return p.cu[s] <= t0; });
  bool more = true;
  while (more) {
    const int64_t k = base + lane, d = (k <= p.nseq ? static_cast<int64_t>(p.cu[k]) : t0 + T + 1) - t0;
    uint32_t mine = 0;
    if (k < p.nseq && d >= 0 && d < T) mine |= 1u << d;
    if (k > 0 && d > 0 && d <= T) mine |= 0x10000u << (d - 1);
    for (uint64_t b = __ballot(mine != 0); b; b &= b - 1)
      bits |= static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(mine), __builtin_ctzll(b)));
    more = __ballot(d <= T) == ~0ull;   // all 64 edges are here or before: there may be others
    base += 64;
  }
  const int64_t from = p.cu[0] - t0, to = (p.cu[p.nseq] < p.total ? p.cu[p.nseq] : p.total) - t0;
  uint32_t live = to <= 0 ? 0u : to >= T ? (1u << T) - 1 : (1u << to) - 1;
  if (from > 0) live &= from >= T ? 0u : ~((1u << from) - 1);
  return {bits & 0xffffu & live, (bits >> 16) & live, live};
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

// (h -> P h + H) behind (h -> p h + v)
__device__ __forceinline__ float through(float P, float H, float h) { return P < 0.0f ? H : fmaf(P, h, H); }
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

// The tile of this workgroup: in the order of the tickets, strip by strip.
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

// What a workgroup's waves tell each other: their pairs, and the states and
// pairs that its tile has to join (place 0 the group before, then the tiles
// before).
template <int NV>
struct Meeting {
  static constexpr int S = 64 * NV;
  float P[kWaves][S], H[kWaves][S];
  float2 came[kGroup][S];
  int fresh;   // nothing that enters the tile is used: a sequence starts (in the scan's direction) with it

  __device__ __forceinline__ void tell(int wave, int lane, const float (&p)[NV], const float (&h)[NV]) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      P[wave][lane * NV + n] = p[n];
      H[wave][lane * NV + n] = h[n];
    }
  }
};

// Publishes the tile's pair and brings in what it joins.  k: the tile, counted
// in the scan's direction (BACK: from the last).  Every thread has to be there;
// afterwards `came` is complete.
template <int NV, bool BACK>
__device__ __forceinline__ void link_tile(const GatedParams &p, Meeting<NV> &m, int k, int64_t strip) {
  constexpr int S = 64 * NV, kParts = 64 * kWaves / S, kEach = kGroup / kParts;
  static_assert(kGroup % kParts == 0, "every thread looks at as many places");
  const int ch = threadIdx.x % S, part = threadIdx.x / S, j = k % kGroup;
  const int64_t c = strip + ch;
  const bool on = c < p.channels, next = k + 1 < p.tiles, closes = j == kGroup - 1;
  const bool looks = k > 0 && !m.fresh;
  float P = 1.0f, H = 0.0f;
  if (part == 0 && next) {
#pragma unroll
    for (int q = 0; q < kWaves; ++q) {
      const int w = BACK ? kWaves - 1 - q : q;
      H = through(m.P[w][ch], m.H[w][ch], H);
      P = joined(P, m.P[w][ch]);
    }
    if (!closes && on) publish(p.pairs + static_cast<int64_t>(k) * p.channels + c, P, H);
  }
  unsigned long long got[kEach];
  const unsigned long long *at[kEach];
  bool wait = false;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int q = part + e * kParts;   // place 0: the group before; place q: the group's tile q - 1
    const bool wants = looks && on && (q == 0 ? k >= kGroup : q <= j);
    at[e] = q == 0 ? p.ends + (static_cast<int64_t>(k / kGroup) - 1) * p.channels + c
                   : p.pairs + (static_cast<int64_t>(k - j) + q - 1) * p.channels + c;
    got[e] = wants ? kNothing : q == 0 ? 0ull : 0x3f800000ull;   // (P, H) = (1, 0)
    wait = wait || wants;
  }
  for (int polls = 0; __ballot(wait); ++polls) {
    wait = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (!there(got[e])) {
        got[e] = polls < kMaxPolls ? look(at[e]) : 0xffc00000bf800000ull;   // (kFresh, NaN)
        wait = wait || !there(got[e]);
      }
    if (__ballot(wait)) __builtin_amdgcn_s_sleep(1);
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    m.came[part + e * kParts][ch] = make_float2(__uint_as_float(static_cast<uint32_t>(got[e])), __uint_as_float(static_cast<uint32_t>(got[e] >> 32)));
  __syncthreads();
  if (part == 0 && next && closes && on) {
    float h = m.came[0][ch].y;
#pragma unroll
    for (int q = 1; q < kGroup; ++q) h = through(m.came[q][ch].x, m.came[q][ch].y, h);
    publish(p.ends + static_cast<int64_t>(k / kGroup) * p.channels + c, 0.0f, through(P, H, h));
  }
}
// The state entering this wave's tokens; j: the tile's place in its group, -1
// where it is the only tile.
template <int NV, bool BACK>
__device__ __forceinline__ void entering(const Meeting<NV> &m, int j, int wave, int lane, float (&h)[NV]) {
#pragma unroll
  for (int n = 0; n < NV; ++n) h[n] = j < 0 ? 0.0f : m.came[0][lane * NV + n].y;
#pragma unroll
  for (int q = 1; q < kGroup; ++q)
    if (q <= j)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const float2 v = m.came[q][lane * NV + n];
        h[n] = through(v.x, v.y, h[n]);
      }
#pragma unroll
  for (int q = 0; q < kWaves - 1; ++q)
    if (q < (BACK ? kWaves - 1 - wave : wave)) {
      const int w = BACK ? kWaves - 1 - q : q;
#pragma unroll
      for (int n = 0; n < NV; ++n) h[n] = through(m.P[w][lane * NV + n], m.H[w][lane * NV + n], h[n]);
    }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <int IO, int NV>
__global__ void __launch_bounds__(64 * kWaves, 4) gated_fwd_kernel(const GatedParams p) {
  constexpr int T = kFwdTok;
  __shared__ Meeting<NV> meet;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int drawn = draw_ticket(p);
  const int k = drawn / p.strips;
  const int64_t strip = static_cast<int64_t>(drawn - k * p.strips) * 64 * NV, c = strip + lane * NV;
  const int64_t t0 = static_cast<int64_t>(k) * kFwdTile + wave * T;
  const bool on = c < p.channels;
  const uint32_t at = on ? lane * NV * sizeof(typename Elem<IO>::type) : 0;   // (other lanes read what the first one does)

  uint32_t xw[T], rw[T], iw[T];
  take_all<IO, NV, T>(rw, p.r, p.rs, t0, strip, p.total, at);
  take_all<IO, NV, T>(iw, p.i, p.is, t0, strip, p.total, at);
  take_all<IO, NV, T>(xw, p.x, p.xs, t0, strip, p.total, at);
  float A[NV], rb[NV], ib[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    A[n] = on ? p.A[c + n] : 0.0f;
    rb[n] = on && p.rb ? p.rb[c + n] : 0.0f;
    ib[n] = on && p.ib ? p.ib[c + n] : 0.0f;
  }
  const Marks marks = marks_of<T>(p, t0);

  float a[T][NV], b[T][NV];
#pragma unroll
  for (int q = 0; q < T; ++q)
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const Gates g = gates_of(part<IO>(rw[q], n) + rb[n], part<IO>(iw[q], n) + ib[n], A[n]);
      a[q][n] = g.a;
      b[q][n] = g.m * (g.iota * part<IO>(xw[q], n));
    }
  float P[NV], H[NV], start[NV];   // start: the state of a sequence that starts at the wave's first token
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    start[n] = H[n] = 0.0f;
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
#pragma unroll
    for (int q = 0; q < T; ++q) {
      const bool first = marks.first >> q & 1;
      if (first && p.state && p.seen) {   // a start's cached state enters with its token's input
        const int64_t s = sequence_of(p, t0 + q), slot = p.slots ? p.slots[s] : s;
        if (slot >= 0 && slot < p.nslots && p.seen[s] > 0 && on)
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const float h = p.state[slot * p.channels + c + n];
            if (q == 0) start[n] = h;
            b[q][n] = fmaf(a[q][n], h, b[q][n]);
          }
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        H[n] = first ? b[q][n] : fmaf(a[q][n], H[n], b[q][n]);
        P[n] = kFresh;
      }
    }
  }
  meet.tell(wave, lane, P, H);
  if (wave == 0) meet.fresh = marks.first & 1;
  __syncthreads();
  if (p.ticket) link_tile<NV, false>(p, meet, k, strip);

  float h[NV];
  entering<NV, false>(meet, p.ticket ? k % kGroup : -1, wave, lane, h);
  if (p.ckpt && t0 % GATED_CHUNK == 0 && t0 < p.total && on) {
#pragma unroll
    for (int n = 0; n < NV; ++n)
      p.ckpt[t0 / GATED_CHUNK * p.channels + c + n] = marks.first & 1 ? start[n] : marks.live & 1 ? h[n] : 0.0f;
  }
  if (marks.first == 0 && marks.last == 0 && marks.live == (1u << T) - 1) {
#pragma unroll
    for (int q = 0; q < T; ++q) {
#pragma unroll
      for (int n = 0; n < NV; ++n) h[n] = fmaf(a[q][n], h[n], b[q][n]);
      if (on) put<IO, NV>(row_at<IO>(p.out, (t0 + q) * p.os + strip), at, h);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < T; ++q) {
    if (!(marks.live >> q & 1)) continue;
#pragma unroll
    for (int n = 0; n < NV; ++n) h[n] = marks.first >> q & 1 ? b[q][n] : fmaf(a[q][n], h[n], b[q][n]);
    if (on) put<IO, NV>(row_at<IO>(p.out, (t0 + q) * p.os + strip), at, h);
    if (p.state && (marks.last >> q & 1)) {
      const int64_t s = sequence_of(p, t0 + q), slot = p.slots ? p.slots[s] : s;
      if (slot >= 0 && slot < p.nslots && on)
#pragma unroll
        for (int n = 0; n < NV; ++n) p.state[slot * p.channels + c + n] = h[n];
    }
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

// Of an element's values the gradient needs after the waves have met: a, and
//   e = m iota     (dx = G e, di = dx x (1 - iota); the input's part of the state is e x)
//   u = a iota / m (q = G rho a (h_{t-1} - u x), dr = A (1 - rho) q)
template <int IO, int NV>
__global__ void __launch_bounds__(64 * kWaves, 4) gated_bwd_kernel(const GatedParams p) {
  constexpr int T = kBwdTok, S = 64 * NV;
  __shared__ Meeting<NV> meet;   // the adjoint's pairs
  __shared__ float2 fore[kWaves][S];   // the states' pairs; then a wave's sums of q and dr
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int drawn = draw_ticket(p);
  const int back = drawn / p.strips, k = p.tiles - 1 - back;   // the last tile first
  const int64_t strip = static_cast<int64_t>(drawn - back * p.strips) * S, c = strip + lane * NV;
  const int64_t t0 = static_cast<int64_t>(k) * kBwdTile + wave * T;
  const bool on = c < p.channels;
  const uint32_t at = on ? lane * NV * sizeof(typename Elem<IO>::type) : 0;   // (other lanes read what the first one does)

  uint32_t xw[T], rw[T], iw[T], gw[T];
  take_all<IO, NV, T>(rw, p.r, p.rs, t0, strip, p.total, at);
  take_all<IO, NV, T>(iw, p.i, p.is, t0, strip, p.total, at);
  take_all<IO, NV, T>(xw, p.x, p.xs, t0, strip, p.total, at);
  take_all<IO, NV, T>(gw, p.dout, p.dos, t0, strip, p.total, at);
  float A[NV], rb[NV], ib[NV], h[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    A[n] = on ? p.A[c + n] : 0.0f;
    rb[n] = on && p.rb ? p.rb[c + n] : 0.0f;
    ib[n] = on && p.ib ? p.ib[c + n] : 0.0f;
    h[n] = on ? p.ckpt[static_cast<int64_t>(k) * p.channels + c + n] : 0.0f;
  }
  const Marks marks = marks_of<T>(p, t0);
  const bool plain = marks.first == 0 && marks.last == 0 && marks.live == (1u << T) - 1;
  // initial states and final states' gradients, where sequences start and end
  auto edge = [&](const float *of, uint32_t bits, int q, float (&v)[NV]) {
#pragma unroll
    for (int n = 0; n < NV; ++n) v[n] = 0.0f;
    if (of && (bits >> q & 1)) {
      const int64_t s = sequence_of(p, t0 + q);
      if (on)
#pragma unroll
        for (int n = 0; n < NV; ++n) v[n] = of[s * p.channels + c + n];
    }
  };

  float a[T][NV], e[T][NV], u[T][NV], rho[T][NV], iota[T][NV];
#pragma unroll
  for (int q = 0; q < T; ++q)
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const Gates g = gates_of(part<IO>(rw[q], n) + rb[n], part<IO>(iw[q], n) + ib[n], A[n]);
      a[q][n] = g.a;
      e[q][n] = g.m * g.iota;
      u[q][n] = g.a * g.inv_m * g.iota;
      rho[q][n] = g.rho;
      iota[q][n] = g.iota;
    }
  {
    float P[NV], H[NV], Pb[NV], Hb[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      P[n] = 1.0f;
      H[n] = Hb[n] = 0.0f;
    }
    if (plain) {
#pragma unroll
      for (int q = 0; q < T; ++q)
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          H[n] = fmaf(a[q][n], H[n], e[q][n] * part<IO>(xw[q], n));
          P[n] *= a[q][n];
        }
#pragma unroll
      for (int q = T - 1; q >= 0; --q)
#pragma unroll
        for (int n = 0; n < NV; ++n) Hb[n] = a[q][n] * (part<IO>(gw[q], n) + Hb[n]);
#pragma unroll
      for (int n = 0; n < NV; ++n) Pb[n] = P[n];
    } else {
#pragma unroll
      for (int q = 0; q < T; ++q) {
        float h0[NV];
        edge(p.h0, marks.first, q, h0);
        const bool first = marks.first >> q & 1;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          H[n] = fmaf(a[q][n], first ? h0[n] : H[n], e[q][n] * part<IO>(xw[q], n));
          P[n] *= a[q][n];
        }
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) Pb[n] = P[n];
#pragma unroll
      for (int q = T - 1; q >= 0; --q) {
        float fin[NV];
        edge(p.dfin, marks.last, q, fin);
        const bool last = marks.last >> q & 1;
#pragma unroll
        for (int n = 0; n < NV; ++n) Hb[n] = a[q][n] * (part<IO>(gw[q], n) + (last ? fin[n] : Hb[n]));
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (marks.first) P[n] = kFresh;
        if (marks.last) Pb[n] = kFresh;
      }
    }
    meet.tell(wave, lane, Pb, Hb);
#pragma unroll
    for (int n = 0; n < NV; ++n) fore[wave][lane * NV + n] = make_float2(P[n], H[n]);
    if (wave == kWaves - 1) meet.fresh = marks.last >> (T - 1) & 1;
  }
  __syncthreads();
  if (p.ticket) link_tile<NV, true>(p, meet, back, strip);

  // u becomes what q's other factors act on, from the states before the tokens
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
    if (w < wave)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const float2 v = fore[w][lane * NV + n];
        h[n] = through(v.x, v.y, h[n]);
      }
#pragma unroll
  for (int q = 0; q < T; ++q) {
    if (marks.first >> q & 1) edge(p.h0, marks.first, q, h);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const float x = part<IO>(xw[q], n);
      u[q][n] = fmaf(-u[q][n], x, h[n]);
      h[n] = fmaf(a[q][n], h[n], e[q][n] * x);
    }
  }
  float come[NV], sum[3][NV];
  entering<NV, true>(meet, p.ticket ? back % kGroup : -1, wave, lane, come);
#pragma unroll
  for (int n = 0; n < NV; ++n) sum[0][n] = sum[1][n] = sum[2][n] = 0.0f;
#pragma unroll
  for (int q = T - 1; q >= 0; --q) {
    float dx[NV], dr[NV], di[NV];
    if (marks.last >> q & 1) edge(p.dfin, marks.last, q, come);
    const bool live = marks.live >> q & 1;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const float adj = part<IO>(gw[q], n) + come[n];
      come[n] = a[q][n] * adj;
      const float w = come[n] * rho[q][n] * u[q][n];
      dx[n] = adj * e[q][n];
      dr[n] = A[n] * (1.0f - rho[q][n]) * w;
      di[n] = dx[n] * (part<IO>(xw[q], n) * (1.0f - iota[q][n]));
      if (!live) dx[n] = dr[n] = di[n] = 0.0f;
      sum[0][n] += live ? w : 0.0f;
      sum[1][n] += dr[n];
      sum[2][n] += di[n];
    }
    if (on && t0 + q < p.total) {
      put<IO, NV>(row_at<IO>(p.dx, (t0 + q) * p.dxs + strip), at, dx);
      put<IO, NV>(row_at<IO>(p.dr, (t0 + q) * p.drs + strip), at, dr);
      put<IO, NV>(row_at<IO>(p.di, (t0 + q) * p.dis + strip), at, di);
    }
    if (p.dinit && (marks.first >> q & 1)) {
      const int64_t s = sequence_of(p, t0 + q);
      if (on)
#pragma unroll
        for (int n = 0; n < NV; ++n) p.dinit[s * p.channels + c + n] = come[n];
    }
  }
  // the tile's sums over its tokens, the waves in order
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    fore[wave][lane * NV + n] = make_float2(sum[0][n], sum[1][n]);
    meet.P[wave][lane * NV + n] = sum[2][n];
  }
  __syncthreads();
  if (wave < 3 && on) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        v += wave == 0 ? fore[w][lane * NV + n].x : wave == 1 ? fore[w][lane * NV + n].y : meet.P[w][lane * NV + n];
      p.part[(static_cast<int64_t>(k) * 3 + wave) * p.channels + c + n] = v;
    }
  }
}

// Sums of the tiles' sums, four threads a column, each its quarter in order, in
// 64 bits; and, by the blocks behind those, what empty sequences pass on.
struct SumParams {
  const float *part, *dfin;
  float *to[3], *dinit;
  const int32_t *cu;
  int64_t tiles, channels, nseq, total;
  int sum_blocks;
};
__global__ void __launch_bounds__(256) gated_sum_kernel(const SumParams p) {
  __shared__ double sum[4][64];
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  if (static_cast<int>(blockIdx.x) >= p.sum_blocks) {
    const int64_t s = blockIdx.x - p.sum_blocks;
    int64_t lo = p.cu[s], hi = p.cu[s + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.total ? p.total : hi;
    if (hi > lo) return;
    for (int64_t c = threadIdx.x; c < p.channels; c += 256)
      p.dinit[s * p.channels + c] = p.dfin ? p.dfin[s * p.channels + c] : 0.0f;
    return;
  }
  const int64_t cols = 3 * p.channels, col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  double v = 0.0;
  if (col < cols) {
    const int64_t to = p.tiles * (q + 1) / 4;
    int64_t r = p.tiles * q / 4;
    for (; r + 8 <= to; r += 8) {   // eight loads in flight
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = p.part[(r + i) * cols + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += f[i];
    }
    for (; r < to; ++r) v += p.part[r * cols + col];
  }
  sum[q][lane] = v;
  __syncthreads();
  if (q == 0 && col < cols) {
    const int64_t j = col / p.channels;
    if (p.to[j]) p.to[j][col - j * p.channels] = static_cast<float>((sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]));
  }
}

struct UpdateParams {
  const void *x, *r, *i;
  void *out;
  const float *A, *rb, *ib;
  float *state;
  const int32_t *seen, *slots;
  int64_t channels, nslots, xs, rs, is, os;
};

template <int IO>
__global__ void __launch_bounds__(64) gated_update_kernel(const UpdateParams p) {
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 64 + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t b = blockIdx.x;
  const int64_t slot = p.slots ? p.slots[b] : b;
  const bool cached = slot >= 0 && slot < p.nslots;
  const Gates g = gates_of(load_io<IO>(p.r, b * p.rs + c) + (p.rb ? p.rb[c] : 0.0f),
                           load_io<IO>(p.i, b * p.is + c) + (p.ib ? p.ib[c] : 0.0f), p.A[c]);
  float h = cached && p.seen && p.seen[b] > 0 ? p.state[slot * p.channels + c] : 0.0f;
  h = fmaf(g.a, h, g.m * (g.iota * load_io<IO>(p.x, b * p.xs + c)));
  store_one<IO>(p.out, b * p.os + c, h);
  if (cached) p.state[slot * p.channels + c] = h;
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
  int64_t tiles, groups, words;   // words: of 16 bytes, without the counter's
  size_t bytes;
};
Tiling tiling(int64_t total, int64_t channels, int tile) {
  Tiling t{};
  t.tiles = (total + tile - 1) / tile;
  t.groups = (t.tiles + kGroup - 1) / kGroup;
  if (t.tiles > 1) {
    t.words = ((t.tiles + t.groups) * channels + 1) / 2;
    t.bytes = static_cast<size_t>(t.words + 1) * 16;
  }
  return t;
}
// Points p at the workspace and enqueues its clearing.  The grid of a launch.
int lay_out(GatedParams &p, const Tiling &t, void *workspace, int nv, hipStream_t stream, unsigned &grid) {
  const int64_t strips = (p.channels + 64 * nv - 1) / (64 * nv);
  if (t.tiles > 0x7fffffffLL / strips || !grid_fits(t.tiles * strips, 64 * kWaves)) return SSM_ERR_SHAPE;
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

extern "C" int gated_scan_varlen_fwd_workspace_size(const gated_scan_varlen_args_t *a, size_t *bytes) {
  const int st = gated_scan_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = tiling(a->total, a->channels, kFwdTile).bytes;
  return SSM_OK;
}

extern "C" int gated_scan_varlen_fwd(const gated_scan_varlen_args_t *a, void *stream_ptr) {
  const int st = gated_scan_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  const Tiling t = tiling(a->total, a->channels, kFwdTile);
  if (t.bytes && (!a->workspace || a->workspace_bytes < t.bytes)) return SSM_ERR_WORKSPACE;
  if (t.bytes && !aligned16(a->workspace)) return SSM_ERR_UNSUPPORTED;
  GatedParams p = gated_params(*a);
  p.out = a->out; p.os = a->out_stride;
  p.state = a->state; p.nslots = a->state_slots; p.seen = a->cache_seqlens; p.slots = a->slots;
  const int32_t io = a->io_dtype;
  const bool two = a->channels % 2 == 0 && pairs_of(io, a->x, a->x_stride) && pairs_of(io, a->r, a->r_stride) &&
                   pairs_of(io, a->i, a->i_stride) && pairs_of(io, a->out, a->out_stride);
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  unsigned grid = 0;
  const int laid = lay_out(p, t, a->workspace, two ? 2 : 1, stream, grid);
  if (laid != SSM_OK) return laid;
  return by_io(io, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    if (two) hipLaunchKernelGGL((gated_fwd_kernel<IO, IO ? 2 : 1>), dim3(grid), dim3(64 * kWaves), 0, stream, p);
    else hipLaunchKernelGGL((gated_fwd_kernel<IO, 1>), dim3(grid), dim3(64 * kWaves), 0, stream, p);
  });
}

extern "C" int gated_scan_varlen_bwd_workspace_size(const gated_scan_varlen_bwd_args_t *a, size_t *bytes) {
  const int st = gated_scan_varlen_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  const Tiling t = tiling(a->fwd.total, a->fwd.channels, kBwdTile);
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
  const Tiling t = tiling(f.total, f.channels, kBwdTile);
  GatedParams p = gated_params(f);
  p.dout = a->dout; p.dos = a->dout_stride;
  p.dx = a->dx; p.dxs = a->dx_stride;
  p.dr = a->dr; p.drs = a->dr_stride;
  p.di = a->di; p.dis = a->di_stride;
  p.h0 = a->initial_states; p.dfin = a->dfinal_states; p.dinit = a->dinitial_states;
  p.part = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + t.bytes);
  const int32_t io = f.io_dtype;
  const bool two = f.channels % 2 == 0 && pairs_of(io, f.x, f.x_stride) && pairs_of(io, f.r, f.r_stride) &&
                   pairs_of(io, f.i, f.i_stride) && pairs_of(io, a->dout, a->dout_stride) && pairs_of(io, a->dx, a->dx_stride) &&
                   pairs_of(io, a->dr, a->dr_stride) && pairs_of(io, a->di, a->di_stride);
  SumParams s{};
  s.part = p.part; s.dfin = p.dfin; s.dinit = p.dinit; s.cu = p.cu;
  s.to[0] = a->dA; s.to[1] = a->dr_bias; s.to[2] = a->di_bias;
  s.tiles = t.tiles; s.channels = p.channels; s.nseq = p.nseq; s.total = p.total;
  const int64_t sums = (3 * p.channels + 63) / 64, blocks = sums + (p.dinit ? p.nseq : 0);
  if (!grid_fits(blocks, 256)) return SSM_ERR_SHAPE;
  s.sum_blocks = static_cast<int>(sums);
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  unsigned grid = 0;
  const int laid = lay_out(p, t, a->workspace, two ? 2 : 1, stream, grid);
  if (laid != SSM_OK) return laid;
  return by_io(io, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    if (two) hipLaunchKernelGGL((gated_bwd_kernel<IO, IO ? 2 : 1>), dim3(grid), dim3(64 * kWaves), 0, stream, p);
    else hipLaunchKernelGGL((gated_bwd_kernel<IO, 1>), dim3(grid), dim3(64 * kWaves), 0, stream, p);
    hipLaunchKernelGGL(gated_sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, s);
  });
}

extern "C" int gated_scan_update(const gated_scan_update_args_t *a, void *stream_ptr) {
  const int st = gated_scan_update_validate(a);
  if (st != SSM_OK) return st;
  const int64_t gy = (a->channels + 63) / 64;
  if (gy > 65535 || !grid_fits(a->batch, 64)) return SSM_ERR_SHAPE;
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
  return by_io(a->io_dtype, [&](auto io) {
    hipLaunchKernelGGL((gated_update_kernel<decltype(io)::value>), grid, dim3(64), 0, stream, p);
  });
}
