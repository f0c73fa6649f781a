// conv_runs.h -- which tokens a run of the packed conv computes, sequence by
// sequence.  Plain index arithmetic, so that it also compiles for the host,
// where every layout can be checked without a GPU.
#pragma once

#include <cstdint>

#ifdef __HIPCC__
#define SSM_RUN_FN __host__ __device__ __forceinline__
#else
#define SSM_RUN_FN inline
#endif

namespace ssm {

constexpr int kTaps = 4;

// A sequence's first token (a negative edge stands for 0).
template <typename Edge>
SSM_RUN_FN int64_t first_token(const Edge &edge, int64_t s) {
  const int64_t at = edge(s);
  return at < 0 ? 0 : at;
}

// Whether the tokens [t0, stop) and the kTaps - 1 before them are tokens of
// sequence s, that of t0.
template <typename Edge>
SSM_RUN_FN bool inside_one(const Edge &edge, int64_t s, int64_t t0, int64_t stop) {
  return t0 - first_token(edge, s) >= kTaps - 1 && stop <= edge(s + 1);
}

// The pieces of the run of tokens [t0, t0 + n) that it computes, in order:
// piece(s, from, to, pos, end) for the tokens t0 + from .. t0 + to - 1 of
// sequence s, the first of them its token pos, end the edge after it.  s0 is the
// sequence of token t0.
//
// A sequence's first kTaps - 1 tokens see its ring, and the run with its first
// token overwrites the ring: so that run takes all of them, up to two behind
// its own end, and the next one leaves them out.  One wave then reads and writes
// a ring, and needs no order against another.
template <typename Edge, typename Piece>
SSM_RUN_FN void run_pieces(const Edge &edge, int64_t nseq, int64_t total, int64_t t0, int n, int64_t s0, Piece &&piece) {
  int64_t s = s0, end = edge(s + 1);
  int64_t pos = t0 - first_token(edge, s);
  int from = 0;
  // where the run with a sequence's first token leaves it, counted from t0
  auto taken = [&](int64_t first) {
    const int64_t stop = end < total ? end : total;
    return (first + (kTaps - 1) < stop ? first + (kTaps - 1) : stop) - t0;
  };
  if (pos > 0 && pos < kTaps - 1) {
    const int64_t skip = taken(t0 - pos);
    if (skip > 0) from = static_cast<int>(skip);   // (edges out of order can give less)
    pos += from;
  }
  while (from < n) {
    while (t0 + from >= end && s + 1 < nseq) {
      ++s;
      end = edge(s + 1);
      pos = t0 + from - first_token(edge, s);
    }
    int to = (s + 1 < nseq && end - t0 < n) ? static_cast<int>(end - t0) : n;
    if (pos == 0) {
      const int64_t more = taken(t0 + from);
      if (more > to) to = static_cast<int>(more);
    }
    piece(s, from, to, pos, end);
    pos += to - from;
    from = to;
  }
}

}  // namespace ssm
