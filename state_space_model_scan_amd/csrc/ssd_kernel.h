// ssd_kernel.h -- the Mamba-2 chunked-scan kernel (included by the sources
// that launch it: ssd.hip for dense rows, ssd_varlen.hip for packed tokens).
// The evaluation, the operand layouts and the work decomposition are
// described at the head of ssd.hip.
#pragma once

#include "ssd_util.h"

namespace ssm {
namespace {

struct SsdParams {
  const uint16_t *x, *dt, *B, *C, *z;
  const float *A, *D, *dt_bias, *init;
  const int32_t *seq_idx;
  uint16_t *out;
  float *fin;
  float *ws_state, *ws_decay;   // sequence split: end states from zero, total decays
  const float *carried;         // chunk scan: the state entering every segment (no fold)
  int64_t seqlen, nheads, ngroups, seg_chunks;
  int D_per_channel, softplus, dt_limit, nseg;
  float dt_min, dt_max;
  // packed tokens (VAR): elements between tokens, the sequences' edges, the
  // cache of states and the chunks' 8-bit states
  int64_t xs, dts, bs, cs, zs, os;
  const int32_t *cu, *seen, *slots;
  int64_t total, max_seqlen, cache_slots;
  float *cache;
  int8_t *codes;
  float *scales;
};

// The two launches of a sequence split: SSD_STATE finds each segment's end
// state from zero and its total decay; SSD_FULL starts every segment from the
// carried state and computes the outputs (one launch of it without a split).
enum { SSD_STATE = 0, SSD_FULL = 1 };

// A state row in 8 bits: v ~ code * 2^e with the smallest e for which every
// |v| <= 127 * 2^e.  The scale is a power of two so that a code's value is
// exact in bf16 (seven bits times a power of two) and can enter a matrix
// product as it is.  Against the scale amax / 127 it costs half a bit on
// average.  e >= -100 keeps the values normal numbers.  A row with an
// infinity or a NaN gets a NaN scale.
__device__ __forceinline__ float row_scale(uint32_t amax_bits, float &inv) {
  if (amax_bits >= 0x7f800000u) {
    inv = 0.0f;
    return __uint_as_float(0x7fc00000u);
  }
  // 127 = 1.984375 * 2^6, and 1.984375 has the fraction bits 0x7e0000
  int e = static_cast<int>(amax_bits >> 23) - 127 - 6 + ((amax_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  e = e < -100 ? -100 : e;
  inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// SEQ: packed sequences (seq_idx given); a template value so that the
// kernel without them keeps its registers.
// VAR: packed tokens.  b is a sequence, which begins at token cu[b]; tensors
// have token strides; states come from and go to a cache; every chunk's
// entering state may be kept in 8 bits.  The steps use the softplus without
// cancellation: a step near 0.001 would lose four digits otherwise, and the
// states are compared in 32 bits.
template <int N, int MODE, bool SEQ, bool VAR = false>
__global__ void __launch_bounds__(256, 2) ssd_kernel(const SsdParams p) {
  constexpr bool FULL = MODE == SSD_FULL;
  constexpr int KN = N / 32;   // K steps over dstate
  constexpr int NT = N / 16;   // state tiles along dstate
  __shared__ __attribute__((aligned(16))) uint16_t sXT[kP * kQ];   // X^T   [p][t]
  __shared__ __attribute__((aligned(16))) uint16_t sBT[N * kQ];    // B^T   [n][t]
  // M [t][tau] as hi / lo bf16, and the chunk's C [t][n] (full pass only)
  __shared__ __attribute__((aligned(16))) uint16_t sM[FULL ? 2 : 1][FULL ? kQ * kQ : 8];
  __shared__ __attribute__((aligned(16))) uint16_t sC[FULL ? kQ * N : 8];
  __shared__ __attribute__((aligned(16))) uint16_t sBrow[FULL ? kQ * N : 8];   // B [t][n] (full pass)
  __shared__ __attribute__((aligned(16))) float sCs[kQ], sDt[kQ], sW[kQ];
  __shared__ __attribute__((aligned(16))) int32_t sSid[SEQ ? kQ : 4];

  const int tid = threadIdx.x;
  const int w = tid >> 6, l = tid & 63, r = l & 15, kq = l >> 4;
  const int64_t bh = blockIdx.x;
  const int64_t BH = gridDim.x;
  // the full pass runs its last (in the library's own plan the longest)
  // segment's workgroups first: they are dispatched in blockIdx order
  const int seg = FULL ? static_cast<int>(gridDim.y) - 1 - static_cast<int>(blockIdx.y)
                       : static_cast<int>(blockIdx.y);
  const int64_t b = bh / p.nheads;
  const int64_t h = bh - b * p.nheads;
  const int64_t g = h / (p.nheads / p.ngroups);
  // packed tokens: an edge outside the tokens, or out of order, is moved
  // inside, so that no access leaves the tensors
  int64_t first = 0, L = p.seqlen;
  int64_t slot = -1;
  if constexpr (VAR) {
    int64_t lo = p.cu[b], hi = p.cu[b + 1];
    lo = lo < 0 ? 0 : lo > p.total ? p.total : lo;
    hi = hi < lo ? lo : hi > p.total ? p.total : hi;
    first = lo;
    L = hi - lo > p.max_seqlen ? p.max_seqlen : hi - lo;
    slot = p.slots ? p.slots[b] : b;
    if (slot >= p.cache_slots) slot = -1;
  }
  const float Ah = p.A[h];
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
  // elements between tokens of x, z, out, B, C and dt
  const int64_t xrow = VAR ? p.xs : p.nheads * kP, zrow = VAR ? p.zs : xrow, orow = VAR ? p.os : xrow;
  const int64_t bcrow = VAR ? p.bs : p.ngroups * N, crow = VAR ? p.cs : bcrow;
  const int64_t dtrow = VAR ? p.dts : p.nheads;
  const uint16_t *xb, *zb, *Bb, *Cb, *dtb;
  uint16_t *ob;
  if constexpr (VAR) {
    xb = p.x + first * xrow + h * kP;
    zb = p.z ? p.z + first * zrow + h * kP : nullptr;
    ob = p.out + first * orow + h * kP;
    Bb = p.B + first * bcrow + g * N;
    Cb = p.C + first * crow + g * N;
    dtb = p.dt + first * dtrow + h;
  } else {
    xb = p.x + (b * L * p.nheads + h) * kP;
    zb = p.z ? p.z + (b * L * p.nheads + h) * kP : nullptr;
    ob = p.out + (b * L * p.nheads + h) * kP;
    Bb = p.B + (b * L * p.ngroups + g) * N;
    Cb = p.C + (b * L * p.ngroups + g) * N;
    dtb = p.dt + b * L * p.nheads + h;
  }
  const int32_t *sidb = SEQ ? p.seq_idx + b * L : nullptr;
  const bf16x8 zero8 = {};

  const int64_t nchunks = (L + kQ - 1) / kQ;
  const int64_t c_begin = seg * p.seg_chunks;
  int64_t c_end = seg + 1 < p.nseg ? c_begin + p.seg_chunks : nchunks;
  // A sequence may be shorter than the longest one's segments.  The state
  // pass runs the segments that have one after them in their sequence.
  bool last_seg = seg + 1 == p.nseg;
  const float *cached = nullptr;   // the state before the sequence's first token (VAR)
  if constexpr (VAR) {
    if (c_end > nchunks) c_end = nchunks;
    last_seg = c_end == nchunks;
    if (seg > 0 && c_begin >= nchunks) return;
    if (!FULL && last_seg) return;
    if (p.cache && slot >= 0 && (p.seen && p.seen[b] > 0)) cached = p.cache + (slot * p.nheads + h) * kP * N;
  }

  // Token pairs and channel groups this thread stages and stores:
  // tokens 2 (tid / 8) + {0, 1}, channels 8 (tid % 8) + 0..7.
  const int xt0 = 2 * (tid >> 3), xp0 = (tid & 7) * 8;
  // D of those channels
  float Dv8[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pp = xp0 + i;
    Dv8[i] = (FULL && p.D) ? (p.D_per_channel ? p.D[h * kP + pp] : p.D[h]) : 0.0f;
  }
  // Y [t][p] (fp32, 16-byte groups permuted by t): in the row-major B copy's
  // space where it fits (dstate 128), which its last reader left before M was
  // stored, so the Y stores need no barrier after the products that read M;
  // otherwise over M
  constexpr bool Y_IN_BR = FULL && kQ * N * 2 >= kQ * kP * 4;
  float *sY = Y_IN_BR ? reinterpret_cast<float *>(sBrow) : reinterpret_cast<float *>(&sM[0][0]);
  uint16_t *sBr = sBrow;   // B row-major [t][n] for the A operand of C B^T

  // state, transposed: wave w holds S[p = 16w + r][n = 16 nt + 4kq + i].
  // The state pass starts every segment from zero; the full pass starts
  // segment k from the initial state carried over segments 0..k-1:
  //   S_in(k) = E_{k-1} + P_{k-1} (E_{k-2} + P_{k-2} (... + P_0 S_init))
  // with E_j segment j's end state from zero and P_j its total decay (zero
  // where a sequence starts inside it).
  // With carried states given (the chunk scan on its own) segment k starts
  // from carried[k] as it is.
  f32x4 accs[NT];
  const int srow = (16 * w + r) * N + 4 * kq;   // this lane's first state element in a (p, n) block
  // Packed tokens: the last segment's workgroup writes the cache while others
  // may still be starting, so a sequence of several segments reads it in the
  // state pass alone: E_0 includes the cached state, and segment 0's start is
  // a copy that the state pass leaves behind the E's.
  const float *start = p.carried ? p.carried + seg * BH * kP * N : p.init;
  if constexpr (VAR) {
    start = nullptr;
    if (cached && seg == 0) {
      if (!FULL || last_seg) start = cached;
      else start = p.ws_state + ((p.nseg - 1) * BH + bh) * kP * N;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 s4 = start ? *reinterpret_cast<const float4 *>(start + srow + 16 * nt) : make_float4(0, 0, 0, 0);
      accs[nt] = (f32x4){s4.x, s4.y, s4.z, s4.w};
      if (!FULL && cached && seg == 0)
        *reinterpret_cast<float4 *>(p.ws_state + ((p.nseg - 1) * BH + bh) * kP * N + srow + 16 * nt) = s4;
    }
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        accs[nt][i] = (FULL && start) ? start[bh * kP * N + srow + 16 * nt + i] : 0.0f;
    }
  }
  if constexpr (FULL) {
    const int nfold = p.carried ? 0 : seg;
    for (int j = 0; j < nfold; ++j) {
      const float P = p.ws_decay[j * BH + bh];
      const float *E = p.ws_state + (j * BH + bh) * kP * N + srow;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 e4 = *reinterpret_cast<const float4 *>(E + 16 * nt);
        accs[nt][0] = fmaf(P, accs[nt][0], e4.x);
        accs[nt][1] = fmaf(P, accs[nt][1], e4.y);
        accs[nt][2] = fmaf(P, accs[nt][2], e4.z);
        accs[nt][3] = fmaf(P, accs[nt][3], e4.w);
      }
    }
  }
  __syncthreads();

  // sequence id the incoming state belongs to: the token before the segment
  // (the first token for the initial state)
  int32_t sid_prev = 0;
  if constexpr (SEQ) sid_prev = sidb[c_begin > 0 ? c_begin * kQ - 1 : 0];
  float seg_decay = 1.0f;   // product of the chunks' decays (state pass)

  constexpr int G8 = N / 8;                      // 16-byte groups per B row
  constexpr int BPIECES = (kQ / 2) * G8;        // (token pair, 16-byte group) pieces of a B tile
  constexpr int BPAIRS = (BPIECES + 255) / 256;  // pieces per thread
  for (int64_t c = c_begin; c < c_end; ++c) {
    const int64_t t0 = c * kQ;
    const int len = static_cast<int>((L - t0 < kQ) ? L - t0 : kQ);

    if constexpr (VAR && FULL) {
      if (p.codes) {
        // the chunk's entering state in 8 bits: this lane holds 4 NT states
        // of row 16w + r, the row's others are 16, 32 and 48 lanes away
        uint32_t top = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = __float_as_uint(accs[nt][i]) & 0x7fffffffu;
            top = v > top ? v : top;
          }
        uint32_t o = __shfl_xor(top, 16);
        top = o > top ? o : top;
        o = __shfl_xor(top, 32);
        top = o > top ? o : top;
        float inv;
        const float scale = row_scale(top, inv);
        const int64_t row = ((first / kQ + b + c) * p.nheads + h) * kP + 16 * w + r;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t word = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            word |= (static_cast<uint32_t>(static_cast<int>(rintf(accs[nt][i] * inv))) & 0xffu) << (8 * i);
          *reinterpret_cast<uint32_t *>(p.codes + row * N + 16 * nt + 4 * kq) = word;
        }
        if (kq == 0) p.scales[row] = scale;
      }
    }

    // ---- every global load of the chunk first, so their latencies overlap
    uint4 xr[2], zr[2], br[BPAIRS][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = xt0 + k;
      xr[k] = t < len ? ld8_raw(xb + (t0 + t) * xrow + xp0) : make_uint4(0, 0, 0, 0);
      zr[k] = (FULL && zb && t < len) ? ld8_raw(zb + (t0 + t) * zrow + xp0) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < BPAIRS; ++j) {
      const int piece = tid + 256 * j;
      const int t = 2 * (piece / G8), n0 = (piece % G8) * 8;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        br[j][k] = (piece < BPIECES && t + k < len) ? ld8_raw(Bb + (t0 + t + k) * bcrow + n0)
                                                     : make_uint4(0, 0, 0, 0);
    }
    bf16x8 cop[FULL ? KN : 1];   // this wave's C rows (tokens 16w + r)
    if constexpr (FULL) {
      const int t = 16 * w + r;
#pragma unroll
      for (int kk = 0; kk < KN; ++kk) cop[kk] = t < len ? ld8(Cb + (t0 + t) * crow + 32 * kk + 8 * kq) : zero8;
    }
    float dtraw = 0.0f;
    int32_t sid = 0;
    if (w == 0 || (VAR && w == 1)) {
      if (l < len) dtraw = bf2f(dtb[(t0 + l) * dtrow]);
      if constexpr (SEQ) sid = sidb[t0 + (l < len ? l : len - 1)];
    }

    // the previous chunk's reads of the staged tiles (and, in the full pass,
    // its epilogue's reads of Y, which shares its space with the row-major B
    // copy at dstate 128 and with M otherwise) are done; the wait overlaps
    // the loads above
    __syncthreads();

    // ---- X^T and B^T into LDS, two tokens per 32-bit store
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t v = (i & 1) ? pair_halves<true>(raw_word(xr[0], i >> 1), raw_word(xr[1], i >> 1))
                                 : pair_halves<false>(raw_word(xr[0], i >> 1), raw_word(xr[1], i >> 1));
      *reinterpret_cast<uint32_t *>(&sXT[swz<kQ>(xp0 + i, xt0)]) = v;
    }
#pragma unroll
    for (int j = 0; j < BPAIRS; ++j) {
      const int piece = tid + 256 * j;
      if (piece >= BPIECES) break;
      const int t = 2 * (piece / G8), n0 = (piece % G8) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = (i & 1) ? pair_halves<true>(raw_word(br[j][0], i >> 1), raw_word(br[j][1], i >> 1))
                                   : pair_halves<false>(raw_word(br[j][0], i >> 1), raw_word(br[j][1], i >> 1));
        *reinterpret_cast<uint32_t *>(&sBT[swz<kQ>(n0 + i, t)]) = v;
      }
      if constexpr (FULL) {
#pragma unroll
        for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4 *>(&sBr[swz<N>(t + k, n0)]) = br[j][k];
      }
    }
    if constexpr (FULL) {
      // this wave's C rows (tokens 16w + r) for every wave's C S^T products
#pragma unroll
      for (int kk = 0; kk < KN; ++kk) {
        const uint4 cw = __builtin_bit_cast(uint4, cop[kk]);
        const int rr = 16 * w + r;
        *reinterpret_cast<uint2 *>(&sC[swz8<N>(rr, 32 * kk + 8 * kq)]) = make_uint2(cw.x, cw.y);
        *reinterpret_cast<uint2 *>(&sC[swz8<N>(rr, 32 * kk + 8 * kq + 4)]) = make_uint2(cw.z, cw.w);
      }
    }
    // ---- the steps and their running sum inside the chunk (padding: dt' = 0).
    // Packed tokens: wave 1 forms the state-update weights from the sum of the
    // later steps themselves; the difference of two running sums would carry
    // the rounding of the larger one.
    if (w == 0 || (VAR && w == 1)) {
      float dtp = 0.0f;
      if (l < len) {
        const float v = dtraw + bias;
        dtp = p.softplus ? (VAR ? softplus_acc(v) : softplus_f(v)) : v;
        if (p.dt_limit) dtp = fminf(fmaxf(dtp, p.dt_min), p.dt_max);
      }
      float cs = dtp * Ah;
      if (VAR && w == 1) {
        cs = __shfl_down(cs, 1);
        if (l == 63) cs = 0.0f;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const float o = __shfl_down(cs, off);
          if (l + off < 64) cs += o;
        }
        sW[l] = fast_exp2(cs * kLog2e) * dtp;
      } else {
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const float o = __shfl_up(cs, off);
          if (l >= off) cs += o;
        }
        sCs[l] = cs;
        sDt[l] = dtp;
        if constexpr (SEQ) sSid[l] = sid;
      }
    }
    __syncthreads();

    const float csl = sCs[kQ - 1];
    // sequences: the chunk's last token's id, and whether the incoming state
    // reaches the end of the chunk (no sequence starts inside it)
    const int32_t sid_last = SEQ ? sSid[len - 1] : 0;
    const bool carry = !SEQ || sid_last == sid_prev;
    // the state-update weights w_t = exp(cs_last - cs_t) * dt'_t, for the
    // tokens of the chunk's last sequence
    if (!VAR && tid < kQ) {
      const bool mine = !SEQ || sSid[tid] == sid_last;
      sW[tid] = mine ? fast_exp2((csl - sCs[tid]) * kLog2e) * sDt[tid] : 0.0f;
    }
    if constexpr (!FULL && !VAR) __syncthreads();

    if constexpr (FULL) {
      // ---- M, from G^T = B C^T: lane holds G[t = 16w + r][tau = 16 tb + 4kq + i],
      // masked to tau <= t (and the same sequence), decayed, split, stored as
      // 4 consecutive tau.  The products read B from its row-major LDS copy,
      // an array of its own, so a wave stores its M as soon as its products
      // are done.
      const int t = 16 * w + r;
      const float cst = sCs[t];
      const int32_t sidt = SEQ ? sSid[t] : 0;
      f32x4 accg[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        accg[tb] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        if (tb <= w) {
          const int tau_row = 16 * tb + r;   // the B row this lane feeds as A operand
#pragma unroll
          for (int kk = 0; kk < KN; ++kk)
            accg[tb] = mfma(ld8(&sBr[swz<N>(tau_row, 32 * kk + 8 * kq)]), cop[kk], accg[tb]);
        }
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const f32x4 acc = accg[tb];
        // the four taus' cumulative steps, steps and ids, one vector read each
        const float4 cs4 = *reinterpret_cast<const float4 *>(&sCs[16 * tb + 4 * kq]);
        const float4 dt4 = *reinterpret_cast<const float4 *>(&sDt[16 * tb + 4 * kq]);
        const float csv[4] = {cs4.x, cs4.y, cs4.z, cs4.w}, dtv[4] = {dt4.x, dt4.y, dt4.z, dt4.w};
        int32_t sdv[4] = {0, 0, 0, 0};
        if constexpr (SEQ) {
          const int4 sd4 = *reinterpret_cast<const int4 *>(&sSid[16 * tb + 4 * kq]);
          sdv[0] = sd4.x; sdv[1] = sd4.y; sdv[2] = sd4.z; sdv[3] = sd4.w;
        }
        // computed for every lane of a block at or before the wave's
        // tokens and selected by the mask (no per-lane branch); the blocks
        // after them are zero
        float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (tb <= w) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tau = 16 * tb + 4 * kq + i;
            const float v = acc[i] * fast_exp2((cst - csv[i]) * kLog2e) * dtv[i];
            m[i] = (tau <= t && (!SEQ || sdv[i] == sidt)) ? v : 0.0f;
          }
        }
        uint2 hi, lo;
        split_bf2(m[0], m[1], hi.x, lo.x);
        split_bf2(m[2], m[3], hi.y, lo.y);
        const int o = swz<kQ>(t, 16 * tb + 4 * kq);
        *reinterpret_cast<uint2 *>(&sM[0][o]) = hi;
        *reinterpret_cast<uint2 *>(&sM[1][o]) = lo;
      }
      __syncthreads();

      // ---- Y^T = S C^T diag(exp(cs)) + X^T M^T for this wave's channels and
      // every token: lane holds Y[t = 16 tb + r][p = 16w + 4kq + i].
      // The state operand comes from this lane's own accumulators,
      // S[p = 16w + r][n = 16 nt + 4kq + i]: the k index of each product runs
      // over the 32 states 32kk + 16a + 4kq + j (a < 2, j < 4) in that order
      // for both operands, a permutation of the states that leaves the sum
      // unchanged; C's are the matching 8-byte pieces of its LDS rows.
      f32x4 accy[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) accy[tb] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < KN; ++kk) {
        uint32_t sh[4], sl[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          split_bf2(accs[2 * kk + i / 4][i % 4], accs[2 * kk + i / 4][i % 4 + 1], sh[i / 2], sl[i / 2]);
        const bf16x8 shi = __builtin_bit_cast(bf16x8, make_uint4(sh[0], sh[1], sh[2], sh[3]));
        const bf16x8 slo = __builtin_bit_cast(bf16x8, make_uint4(sl[0], sl[1], sl[2], sl[3]));
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const int row = 16 * tb + r;
          const uint2 c0 = *reinterpret_cast<const uint2 *>(&sC[swz8<N>(row, 32 * kk + 4 * kq)]);
          const uint2 c1 = *reinterpret_cast<const uint2 *>(&sC[swz8<N>(row, 32 * kk + 16 + 4 * kq)]);
          const bf16x8 cop8 = __builtin_bit_cast(bf16x8, make_uint4(c0.x, c0.y, c1.x, c1.y));
          accy[tb] = mfma(shi, cop8, accy[tb]);
          accy[tb] = mfma(slo, cop8, accy[tb]);
        }
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        // the incoming state reaches token t only inside its own sequence
        const int tt = 16 * tb + r;
        const float e = (!SEQ || sSid[SEQ ? tt : 0] == sid_prev) ? fast_exp2(sCs[tt] * kLog2e) : 0.0f;
        accy[tb] *= e;
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const bf16x8 xop = ld8(&sXT[swz<kQ>(16 * w + r, 32 * kk + 8 * kq)]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          if (32 * kk < 16 * (tb + 1)) {   // tau blocks at or before the token block
            const int o = swz<kQ>(16 * tb + r, 32 * kk + 8 * kq);
            accy[tb] = mfma(xop, ld8(&sM[0][o]), accy[tb]);
            accy[tb] = mfma(xop, ld8(&sM[1][o]), accy[tb]);
          }
        }
      }
      if constexpr (!Y_IN_BR) __syncthreads();   // every read of M is done

      // ---- Y into LDS (the B copy's space or over M), four consecutive channels per store
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const int ty = 16 * tb + r;
        const int grp = (4 * w + kq) ^ (ty & 15);   // 16-byte group of channels 16w + 4kq, permuted by t
        *reinterpret_cast<float4 *>(&sY[ty * kP + 4 * grp]) =
            make_float4(accy[tb][0], accy[tb][1], accy[tb][2], accy[tb][3]);
      }
    }
    // ---- S^T <- exp(cs_last) S^T + B^T (X w); the old state only if no
    // sequence starts inside the chunk
    const float dec = carry ? fast_exp2(csl * kLog2e) : 0.0f;
    if constexpr (!FULL) seg_decay *= dec;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) accs[nt] *= dec;
#pragma unroll
    for (int kk = 0; kk < kQ / 32; ++kk) {
      // B operand: (X w) at tokens 32kk + 8kq + i, channel 16w + r, split into
      // hi and lo; packed tokens: into three parts (all 24 bits), because the
      // state is a 32-bit output and its 8-bit form is decided by it
      const uint4 xt = ld8_raw(&sXT[swz<kQ>(16 * w + r, 32 * kk + 8 * kq)]);
      uint32_t xh[4], xl[4], xr2[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float a = bf2f(raw_bits(xt, i)) * sW[32 * kk + 8 * kq + i];
        const float b = bf2f(raw_bits(xt, i + 1)) * sW[32 * kk + 8 * kq + i + 1];
        split_bf2(a, b, xh[i / 2], xl[i / 2]);
        if constexpr (VAR)
          xr2[i / 2] = pack_bf2(a - __uint_as_float(xh[i / 2] << 16) - __uint_as_float(xl[i / 2] << 16),
                                b - __uint_as_float(xh[i / 2] & 0xffff0000u) - __uint_as_float(xl[i / 2] & 0xffff0000u));
      }
      const bf16x8 xhi = __builtin_bit_cast(bf16x8, make_uint4(xh[0], xh[1], xh[2], xh[3]));
      const bf16x8 xlo = __builtin_bit_cast(bf16x8, make_uint4(xl[0], xl[1], xl[2], xl[3]));
      bf16x8 xrest = zero8;
      if constexpr (VAR) xrest = __builtin_bit_cast(bf16x8, make_uint4(xr2[0], xr2[1], xr2[2], xr2[3]));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bf16x8 bop = ld8(&sBT[swz<kQ>(16 * nt + r, 32 * kk + 8 * kq)]);
        accs[nt] = mfma(bop, xhi, accs[nt]);
        accs[nt] = mfma(bop, xlo, accs[nt]);
        if constexpr (VAR) accs[nt] = mfma(bop, xrest, accs[nt]);
      }
    }
    sid_prev = sid_last;
    if constexpr (FULL) {
      __syncthreads();   // Y is in LDS

      // ---- out = (Y + D x) * silu(z): this thread's x / z pieces, 16-byte stores
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = xt0 + k;
        if (t < len) {
          const int g0 = (xp0 >> 2) ^ (t & 15), g1 = ((xp0 >> 2) + 1) ^ (t & 15);
          const float4 y0 = *reinterpret_cast<const float4 *>(&sY[t * kP + 4 * g0]);
          const float4 y1 = *reinterpret_cast<const float4 *>(&sY[t * kP + 4 * g1]);
          float yv[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
          // the uniform conditions outside the element loops, so the eight
          // gates' exp / rcp chains interleave
          if (p.D) {
#pragma unroll
            for (int i = 0; i < 8; ++i) yv[i] = fmaf(Dv8[i], bf2f(raw_bits(xr[k], i)), yv[i]);
          }
          if (zb) {
#pragma unroll
            for (int i = 0; i < 8; ++i) yv[i] *= silu_f(bf2f(raw_bits(zr[k], i)));
          }
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 8; i += 2) pk[i / 2] = pack_bf2(yv[i], yv[i + 1]);
          *reinterpret_cast<uint4 *>(ob + (t0 + t) * orow + xp0) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
    }
  }

  if constexpr (FULL && VAR) {
    if (p.cache && slot >= 0 && last_seg) {
      float *end = p.cache + (slot * p.nheads + h) * kP * N + srow;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float4 *>(end + 16 * nt) = make_float4(accs[nt][0], accs[nt][1], accs[nt][2], accs[nt][3]);
    }
  } else if constexpr (FULL) {
    if (p.fin && seg + 1 == p.nseg) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p.fin[(bh * kP + 16 * w + r) * N + 16 * nt + 4 * kq + i] = accs[nt][i];
      }
    }
  } else {
    float *E = p.ws_state + (seg * BH + bh) * kP * N + srow;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      *reinterpret_cast<float4 *>(E + 16 * nt) = make_float4(accs[nt][0], accs[nt][1], accs[nt][2], accs[nt][3]);
    if (tid == 0) p.ws_decay[seg * BH + bh] = seg_decay;
  }
}

}  // namespace
}  // namespace ssm
