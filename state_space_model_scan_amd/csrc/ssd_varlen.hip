// ssd_varlen.hip -- the Mamba-2 chunked scan over packed tokens
// (ssd_varlen_fwd): prompts of several lengths from and to a cache of states,
// and the training forward, which keeps every chunk's entering state in 8
// bits.
//
// The evaluation is ssd.hip's: per chunk of Q = 64 tokens with dt' the step,
// cs its running sum times A, S the (headdim x dstate) state entering it,
//   M[t][tau] = (C_t . B_tau) exp(cs_t - cs_tau) dt'_tau      (tau <= t)
//   Y         = M X + diag(exp(cs)) C S^T
//   S        <- exp(cs_end) S + X^T diag(exp(cs_end - cs) dt') B
// with M and S entering their products as a bf16 head and tail.  The weighted
// X of the state update enters in three parts (all 24 bits) and the running
// sum is kept in two floats, whose difference gives every decay: the state is a
// 32-bit output, and its 8-bit form is decided by it.
//
// What bounds it is the chain of a chunk's dependent steps, not HBM: the chunks
// of a (sequence, head) follow each other.  So:
// - a workgroup of four waves walks a head's chunks, and 79 KB of LDS let two
//   run on a compute unit, each in its own phase (one workgroup of eight
//   waves for two heads, which shares B and C, took 707 us where this took
//   650: 32768 tokens, 80 heads);
// - the next chunk's x and B go from global memory straight into the other
//   half of a double buffer in LDS while this chunk is computed, its C as soon
//   as C has been read, before the outputs are stored, and its steps are summed
//   at this chunk's end.  A wave waits for loads twice a chunk, and for stores
//   not at all (with C behind the stores, and so waiting for them, 654 us);
// - what the loop does is fixed by template values (gated or not, with or
//   without the 8-bit states: 630 -> 601 us for the first, and a prompts' batch
//   of 24 x 32 heads 53 -> 50 us for the second): a branch ends what the
//   compiler may interleave;
// - tiles stay as they lie in memory, token by token, and are read across by
//   the transposing LDS load, so nothing is rearranged on the way;
// - three barriers a chunk: data there, M there, C done with.
// Now 595 to 615 us, from card to card; the 24 prompts 50.
// With few (sequence, head) pairs the sequence is cut into segments; a first
// launch finds their end states from zero (FULL false), and
// the second starts every segment from the states carried over.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_util.h"
#include "packed_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

struct ScanParams {
  const uint16_t *x, *dt, *B, *C, *z;
  const float *A, *D, *dt_bias;
  uint16_t *out;
  float *ws_state, *ws_decay;   // segments: end states (and the cached states' copies), decays
  const int32_t *cu, *seen, *slots;
  float *cache;
  int8_t *codes;
  float *scales;
  int64_t xs, dts, bs, cs, zs, os;
  int64_t total, max_seqlen, cache_slots, nheads, seg_chunks;
  uint32_t heads, per_group;   // nheads, heads of a group
  int D_per_channel, nseg;
  StepRule step;
};

// M keeps its ten 16 x 16 tiles on and below the diagonal, and a zero one for
// the half of an operand that reaches above it.
constexpr int kTile = 256, kZeroTile = 10;
// tile of the (token block, tau block), element of (token, tau) inside a tile
__device__ __forceinline__ constexpr int m_tile(int tb, int ub) { return ub <= tb ? tb * (tb + 1) / 2 + ub : kZeroTile; }
__device__ __forceinline__ int m_at(int t, int tau) { return t * 16 + (tau ^ (((t >> 2) & 1) << 3)); }

template <int N, bool FULL>
struct ScanLds {
  uint16_t B[2][kQ * N];                              // [t][n]
  uint16_t x[2][kQ * kP];                             // [t][p]
  uint16_t C[FULL ? kQ * N : 8];                      // [t][n]
  uint16_t M[2][FULL ? (kZeroTile + 1) * kTile : 8];    // head, tail
  // running sum times log2 e (two floats), step, exp(cs), and the state update's weight, per token
  float cs[2][kQ], cl[2][kQ], dt[2][kQ], e[2][kQ], w[2][kQ];
};

// The transposed operand of B for state tile a of the k step kk: lane m's row
// is the state n = 32kk + 8 (m / 4) + 4a + m % 4, so that a lane's accumulators
// of tiles a = 0 and 1 are eight neighbouring states, 32kk + 8kq + 0..7.
template <int N>
__device__ __forceinline__ bf16x8 frag_states(int l, uint16_t *tile, int row0, int kk, int a) {
  typedef __attribute__((address_space(3))) s16x4 *lds;
  const int i = l & 15, kq = l >> 4;
  const int row = row0 + 8 * kq + (i >> 2), col = 32 * kk + 8 * (i & 3) + 4 * a;
  const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(tile + tile_at<N>(row, col)));
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(tile + tile_at<N>(row + 4, col)));
  const uint2 uu = __builtin_bit_cast(uint2, u), uv = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(bf16x8, make_uint4(uu.x, uu.y, uv.x, uv.y));
}

template <int N, bool FULL, bool GATED = false, bool KEEP = false>
__global__ void __launch_bounds__(256, FULL ? 2 : 3) packed_scan_kernel(const ScanParams p) {
  constexpr int KN = N / 32;   // K steps over dstate
  constexpr int NT = N / 16;   // state tiles along dstate
  extern __shared__ __attribute__((aligned(16))) char smem[];
  ScanLds<N, FULL> &sm = *reinterpret_cast<ScanLds<N, FULL> *>(smem);
  const int tid = threadIdx.x, l = tid & 63, r = l & 15, kq = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);   // channels 16w..16w+15
  const int64_t SH = gridDim.x;
  const uint32_t sh = blockIdx.x, s = sh / p.heads, h = sh - s * p.heads, g = h / p.per_group;
  const Seq q = sequence(p.cu, p.total, p.max_seqlen, s);
  // the full pass dispatches its last segments first: those of the longest sequences
  const int64_t seg = FULL ? static_cast<int64_t>(gridDim.y) - 1 - blockIdx.y : blockIdx.y;
  const int64_t c_begin = seg * p.seg_chunks;
  const int64_t c_end = c_begin + p.seg_chunks < q.chunks ? c_begin + p.seg_chunks : q.chunks;
  const bool last_seg = c_end >= q.chunks;
  if (seg > 0 && c_begin >= q.chunks) return;
  if (!FULL && last_seg) return;   // the first launch runs the segments that have one after them
  int64_t slot = p.slots ? p.slots[s] : s;
  if (slot >= p.cache_slots) slot = -1;
  const bool cached = p.cache && slot >= 0 && p.seen && p.seen[s] > 0;

  // the segment's chunks and, from its first token, the tokens and the rows;
  // what the loop counts and steps through is 32 bits or a pointer, for a
  // wave's scalar instructions hold up its others
  const int nchunks = static_cast<int>(c_end - c_begin), ntokens = static_cast<int>(q.len - c_begin * kQ);
  const int64_t first = q.first + c_begin * kQ;
  const uint16_t *xb = p.x + first * p.xs + h * kP;   // of the next tiles
  const uint16_t *Bb = p.B + first * p.bs + g * N, *Cb = p.C + first * p.cs + g * N;
  const uint16_t *dtb = p.dt + first * p.dts + h;
  const uint16_t *zb = GATED ? p.z + first * p.zs + h * kP : nullptr;   // of this chunk
  uint16_t *ob = p.out + first * p.os + h * kP;
  const float Ah = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
  float *state_ws = p.ws_state + static_cast<int64_t>(sh) * kP * N;   // segment k's at k * SH * kP * N
  const int srow = (16 * w + r) * N + (FULL ? 8 : 4) * kq;   // this lane's first state element in a (p, n) block

  TileLoad<kP> lx;
  TileLoad<N> lb, lc;
  auto place = [&](int len) {
    lx.place(p.xs, len, w, l);
    lb.place(p.bs, len, w, l);
    if constexpr (FULL) lc.place(p.cs, len, w, l);
  };
  place(ntokens < kQ ? ntokens : kQ);
  auto fetch = [&](int b) {
    lx.fetch(sm.x[b], xb, w);
    lb.fetch(sm.B[b], Bb, w);
    xb += kQ * p.xs;
    Bb += kQ * p.bs;
  };
  auto fetch_C = [&] {
    if constexpr (FULL) lc.fetch(sm.C, Cb, w);
    Cb += kQ * p.cs;
  };
  // a chunk's raw steps, and what the chunk needs of them (wave 0)
  auto raw_steps = [&](int len) {   // (of the last token beyond the end; as loaded: a conversion would wait for it)
    const uint32_t raw = dtb[(l < len ? l : len - 1) * p.dts];
    dtb += kQ * p.dts;
    return raw;
  };
  auto put_steps = [&](int len, int b, uint32_t raw) {
    asm volatile("" : "+v"(raw));   // or it is converted, and waited for, where it is loaded
    float v;
    const float d = chunk_step(p.step, bf2f(static_cast<uint16_t>(raw)), bias, l < len, v);
    const TwoSum cs = running_sum(d, Ah);
    const TwoSum end = {__int_as_float(__builtin_amdgcn_readlane(__float_as_int(cs.hi), 63)),
                        __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cs.lo), 63))};
    const TwoSum turns = times_log2e(cs);
    sm.cs[b][l] = turns.hi;
    sm.cl[b][l] = turns.lo;
    sm.dt[b][l] = d;
    sm.e[b][l] = exp_sum(cs);
    sm.w[b][l] = exp_sum(diff(end, cs)) * d;
  };

  // ---- state, transposed: wave w holds S[p = 16w + r][n = 32 kk + 8kq + 4a + i]
  // in accs[2 kk + a][i]; the state pass, which feeds no product from it, holds
  // n = 16 nt + 4kq + i in accs[nt][i], whose operands meet in no LDS bank.
  // The state pass starts segment 0 from the cached state and the others from
  // zero; the full pass starts segment k from E_{k-1} + P_{k-1} (E_{k-2} + ...).
  // The last segment's workgroup writes the cache while others may still be
  // starting, so a sequence of several segments reads it in the state pass
  // alone: segment 0's start is a copy that the state pass leaves behind the
  // E's.
  auto state_at = [](int nt) { return FULL ? 32 * (nt >> 1) + 4 * (nt & 1) : 16 * nt; };
  f32x4 accs[NT];
  {
    const float *start = nullptr;
    if (cached && seg == 0)
      start = (!FULL || last_seg) ? p.cache + (slot * p.nheads + h) * kP * N : state_ws + (p.nseg - 1) * SH * kP * N;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 v = start ? *reinterpret_cast<const float4 *>(start + srow + state_at(nt)) : make_float4(0, 0, 0, 0);
      accs[nt] = (f32x4){v.x, v.y, v.z, v.w};
      if (!FULL && start)
        *reinterpret_cast<float4 *>(state_ws + (p.nseg - 1) * SH * kP * N + srow + state_at(nt)) = v;
    }
  }
  if (FULL) {
    for (int64_t j = 0; j < seg; ++j) {
      const float P = p.ws_decay[j * SH + sh];
      const float *E = state_ws + j * SH * kP * N + srow;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 e = *reinterpret_cast<const float4 *>(E + state_at(nt));
        accs[nt] = (f32x4){fmaf(P, accs[nt][0], e.x), fmaf(P, accs[nt][1], e.y), fmaf(P, accs[nt][2], e.z),
                           fmaf(P, accs[nt][3], e.w)};
      }
    }
  }
  if constexpr (FULL) {   // M's zero tile
    if (tid < 2 * kTile / 8) *reinterpret_cast<uint4 *>(&sm.M[tid / (kTile / 8)][kZeroTile * kTile + tid % (kTile / 8) * 8]) = make_uint4(0, 0, 0, 0);
  }
  float Dv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int pc = 16 * w + 4 * kq;   // this lane's channels of Y
  if (FULL && p.D) {
#pragma unroll
    for (int i = 0; i < 4; ++i) Dv[i] = p.D_per_channel ? p.D[h * kP + pc + i] : p.D[h];
  }
  float seg_decay = 1.0f;

  // the entering states' 8-bit form, this lane's piece of it
  int8_t *codes = nullptr;
  float *scales = nullptr;
  if constexpr (KEEP) {
    const int64_t row = ((q.entry + c_begin) * p.nheads + h) * kP + 16 * w + r;
    codes = p.codes + row * N + 8 * kq;
    scales = p.scales + row;
  }

  if (nchunks > 0) {
    const int len = ntokens < kQ ? ntokens : kQ;
    fetch(0);
    fetch_C();
    if (w == 0) put_steps(len, 0, raw_steps(len));
  }
  loads_landed();
  for (int c = 0, left = ntokens; c < nchunks; ++c, left -= kQ) {
    const int b = c & 1;
    const int len = left < kQ ? left : kQ, next = left - kQ < kQ ? left - kQ : kQ;
    // every wave's part of the chunk's tiles is there, and the last chunk's
    // readers are done
    lds_barrier();
    uint32_t raw = 0;
    const bool more = c + 1 < nchunks;
    if (w == 0 && more) raw = raw_steps(next);
    uint2 zv[4] = {};
    if constexpr (GATED) {
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
        if (16 * tb + r < len) zv[tb] = *reinterpret_cast<const uint2 *>(zb + (16 * tb + r) * p.zs + pc);
      zb += kQ * p.zs;
    }
    if (more) {
      if (next < kQ) place(next);   // the sequence's end
      fetch(b ^ 1);
    }
    const float *cs = sm.cs[b], *cl = sm.cl[b], *dt = sm.dt[b], *e0 = sm.e[b], *we = sm.w[b];
    uint16_t *X = sm.x[b], *B = sm.B[b];

    if constexpr (FULL) {
      if constexpr (KEEP) {
        // the chunk's entering state in 8 bits: this lane holds 4 NT states of
        // row 16w + r, the row's others are 16, 32 and 48 lanes away
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
#pragma unroll
        for (int kk = 0; kk < KN; ++kk) {
          uint32_t word[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            word[i >> 2] |= (static_cast<uint32_t>(static_cast<int>(rintf(accs[2 * kk + (i >> 2)][i & 3] * inv))) & 0xffu) << (8 * (i & 3));
          *reinterpret_cast<uint2 *>(codes + 32 * kk) = make_uint2(word[0], word[1]);
        }
        if (kq == 0) *scales = scale;
        codes += p.nheads * kP * N;
        scales += p.nheads * kP;
      }

      // ---- M, from G^T = B C^T: lane holds (t = 16 wt + r, tau = 16 tb + 4kq + i),
      // tau <= t.  Every second head's waves take the token blocks in the other
      // order, so that the waves of a SIMD share the triangle's work.
      // (One copy of the code for each block: with the block a variable, a
      // branch stood between any two products.)
      auto form_M = [&](auto block) {
        constexpr int WT = decltype(block)::value;
        const int t = 16 * WT + r;
        bf16x8 cop[KN];
#pragma unroll
        for (int kk = 0; kk < KN; ++kk) cop[kk] = frag<N>(l, sm.C, 16 * WT, 32 * kk);
        f32x4 acc[WT + 1];
#pragma unroll
        for (int tb = 0; tb <= WT; ++tb) acc[tb] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < KN; ++kk)
#pragma unroll
          for (int tb = 0; tb <= WT; ++tb) acc[tb] = mfma(frag<N>(l, B, 16 * tb, 32 * kk), cop[kk], acc[tb]);
        const float cst = cs[t], clt = cl[t];
#pragma unroll
        for (int tb = 0; tb <= WT; ++tb) {
          const float4 cs4 = *reinterpret_cast<const float4 *>(&cs[16 * tb + 4 * kq]);
          const float4 cl4 = *reinterpret_cast<const float4 *>(&cl[16 * tb + 4 * kq]);
          const float4 dt4 = *reinterpret_cast<const float4 *>(&dt[16 * tb + 4 * kq]);
          const float csv[4] = {cs4.x, cs4.y, cs4.z, cs4.w}, clv[4] = {cl4.x, cl4.y, cl4.z, cl4.w}, dtv[4] = {dt4.x, dt4.y, dt4.z, dt4.w};
          float m[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = acc[tb][i] * fast_exp2((cst - csv[i]) + (clt - clv[i])) * dtv[i];
            m[i] = (tb < WT || 4 * kq + i <= r) ? v : 0.0f;
          }
          uint2 hi, lo;
          split_bf2(m[0], m[1], hi.x, lo.x);
          split_bf2(m[2], m[3], hi.y, lo.y);
          const int o = m_tile(WT, tb) * kTile + m_at(r, 4 * kq);
          *reinterpret_cast<uint2 *>(&sm.M[0][o]) = hi;
          *reinterpret_cast<uint2 *>(&sm.M[1][o]) = lo;
        }
      };
      switch ((h & 1) ? 3 - w : w) {
        case 0: form_M(std::integral_constant<int, 0>{}); break;
        case 1: form_M(std::integral_constant<int, 1>{}); break;
        case 2: form_M(std::integral_constant<int, 2>{}); break;
        default: form_M(std::integral_constant<int, 3>{}); break;
      }
      lds_barrier();
    }

    // X across: lane (channel 16w + r, tokens 32kk + 8kq + i)
    bf16x8 xt[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) xt[kk] = frag_t<kP>(l, X, 32 * kk, 16 * w);

    if constexpr (FULL) {
      // ---- Y^T = S C^T diag(exp(cs)) + X^T M^T for this wave's channels and
      // every token: lane holds Y[t = 16 tb + r][p = 16w + 4kq + i].  The state
      // operand is this lane's own accumulators.
      f32x4 acc[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) acc[tb] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < KN; ++kk) {
        uint32_t sh_[4], sl_[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          split_bf2(accs[2 * kk + i / 4][i % 4], accs[2 * kk + i / 4][i % 4 + 1], sh_[i / 2], sl_[i / 2]);
        const bf16x8 shi = __builtin_bit_cast(bf16x8, make_uint4(sh_[0], sh_[1], sh_[2], sh_[3]));
        const bf16x8 slo = __builtin_bit_cast(bf16x8, make_uint4(sl_[0], sl_[1], sl_[2], sl_[3]));
        bf16x8 cf[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          cf[tb] = frag<N>(l, sm.C, 16 * tb, 32 * kk);
          acc[tb] = mfma(shi, cf[tb], acc[tb]);
        }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) acc[tb] = mfma(slo, cf[tb], acc[tb]);
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) acc[tb] *= e0[16 * tb + r];
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int tb = 0; tb < 4; ++tb)
            if (32 * kk < 16 * (tb + 1)) {   // tau blocks at or before the token block
              const int o = (kq < 2 ? m_tile(tb, 2 * kk) : m_tile(tb, 2 * kk + 1)) * kTile + m_at(r, 8 * (kq & 1));
              acc[tb] = mfma(xt[kk], ld8(&sm.M[part][o]), acc[tb]);
            }
      // z and the next steps are there, and the next tiles (whose loads followed
      // theirs); asked for behind C's loads, they would wait for those too
      loads_landed();
      if (more) {
        lds_barrier();   // C's readers are done
        fetch_C();
      }
      // ---- out = (Y + D x) * silu(z), four channels of a token
      if (p.D) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          float xv[4];
          four(&X[tile_at<kP>(16 * tb + r, pc)], xv);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[tb][i] = fmaf(Dv[i], xv[i], acc[tb][i]);
        }
      }
      if constexpr (GATED) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const float zf[4] = {__uint_as_float(zv[tb].x << 16), __uint_as_float(zv[tb].x & 0xffff0000u),
                               __uint_as_float(zv[tb].y << 16), __uint_as_float(zv[tb].y & 0xffff0000u)};
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[tb][i] *= silu_f(zf[i]);
        }
      }
      uint16_t *to = ob + r * p.os + pc;
      ob += kQ * p.os;
      auto put = [&](int tb) {
        *reinterpret_cast<uint2 *>(to + 16 * tb * p.os) = make_uint2(pack_bf2(acc[tb][0], acc[tb][1]), pack_bf2(acc[tb][2], acc[tb][3]));
      };
      if (len == kQ) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) put(tb);
      } else {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
          if (16 * tb + r < len) put(tb);
      }
    }

    // ---- S^T <- exp(cs_end) S^T + B^T (X w), X w in three bf16 parts.  The
    // matrix unit rounds its accumulator four times a product, so the small parts
    // come first and the state is added at the end, with one rounding.
    const float dec = e0[kQ - 1];
    if constexpr (!FULL) seg_decay *= dec;
    bf16x8 part[3][2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const uint4 xw = __builtin_bit_cast(uint4, xt[kk]);
      uint32_t x0[4], x1[4], x2[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float a = bf2f(raw_bits(xw, i)) * we[32 * kk + 8 * kq + i];
        const float d = bf2f(raw_bits(xw, i + 1)) * we[32 * kk + 8 * kq + i + 1];
        split_bf2(a, d, x0[i / 2], x1[i / 2]);
        x2[i / 2] = third_bf2(a, d, x0[i / 2], x1[i / 2]);
      }
      part[0][kk] = __builtin_bit_cast(bf16x8, make_uint4(x0[0], x0[1], x0[2], x0[3]));
      part[1][kk] = __builtin_bit_cast(bf16x8, make_uint4(x1[0], x1[1], x1[2], x1[3]));
      part[2][kk] = __builtin_bit_cast(bf16x8, make_uint4(x2[0], x2[1], x2[2], x2[3]));
    }
    constexpr int AT = 2;   // tiles at a time (4 and 8 take registers: 606 and 709 us where this takes 602)
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += AT) {
      bf16x8 bt[AT][2];
      f32x4 sum[AT];
#pragma unroll
      for (int a = 0; a < AT; ++a) {
        sum[a] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          bt[a][kk] = FULL ? frag_states<N>(l, B, 32 * kk, (n0 + a) >> 1, a & 1) : frag_t<N>(l, B, 32 * kk, 16 * (n0 + a));
      }
#pragma unroll
      for (int k = 2; k >= 0; --k)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int a = 0; a < AT; ++a) sum[a] = mfma(bt[a][kk], part[k][kk], sum[a]);
#pragma unroll
      for (int a = 0; a < AT; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) accs[n0 + a][i] = fmaf(accs[n0 + a][i], dec, sum[a][i]);
    }
    if (w == 0 && more) put_steps(next, b ^ 1, raw);
    // C is there, whatever the four stores after it do (a chunk with one after
    // it is whole)
    loads_landed<FULL ? 4 : 0>();
  }

  float *end = nullptr;
  if constexpr (FULL) {
    if (p.cache && slot >= 0 && last_seg) end = p.cache + (slot * p.nheads + h) * kP * N + srow;
  } else {
    end = state_ws + seg * SH * kP * N + srow;
    if (w == 0 && l == 0) p.ws_decay[seg * SH + sh] = seg_decay;
  }
  if (end) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      *reinterpret_cast<float4 *>(end + state_at(nt)) = make_float4(accs[nt][0], accs[nt][1], accs[nt][2], accs[nt][3]);
  }
}

using VarFn = void (*)(const ScanParams);

template <int N>
VarFn var_fn_n(bool full, bool gated, bool keep) {
  if (!full) return packed_scan_kernel<N, false>;
  if (keep) return gated ? packed_scan_kernel<N, true, true, true> : packed_scan_kernel<N, true, false, true>;
  return gated ? packed_scan_kernel<N, true, true, false> : packed_scan_kernel<N, true, false, false>;
}
VarFn var_fn(int64_t dstate, bool full, const ScanParams &p) {
  const bool gated = p.z != nullptr, keep = p.codes != nullptr;
  switch (dstate) {
    case 32: return var_fn_n<32>(full, gated, keep);
    case 64: return var_fn_n<64>(full, gated, keep);
    default: return var_fn_n<128>(full, gated, keep);
  }
}

unsigned var_lds(int64_t dstate, bool full) {
  switch (dstate) {
    case 32: return full ? sizeof(ScanLds<32, true>) : sizeof(ScanLds<32, false>);
    case 64: return full ? sizeof(ScanLds<64, true>) : sizeof(ScanLds<64, false>);
    default: return full ? sizeof(ScanLds<128, true>) : sizeof(ScanLds<128, false>);
  }
}

hipError_t launch_var(int64_t dstate, bool full, dim3 grid, hipStream_t stream, const ScanParams &p) {
  const VarFn fn = var_fn(dstate, full, p);
  const unsigned lds = var_lds(dstate, full);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(lds));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, grid, dim3(256), lds, stream, p);
  return hipGetLastError();
}

struct VarPlan {
  int nseg;
  int64_t seg_chunks;
  size_t off_decay, ws_bytes;
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The whole call with segments of seg chunks.  The chunk times (full pass 3.4
// and 4.6 us, state pass 1.5 and 2.7) are those measured at dstate 128.  A
// smaller one takes less of each, in about their ratios: the choices below hold
// at 64 too, and at 32 are up to 17% from the best.  Each segment costs about 0.8
// chunks to start, segment k reads the k end states before it (32 KB each, from
// the caches mostly), and a second launch about 5 us.
double split_us(int64_t blocks, int64_t nchunks, int64_t seg, int64_t dstate, int64_t cus) {
  const int64_t G = (nchunks + seg - 1) / seg;
  const double len = static_cast<double>(seg) + 0.8;
  double t = rounds_us(blocks * G, len, 3.4, 4.6, 2, cus);
  if (G > 1) {
    const double block_bytes = static_cast<double>(blocks) * kP * dstate * sizeof(float);
    t += rounds_us(blocks * (G - 1), len, 1.5, 2.7, 3, cus) + 5.0 +
         block_bytes * (static_cast<double>(G) * (G - 1) / 2 / 1e7 + (G - 1) / 5e6);
  }
  return t;
}

// Segments of the longest sequence; a shorter one has fewer.  The library's own
// count is the one that split_us finds fastest.  Measured (us, chosen / best of
// a sweep), at dstate 128, 64 and 32: 1 x 32768 tokens x 80 heads 590 / 576,
// 418 / 418, 344 / 327; 4 x 2048 x 80 141 / 137, 102 / 101, 78 / 72; 1 x 2048 x 80
// 55 / 52, 41 / 39, 34 / 29; 1 x 16384 x 16 97 / 95, 63 / 63, 47 / 47; 5 x 200 x 8
// 16 / 16, 13 / 13, 11 / 11.
VarPlan var_plan(const ssd_varlen_args_t *a, int cus) {
  VarPlan pl{};
  int64_t nchunks = (a->max_seqlen + kQ - 1) / kQ;
  if (nchunks < 1) nchunks = 1;
  const int64_t SH = a->nseq * a->nheads;
  int64_t G = 1;
  if (a->seq_segments >= 1) {
    G = a->seq_segments;
  } else {
    // sequences of the longest one's length that hold all tokens
    const int64_t rows = (a->total / kQ + a->nseq + nchunks - 1) / nchunks;
    const int64_t blocks = (rows < a->nseq ? rows : a->nseq) * a->nheads;
    double best = 1e300;
    for (int64_t k = 1; k <= 64 && (k == 1 || 2 * k <= nchunks); ++k) {
      const double t = split_us(blocks, nchunks, (nchunks + k - 1) / k, a->dstate, cus);
      if (t < best) {
        best = t;
        G = k;
      }
    }
  }
  if (G > nchunks) G = nchunks;
  if (G > 65535) G = 65535;
  pl.seg_chunks = (nchunks + G - 1) / G;
  pl.nseg = static_cast<int>((nchunks + pl.seg_chunks - 1) / pl.seg_chunks);
  if (pl.nseg > 1) {
    // the segments' end states, and behind them a copy of the cached states
    pl.off_decay = up256(static_cast<size_t>(pl.nseg) * SH * kP * a->dstate * sizeof(float));
    pl.ws_bytes = pl.off_decay + up256(static_cast<size_t>(pl.nseg - 1) * SH * sizeof(float));
  }
  return pl;
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int ssd_varlen_fwd_workspace_size(const ssd_varlen_args_t *a, size_t *bytes) {
  const int st = ssd_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = var_plan(a, cu_count_cached()).ws_bytes;
  return SSM_OK;
}

extern "C" int ssd_varlen_fwd(const ssd_varlen_args_t *a, void *stream_ptr) {
  const int st = ssd_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  const int64_t blocks = a->nseq * a->nheads;
  if (!grid_fits(blocks, 256)) return SSM_ERR_SHAPE;
  const VarPlan pl = var_plan(a, cu_count_cached());
  if (pl.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < pl.ws_bytes)) return SSM_ERR_WORKSPACE;
  if (pl.ws_bytes > 0 && !aligned16(a->workspace)) return SSM_ERR_UNSUPPORTED;
  ScanParams p{};
  p.x = static_cast<const uint16_t *>(a->x); p.xs = a->x_stride;
  p.dt = static_cast<const uint16_t *>(a->dt); p.dts = a->dt_stride;
  p.B = static_cast<const uint16_t *>(a->B); p.bs = a->B_stride;
  p.C = static_cast<const uint16_t *>(a->C); p.cs = a->C_stride;
  p.z = static_cast<const uint16_t *>(a->z); p.zs = a->z_stride;
  p.out = static_cast<uint16_t *>(a->out); p.os = a->out_stride;
  p.A = a->A; p.D = a->D; p.dt_bias = a->dt_bias;
  p.D_per_channel = a->D_per_channel;
  p.step = {a->dt_softplus, a->dt_limit, a->dt_min, a->dt_max};
  p.nheads = a->nheads;
  p.heads = static_cast<uint32_t>(a->nheads);
  p.per_group = static_cast<uint32_t>(a->nheads / a->ngroups);
  p.cu = a->cu_seqlens; p.total = a->total; p.max_seqlen = a->max_seqlen;
  p.cache = a->ssm_state; p.cache_slots = a->state_slots; p.seen = a->cache_seqlens; p.slots = a->slots;
  p.codes = a->checkpoints; p.scales = a->checkpoint_scales;
  p.nseg = pl.nseg; p.seg_chunks = pl.seg_chunks;
  if (pl.nseg > 1) {
    char *ws = static_cast<char *>(a->workspace);
    p.ws_state = reinterpret_cast<float *>(ws);
    p.ws_decay = reinterpret_cast<float *>(ws + pl.off_decay);
  }
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const unsigned gx = static_cast<unsigned>(blocks);
  if (pl.nseg > 1) {
    const hipError_t e = launch_var(a->dstate, false, dim3(gx, pl.nseg - 1), stream, p);
    if (e != hipSuccess) return hip_fail(e);
  }
  const hipError_t e = launch_var(a->dstate, true, dim3(gx, pl.nseg), stream, p);
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}
