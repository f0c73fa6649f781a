// ssd_varlen_bwd.hip -- the gradient of the packed chunked scan
// (ssd_varlen_bwd), on the gfx950 matrix cores.
//
// With the steps dt', cs their running sum times A inside a chunk of Q = 64
// tokens, H the state entering the chunk (from its 8-bit checkpoint), dH the
// adjoint of the state leaving it, g = dout, e_i = exp(cs_i),
// w_j = exp(cs_end - cs_j), and for i >= j
//   L_ij = exp(cs_i - cs_j), S_ij = C_i . B_j, M_ij = g_i . x_j:
//   dx_j = dt'_j (sum_i S_ij L_ij g_i + w_j dH B_j) + D g_j
//   dB_j = sum_heads [ sum_i (M_ij L_ij dt'_j) C_i + dt'_j w_j dH^T x_j ]
//   dC_i = sum_heads [ sum_j (M_ij L_ij dt'_j) B_j + e_i H^T g_i ]
//   dH  <- exp(cs_end) dH + sum_i e_i g_i C_i^T
// and, for the steps, with G_ij = S_ij L_ij M_ij, q_i = e_i g_i . (H C_i) and
// r_j = w_j x_j . (dH B_j):
//   direct_j = sum_i G_ij + r_j
//   da_t = sum_{i >= t > j} G_ij dt'_j + sum_{i >= t} q_i + sum_{j < t} dt'_j r_j + exp(cs_end) <dH, H>
//   ddt'_t = direct_t + A da_t,  dA = sum dt' da.
// da_t is the gradient of token t's decay exponent, and these are the paths
// that pass it.  (As sums from t on of d cs, every path between two tokens at or
// after t would be added at its end and taken off again at its start, a token's
// way into its own output first of all: what their roundings leave is then the
// whole of a gradient that has to vanish, as for a sequence of one token.)
//
// Three launches.  (1) adjoint_kernel walks every (sequence, head)'s chunks
// backwards and leaves each chunk's dH in the workspace; with few (sequence, head) pairs the
// sequence is cut into segments as in the forward.  (2) chunk_kernel takes one
// chunk and a block of heads of one group: everything but dH is local to the
// chunk.  S is formed once for the group.  dB's and dC's pair products are
// linear in M L dt', so that sum over the heads is kept (64 x 64, in
// registers) and multiplied with C and B once at the end; their state parts
// are summed over the heads in registers too.  (3) small kernels add the head
// blocks' dB and dC and the chunks' dA, dD and ddt_bias, in a fixed order.
//
// Precision: x, B, C, g and the dequantised H (seven bits times a power of
// two) are exact in bf16.  dA and ddt_bias are 32-bit sums, so what they take
// from a product is formed from all 24 bits: dH enters r and <dH, H> in three
// parts (with a head and a tail, 2^-17 of it, r alone put 1e-6 into dA).  What
// only reaches an output in bf16 enters as head and tail: dH in dB, S L and the
// summed M L dt'.  The matrix unit rounds an accumulator that is below the
// products' sum towards minus infinity (measured on the device), so that sums of
// products would all be off to one side, and the sums over tokens with them: dA
// by 9e-7 at 8 x 2048 tokens, whatever the sign of g.  So every second token's B
// and every second state's H enter negated, and the adjoint changes its sign from
// chunk to chunk (7e-8).
//
// Operand layout of the 16x16x32 product as in ssd.hip.  Tiles are kept
// row-major in LDS, and an operand that runs along the other index is read
// with the transposing LDS load (ds_read_b64_tr_b16: of four rows by sixteen
// columns, lane l of sixteen receives column l; checked on the device), so no
// tile is stored twice.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_util.h"
#include "packed_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kMaxHeads = 16;   // heads of a chunk_kernel workgroup

struct BwdParams {
  const uint16_t *x, *dt, *B, *C, *g;
  const float *A, *D, *dt_bias, *dfin;
  const int32_t *cu;
  const int8_t *codes;
  const float *scales;
  uint16_t *dx, *ddt, *dB, *dC;
  float *dinit;
  float *ws_dh;                  // (entries, heads, p, n), as adjoint_kernel's lanes hold it
  float *ws_state, *ws_decay;    // adjoint segments
  float *ws_bc;                  // (2, head blocks of a group, total, groups, n) or NULL (one block: dB, dC directly)
  float *ws_sum;                 // (entries, heads, 2): dA, ddt_bias
  float *ws_dd;                  // (entries, heads) or (entries, heads, p): dD
  int64_t xs, dts, bs, cs, gs, dxs, ddts, dbs, dcs;
  int64_t code_entry, code_head, scale_entry, scale_head;
  int64_t total, nseq, max_seqlen, nheads, ngroups, seg_chunks, entries;
  uint32_t heads, per_group;   // nheads, heads of a group
  int nseg, D_per_channel, hb_heads, hb_per_group;
  StepRule step;
};

// ---------------------------------------------------------------------------
// (1) the adjoint of the states.  One workgroup of four waves per (sequence,
// head, segment); wave w holds dH rows p = 16w + r, n = 16 nt + 4 kq + i, as
// the forward holds the state.  STORE: write every chunk's dH; otherwise find
// the segment's adjoint from zero and its decay.
// ---------------------------------------------------------------------------
// The sign with which an entry's dH is kept (see Precision).
__device__ __forceinline__ float entry_sign(int64_t entry) { return entry & 1 ? -1.0f : 1.0f; }

template <int N>
struct AdjointLds {
  uint16_t C[2][kQ * N], g[2][kQ * kP];   // [t][n], [t][p]; the next chunk's are on their way into the other half
  float e[2][kQ], end[2];                 // exp(cs), and at the chunk's end
};

template <int N, bool STORE>
__global__ void __launch_bounds__(256, 3) adjoint_kernel(const BwdParams p) {
  constexpr int NT = N / 16;
  __shared__ __attribute__((aligned(16))) AdjointLds<N> sm;
  const int tid = threadIdx.x, l = tid & 63, r = l & 15, kq = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t SH = gridDim.x;
  const uint32_t sh = blockIdx.x, s = sh / p.heads, h = sh - s * p.heads, gr = h / p.per_group;
  const Seq q = sequence(p.cu, p.total, p.max_seqlen, s);
  // the first launch runs the segments that have one before them
  const int64_t seg = STORE ? blockIdx.y : blockIdx.y + 1;
  const int64_t c_begin = seg * p.seg_chunks;
  if (seg > 0 && c_begin >= q.chunks) return;
  const int64_t c_end = c_begin + p.seg_chunks < q.chunks ? c_begin + p.seg_chunks : q.chunks;
  const float Ah = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
  const uint16_t *gb = p.g + q.first * p.gs + h * kP;
  const uint16_t *Cb = p.C + q.first * p.cs + gr * N;
  const uint16_t *dtb = p.dt + q.first * p.dts + h;
  const int srow = (16 * w + r) * N + 4 * kq;

  auto chunk_len = [&](int64_t c) { return static_cast<int>(q.len - c * kQ < kQ ? q.len - c * kQ : kQ); };
  TileLoad<kP> lg;
  TileLoad<N> lc;
  auto fetch = [&](int64_t c, int b) {   // from the last chunk down: only the first one fetched can be short
    lg.fetch(sm.g[b], gb + c * kQ * p.gs, w);
    lc.fetch(sm.C[b], Cb + c * kQ * p.cs, w);
  };
  auto raw_steps = [&](int64_t c) {   // (of the last token beyond the end; as loaded: a conversion would wait for it)
    const int len = chunk_len(c);
    return static_cast<uint32_t>(dtb[(c * kQ + (l < len ? l : len - 1)) * p.dts]);
  };
  // tokens beyond the chunk's end repeat its last one and weigh nothing
  auto put_steps = [&](int64_t c, int b, uint32_t raw) {
    asm volatile("" : "+v"(raw));   // or it is converted, and waited for, where it is loaded
    float v;
    const TwoSum cs = running_sum(chunk_step(p.step, bf2f(static_cast<uint16_t>(raw)), bias, l < chunk_len(c), v), Ah);
    const float e = exp_sum(cs);
    sm.e[b][l] = l < chunk_len(c) ? entry_sign(q.entry + c - 1) * e : 0.0f;
    if (l == 63) sm.end[b] = e;
  };
  if (c_begin < c_end) {
    const int len = chunk_len(c_end - 1);
    lg.place(p.gs, len, w, l);
    lc.place(p.cs, len, w, l);
    fetch(c_end - 1, 0);
    if (len < kQ) {
      lg.place(p.gs, kQ, w, l);
      lc.place(p.cs, kQ, w, l);
    }
    if (w == 0) put_steps(c_end - 1, 0, raw_steps(c_end - 1));
  }

  f32x4 acc[NT];
  const bool from_end = c_end >= q.chunks && p.dfin;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float4 v = from_end ? *reinterpret_cast<const float4 *>(p.dfin + static_cast<int64_t>(sh) * kP * N + srow + 16 * nt)
                              : make_float4(0, 0, 0, 0);
    acc[nt] = (f32x4){v.x, v.y, v.z, v.w};
  }
  if constexpr (STORE) {
    // the carry of the later segments, the last one's first
    int64_t j = p.nseg - 1;
    while (j > seg && j * p.seg_chunks >= q.chunks) --j;
    for (; j > seg; --j) {
      const float P = p.ws_decay[(j - 1) * SH + sh];
      const float *E = p.ws_state + ((j - 1) * SH + sh) * kP * N + srow;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 e = *reinterpret_cast<const float4 *>(E + 16 * nt);
        acc[nt] = (f32x4){fmaf(P, acc[nt][0], e.x), fmaf(P, acc[nt][1], e.y), fmaf(P, acc[nt][2], e.z),
                          fmaf(P, acc[nt][3], e.w)};
      }
    }
  }
  {
    const float sign = entry_sign(q.entry + c_end - 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt] *= sign;
  }
  float decay = 1.0f;
  for (int64_t c = c_end - 1; c >= c_begin; --c) {
    const int b = static_cast<int>((c_end - 1 - c) & 1);
    loads_landed();
    __syncthreads();   // the chunk's tiles are there; the other half's readers are done
    const bool more = c > c_begin;
    uint32_t raw = 0;
    if (w == 0 && more) raw = raw_steps(c - 1);
    if (more) fetch(c - 1, b ^ 1);
    const float end = sm.end[b];
    decay *= end;
    bf16x8 part[kQ / 32][3];   // e g across, in three parts: all 24 bits
#pragma unroll
    for (int kk = 0; kk < kQ / 32; ++kk) {
      const uint4 gt = __builtin_bit_cast(uint4, frag_t<kP>(l, sm.g[b], 32 * kk, 16 * w));
      const float *e = &sm.e[b][32 * kk + 8 * kq];
      uint32_t g0[4], g1[4], g2[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float x = bf2f(raw_bits(gt, i)) * e[i], y = bf2f(raw_bits(gt, i + 1)) * e[i + 1];
        split_bf2(x, y, g0[i / 2], g1[i / 2]);
        g2[i / 2] = third_bf2(x, y, g0[i / 2], g1[i / 2]);
      }
      part[kk][0] = __builtin_bit_cast(bf16x8, make_uint4(g0[0], g0[1], g0[2], g0[3]));
      part[kk][1] = __builtin_bit_cast(bf16x8, make_uint4(g1[0], g1[1], g1[2], g1[3]));
      part[kk][2] = __builtin_bit_cast(bf16x8, make_uint4(g2[0], g2[1], g2[2], g2[3]));
    }
    // Two tiles at a time: their states out, then their products.  Every
    // workgroup is at about the same place of its chunk, so stores that all come
    // at its start leave the memory idle for the rest of it (213 us where this
    // took 196 at 8 x 2048 tokens, 80 heads, and without any store 108; 186 now).
    float *dh = STORE ? p.ws_dh + ((q.entry + c) * p.nheads + h) * kP * N + (16 * w * N + 4 * l) : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; nt += 2) {
      if constexpr (STORE) {
        // as the lanes hold it: a lane's four states of a tile are 16 bytes, and
        // a wave's store one KiB in a row
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4 *>(dh + 256 * (nt + j)) = make_float4(acc[nt + j][0], acc[nt + j][1], acc[nt + j][2], acc[nt + j][3]);
      }
      bf16x8 ct[2][kQ / 32];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[nt + j] *= -end;
#pragma unroll
        for (int kk = 0; kk < kQ / 32; ++kk) ct[j][kk] = frag_t<N>(l, sm.C[b], 32 * kk, 16 * (nt + j));
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int kk = 0; kk < kQ / 32; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[nt + j] = mfma(ct[j][kk], part[kk][k], acc[nt + j]);
    }
    if (w == 0 && more) put_steps(c - 1, b ^ 1, raw);
  }
  float *to = nullptr;
  if constexpr (STORE) {
    if (p.dinit && seg == 0) to = p.dinit + static_cast<int64_t>(sh) * kP * N + srow;
  } else {
    to = p.ws_state + ((seg - 1) * SH + sh) * kP * N + srow;
    if (tid == 0) p.ws_decay[(seg - 1) * SH + sh] = decay;
  }
  if (to) {
    const float sign = entry_sign(q.entry + c_begin - 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      acc[nt] *= sign;
      *reinterpret_cast<float4 *>(to + 16 * nt) = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    }
  }
}

// ---------------------------------------------------------------------------
// (2) one chunk and hb_heads heads of a group: eight waves.
// ---------------------------------------------------------------------------

template <int N>
struct ChunkLds {
  uint16_t B[kQ * N], C[kQ * N];          // [t][n]; from head to head B's place holds dH's third part [p][n]
  uint16_t x[kQ * kP], g[kQ * kP];        // [t][p]
  uint16_t H[kP * N];                     // [p][n]
  uint16_t dh[2][kP * N > kQ * kQ ? kP * N : kQ * kQ];   // [p][n] head, tail; at the end M L dt' [j][i]
  // per head and token: the running sum, the step, exp(cs) to the chunk's
  // start, to the 16-token block's start, and from the chunk's end
  float ch[kMaxHeads][kQ], cl[kMaxHeads][kQ], dt[kMaxHeads][kQ], e0[kMaxHeads][kQ], eb[kMaxHeads][kQ], we[kMaxHeads][kQ];
  // one head's partial sums, and what the heads' steps need of them
  float row[4][kQ], col[4][kQ], q[N / 16][kQ], r[2][kQ], dd[4][kP], hh[8];
  float D[kMaxHeads][kP];   // (a load of D among the products would wait for the next head's tiles)
  // (a token's block is the 16-token one it is in.)  direct and r; the paths
  // through the token: inside its block; and of those to the token, from the
  // blocks before and the entering state, and from it to the blocks after
  float direct[kMaxHeads][kQ], rs[kMaxHeads][kQ], inside[kMaxHeads][kQ], into[kMaxHeads][kQ], from[kMaxHeads][kQ];
  float past[kMaxHeads][4];   // paths from before block k to after it
  float ddc[kMaxHeads][kP], hhs[kMaxHeads];
};

// One workgroup of eight waves.  For a head, between two barriers:
//   a wave forms the pair tiles (i block >= j block) of one j block, M = g x^T,
//     and multiplies S L straight from its registers (a product's result lies
//     as the 16x16x16 product's second operand does) with one half of the
//     channels of g: dx of its j block and half.  Two waves form each tile,
//     which costs less than an LDS round trip and a third barrier; each keeps
//     every second tile's sums.  Wave w takes block w of the first half, wave
//     4 + w block 3 - w of the second, so that the two waves of a SIMD have
//     five tiles together (four waves to a tile, ten to a SIMD, took 659 us
//     where this took 600 at 8 x 2048 tokens, 80 heads);
//   and the state products of its n tile, dH^T x and H^T g.
// The partial sums over tiles meet in LDS; the steps' gradients, chains of
// lane sums, wait until the end and are then done for all heads at once.  545 us
// at 8 x 2048 tokens, 80 heads, of them 45 for dH's third part; vector
// instructions issue 52% of the time, one workgroup a compute unit.
template <int N>
__global__ void __launch_bounds__(512, 2) chunk_kernel(const BwdParams p) {
  constexpr int NT = N / 16;          // n tiles
  constexpr int KN = N / 32;          // k steps over n
  constexpr int IT = NT / 2;          // token tiles of a wave in the (n, token) products
  constexpr int G8 = N / 8;
  constexpr int BC = (kQ * G8 + 511) / 512;     // 16-byte pieces of a B or C tile per thread
  constexpr int HPIECES = kP * N / 16;          // 16-code pieces of H
  static_assert(kP == kQ, "dH's third part in B's place");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  ChunkLds<N> &sm = *reinterpret_cast<ChunkLds<N> *>(smem);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

  // the entry's sequence: the last s whose first entry is at or before it
  const int64_t entry = blockIdx.x;
  const int64_t lo = wave_search(p.nseq, [&](int64_t i) {
    const int at = p.cu[i];
    return (at < 0 ? 0 : at) / kQ + i <= entry;
  });
  const Seq q = sequence(p.cu, p.total, p.max_seqlen, lo);
  const int64_t chunk = entry - q.entry;
  const int64_t hpg = p.per_group;
  const uint32_t gr = blockIdx.y / static_cast<uint32_t>(p.hb_per_group), hb = blockIdx.y - gr * p.hb_per_group;
  const int64_t h0 = gr * hpg + static_cast<int64_t>(hb) * p.hb_heads;
  const int64_t h1 = h0 + p.hb_heads < (gr + 1) * hpg ? h0 + p.hb_heads : (gr + 1) * hpg;
  const int nh = static_cast<int>(h1 - h0);
  if (chunk < 0 || chunk >= q.chunks) {   // an entry of no chunk: nothing to add
    for (int i = tid; i < nh; i += 512) {
      p.ws_sum[(entry * p.nheads + h0 + i) * 2] = 0.0f;
      p.ws_sum[(entry * p.nheads + h0 + i) * 2 + 1] = 0.0f;
    }
    if (p.D) {
      const int64_t per = p.D_per_channel ? kP : 1;
      for (int64_t i = tid; i < nh * per; i += 512) p.ws_dd[(entry * p.nheads + h0) * per + i] = 0.0f;
    }
    return;
  }
  const int64_t t0 = q.first + chunk * kQ;      // the chunk's first token
  const int len = static_cast<int>(q.len - chunk * kQ < kQ ? q.len - chunk * kQ : kQ);
  int l = lane, r = l & 15, kq = l >> 4;

  // ---- this thread's pieces of a head's tiles, loaded one head ahead
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 xv, gv, hv;
  float4 dv[KN];   // of dH: kP N / 4 pieces of four
  float sc = 0.0f;
  // what is the same for the wave steps from head to head, what is the lane's stays
  const int my_t = tid >> 3, my_p = (tid & 7) * 8, my_row = my_t < len ? my_t : len - 1;
  const uint32_t x_at = static_cast<uint32_t>(my_row) * static_cast<uint32_t>(p.xs) + my_p;
  const uint32_t g_at = static_cast<uint32_t>(my_row) * static_cast<uint32_t>(p.gs) + my_p;
  const uint16_t *xh = p.x + t0 * p.xs + h0 * kP, *gh = p.g + t0 * p.gs + h0 * kP;
  const int8_t *code_h = p.codes + entry * p.code_entry + h0 * p.code_head;
  const float *scale_h = p.scales + entry * p.scale_entry + h0 * p.scale_head;
  const float *dh_h = p.ws_dh + (entry * p.nheads + h0) * kP * N;
  auto load_head = [&] {   // tokens beyond the chunk's end repeat the last one here
    xv = ld8_raw(xh + x_at);
    gv = ld8_raw(gh + g_at);
    if (tid < HPIECES) {
      hv = *reinterpret_cast<const uint4 *>(code_h + 16 * tid);
      sc = scale_h[16 * tid / N];
    }
#pragma unroll
    for (int k = 0; k < KN; ++k) dv[k] = *reinterpret_cast<const float4 *>(dh_h + 4 * (tid + 512 * k));
    xh += kP;
    gh += kP;
    code_h += p.code_head;
    scale_h += p.scale_head;
    dh_h += kP * N;
  };
  load_head();

  // ---- B, C, and every head's steps
#pragma unroll
  for (int k = 0; k < BC; ++k) {
    const int piece = tid + 512 * k, t = piece / G8, n0 = (piece % G8) * 8;
    if (piece < kQ * G8) {
      *reinterpret_cast<uint4 *>(&sm.B[tile_at<N>(t, n0)]) = t < len ? ld8_raw(p.B + (t0 + t) * p.bs + gr * N + n0) : zero;
      *reinterpret_cast<uint4 *>(&sm.C[tile_at<N>(t, n0)]) = t < len ? ld8_raw(p.C + (t0 + t) * p.cs + gr * N + n0) : zero;
    }
  }
  for (int k = w; k < nh; k += 8) {
    const int64_t h = h0 + k;
    const float raw = l < len ? bf2f(p.dt[(t0 + l) * p.dts + h]) : 0.0f;
    float v;
    const float d = chunk_step(p.step, raw, p.dt_bias ? p.dt_bias[h] : 0.0f, l < len, v);
    const TwoSum cs = running_sum(d, p.A[h]);
    sm.ch[k][l] = cs.hi;
    sm.cl[k][l] = cs.lo;
    sm.dt[k][l] = d;
    sm.e0[k][l] = exp_sum(cs);
    sm.eb[k][l] = exp_sum(diff(cs, {__shfl(cs.hi, l & 48), __shfl(cs.lo, l & 48)}));
    if (p.D) sm.D[k][l] = p.D_per_channel ? p.D[h * kP + l] : p.D[h];
    sm.we[k][l] = exp_sum(diff({__shfl(cs.hi, 63), __shfl(cs.lo, 63)}, cs));
  }
  if (tid < kQ) {   // no pair tile above the diagonal adds to these
    for (int k = 0; k < 4; ++k) sm.row[k][tid] = sm.col[k][tid] = 0.0f;
  }

  const int ph = w >> 2, jb = ph ? 7 - w : w;   // channel half, j block
  const int nt = w % NT, ti0 = (w / NT) * IT;
  f32x4 S[4], V[2], dBa[IT], dCa[IT];
  const f32x4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 4; ++k) S[k] = zero4;
  V[0] = V[1] = zero4;
#pragma unroll
  for (int k = 0; k < IT; ++k) dBa[k] = dCa[k] = zero4;
  __syncthreads();
  // one copy of the code for each j block
  auto for_block = [&](auto &&f) {
    if (jb == 0) f(std::integral_constant<int, 0>{});
    else if (jb == 1) f(std::integral_constant<int, 1>{});
    else if (jb == 2) f(std::integral_constant<int, 2>{});
    else f(std::integral_constant<int, 3>{});
  };
  for_block([&](auto block) {
    constexpr int JB = decltype(block)::value;
#pragma unroll
    for (int kk = 0; kk < KN; ++kk) {
      const bf16x8 bf = frag<N>(l, sm.B, 16 * JB, 32 * kk);
#pragma unroll
      for (int it = JB; it < 4; ++it) S[it - JB] = mfma(frag<N>(l, sm.C, 16 * it, 32 * kk), bf, S[it - JB]);
    }
  });
  // the wave's block of B, which every head's dH is multiplied with
  bf16x8 Bj[KN];
#pragma unroll
  for (int kk = 0; kk < KN; ++kk) {
    const uint4 b = __builtin_bit_cast(uint4, frag<N>(l, sm.B, 16 * jb, 32 * kk));
    const uint32_t sign = ((l ^ static_cast<int>(entry)) & 1) * 0x80008000u;   // negated for every second token, and as dH
    Bj[kk] = __builtin_bit_cast(bf16x8, make_uint4(b.x ^ sign, b.y ^ sign, b.z ^ sign, b.w ^ sign));
  }
  __syncthreads();   // and B's place is free

  uint16_t *dx_h = p.dx + t0 * p.dxs + h0 * kP;
  const float sign = entry_sign(entry);   // dH's
  for (int k = 0; k < nh; ++k, dx_h += kP) {
    // the lane anew for every head: the tiles' addresses are then formed where
    // they are used; kept over the loop they would take the registers
    asm volatile("" : "+v"(l));
    r = l & 15;
    kq = l >> 4;
    const float *dt = sm.dt[k];
    // ---- stage the head (its tiles' last readers passed the barrier before)
    {
      if (my_t >= len) xv = gv = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(&sm.x[tile_at<kP>(my_t, my_p)]) = xv;
      *reinterpret_cast<uint4 *>(&sm.g[tile_at<kP>(my_t, my_p)]) = gv;
    }
    if (tid < HPIECES) {
      // codes as unsigned bytes (code + 128), one conversion each
      const int row = 16 * tid / N, n0 = (16 * tid) % N;
      const float off = -128.0f * sc;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t word = raw_word(hv, 2 * hf + (i >> 1)) ^ 0x80808080u;
          const int sh = (i & 1) * 16;
          o[i] = pack_bf2(fmaf(static_cast<float>((word >> sh) & 0xffu), sc, off),
                          fmaf(static_cast<float>((word >> (sh + 8)) & 0xffu), -sc, -off));   // every second state negated
        }
        *reinterpret_cast<uint4 *>(&sm.H[tile_at<N>(row, n0 + 8 * hf)]) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
#pragma unroll
    for (int b = 0; b < KN; ++b) {   // out of adjoint_kernel's order: 16 x 16 tiles, four states a lane
      const int tile = (tid >> 6) + 8 * b;
      const int o = tile_at<N>(tile / NT * 16 + (tid & 15), tile % NT * 16 + (tid >> 4 & 3) * 4);
      const float4 v = dv[b];
      uint2 part[3];
      split_bf2(v.x, v.y, part[0].x, part[1].x);
      split_bf2(v.z, v.w, part[0].y, part[1].y);
      part[2].x = third_bf2(v.x, v.y, part[0].x, part[1].x);
      part[2].y = third_bf2(v.z, v.w, part[0].y, part[1].y);
#pragma unroll
      for (int a = 0; a < 2; ++a) *reinterpret_cast<uint2 *>(&sm.dh[a][o]) = part[a];
      *reinterpret_cast<uint2 *>(&sm.B[o]) = part[2];
    }
    __syncthreads();
    if (k + 1 < nh) load_head();

    // ---- the pairs, and dx: pair tiles lie as (i = 16 it + 4 kq + ii,
    // j = 16 JB + r), dx as (p = 16 (2 ph + a) + 4 kq + ii, j = 16 JB + r)
    for_block([&](auto block) {
      constexpr int JB = decltype(block)::value;
      const int j = 16 * JB + r;
      const float jh = sm.ch[k][j], jl = sm.cl[k][j], dj = dt[j];
      f32x4 pr[2] = {zero4, zero4}, st[2] = {zero4, zero4};
#pragma unroll
      for (int kk = 0; kk < KN; ++kk) {
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int a = 0; a < 2; ++a)
            st[a] = mfma(frag<N>(l, part < 2 ? sm.dh[part] : sm.B, 32 * ph + 16 * a, 32 * kk), Bj[kk], st[a]);
      }
      bf16x8 xf[2];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) xf[kk] = frag<kP>(l, sm.x, 16 * JB, 32 * kk);
#pragma unroll
      for (int it = JB; it < 4; ++it) {
        if ((it - JB) % 2 == 0) __builtin_amdgcn_sched_barrier(0);   // bounds the operands in flight
        const int t = it - JB, i0 = 16 * it + 4 * kq;
        f32x4 m = zero4;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) m = mfma(frag<kP>(l, sm.g, 16 * it, 32 * kk), xf[kk], m);
        float L[4];
        if (it == JB) {
          const float4 ih = *reinterpret_cast<const float4 *>(&sm.ch[k][i0]), il = *reinterpret_cast<const float4 *>(&sm.cl[k][i0]);
          const float ihv[4] = {ih.x, ih.y, ih.z, ih.w}, ilv[4] = {il.x, il.y, il.z, il.w};
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) L[ii] = exp_diff(ihv[ii], ilv[ii], jh, jl);
        } else {
          // the decay from j to block i's start, and from there to i
          const float f = exp_diff(sm.ch[k][16 * it], sm.cl[k][16 * it], jh, jl);
          const float4 e = *reinterpret_cast<const float4 *>(&sm.eb[k][i0]);
          L[0] = e.x * f; L[1] = e.y * f; L[2] = e.z * f; L[3] = e.w * f;
        }
        float u[4];
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          u[ii] = S[t][ii] * L[ii];
          if (it == JB && 4 * kq + ii < r) u[ii] = 0.0f;
        }
        uint2 uh, ul;
        split_bf2(u[0], u[1], uh.x, ul.x);
        split_bf2(u[2], u[3], uh.y, ul.y);
        s16x4 gt[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          gt[a] = frag_t4<kP>(l, sm.g, 16 * it, 32 * ph + 16 * a);
          pr[a] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(gt[a], __builtin_bit_cast(s16x4, uh), pr[a], 0, 0, 0);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
          pr[a] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(gt[a], __builtin_bit_cast(s16x4, ul), pr[a], 0, 0, 0);
        if (ph == ((it + JB) & 1)) {
          float col = 0.0f, rows[4];
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            const bool out = it == JB && 4 * kq + ii < r;
            V[t >> 1][ii] = fmaf(out ? 0.0f : m[ii] * L[ii], dj, V[t >> 1][ii]);
            const float G = out ? 0.0f : u[ii] * m[ii];
            col += G;
            rows[ii] = G * dj;
          }
          if (it == JB) {   // of row i, the pairs from before token i to it or after it
            rows[2] += rows[3];
            rows[1] += rows[2];
            rows[0] += rows[1];
            const float after = sum_later_kq(rows[0], kq);
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) rows[ii] = r < 4 * kq + ii ? rows[ii] + after : 0.0f;
          }
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) rows[ii] = sum_r(rows[ii]);
          col = sum_kq(col);
          if (kq == 0) sm.col[it][j] = col;
          if (r == 0) *reinterpret_cast<float4 *>(&sm.row[JB][i0]) = make_float4(rows[0], rows[1], rows[2], rows[3]);
        }
      }
      const float wj = r & 1 ? -sm.we[k][j] : sm.we[k][j];   // (as Bj)
      float rs = 0.0f, gxs = 0.0f, dxv[2][4];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int pc = 32 * ph + 16 * a + 4 * kq;
        float xv4[4], gv4[4], gx[4];
        float (&o)[4] = dxv[a];
        four(&sm.x[tile_at<kP>(j, pc)], xv4);
        four(&sm.g[tile_at<kP>(j, pc)], gv4);
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const float sv = st[a][ii] * wj;
          rs = fmaf(xv4[ii], sv, rs);
          o[ii] = dj * (pr[a][ii] + sv);
        }
        if (p.D) {
          const float4 D4 = *reinterpret_cast<const float4 *>(&sm.D[k][pc]);
          o[0] = fmaf(D4.x, gv4[0], o[0]);
          o[1] = fmaf(D4.y, gv4[1], o[1]);
          o[2] = fmaf(D4.z, gv4[2], o[2]);
          o[3] = fmaf(D4.w, gv4[3], o[3]);
        }
        // and these tokens' part of dD: of each channel's, or of the head's
        if (p.D_per_channel) {
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            gx[ii] = sum_r(gv4[ii] * xv4[ii]);
          }
          if (r == 0) *reinterpret_cast<float4 *>(&sm.dd[JB][pc]) = make_float4(gx[0], gx[1], gx[2], gx[3]);
        } else if (p.D) {
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            gxs = fmaf(gv4[ii], xv4[ii], gxs);
          }
        }
      }
      uint16_t *to = dx_h + j * p.dxs + 32 * ph + 4 * kq;
      if (j < len) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
          *reinterpret_cast<uint2 *>(to + 16 * a) = make_uint2(pack_bf2(dxv[a][0], dxv[a][1]), pack_bf2(dxv[a][2], dxv[a][3]));
      }
      rs = sum_kq(rs);
      if (kq == 0) sm.r[ph][j] = rs;
      if (p.D && !p.D_per_channel) {   // (sixteen token sums of each channel half, in the places of 32 channels)
        gxs = sum_kq(gxs);
        if (kq == 0) {
          sm.dd[JB][32 * ph + r] = gxs;
          sm.dd[JB][32 * ph + 16 + r] = 0.0f;
        }
      }
    });

    // ---- H^T g and dH^T x: lane holds (n = 16 nt + 4 kq + ii, token = 16 ti + r)
    __builtin_amdgcn_sched_barrier(0);
    {
      bf16x8 hf[2], df[2][2];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        hf[kk] = frag_t<N>(l, sm.H, 32 * kk, 16 * nt);
        df[0][kk] = frag_t<N>(l, sm.dh[0], 32 * kk, 16 * nt);
        df[1][kk] = frag_t<N>(l, sm.dh[1], 32 * kk, 16 * nt);
      }
      if (ti0 == 0) {   // <dH, H> over these n: the diagonal of the tiles' product
        f32x4 t = zero4;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          t = mfma(hf[kk], df[0][kk], t);
          t = mfma(hf[kk], df[1][kk], t);
          t = mfma(hf[kk], frag_t<N>(l, sm.B, 32 * kk, 16 * nt), t);
        }
        const int ii = r - 4 * kq;
        const float d = ii == 0 ? t[0] : ii == 1 ? -t[1] : ii == 2 ? t[2] : ii == 3 ? -t[3] : 0.0f;
        const float hh = sum_wave(d);
        if (l == 0) sm.hh[w] = hh;
      }
#pragma unroll
      for (int a = 0; a < IT; ++a) {
        if (a % 2 == 0) __builtin_amdgcn_sched_barrier(0);
        const int t = 16 * (ti0 + a) + r;
        f32x4 c = zero4, b = zero4;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const bf16x8 gf = frag<kP>(l, sm.g, 16 * (ti0 + a), 32 * kk), xf = frag<kP>(l, sm.x, 16 * (ti0 + a), 32 * kk);
          c = mfma(hf[kk], gf, c);
          b = mfma(df[0][kk], xf, b);
          b = mfma(df[1][kk], xf, b);
        }
        const float e = sm.e0[k][t], wj = sm.we[k][t] * dt[t] * sign;
        float cf[4], qs = 0.0f;
        four(&sm.C[tile_at<N>(t, 16 * nt + 4 * kq)], cf);
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const float ce = ii & 1 ? -c[ii] * e : c[ii] * e;   // (as H)
          dCa[a][ii] += ce;
          dBa[a][ii] = fmaf(b[ii], wj, dBa[a][ii]);
          qs = fmaf(ce, cf[ii], qs);
        }
        qs = sum_kq(qs);
        if (kq == 0) sm.q[nt][t] = qs;
      }
    }
    __syncthreads();
    // ---- add up the head's partial sums (read before the next barrier, after
    // which the next head writes its own), each wave a part: by one wave alone
    // they held up the others at that barrier (8 x 2048 tokens, 80 heads: 712 us
    // for 684)
    const int own = l >> 4, part = (w - k) & 7;
    if (part == 0) {
      const float rs = sm.r[0][l] + sm.r[1][l];
      float from = 0.0f;
#pragma unroll
      for (int it = 1; it < 4; ++it) from += it > own ? sm.col[it][l] : 0.0f;
      sm.rs[k][l] = rs;
      sm.direct[k][l] = from + sm.col[own][l] + rs;
      sm.inside[k][l] = sm.row[own][l];
      sm.from[k][l] = from;
    } else if (part < 5) {
      // to this token from before block part - 1 (at most its own)
      const int b = part - 1;
      float into = 0.0f;
#pragma unroll
      for (int a = 0; a < NT; ++a) into += sm.q[a][l];
#pragma unroll
      for (int a = 0; a < 3; ++a)
        if (a < b) into += own > a ? sm.row[a][l] : 0.0f;
      if (b == 3) sm.into[k][l] = into;
      const float past = sum_wave(own > b ? into : 0.0f);
      if (l == 0) sm.past[k][b] = past;
    } else if (part == 5) {
      if (p.D) sm.ddc[k][l] = (sm.dd[0][l] + sm.dd[1][l]) + (sm.dd[2][l] + sm.dd[3][l]);
    } else if (part == 6) {
      if (l == 0) {
        float hh = 0.0f;
#pragma unroll
        for (int a = 0; a < NT; ++a) hh += sm.hh[a];
        sm.hhs[k] = sign * hh;
      }
    }
  }
  __syncthreads();
  uint4 bv[BC];   // B again
#pragma unroll
  for (int k = 0; k < BC; ++k) {
    const int piece = tid + 512 * k, t = piece / G8;
    bv[k] = piece < kQ * G8 && t < len ? ld8_raw(p.B + (t0 + t) * p.bs + gr * N + (piece % G8) * 8) : zero;
  }

  // ---- the heads' steps: lane = token
  for (int k = w; k < nh; k += 8) {
    const int64_t h = h0 + k;
    const float Ah = p.A[h], d = sm.dt[k][l], rs = sm.rs[k][l], direct = sm.direct[k][l];
    const float raw = l < len ? bf2f(p.dt[(t0 + l) * p.dts + h]) : 0.0f;
    const float da = ((sm.inside[k][l] + sums_before<16>(d * sm.from[k][l])) + (row_suffix(sm.into[k][l]) + sm.past[k][l >> 4])) +
                     fmaf(sm.e0[k][kQ - 1], sm.hhs[k], sums_before<64>(d * rs));
    float v, dd = fmaf(Ah, da, direct);
    chunk_step(p.step, raw, p.dt_bias ? p.dt_bias[h] : 0.0f, true, v);
    if (p.step.limit) {
      const float sp = p.step.softplus ? softplus_step(v) : v;
      if (!(sp >= p.step.lo && sp <= p.step.hi)) dd = 0.0f;
    }
    if (p.step.softplus) dd *= fast_rcp(1.0f + fast_exp2(-v * kLog2e));
    if (l >= len) dd = 0.0f;
    else p.ddt[(t0 + l) * p.ddts + h] = static_cast<uint16_t>(float_to_half_bits<1>(dd));
    const float dA = sum_wave(d * da), db = sum_wave(dd);
    if (l == 0) {
      p.ws_sum[(entry * p.nheads + h) * 2] = dA;
      p.ws_sum[(entry * p.nheads + h) * 2 + 1] = db;
    }
    if (p.D) {
      const float s = sm.ddc[k][l];
      if (p.D_per_channel) p.ws_dd[(entry * p.nheads + h) * kP + l] = s;
      else if (const float all = sum_wave(s); l == 0) p.ws_dd[entry * p.nheads + h] = all;
    }
  }

  // ---- the pair parts of dB and dC, from the heads' summed M L dt'
#pragma unroll
  for (int k = 0; k < BC; ++k) {
    const int piece = tid + 512 * k;
    if (piece < kQ * G8) *reinterpret_cast<uint4 *>(&sm.B[tile_at<N>(piece / G8, (piece % G8) * 8)]) = bv[k];
  }
  uint16_t *Vh = sm.dh[0], *Vl = sm.dh[1];
  *reinterpret_cast<uint4 *>(Vh + 8 * tid) = zero;
  *reinterpret_cast<uint4 *>(Vl + 8 * tid) = zero;
  __syncthreads();
  for_block([&](auto block) {
    constexpr int JB = decltype(block)::value;
#pragma unroll
    for (int it = JB; it < 4; ++it) {
      if (ph != ((it + JB) & 1)) continue;
      const f32x4 &v = V[(it - JB) >> 1];
      uint2 vh, vl;
      split_bf2(v[0], v[1], vh.x, vl.x);
      split_bf2(v[2], v[3], vh.y, vl.y);
      const int o = tile_at<kQ>(16 * JB + r, 16 * it + 4 * kq);
      *reinterpret_cast<uint2 *>(&Vh[o]) = vh;
      *reinterpret_cast<uint2 *>(&Vl[o]) = vl;
    }
  });
  __syncthreads();
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const bf16x8 bt = frag_t<N>(l, sm.B, 32 * kk, 16 * nt), ct = frag_t<N>(l, sm.C, 32 * kk, 16 * nt);
#pragma unroll
    for (int a = 0; a < IT; ++a) {
      const int tt = 16 * (ti0 + a);
      dCa[a] = mfma(bt, frag_t<kQ>(l, Vh, 32 * kk, tt), dCa[a]);
      dCa[a] = mfma(bt, frag_t<kQ>(l, Vl, 32 * kk, tt), dCa[a]);
      dBa[a] = mfma(ct, frag<kQ>(l, Vh, tt, 32 * kk), dBa[a]);
      dBa[a] = mfma(ct, frag<kQ>(l, Vl, tt, 32 * kk), dBa[a]);
    }
  }
#pragma unroll
  for (int a = 0; a < IT; ++a) {
    const int t = 16 * (ti0 + a) + r, n0 = 16 * nt + 4 * kq;
    if (t < len) {
      if (p.ws_bc) {
        const int64_t plane = p.hb_per_group * p.total * p.ngroups * N;
        float *o = p.ws_bc + ((static_cast<int64_t>(hb) * p.total + t0 + t) * p.ngroups + gr) * N + n0;
        *reinterpret_cast<float4 *>(o) = make_float4(dBa[a][0], dBa[a][1], dBa[a][2], dBa[a][3]);
        *reinterpret_cast<float4 *>(o + plane) = make_float4(dCa[a][0], dCa[a][1], dCa[a][2], dCa[a][3]);
      } else {
        *reinterpret_cast<uint2 *>(p.dB + (t0 + t) * p.dbs + gr * N + n0) =
            make_uint2(pack_bf2(dBa[a][0], dBa[a][1]), pack_bf2(dBa[a][2], dBa[a][3]));
        *reinterpret_cast<uint2 *>(p.dC + (t0 + t) * p.dcs + gr * N + n0) =
            make_uint2(pack_bf2(dCa[a][0], dCa[a][1]), pack_bf2(dCa[a][2], dCa[a][3]));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// (3) the sums over head blocks and chunks
// ---------------------------------------------------------------------------
// One launch for all of them: workgroups [0, 2 bc_blocks) add the head blocks'
// dB and dC (1024 elements each), the next ones the chunks' (dA, ddt_bias),
// the last ones the chunks' dD: 8 columns each, 32 threads a column, every
// thread its chunks in order and then the 32 in order, in 64 bits.
struct SumParams {
  const float *bc, *sum, *dd;
  uint16_t *dB, *dC;
  float *dA, *ddt_bias, *dD;
  int64_t total, row, dbs, dcs, entries, nheads, dd_cols, bc_blocks, sum_blocks;
  int hb;
};

__global__ void __launch_bounds__(256) sum_kernel(const SumParams p) {
  __shared__ double part[32][8];
  const int tid = threadIdx.x;
  int64_t blk = blockIdx.x;
  if (blk < 2 * p.bc_blocks) {
    const bool second = blk >= p.bc_blocks;
    const int64_t plane = p.total * p.row;
    const float *from = p.bc + (second ? p.hb * plane : 0);
    const int64_t i = ((blk - (second ? p.bc_blocks : 0)) * 256 + tid) * 4;
    if (i >= plane) return;
    float4 a = *reinterpret_cast<const float4 *>(from + i);
    for (int k = 1; k < p.hb; ++k) {
      const float4 b = *reinterpret_cast<const float4 *>(from + k * plane + i);
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    const int64_t t = i / p.row, c = i - t * p.row;
    *reinterpret_cast<uint2 *>((second ? p.dC + t * p.dcs : p.dB + t * p.dbs) + c) =
        make_uint2(pack_bf2(a.x, a.y), pack_bf2(a.z, a.w));
    return;
  }
  blk -= 2 * p.bc_blocks;
  const bool steps = blk < p.sum_blocks;
  const float *from = steps ? p.sum : p.dd;
  const int64_t cols = steps ? 2 * p.nheads : p.dd_cols;
  const int64_t col = (steps ? blk : blk - p.sum_blocks) * 8 + (tid & 7);
  double v = 0.0;
  if (col < cols) {
#pragma unroll 4
    for (int64_t e = tid >> 3; e < p.entries; e += 32) v += from[e * cols + col];
  }
  part[tid >> 3][tid & 7] = v;
  __syncthreads();
  if (tid >= 8 || col >= cols) return;
  v = 0.0;
  for (int k = 0; k < 32; ++k) v += part[k][tid];
  const float out = static_cast<float>(v);
  if (!steps) p.dD[col] = out;
  else if (!(col & 1)) p.dA[col >> 1] = out;
  else if (p.ddt_bias) p.ddt_bias[col >> 1] = out;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct BwdPlan {
  int nseg, hb_heads, hb_per_group;
  int64_t seg_chunks, entries;
  size_t off_state, off_decay, off_bc, off_sum, off_dd, bytes;
};

// Time in us of the adjoint pass with segments of seg chunks.  Storing every
// chunk's dH (32 KB at dstate 128, beside 24 KB read) goes at about 4 TB/s; a
// workgroup's chain takes 2.2 us a chunk, or 1.6 where nothing is stored, in
// the launch that finds the segments' ends, at dstate 128.  Measured (us of the
// whole backward, one segment / chosen / best of a sweep), at dstate 128, 64 and
// 32: 4 x 2048 tokens x 80 heads 403 / 403 / 403, 270 / 269 / 270, 216 / 215 / 216;
// 1 x 2048 x 80 168 / 158 / 158, 120 / 111 / 109, 101 / 90 / 91; 1 x 16384 x 16
// 508 / 234 / 230, 378 / 148 / 146, 301 / 117 / 117.
double adjoint_us(int64_t blocks, int64_t nchunks, int64_t seg, int64_t dstate, int64_t cus) {
  const int64_t G = (nchunks + seg - 1) / seg;
  const double len = static_cast<double>(seg) + 0.8, state = static_cast<double>(kP) * dstate * sizeof(float);
  const double store = static_cast<double>(blocks) * nchunks * (state + kP * kQ * 2 + 2.0 * dstate * kQ) / 4e6;
  double t = rounds_us(blocks * G, len, 2.2, 2.2, 3, cus);
  if (t < store) t = store;
  if (G > 1)
    t += rounds_us(blocks * (G - 1), len, 1.6, 1.6, 3, cus) + 5.0 +
         blocks * state * (static_cast<double>(G) * (G - 1) / 2 / 1e7 + (G - 1) / 5e6);
  return t;
}

BwdPlan bwd_plan(const ssd_varlen_args_t *a, int cus) {
  BwdPlan pl{};
  pl.entries = ssd_checkpoint_slots(a->total, a->nseq);
  const int64_t SH = a->nseq * a->nheads, hpg = a->nheads / a->ngroups;
  // adjoint segments
  int64_t nchunks = (a->max_seqlen + kQ - 1) / kQ;
  if (nchunks < 1) nchunks = 1;
  int64_t G = 1;
  if (a->seq_segments >= 1) {
    G = a->seq_segments;
  } else {
    const int64_t rows = (pl.entries + nchunks - 1) / nchunks;
    const int64_t blocks = (rows < a->nseq ? rows : a->nseq) * a->nheads;
    double best = 1e300;
    for (int64_t k = 1; k <= 64 && (k == 1 || 2 * k <= nchunks); ++k) {
      const double t = adjoint_us(blocks, nchunks, (nchunks + k - 1) / k, a->dstate, cus);
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
  // head blocks: enough workgroups for four rounds, as few partial dB and dC
  // as that allows
  int64_t per = (4LL * cus + pl.entries * a->ngroups - 1) / (pl.entries * a->ngroups);
  if (per < (hpg + kMaxHeads - 1) / kMaxHeads) per = (hpg + kMaxHeads - 1) / kMaxHeads;
  if (per > hpg) per = hpg;
  pl.hb_heads = static_cast<int>((hpg + per - 1) / per);
  pl.hb_per_group = static_cast<int>((hpg + pl.hb_heads - 1) / pl.hb_heads);
  size_t at = up256(static_cast<size_t>(pl.entries) * a->nheads * kP * a->dstate * sizeof(float));
  pl.off_state = at;
  if (pl.nseg > 1) at += up256(static_cast<size_t>(pl.nseg - 1) * SH * kP * a->dstate * sizeof(float));
  pl.off_decay = at;
  if (pl.nseg > 1) at += up256(static_cast<size_t>(pl.nseg - 1) * SH * sizeof(float));
  pl.off_bc = at;
  if (pl.hb_per_group > 1)
    at += up256(2 * static_cast<size_t>(pl.hb_per_group) * a->total * a->ngroups * a->dstate * sizeof(float));
  pl.off_sum = at;
  at += up256(static_cast<size_t>(pl.entries) * a->nheads * 2 * sizeof(float));
  pl.off_dd = at;
  if (a->D) at += up256(static_cast<size_t>(pl.entries) * a->nheads * (a->D_per_channel ? kP : 1) * sizeof(float));
  pl.bytes = at;
  return pl;
}

template <int N>
hipError_t launch_bwd(const BwdParams &p, const BwdPlan &pl, hipStream_t stream) {
  const unsigned sh = static_cast<unsigned>(p.nseq * p.nheads);
  hipError_t e;
  if (pl.nseg > 1) {
    hipLaunchKernelGGL((adjoint_kernel<N, false>), dim3(sh, pl.nseg - 1), dim3(256), 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((adjoint_kernel<N, true>), dim3(sh, pl.nseg), dim3(256), 0, stream, p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned lds = sizeof(ChunkLds<N>);
  const auto chunk = chunk_kernel<N>;
  e = hipFuncSetAttribute(reinterpret_cast<const void *>(chunk), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(lds));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(chunk, dim3(static_cast<unsigned>(pl.entries), static_cast<unsigned>(p.ngroups * pl.hb_per_group)),
                     dim3(512), lds, stream, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int ssd_varlen_bwd_workspace_size(const ssd_varlen_bwd_args_t *a, size_t *bytes) {
  const int st = ssd_varlen_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = bwd_plan(&a->fwd, cu_count_cached()).bytes;
  return SSM_OK;
}

extern "C" int ssd_varlen_bwd(const ssd_varlen_bwd_args_t *a, void *stream_ptr) {
  const int st = ssd_varlen_bwd_validate(a);
  if (st != SSM_OK) return st;
  const ssd_varlen_args_t &f = a->fwd;
  const BwdPlan pl = bwd_plan(&f, cu_count_cached());
  // sum_kernel's workgroups for dB and dC, where there are head blocks to add
  const int64_t bc_blocks = pl.hb_per_group > 1 ? (f.total * f.ngroups * f.dstate + 1023) / 1024 : 0;
  if (!grid_fits(f.nseq * f.nheads, 256) || !grid_fits(pl.entries, 512) || f.ngroups * pl.hb_per_group > 65535 ||
      !grid_fits(2 * bc_blocks + f.nheads * kP, 256))
    return SSM_ERR_SHAPE;
  if (!a->workspace || a->workspace_bytes < pl.bytes) return SSM_ERR_WORKSPACE;
  if (!aligned16(a->workspace)) return SSM_ERR_UNSUPPORTED;
  char *ws = static_cast<char *>(a->workspace);
  BwdParams p{};
  p.x = static_cast<const uint16_t *>(f.x); p.xs = f.x_stride;
  p.dt = static_cast<const uint16_t *>(f.dt); p.dts = f.dt_stride;
  p.B = static_cast<const uint16_t *>(f.B); p.bs = f.B_stride;
  p.C = static_cast<const uint16_t *>(f.C); p.cs = f.C_stride;
  p.g = static_cast<const uint16_t *>(a->dout); p.gs = a->dout_stride;
  p.A = f.A; p.D = f.D; p.dt_bias = f.dt_bias; p.dfin = a->dfinal_states;
  p.cu = f.cu_seqlens; p.codes = f.checkpoints; p.scales = f.checkpoint_scales;
  p.dx = static_cast<uint16_t *>(a->dx); p.dxs = a->dx_stride;
  p.ddt = static_cast<uint16_t *>(a->ddt); p.ddts = a->ddt_stride;
  p.dB = static_cast<uint16_t *>(a->dB); p.dbs = a->dB_stride;
  p.dC = static_cast<uint16_t *>(a->dC); p.dcs = a->dC_stride;
  p.dinit = a->dinitial_states;
  p.ws_dh = reinterpret_cast<float *>(ws);
  p.ws_state = reinterpret_cast<float *>(ws + pl.off_state);
  p.ws_decay = reinterpret_cast<float *>(ws + pl.off_decay);
  p.ws_bc = pl.hb_per_group > 1 ? reinterpret_cast<float *>(ws + pl.off_bc) : nullptr;
  p.ws_sum = reinterpret_cast<float *>(ws + pl.off_sum);
  p.ws_dd = reinterpret_cast<float *>(ws + pl.off_dd);
  p.total = f.total; p.nseq = f.nseq; p.max_seqlen = f.max_seqlen;
  p.nheads = f.nheads; p.ngroups = f.ngroups;
  p.heads = static_cast<uint32_t>(f.nheads);
  p.per_group = static_cast<uint32_t>(f.nheads / f.ngroups);
  p.code_entry = a->code_entry_stride; p.code_head = a->code_head_stride;
  p.scale_entry = a->scale_entry_stride; p.scale_head = a->scale_head_stride;
  p.seg_chunks = pl.seg_chunks; p.nseg = pl.nseg; p.entries = pl.entries;
  p.hb_heads = pl.hb_heads; p.hb_per_group = pl.hb_per_group;
  p.step = {f.dt_softplus, f.dt_limit, f.dt_min, f.dt_max};
  p.D_per_channel = f.D && f.D_per_channel;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  hipError_t e = f.dstate == 32 ? launch_bwd<32>(p, pl, stream)
                 : f.dstate == 64 ? launch_bwd<64>(p, pl, stream) : launch_bwd<128>(p, pl, stream);
  if (e != hipSuccess) return hip_fail(e);
  SumParams q{};
  q.bc = p.ws_bc; q.sum = p.ws_sum; q.dd = p.ws_dd;
  q.dB = p.dB; q.dC = p.dC; q.dbs = p.dbs; q.dcs = p.dcs;
  q.dA = a->dA; q.ddt_bias = f.dt_bias ? a->ddt_bias : nullptr; q.dD = a->dD;
  q.total = f.total; q.row = f.ngroups * f.dstate; q.entries = pl.entries; q.nheads = f.nheads;
  q.hb = pl.hb_per_group;
  q.bc_blocks = bc_blocks;
  q.sum_blocks = (2 * f.nheads + 7) / 8;
  q.dd_cols = f.D ? f.nheads * (f.D_per_channel ? kP : 1) : 0;
  const int64_t blocks = 2 * q.bc_blocks + q.sum_blocks + (q.dd_cols + 7) / 8;
  hipLaunchKernelGGL(sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, q);
  e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}
