// packed_util.h -- what the packed-token scan's forward and backward share
// (gfx950): sequences, steps, LDS tiles and their operand fragments, lane sums.
#pragma once

#include "ssd_util.h"

namespace ssm {

struct Seq {
  int64_t first, len, chunks, entry;   // entry: its first checkpoint
};
// A sequence's tokens, kept inside the tensors whatever cu holds.
__device__ __forceinline__ Seq sequence(const int32_t *cu, int64_t total, int64_t max_seqlen, int64_t s) {
  int64_t lo = cu[s], hi = cu[s + 1];
  lo = lo < 0 ? 0 : lo > total ? total : lo;
  hi = hi < lo ? lo : hi > total ? total : hi;
  const int64_t len = hi - lo > max_seqlen ? max_seqlen : hi - lo;
  return {lo, len, (len + kQ - 1) / kQ, lo / kQ + s};
}

// How a step comes from dt.
struct StepRule {
  int softplus, limit;
  float lo, hi;
};
// The value before softplus of a token's step, and the step (0 beyond the
// chunk's end).
__device__ __forceinline__ float chunk_step(const StepRule &s, float raw, float bias, bool live, float &v) {
  v = raw + bias;
  float d = s.softplus ? softplus_step(v) : v;
  if (s.limit) d = fminf(fmaxf(d, s.lo), s.hi);
  return live ? d : 0.0f;
}

// Running sum over the wave's lanes of d A, as an unevaluated sum of two
// floats: decays are exponentials of its differences, whose error would
// otherwise be the rounding of a sum that reaches 100 and more.  (Without
// contraction: with the product d A inside the first sum's fma, its rounding was
// counted there and in lo.)
struct TwoSum {
  float hi, lo;
};
// lane n's value from the lane that CTRL names, 0 where there is none
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float from_lane(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROW_MASK, 0xf, false));
}
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ void add_lane(TwoSum &s) {
#pragma clang fp contract(off)
  const float oh = from_lane<CTRL, ROW_MASK>(s.hi), ol = from_lane<CTRL, ROW_MASK>(s.lo);
  const float t = s.hi + oh, b = t - s.hi;
  s.lo += ol + ((s.hi - (t - b)) + (oh - b));
  s.hi = t;
}
__device__ __forceinline__ TwoSum running_sum(float d, float A) {
#pragma clang fp contract(off)
  TwoSum s;
  s.hi = d * A;
  s.lo = fmaf(d, A, -s.hi);
  add_lane<0x111, 0xf>(s);   // the lanes 1, 2, 4 and 8 before, inside a row of 16
  add_lane<0x112, 0xf>(s);
  add_lane<0x114, 0xf>(s);
  add_lane<0x118, 0xf>(s);
  add_lane<0x142, 0xa>(s);   // row 0's sum to row 1, row 2's to row 3
  add_lane<0x143, 0xc>(s);   // the first half's to the second
  return s;
}
// s log2 e, as an unevaluated sum: the rounding of the product, which a sum of
// -10 makes ten times 2^-24, is recovered with an fma.
__device__ __forceinline__ TwoSum times_log2e(TwoSum s) {
  constexpr float kLog2eLo = 1.9259630e-8f;   // log2 e - kLog2e
  const float t = s.hi * kLog2e;
  return {t, fmaf(s.hi, kLog2e, -t) + fmaf(s.hi, kLog2eLo, s.lo * kLog2e)};
}
// exp of an unevaluated sum, to the hardware exp2's own rounding.
__device__ __forceinline__ float exp_sum(TwoSum s) {
  const TwoSum t = times_log2e(s);
  const float e = fast_exp2(t.hi);
  return fmaf(e, t.lo * kLn2, e);
}
// a - b
__device__ __forceinline__ TwoSum diff(TwoSum a, TwoSum b) {
#pragma clang fp contract(off)
  const float t = a.hi - b.hi, v = t - a.hi;
  return {t, ((a.hi - (t - v)) - (b.hi + v)) + (a.lo - b.lo)};
}
// exp(a - b), without that recovery
__device__ __forceinline__ float exp_diff(float ah, float al, float bh, float bl) {
  return fast_exp2(((ah - bh) + (al - bl)) * kLog2e);
}

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

// Element offset of (row, col) in a row-major tile of ROW_LEN bf16.  A row's
// 16-byte groups are permuted by g = the row's last three bits rotated, so
// that eight consecutive rows at one column (an operand read row by row) have
// eight values of g, and four consecutive rows (a transposing read: 32 bytes
// of each) four values of g / 2.  Rows r and r + 8 of an operand still meet:
// conflicts are 42 to 52% of the LDS's active cycles in the scan and its gradient.
template <int ROW_LEN>
__device__ __forceinline__ int tile_at(int row, int col) {
  constexpr int GROUPS = ROW_LEN / 8;
  const int g = (((row & 3) << 1) | ((row >> 2) & 1)) & (GROUPS - 1);
  return row * ROW_LEN + (col & ~63) + ((col & 63) ^ (g << 3));
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
// The operand fragment that a row-major tile holds column by column: lane
// (r, kq) receives tile[row0 + 8 kq + i][col0 + r], i < 8.
template <int ROW_LEN>
__device__ __forceinline__ bf16x8 frag_t(int l, uint16_t *tile, int row0, int col0) {
  typedef __attribute__((address_space(3))) s16x4 *lds;
  const int i = l & 15, kq = l >> 4;
  const int row = row0 + 8 * kq + (i >> 2), col = col0 + 4 * (i & 3);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(tile + tile_at<ROW_LEN>(row, col)));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(tile + tile_at<ROW_LEN>(row + 4, col)));
  const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
  return __builtin_bit_cast(bf16x8, make_uint4(ua.x, ua.y, ub.x, ub.y));
}
// ... of four rows only: lane (r, kq) receives tile[row0 + 4 kq + i][col0 + r], i < 4.
template <int ROW_LEN>
__device__ __forceinline__ s16x4 frag_t4(int l, uint16_t *tile, int row0, int col0) {
  typedef __attribute__((address_space(3))) s16x4 *lds;
  const int i = l & 15, kq = l >> 4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(tile + tile_at<ROW_LEN>(row0 + 4 * kq + (i >> 2), col0 + 4 * (i & 3))));
}
// ... and row by row: lane (r, kq) receives tile[row0 + r][col0 + 8 kq + i].
template <int ROW_LEN>
__device__ __forceinline__ bf16x8 frag(int l, const uint16_t *tile, int row0, int col0) {
  return ld8(tile + tile_at<ROW_LEN>(row0 + (l & 15), col0 + 8 * (l >> 4)));
}

// sum over the four kq lanes of a column r: neighbouring rows of 16 lanes swap,
// then the halves
__device__ __forceinline__ float sum_kq(float v) {
  const uint32_t a = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(__uint_as_float(x[0]) + __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}
// sum over the sixteen r lanes of a row kq: rotations of the row
template <int N>
__device__ __forceinline__ float row_rotate(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum_r(float v) {
  v += row_rotate<8>(v);
  v += row_rotate<4>(v);
  v += row_rotate<2>(v);
  return v + row_rotate<1>(v);
}
__device__ __forceinline__ float sum_wave(float v) { return sum_kq(sum_r(v)); }
// sum over the kq lanes of a column after this one
__device__ __forceinline__ float sum_later_kq(float v, int kq) {
  const uint32_t a = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);   // each pair of rows: the first, the second
  const float second = __uint_as_float(x[1]);
  const uint32_t b = __float_as_uint(__uint_as_float(x[0]) + second);
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return (kq & 1 ? 0.0f : second) + (kq < 2 ? __uint_as_float(y[1]) : 0.0f);
}
// sum over the lanes of a row of 16 from this one on
__device__ __forceinline__ float row_suffix(float v) {
  v += from_lane<0x101, 0xf>(v);
  v += from_lane<0x102, 0xf>(v);
  v += from_lane<0x104, 0xf>(v);
  return v + from_lane<0x108, 0xf>(v);
}
// sum over the lanes before this one, in its row of 16 or in the wave
template <int LANES>
__device__ __forceinline__ float sums_before(float v) {
  v = LANES == 16 ? from_lane<0x111, 0xf>(v) : from_lane<0x138, 0xf>(v);   // one lane on
  v += from_lane<0x111, 0xf>(v);
  v += from_lane<0x112, 0xf>(v);
  v += from_lane<0x114, 0xf>(v);
  v += from_lane<0x118, 0xf>(v);
  if constexpr (LANES == 64) {
    v += from_lane<0x142, 0xa>(v);
    v += from_lane<0x143, 0xc>(v);
  }
  return v;
}

// four bf16 of one 8-byte piece
__device__ __forceinline__ void four(const uint16_t *p, float (&v)[4]) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  v[0] = __uint_as_float(w.x << 16);
  v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16);
  v[3] = __uint_as_float(w.y & 0xffff0000u);
}

// A row-major tile's 16-byte pieces straight into LDS.  A wave writes one KiB
// in order, so the tile's permutation (tile_at, its own inverse) is applied to
// where each lane reads: `at` holds a lane's byte offsets from the tile's
// first token, which only a sequence's last chunk changes.  Tokens at and
// after `len` repeat the last one: their steps are 0, and what they give
// reaches no output.
template <int ROW_LEN>
struct TileLoad {
  static constexpr int G = ROW_LEN / 8, ALL = kQ * G / 64, PER = (ALL + 3) / 4;
  uint32_t at[PER];
  __device__ __forceinline__ void place(int64_t stride, int len, int w, int lane) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int piece = (w + 4 * i) * 64 + lane, row = piece / G, t = row < len ? row : len - 1;
      at[i] = 2u * (static_cast<uint32_t>(t) * static_cast<uint32_t>(stride) +
                    static_cast<uint32_t>(tile_at<ROW_LEN>(row, (piece % G) * 8) - row * ROW_LEN));
    }
  }
  // In assembly, because the compiler cannot tell the two halves of a double
  // buffer apart and waits for the loads at the first LDS read after them; the
  // reader of the tile waits itself (loads_landed, then a barrier).  Such a
  // load writes no register.  The compiler's own counted waits stay right:
  // loads return in order, so an unknown one can only make them wait longer.
  // The wait states are those a load needs after a vector instruction wrote its
  // scalar address (five) or a scalar one m0 (one).
  __device__ __forceinline__ void fetch(uint16_t *tile, const uint16_t *from, int w) const {
    const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint16_t *)tile));
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (w + 4 * i < ALL)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(__builtin_amdgcn_readfirstlane(lds + (w + 4 * i) * 1024)), "v"(at[i]), "s"(from)
                     : "m0", "memory");
  }
};

// This wave's part of the tiles is in LDS (every wave's after a barrier), and
// what else it loaded before its last LATER stores is there: loads and stores
// are counted together and return in order, so stores that follow the loads
// need not have ended.
template <int LATER = 0>
__device__ __forceinline__ void loads_landed() {
  static_assert(LATER < 16, "the count's low bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70 | LATER);   // vmcnt(LATER); the compiler counts on from here
  asm volatile("" ::: "memory");
}

// A barrier for LDS alone: what is on its way from global memory stays so.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace ssm
