// ssd_util.h -- matrix-core, LDS-layout and bf16 head/tail helpers shared by
// the Mamba-2 chunked-scan kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_util.h"
#include "ssmscan.h"

namespace ssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kQ = SSD_CHUNK;     // tokens per chunk
constexpr int kP = SSD_HEADDIM;   // channels per head

// element offset of (row, col) in a row-major LDS matrix whose rows hold
// ROW_LEN bf16 elements: the row's 16-byte groups are permuted by
// (row ^ row / 8) mod 8, so that both the operand reads (16 rows, one group
// each) and the transposed stores (8 rows 8 apart, 8 consecutive columns)
// spread over the banks
template <int ROW_LEN>
__device__ __forceinline__ int swz(int row, int col) {
  constexpr int GROUPS = ROW_LEN / 8;
  const int gsw = ((row ^ (row >> 3)) & 7) & (GROUPS - 1);
  return row * ROW_LEN + (col ^ (gsw << 3));
}

// element offset of (row, col) in a row-major LDS matrix of ROW_LEN bf16
// whose rows are read in 8-byte pieces: the row's 8-byte pieces are permuted
// by the row (mod 16), so 16 consecutive rows read at one column land on
// different banks (measured: permuting 16-byte groups instead left these
// reads with as many bank conflicts as no permutation)
template <int ROW_LEN>
__device__ __forceinline__ int swz8(int row, int col) {
  constexpr int PIECES = ROW_LEN / 4;
  constexpr int MASK = PIECES > 16 ? 15 : PIECES - 1;
  return row * ROW_LEN + (col ^ ((row & MASK) << 2));
}

__device__ __forceinline__ float bf2f(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }
__device__ __forceinline__ bf16x8 ld8(const uint16_t *p) { return *reinterpret_cast<const bf16x8 *>(p); }
// 8 consecutive bf16 as raw words (element i in the low / high half of word i/2)
__device__ __forceinline__ uint4 ld8_raw(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ uint32_t raw_word(const uint4 &q, int j) {
  return j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
}
__device__ __forceinline__ uint16_t raw_bits(const uint4 &q, int i) {
  const uint32_t wd = raw_word(q, i >> 1);
  return static_cast<uint16_t>((i & 1) ? (wd >> 16) : (wd & 0xffffu));
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// two floats rounded to bf16 (to nearest, ties to even) by one paired
// conversion; a in the low half
__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
// a ~ hi + lo and b ~ hi + lo with all four halves bf16 (hi rounded to
// nearest, lo the rounded rest), as two packed pairs: the same values as
// rounding each element on its own, in three operations per element
__device__ __forceinline__ void split_bf2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf2(a, b);
  lo = pack_bf2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
// ... and what head and tail leave of a and b: with it all 24 bits
__device__ __forceinline__ uint32_t third_bf2(float a, float b, uint32_t hi, uint32_t lo) {
  return pack_bf2(a - __uint_as_float(hi << 16) - __uint_as_float(lo << 16),
                  b - __uint_as_float(hi & 0xffff0000u) - __uint_as_float(lo & 0xffff0000u));
}
// the 16-bit halves of two words side by side (one byte permute): the low
// halves (HIGH = false) or the high halves of a and b, a's in the low half
template <bool HIGH>
__device__ __forceinline__ uint32_t pair_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, HIGH ? 0x07060302u : 0x05040100u);
}

__device__ __forceinline__ f32x4 mfma(const bf16x8 &a, const bf16x8 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

}  // namespace ssm
