// Microscaled 4-bit matrices (OCP Microscaling Formats v1.0, MXFP4): E2M1 elements
// with one E8M0 scale, a power of two, for each 32 consecutive elements of a row.
//
// Packed form of a matrix of R rows of L elements, L padded with zeros to
// Lp = 128 ceil(L / 128):
//   codes  [Lp / 32][R][16]  16 bytes a block, even element in the low nibble;
//   scales [Lp / 128][R][4]  the scale bytes of four consecutive blocks of a row.
// Blocks of one position along the rows lie together because a lane of the
// 32x32x64 matrix instruction takes exactly one block (16 bytes) of one row: 32
// consecutive rows are 512 consecutive bytes, from memory to LDS to registers
// with no swizzle and no bank conflict, and a reduction step of 128 reads four
// such runs and one run of scale words.
#pragma once

#include "common.h"

namespace mx4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 32;      // elements of one scale
constexpr int kPad = 128;       // padding of the packed length: the four blocks of a scale word

inline int64_t padded(int64_t len) { return (len + kPad - 1) / kPad * kPad; }
inline int64_t code_bytes(int64_t rows, int64_t len) { return padded(len) / 2 * rows; }
inline int64_t scale_bytes(int64_t rows, int64_t len) { return padded(len) / kBlock * rows; }

// Scale byte of a block whose largest magnitude has the fp32 bits `top`: the
// exponent floor(log2 top) - 2 puts it in [4, 8), where E2M1 ends (at 6).  The
// exponent is at least -123, so that no value of a packed matrix, and no element
// that does not round to 0, is subnormal in fp32 or bf16 (the smallest value is
// 2^-124; elements below 2^-125 round to 0 under any treatment of subnormals).
// 255 marks a block with an infinity or NaN: all its values are NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : (e > 6u ? e - 2u : 4u);
}

// The scale operand of the conversions, which read its exponent bits alone: byte 0 stands
// for 2^-127 there as in the matrix instruction.
__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

// Largest over lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ uint32_t max_over_rows(uint32_t v) {
  u32x2 s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(s[0], s[1]);
  s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(s[0], s[1]);
}

// Eight bf16 (four words) -> eight codes, nearest with ties to even, at most 6.
__device__ __forceinline__ uint32_t encode8(u32x4 v, float s) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[0]), s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[1]), s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[2]), s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)v[3]), s, 3);
  return c;
}

__device__ __forceinline__ uint32_t encode8(const float (&v)[8], float s) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return c;
}

// Eight codes -> eight bf16 (exact: two significant bits times a power of two).
__device__ __forceinline__ u32x4 decode8(uint32_t c, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
}

// acc += (A 2^sa) (B 2^sb) over 64 of the reduction: lane l holds 32 elements
// (16 bytes) of row / column l % 32 from position 32 (l / 32), its scale byte
// being byte `ia` / `ib` of sa / sb.
template <int ia, int ib>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x16 acc) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc, 4, 4, ia, (int)sa, ib, (int)sb);
}

// The same over 128 for 16 x 16 tiles: lane l holds row / column l % 16, block l / 16.
__device__ __forceinline__ f32x4 mfma16(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 acc) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 4, 0, (int)sa, 0, (int)sb);
}

}  // namespace mx4
