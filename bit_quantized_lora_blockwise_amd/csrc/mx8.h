// Microscaled 8-bit matrices (OCP Microscaling Formats v1.0, MXFP8 with E4M3 elements): one
// E8M0 scale, a power of two, for each 32 consecutive elements of a row.  The form that
// activations are kept in for the backward.
//
// Packed form of a matrix of R rows of L elements, L padded with zeros to Lp = 32 ceil(L / 32):
//   codes  [R][Lp]       one byte an element;
//   scales [R][Lp / 32]  one byte a block.
// Row-major, so that a pass that reads a bf16 matrix by rows or a tile at a time reads this
// one with the same indices, and every row begins at a multiple of 32 bytes.
#pragma once

#include "common.h"

namespace mx8 {

constexpr int kBlock = 32;

__host__ __device__ inline int64_t padded(int64_t len) { return (len + kBlock - 1) / kBlock * kBlock; }
inline int64_t code_bytes(int64_t rows, int64_t len) { return padded(len) * rows; }
inline int64_t scale_bytes(int64_t rows, int64_t len) { return padded(len) / kBlock * rows; }

// Scale byte of a block whose largest magnitude has the fp32 bits `top`: the least exponent
// e with max <= 448 2^e (E4M3 ends at 448 = 1.75 2^8), so that nothing saturates; the sum
// carries into the exponent where the mantissa is past 1.75.  (The format's own
// floor(log2 max) - 8 puts maxima in (448, 512) 2^e, which lose up to an eighth.)  At least
// -117, so that the smallest element, 2^-9 of the scale, is a normal bf16.  255 marks a
// block with an infinity or NaN: all its values are NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t e = (top + 0x1FFFFFu) >> 23;
  return top >= 0x7F800000u ? 255u : (e > 18u ? e - 8u : 10u);
}

// 2^(127 - byte), by which elements are multiplied before they are rounded (0 for 255: codes 0).
__device__ __forceinline__ float inverse(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float scale_f32(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte ? byte << 23 : 0x00400000u);
}

// Largest magnitude bits of values; a NaN's are the largest of all.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// max over aligned groups of 4 lanes
__device__ __forceinline__ uint32_t max4(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad_perm [1,0,3,2]
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad_perm [2,3,0,1]
}

// Four values to four codes, nearest with ties to even.  In a block with an infinity or NaN (inv
// = 0) they are 0: that product would be NaN there.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return inv == 0.0f ? 0u : (uint32_t)w;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Four codes to their values over the scale.
__device__ __forceinline__ void decode4(uint32_t w, float s, float* v) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0] * s;
  v[1] = lo[1] * s;
  v[2] = hi[0] * s;
  v[3] = hi[1] * s;
}

}  // namespace mx8
