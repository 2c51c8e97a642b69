// Dropout mask of an adapter's input from a counter-based generator: element
// (m, k) is kept when the 16-bit number drawn for it is at least `cut`.  Nothing
// of the mask is stored: forward and backward draw the same numbers again.
//
// Generator: Philox4x32 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011) with seven rounds, the fewest for which
// the paper reports that it passes BigCrush.  Counter (k / 8, m, offset low,
// offset high), key (seed low, seed high); element k takes half k % 2 (low half
// first) of output word (k % 8) / 2, so one call decides the eight elements that
// a 16-byte load of bf16 brings.  32-bit products run at a quarter of the VALU
// rate, which makes the seven rounds about 340 cycles a wave (12 us for the 45 M
// elements of 4096 x 11008 on the whole chip); 16 bits a decision rather than 32 halve
// that, and leave p a step of 2^-16.
#pragma once

#include "common.h"

namespace drop {

// cut = 0: nothing is dropped and nothing is drawn.
struct Params {
  uint32_t k0, k1;      // key
  uint32_t o0, o1;      // offset
  uint32_t cut;         // round(65536 p), below 65536
  float scale;          // 65536 / (65536 - cut)
};

// A call in flight: counter words and the key of the next round.
struct State {
  uint32_t c0, c1, c2, c3, k0, k1;
};

__device__ __forceinline__ State begin(const Params& d, uint32_t m, uint32_t q) {
  return State{q, m, d.o0, d.o1, d.k0, d.k1};
}

// In one instruction (the compiler makes two of a ^ b ^ c).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);
}

__device__ __forceinline__ void round(State& s) {
  const uint64_t a = (uint64_t)s.c0 * 0xD2511F53u, b = (uint64_t)s.c2 * 0xCD9E8D57u;
  s.c0 = xor3((uint32_t)(b >> 32), s.c1, s.k0);
  s.c2 = xor3((uint32_t)(a >> 32), s.c3, s.k1);
  s.c1 = (uint32_t)b;
  s.c3 = (uint32_t)a;
  s.k0 += 0x9E3779B9u;
  s.k1 += 0xBB67AE85u;
}

// The numbers of elements (m, 8 q) .. (m, 8 q + 7).
__device__ __forceinline__ u32x4 draw8(const Params& d, uint32_t m, uint32_t q) {
  State s = begin(d, m, q);
#pragma unroll
  for (int n = 0; n < 7; ++n) round(s);
  return u32x4{s.c0, s.c1, s.c2, s.c3};
}

// 0xFFFF in each half of a word whose number keeps its element, else 0.
__device__ __forceinline__ uint32_t keep2(uint32_t u, uint32_t cut) {
  return ((u & 0xFFFFu) >= cut ? 0xFFFFu : 0u) | (u >= (cut << 16) ? 0xFFFF0000u : 0u);
}

// Eight bf16 of row m from column 8 q with the dropped ones zeroed (not scaled).
__device__ __forceinline__ u32x4 mask8(u32x4 v, const Params& d, uint32_t m, uint32_t q) {
  const u32x4 u = draw8(d, m, q);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] &= keep2(u[j], d.cut);
  return v;
}

// Eight numbers' decisions as bits 0 .. 7.
__device__ __forceinline__ uint32_t bits8_of(u32x4 u, uint32_t cut) {
  uint32_t b = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    b |= ((u[j] & 0xFFFFu) >= cut ? 1u << (2 * j) : 0u) | (u[j] >= (cut << 16) ? 2u << (2 * j) : 0u);
  return b;
}

__device__ __forceinline__ uint32_t bits8(const Params& d, uint32_t m, uint32_t q) {
  return bits8_of(draw8(d, m, q), d.cut);
}

// A tile's decisions in LDS, a bit an element: row i at byte i * bit_pitch(cols),
// column c in bit c % 8 of byte c / 8.  One word of padding a row keeps rows that
// lanes read together on different banks.
__host__ __device__ constexpr int bit_pitch(int cols) { return cols / 8 + 4; }

// Decisions of elements (m0 + i, k0 + c) of a kRows x kCols tile (k0 % 8 == 0), by
// threads t of n.
template <int kRows, int kCols>
__device__ __forceinline__ void fill_bits(LDS_AS uint8_t* lds, const Params& d, int64_t m0, int64_t k0, int t, int n) {
  for (int i = t; i < kRows * (kCols / 8); i += n) {
    const int row = i / (kCols / 8), q = i % (kCols / 8);
    lds[row * bit_pitch(kCols) + q] = (uint8_t)bits8(d, (uint32_t)(m0 + row), (uint32_t)(k0 >> 3) + q);
  }
}

template <int kCols>
__device__ __forceinline__ bool kept(const LDS_AS uint8_t* lds, int row, int col) {
  return (lds[row * bit_pitch(kCols) + (col >> 3)] >> (col & 7)) & 1;
}

}  // namespace drop
