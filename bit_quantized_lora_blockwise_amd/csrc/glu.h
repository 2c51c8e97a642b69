// The gated activation H = silu(G) U and its gradients, in fp32.
#pragma once

#include "common.h"
#include "mx8.h"

namespace glu {

// 1 / (1 + e^-g), off by at most (|g| + 4) 2^-23 of itself: the exponent's product is rounded once, 2^-24 of
// |g| log2(e), which the exponential turns into as large a share; exp2 and the reciprocal add about one unit in
// the last place each.  H's rounding to bf16 does not see that before |g| is in the thousands.  For g below -88 the exponential is infinite and the result 0, as in the limit.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.442695041f * g));
}

__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

// dG = dH U sig (1 + G (1 - sig)), dU = dH G sig
__device__ __forceinline__ void back(float g, float u, float dh, float& dg, float& du) {
  const float s = sigmoid(g), gs = g * s;
  du = dh * gs;
  dg = dh * u * fmaf(gs, 1.0f - s, s);
}

constexpr uint32_t kOOB = 0x80000000u;     // a buffer offset past every range: the load returns 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// Elements c .. c + 7 of a row of `cols` bf16 that begins at byte `row`, in two halves: the load, which waits for
// nothing, and what fits it when it is used.  kVec: rows of whole 16-byte pieces.  Otherwise a piece that
// crosses the row's end is read as the row's last eight and moved; rows of fewer are read one by one.
template <bool kVec>
__device__ __forceinline__ u32x4 load8(__amdgpu_buffer_rsrc_t rs, uint32_t row, int c, int cols, bool on) {
  const bool in = on && c < cols;
  if constexpr (kVec) return __builtin_amdgcn_raw_buffer_load_b128(rs, in ? row + 2 * c : kOOB, 0, 0);
  if (cols >= 8) return __builtin_amdgcn_raw_buffer_load_b128(rs, in ? row + 2 * min(c, cols - 8) : kOOB, 0, 0);
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    e[j] = __builtin_amdgcn_raw_buffer_load_b16(rs, in && c + j < cols ? row + 2 * (c + j) : kOOB, 0, 0);
  return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}
template <bool kVec>
__device__ __forceinline__ u32x4 fit8(u32x4 v, int c, int cols) {
  if (kVec || cols < 8 || c + 8 <= cols || c >= cols) return v;
  return qk::drop_front8(v, c + 8 - cols);
}

// Eight fp32 as bf16, which they keep the rest of.
__device__ __forceinline__ u32x4 take_plane(float (&v)[8]) {
  u32x4 p;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    p[k] = qk::pack_bf16x2(v[2 * k], v[2 * k + 1]);
    v[2 * k] -= __uint_as_float(p[k] << 16);
    v[2 * k + 1] -= __uint_as_float(p[k] & 0xFFFF0000u);
  }
  return p;
}

// ---- what a gated product does with 32 rows of G and U ---------------------------------
// Lane (x, h) of a wave holds row m (x of 32) and, of 32 columns from c0 (a multiple of 32) on,
// columns 8 q + 4 h + e at accumulator 4 q + e.

// H = bf16(silu(G) U): the wave's halves exchange groups of four columns, so that a lane stores
// eight consecutive ones.
__device__ __forceinline__ void store_h(const f32x16& g, const f32x16& u, uint16_t* __restrict__ H, int64_t m, int64_t M,
                                        int64_t c0, int64_t F) {
  const int h = (threadIdx.x & 63) >> 5;
  u32x2 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      o[q][e] = qk::pack_bf16x2(silu(g[4 * q + 2 * e]) * u[4 * q + 2 * e], silu(g[4 * q + 2 * e + 1]) * u[4 * q + 2 * e + 1]);
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    const u32x2 s0 = __builtin_amdgcn_permlane32_swap(o[q][0], o[q + 1][0], false, false);
    const u32x2 s1 = __builtin_amdgcn_permlane32_swap(o[q][1], o[q + 1][1], false, false);
    const int64_t c = c0 + 8 * q + 8 * h;
    if (m < M && c < F) qk::store8_row(H + m * F + c, u32x4{s0[0], s1[0], s0[1], s1[1]}, (int)min((int64_t)8, F - c));
  }
}

// G or U in 8 bits: half the block's maximum is in the lane, and after two exchanges so are 16
// consecutive codes.  codes, scales: of the packed matrix's row 0 of this half.
__device__ __forceinline__ void store_8(f32x16 v, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t m,
                                        int64_t M, int64_t c0, int64_t F) {
  const int h = (threadIdx.x & 63) >> 5;
  const int64_t fp = mx8::padded(F);
  if (c0 + 32 > F) {                       // zeros past the end of the row
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = c0 + 8 * (e >> 2) + 4 * h + (e & 3) < F ? v[e] : 0.0f;
  }
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, mx8::mag(v[e]));
  const u32x2 both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
  const uint32_t sb = mx8::scale_byte(max(both[0], both[1]));
  const float inv = mx8::inverse(sb);
  uint32_t k[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) k[q] = mx8::encode4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3], inv);
  const u32x2 s01 = __builtin_amdgcn_permlane32_swap(k[0], k[1], false, false);
  const u32x2 s23 = __builtin_amdgcn_permlane32_swap(k[2], k[3], false, false);
  const u32x2 t0 = __builtin_amdgcn_permlane32_swap(s01[0], s23[0], false, false);
  const u32x2 t1 = __builtin_amdgcn_permlane32_swap(s01[1], s23[1], false, false);
  if (m < M) {
    *(u32x4*)(codes + m * fp + c0 + 16 * h) = u32x4{t0[0], t1[0], t0[1], t1[1]};
    if (h == 0) scales[m * (fp / 32) + (c0 >> 5)] = (uint8_t)sb;
  }
}

}  // namespace glu
