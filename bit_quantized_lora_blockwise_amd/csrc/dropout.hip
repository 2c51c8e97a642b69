// Elementwise dropout, Y = D o X with D the mask of philox.h: kept elements times
// 65536 / (65536 - cut), dropped ones 0 whatever they hold.  D o is its own
// transpose, so the same call is the backward.
//
// One thread takes the eight elements of a row that share a draw.  Bound: HBM for
// large bf16 matrices; the draws' quarter-rate products cost about the same time
// as the traffic of a bf16 element (4 bytes), and overlap with it.
#include "philox.h"

#include "kernels.h"

namespace {

constexpr int kThreads = 256;

// kVec: rows of whole 16-byte pieces (cols % 8 == 0, both rows' starts aligned).
template <bool kBf16, bool kVec>
__global__ __launch_bounds__(kThreads) void k_dropout(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                      int64_t ld, drop::Params d, void* __restrict__ Y) {
  const int64_t octs = (cols + 7) / 8;
  const int64_t total = rows * octs, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
    const int64_t m = i / octs, q = i - m * octs;
    u32x4 u = {};
    if (d.cut) u = drop::draw8(d, (uint32_t)m, (uint32_t)q);
    const int64_t src = m * ld + 8 * q, dst = m * cols + 8 * q;
    const int n = (int)min((int64_t)8, cols - 8 * q);
    if constexpr (kBf16) {
      u32x4 v = {};
      if constexpr (kVec) {
        v = *(const u32x4*)((const uint16_t*)X + src);
      } else {
        for (int j = 0; j < n; ++j) v[j >> 1] |= (uint32_t)((const uint16_t*)X)[src + j] << (16 * (j & 1));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (d.cut) {
          v[j] &= drop::keep2(u[j], d.cut);
          v[j] = qk::pack_bf16x2(__uint_as_float(v[j] << 16) * d.scale, __uint_as_float(v[j] & 0xFFFF0000u) * d.scale);
        }
      }
      if constexpr (kVec) {
        *(u32x4*)((uint16_t*)Y + dst) = v;
      } else {
        for (int j = 0; j < n; ++j) ((uint16_t*)Y)[dst + j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
      }
    } else {
      float v[8];
      if constexpr (kVec) {
        *(f32x4*)v = *(const f32x4*)((const float*)X + src);
        *(f32x4*)(v + 4) = *(const f32x4*)((const float*)X + src + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? ((const float*)X)[src + j] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (d.cut) v[j] = ((u[j >> 1] >> (16 * (j & 1))) & 0xFFFFu) >= d.cut ? v[j] * d.scale : 0.0f;
      if constexpr (kVec) {
        *(f32x4*)((float*)Y + dst) = *(f32x4*)v;
        *(f32x4*)((float*)Y + dst + 4) = *(f32x4*)(v + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) ((float*)Y)[dst + j] = v[j];
      }
    }
  }
}

}  // namespace

hipError_t launch_dropout(const void* X, bool bf16, int64_t rows, int64_t cols, int64_t ld, const drop::Params& d,
                          void* Y, hipStream_t s) {
  const int64_t octs = rows * ((cols + 7) / 8);
  int64_t grid = (octs + kThreads - 1) / kThreads;
  if (grid > 8192) grid = 8192;
  const bool vec = (cols % 8) == 0 && (ld % 8) == 0;
#define QL_DROP(B, V) \
  hipLaunchKernelGGL((k_dropout<B, V>), dim3((unsigned)grid), dim3(kThreads), 0, s, X, rows, cols, ld, d, Y)
  if (bf16) {
    if (vec) QL_DROP(true, true);
    else QL_DROP(true, false);
  } else {
    if (vec) QL_DROP(false, true);
    else QL_DROP(false, false);
  }
#undef QL_DROP
  return hipGetLastError();
}
