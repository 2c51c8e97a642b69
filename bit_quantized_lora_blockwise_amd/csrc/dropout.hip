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

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_dropout(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                      int64_t ld, drop::Params d, void* __restrict__ Y) {
  const int64_t octs = (cols + 7) / 8;
  const int64_t total = rows * octs, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
    const int64_t m = i / octs, q = i - m * octs;
    const int n = (int)min((int64_t)8, cols - 8 * q);
    u32x4 u = {};
    if constexpr (kBf16) {
      const uint16_t* src = (const uint16_t*)X + m * ld;
      u32x4 v;
      if (n == 8) v = *(const u32x4_a2*)(src + 8 * q);
      else v = qk::load8_row(src, 8 * q, cols);
      if (d.cut) {
        u = drop::draw8(d, (uint32_t)m, (uint32_t)q);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] &= drop::keep2(u[j], d.cut);
          v[j] = qk::pack_bf16x2(__uint_as_float(v[j] << 16) * d.scale, __uint_as_float(v[j] & 0xFFFF0000u) * d.scale);
        }
      }
      qk::store8_row((uint16_t*)Y + m * cols + 8 * q, v, n);
    } else {
      const float* src = (const float*)X + m * ld + 8 * q;
      float* dst = (float*)Y + m * cols + 8 * q;
      float v[8];
      if (n == 8) {
        *(f32x4*)v = *(const f32x4_a4*)src;
        *(f32x4*)(v + 4) = *(const f32x4_a4*)(src + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? src[j] : 0.0f;
      }
      if (d.cut) {
        u = drop::draw8(d, (uint32_t)m, (uint32_t)q);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ((u[j >> 1] >> (16 * (j & 1))) & 0xFFFFu) >= d.cut ? v[j] * d.scale : 0.0f;
      }
      if (n == 8) {
        *(f32x4_a4*)dst = *(f32x4*)v;
        *(f32x4_a4*)(dst + 4) = *(f32x4*)(v + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) dst[j] = v[j];
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
  if (bf16)
    hipLaunchKernelGGL(k_dropout<true>, dim3((unsigned)grid), dim3(kThreads), 0, s, X, rows, cols, ld, d, Y);
  else
    hipLaunchKernelGGL(k_dropout<false>, dim3((unsigned)grid), dim3(kThreads), 0, s, X, rows, cols, ld, d, Y);
  return hipGetLastError();
}
