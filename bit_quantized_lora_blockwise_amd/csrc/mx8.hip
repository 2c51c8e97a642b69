// mx8_quantize and mx8_dequantize: activations to microscaled 8-bit and back (layout and
// rounding: mx8.h).  Bound: HBM, one read and one write of each element.  A thread takes
// eight elements of a row, four lanes a block: the block's largest magnitude is two
// register exchanges away.  4096 x 11008 bf16: packing 28 us (137 MB, 4.9 TB/s), unpacking 21.
#include "kernels.h"
#include "mx8.h"

namespace {

constexpr int kT = 256;

// Eight values of a row as fp32, zeros past its end.
__device__ __forceinline__ void load8(const uint16_t* row, int64_t c, int64_t cols, float* v) {
  const u32x4 x = qk::load8_row(row, c, cols);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(x[j] << 16);
    v[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* row, int64_t c, int64_t cols, float* v) {
  if (c + 8 <= cols) {
    const f32x4 a = *(const f32x4_a4*)(row + c), b = *(const f32x4_a4*)(row + c + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? row[c + j] : 0.0f;
  }
}

// A work group is `1 << lg` threads along the rows by kT >> lg rows.
template <typename T>
__global__ __launch_bounds__(kT) void k_mx8_quant(const T* __restrict__ X, int64_t rows, int64_t cols, int64_t ld,
                                                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int lg) {
  const int64_t pc = mx8::padded(cols);
  const int64_t c = 8 * (((int64_t)blockIdx.x << lg) + (threadIdx.x & ((1 << lg) - 1)));
  if (c >= pc) return;                               // whole blocks: pc is a multiple of 32
  for (int64_t m = (int64_t)blockIdx.y * (kT >> lg) + (threadIdx.x >> lg); m < rows; m += (int64_t)gridDim.y * (kT >> lg)) {
    float v[8];
    if (c < cols) load8(X + m * ld, c, cols, v);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, mx8::mag(v[j]));
    const uint32_t sb = mx8::scale_byte(mx8::max4(top));
    const float inv = mx8::inverse(sb);
    *(u32x2*)(codes + m * pc + c) =
        u32x2{mx8::encode4(v[0], v[1], v[2], v[3], inv), mx8::encode4(v[4], v[5], v[6], v[7], inv)};
    if ((c & 31) == 0) scales[m * (pc / 32) + (c >> 5)] = (uint8_t)sb;
  }
}

__global__ __launch_bounds__(kT) void k_mx8_dequant(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                    int64_t rows, int64_t cols, uint16_t* __restrict__ out, int lg) {
  const int64_t pc = mx8::padded(cols);
  const int64_t c = 8 * (((int64_t)blockIdx.x << lg) + (threadIdx.x & ((1 << lg) - 1)));
  if (c >= cols) return;
  for (int64_t m = (int64_t)blockIdx.y * (kT >> lg) + (threadIdx.x >> lg); m < rows; m += (int64_t)gridDim.y * (kT >> lg)) {
    const u32x2 w = *(const u32x2*)(codes + m * pc + c);
    const float s = mx8::scale_f32(scales[m * (pc / 32) + (c >> 5)]);
    float v[8];
    mx8::decode4(w[0], s, v);
    mx8::decode4(w[1], s, v + 4);
    const u32x4 o = {qk::pack_bf16x2(v[0], v[1]), qk::pack_bf16x2(v[2], v[3]), qk::pack_bf16x2(v[4], v[5]),
                     qk::pack_bf16x2(v[6], v[7])};
    qk::store8_row(out + m * cols + c, o, (int)min((int64_t)8, cols - c));
  }
}

// Threads along a row: the power of two that covers it, 4 (a block) to kT.
dim3 grid_of(int64_t rows, int64_t cols, int* lg) {
  const int64_t n = mx8::padded(cols) / 8;
  *lg = 2;
  while ((1 << *lg) < n && (1 << *lg) < kT) ++*lg;
  const int64_t per = kT >> *lg, y = (rows + per - 1) / per;
  return dim3((unsigned)((n + (1 << *lg) - 1) >> *lg), (unsigned)(y < 65535 ? y : 65535));
}

}  // namespace

hipError_t launch_mx8_quant(const void* X, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                            uint8_t* scales, hipStream_t s) {
  int lg;
  const dim3 grid = grid_of(rows, cols, &lg);
  if (bf16)
    hipLaunchKernelGGL(k_mx8_quant<uint16_t>, grid, dim3(kT), 0, s, (const uint16_t*)X, rows, cols, ld, codes, scales, lg);
  else
    hipLaunchKernelGGL(k_mx8_quant<float>, grid, dim3(kT), 0, s, (const float*)X, rows, cols, ld, codes, scales, lg);
  return hipGetLastError();
}

hipError_t launch_mx8_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* out,
                              hipStream_t s) {
  int lg;
  const dim3 grid = grid_of(rows, cols, &lg);
  hipLaunchKernelGGL(k_mx8_dequant, grid, dim3(kT), 0, s, codes, scales, rows, cols, out, lg);
  return hipGetLastError();
}
