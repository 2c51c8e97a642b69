// Root-mean-square norm with the residual's addition, and its backward:
//   forward   S = rnd(X + R);  inv = 1 / sqrt(mean(S^2) + eps);  Y = bf16(S w inv), and
//             the same values in microscaled 8-bit (mx8.h) for the backward of what reads Y
//   backward  n = S inv, d = w dY:  dX = inv (d - n mean(n d)) + dS,  dw = sum over rows of n dY
// Bound: HBM, each matrix read or written once: a row stays in registers between the sum
// over it and the pass that uses the sum.  Sums and statistics are fp32 (a thread's at most
// 32 squares, then a tree), the root fp64: one of them a row.
//
// A row belongs to a wave (up to 2048 columns), to 256 threads (8192) or to 1024 (32768), up
// to four chunks of eight columns a thread.
#include <algorithm>

#include "kernels.h"
#include "mx8.h"

namespace {

// Eight values of a row as fp32, zeros past its end.
__device__ __forceinline__ void load8(const uint16_t* row, int c, int cols, float* v) {
  const u32x4 x = qk::load8_row(row, c, cols);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(x[j] << 16);
    v[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* row, int c, int cols, float* v) {
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

__device__ __forceinline__ u32x4 pack8(const float* v) {
  return u32x4{qk::pack_bf16x2(v[0], v[1]), qk::pack_bf16x2(v[2], v[3]), qk::pack_bf16x2(v[4], v[5]),
               qk::pack_bf16x2(v[6], v[7])};
}

__device__ __forceinline__ void store8(uint16_t* row, int c, int cols, const float* v) {
  qk::store8_row(row + c, pack8(v), min(8, cols - c));
}
__device__ __forceinline__ void store8(float* row, int c, int cols, const float* v) {
  if (c + 8 <= cols) {
    *(f32x4_a4*)(row + c) = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4_a4*)(row + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) row[c + j] = v[j];
  }
}

// Rounds to the type the values are stored in.
__device__ __forceinline__ void round8(const uint16_t*, float* v) {
  const u32x4 p = pack8(v);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(p[j] << 16);
    v[2 * j + 1] = __uint_as_float(p[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void round8(const float*, float*) {}

// Eight weights, fp32 or bf16.
__device__ __forceinline__ void weight8(const void* w, bool bf16, int c, int cols, float* v) {
  if (bf16) load8((const uint16_t*)w, c, cols, v);
  else load8((const float*)w, c, cols, v);
}

// The sum of v over the kRow threads of a row, in all of them.  slot: kRow / 64 floats (unused for a wave).
template <int kRow>
__device__ __forceinline__ float row_sum(float v, float* slot) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  if constexpr (kRow > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();                       // the slots' last readers are done
    if ((threadIdx.x & 63) == 0) slot[w] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int i = 1; i < kRow / 64; ++i) v += slot[i];
  }
  return v;
}

// 1 / sqrt(sum / cols + eps): once a row, in fp64, so that it is off by its rounding alone.
__device__ __forceinline__ float inverse_rms(float sum, int cols, float eps) {
  return (float)(1.0 / sqrt((double)sum / cols + (double)eps));
}

// kRow threads a row (four rows a work group of 256 if 64), kC chunks a thread.  S may be X or R
// (no __restrict__; a thread has read what it overwrites, and of other threads' columns uses none).
template <typename T, int kRow, int kC>
__global__ __launch_bounds__(kRow < 256 ? 256 : kRow) void k_norm_fwd(const T* X, const T* R, int64_t rows, int cols,
                                                                     const void* __restrict__ w, bool w_bf16, float eps,
                                                                     T* S, uint16_t* __restrict__ Y,
                                                                     uint8_t* __restrict__ codes,
                                                                     uint8_t* __restrict__ scales) {
  constexpr int kRows = kRow < 256 ? 256 / kRow : 1;
  __shared__ float slot[kRow / 64];
  const int t = threadIdx.x % kRow;
  // a row (four) a work group while the launch can count them; m is uniform over a row's threads
  for (int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow; m < rows; m += (int64_t)gridDim.x * kRows) {
    float v[kC][8], u[kC][8];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = u[i][j] = 0.0f;
      if (c < cols) {
        load8(X + m * cols, c, cols, v[i]);
        if (R) load8(R + m * cols, c, cols, u[i]);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      if (R && c < cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += u[i][j];
        round8(X, v[i]);                     // the norm is that of the sum as stored, which the backward reads
        store8(S + m * cols, c, cols, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    }
    const float inv = inverse_rms(row_sum<kRow>(sum, slot), cols, eps);
    const int pc = (int)mx8::padded(cols);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      if (c >= pc) break;
      float y[8];
      if (c < cols) weight8(w, w_bf16, c, cols, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = c + j < cols ? v[i][j] * y[j] * inv : 0.0f;   // bf16 times bf16 is exact
      if (Y && c < cols) store8(Y + m * cols, c, cols, y);
      if (codes) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, mx8::mag(y[j]));
        const uint32_t sb = mx8::scale_byte(mx8::max4(top));
        const float k = mx8::inverse(sb);
        *(u32x2*)(codes + m * pc + c) =
            u32x2{mx8::encode4(y[0], y[1], y[2], y[3], k), mx8::encode4(y[4], y[5], y[6], y[7], k)};
        if ((c & 31) == 0) scales[m * (pc / 32) + (c >> 5)] = (uint8_t)sb;
      }
    }
  }
}

// A work group takes rows blockIdx.x, + gridDim.x, .. and keeps its share of dw in registers; the
// shares, part[gridDim.x rows][cols], are added in order by k_norm_dw.  dX may be dS or S.
template <typename T, int kRow, int kC>
__global__ __launch_bounds__(kRow < 256 ? 256 : kRow) void k_norm_bwd(const uint16_t* __restrict__ dY, const T* S,
                                                                     const T* dS, int64_t rows, int cols,
                                                                     const void* __restrict__ w, bool w_bf16, float eps,
                                                                     T* dX, float* __restrict__ part) {
  constexpr int kRows = kRow < 256 ? 256 / kRow : 1;
  __shared__ float slot[2][kRow / 64];
  const int t = threadIdx.x % kRow;
  float dw[kC][8], k[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int c = 8 * (t + kRow * i);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = k[i][j] = 0.0f;
    if (c < cols) weight8(w, w_bf16, c, cols, k[i]);
  }
  const int64_t first = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow;
  for (int64_t m = first; m < rows; m += (int64_t)gridDim.x * kRows) {
    float s[kC][8], d[kC][8], g[kC][8];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = d[i][j] = g[i][j] = 0.0f;
      if (c < cols) {
        load8(S + m * cols, c, cols, s[i]);
        load8(dY + m * cols, c, cols, d[i]);
        if (dS) load8(dS + m * cols, c, cols, g[i]);
      }
    }
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(s[i][j], s[i][j], sum);
        dot = fmaf(s[i][j] * k[i][j], d[i][j], dot);
      }
    const float inv = inverse_rms(row_sum<kRow>(sum, slot[0]), cols, eps);
    const float mean = (float)((double)row_sum<kRow>(dot, slot[1]) * inv / cols);   // of n d
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = s[i][j] * inv;
        dw[i][j] = fmaf(n, d[i][j], dw[i][j]);
        g[i][j] = fmaf(inv, k[i][j] * d[i][j] - n * mean, g[i][j]);
      }
      if (dX && c < cols) store8(dX + m * cols, c, cols, g[i]);
    }
  }
  if (!part) return;
  if constexpr (kRows > 1) {               // the waves' shares, added in order
    __shared__ float share[kRows][64 * 8 * kC];
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) share[threadIdx.x / kRow][8 * (t + kRow * i) + j] = dw[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += 256) {
      float u = share[0][c];
#pragma unroll
      for (int i = 1; i < kRows; ++i) u += share[i][c];
      part[(int64_t)blockIdx.x * cols + c] = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      if (c < cols) store8(part + (int64_t)blockIdx.x * cols, c, cols, dw[i]);
    }
  }
}

// dw[c] = the shares' sum: 64 columns a work group, sixteen waves of them a sixteenth of the shares each.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* __restrict__ part, int shares, int cols,
                                                  float* __restrict__ dw) {
  __shared__ float sum[16][64];
  const int c = 64 * (int)blockIdx.x + (threadIdx.x & 63), w = threadIdx.x >> 6;
  float u = 0.0f;
  if (c < cols) {
    const int per = (shares + 15) / 16, end = min(shares, per * (w + 1));
    int i = per * w;
    for (; i + 4 <= end; i += 4) {
      const float a = part[(int64_t)i * cols + c], b = part[(int64_t)(i + 1) * cols + c];
      const float d = part[(int64_t)(i + 2) * cols + c], e = part[(int64_t)(i + 3) * cols + c];
      u += (a + b) + (d + e);
    }
    for (; i < end; ++i) u += part[(int64_t)i * cols + c];
  }
  sum[w][threadIdx.x & 63] = u;
  __syncthreads();
  if (w == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) u += sum[i][threadIdx.x];
    dw[c] = u;
  }
}

int64_t shares_of(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 2048 ? 4 : 1;
  return std::min<int64_t>((rows + per - 1) / per, 512);
}

template <typename T>
hipError_t fwd(const T* X, const T* R, int64_t rows, int cols, const void* w, bool w_bf16, float eps, T* S, uint16_t* Y,
               uint8_t* codes, uint8_t* scales, hipStream_t s) {
#define QL_NORM(R_, C_)                                                                                             \
  hipLaunchKernelGGL((k_norm_fwd<T, R_, C_>), dim3((unsigned)std::min<int64_t>(R_ == 64 ? (rows + 3) / 4 : rows, 1 << 20)),  \
                     dim3(R_ < 256 ? 256 : R_), 0, s, X, R, rows, cols, w, w_bf16, eps, S, Y, codes, scales)
  if (cols <= 512) QL_NORM(64, 1);
  else if (cols <= 1024) QL_NORM(64, 2);
  else if (cols <= 2048) QL_NORM(64, 4);
  else if (cols <= 4096) QL_NORM(256, 2);
  else if (cols <= 8192) QL_NORM(256, 4);
  else if (cols <= 16384) QL_NORM(1024, 2);
  else QL_NORM(1024, 4);
#undef QL_NORM
  return hipGetLastError();
}

template <typename T>
hipError_t bwd(const uint16_t* dY, const T* S, const T* dS, int64_t rows, int cols, const void* w, bool w_bf16, float eps,
               T* dX, float* dw, float* ws, hipStream_t s) {
  const int shares = (int)shares_of(rows, cols);
  float* part = dw ? ws : nullptr;
#define QL_NORM(R_, C_)                                                                                            \
  hipLaunchKernelGGL((k_norm_bwd<T, R_, C_>), dim3((unsigned)shares), dim3(R_ < 256 ? 256 : R_), 0, s, dY, S, dS,  \
                     rows, cols, w, w_bf16, eps, dX, part)
  if (cols <= 512) QL_NORM(64, 1);
  else if (cols <= 1024) QL_NORM(64, 2);
  else if (cols <= 2048) QL_NORM(64, 4);
  else if (cols <= 4096) QL_NORM(256, 2);
  else if (cols <= 8192) QL_NORM(256, 4);
  else if (cols <= 16384) QL_NORM(1024, 2);
  else QL_NORM(1024, 4);
#undef QL_NORM
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dw) return e;
  hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, s, ws, shares, cols, dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const void* X, const void* R, bool bf16, int64_t rows, int64_t cols, const void* w, bool w_bf16,
                           float eps, void* S, uint16_t* Y, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  if (bf16)
    return fwd((const uint16_t*)X, (const uint16_t*)R, rows, (int)cols, w, w_bf16, eps, (uint16_t*)S, Y, codes, scales, s);
  return fwd((const float*)X, (const float*)R, rows, (int)cols, w, w_bf16, eps, (float*)S, Y, codes, scales, s);
}

size_t norm_bwd_ws(int64_t rows, int64_t cols) { return (size_t)shares_of(rows, cols) * cols * sizeof(float); }

hipError_t launch_norm_bwd(const uint16_t* dY, const void* S, const void* dS, bool bf16, int64_t rows, int64_t cols,
                           const void* w, bool w_bf16, float eps, void* dX, float* dw, float* ws, hipStream_t s) {
  if (bf16)
    return bwd(dY, (const uint16_t*)S, (const uint16_t*)dS, rows, (int)cols, w, w_bf16, eps, (uint16_t*)dX, dw, ws, s);
  return bwd(dY, (const float*)S, (const float*)dS, rows, (int)cols, w, w_bf16, eps, (float*)dX, dw, ws, s);
}
