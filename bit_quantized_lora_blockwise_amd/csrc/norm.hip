// Root-mean-square norm with the residual's addition, and its backward:
//   forward   S = rnd(X + R);  inv = 1 / sqrt(mean(S^2) + eps);  Y = bf16(S w inv), and
//             the same values in microscaled 8-bit (mx8.h) for the backward of what reads Y
//   backward  n = S inv, d = w dY:  dX = inv (d - n mean(n d)) + dS,  dw = sum over rows of n dY
// Bound up to 8192 columns: HBM, each matrix read or written once: a row stays in registers
// between the sum over it and the pass that uses the sum.  Sums and statistics are fp32 (a thread's at most
// 32 squares, then a tree), the root fp64: one of them a row.
//
// bf16: 2048 x 8192 with the residual and 8-bit copies 30 us, 5.0 TB/s; backward 4096 x 4096 with dS
// 26.5 us, 5.1 TB/s, and 4 us for dw.
//
// Past 8192 columns the 1024 threads of a row have 128 registers each.  The backward keeps two rows,
// the weights and dw, and spills: 13 registers with two chunks of bf16 (42 if cols % 8), 41 (123) of
// fp32, 183 (355) and 263 (708) with four; the forward 32 and 75 with four chunks if cols % 8.  Bound by
// those there: 4096 rows, bf16 / fp32, us (a copy's time for the same bytes): backward 8192 columns 50 / 96
// (52 / 91), 12288 107 / 310 (78 / 136), 16384 138 / 363 (103 / 181), 16390 867 / 1923, 22016 676 / 1245
// (139 / 243); forward with residual and 8-bit copy 8192 53 / 93, 16384 118 / 184, 22016 169 / 254, 22018
// 253 / 489.
//
// A row belongs to a wave (up to 1024 columns) or to 256, 512 or 1024 threads, one or two
// chunks of eight columns a thread (four past 16384 columns).  Rows are read through a
// descriptor of their own, so that no load stands behind a branch.
#include <algorithm>

#include "kernels.h"
#include "mx8.h"

namespace {

constexpr uint32_t kOOB = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// Eight values of a row of `cols` as they lie in memory, from column c on.  kVec: cols % 8 == 0.  Otherwise a chunk
// that crosses the end is read as the row's last eight and moved when it is used; rows of fewer are read one by one.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 v;
};
template <>
struct Raw<float> {
  f32x4 v[2];
};

template <bool kVec>
__device__ __forceinline__ void load8(Raw<uint16_t>& r, __amdgpu_buffer_rsrc_t rs, int c, int cols) {
  if (kVec || cols >= 8) {
    r.v = __builtin_amdgcn_raw_buffer_load_b128(rs, c < cols ? 2u * (kVec ? c : min(c, cols - 8)) : kOOB, 0, 0);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_raw_buffer_load_b16(rs, c + j < cols ? 2u * (c + j) : kOOB, 0, 0);
    r.v = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
  }
}
template <bool kVec>
__device__ __forceinline__ void load8(Raw<float>& r, __amdgpu_buffer_rsrc_t rs, int c, int cols) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (kVec || cols >= 8) {
      const uint32_t at = c < cols ? 4u * (kVec ? c : min(c, cols - 8)) + 16u * h : kOOB;
      r.v[h] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = c + 4 * h + j;
        r.v[h][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, k < cols ? 4u * k : kOOB, 0, 0));
      }
    }
  }
}

template <bool kVec>
__device__ __forceinline__ void values8(const Raw<uint16_t>& r, int c, int cols, float* v) {
  u32x4 x = r.v;
  if (!kVec && cols >= 8 && c + 8 > cols && c < cols) x = qk::drop_front8(x, c + 8 - cols);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(x[j] << 16);
    v[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
  }
}
template <bool kVec>
__device__ __forceinline__ void values8(const Raw<float>& r, int c, int cols, float* v) {
  f32x4 a = r.v[0], b = r.v[1];
  if (!kVec && cols >= 8 && c + 8 > cols && c < cols) qk::drop_front8(a, b, c + 8 - cols);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}

__device__ __forceinline__ u32x4 pack8(const float* v) {
  return u32x4{qk::pack_bf16x2(v[0], v[1]), qk::pack_bf16x2(v[2], v[3]), qk::pack_bf16x2(v[4], v[5]),
               qk::pack_bf16x2(v[6], v[7])};
}

template <bool kVec>
__device__ __forceinline__ void store8(uint16_t* row, int c, int cols, const float* v) {
  if constexpr (kVec) *(u32x4*)(row + c) = pack8(v);
  else qk::store8_row(row + c, pack8(v), min(8, cols - c));
}
template <bool kVec>
__device__ __forceinline__ void store8(float* row, int c, int cols, const float* v) {
  if (kVec || c + 8 <= cols) {
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

// Sums of two values over the kRow threads of a row, in all of them.  slot: two floats for each of the row's waves, not
// those of the call before: its readers need not be done (one barrier a call).
template <int kRow>
__device__ __forceinline__ void row_sums(float& a, float& b, f32x4* slot) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (kRow > 64) {
    float* s = (float*)slot;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      s[2 * w] = a;
      s[2 * w + 1] = b;
    }
    __syncthreads();
    a = s[0];
    b = s[1];
#pragma unroll
    for (int i = 1; i < kRow / 64; ++i) {
      a += s[2 * i];
      b += s[2 * i + 1];
    }
  }
}

// 1 / sqrt(sum / cols + eps): once a row, in fp64, so that it is off by its rounding alone.
__device__ __forceinline__ float inverse_rms(float sum, double per, float eps) {
  return (float)rsqrt((double)sum * per + (double)eps);
}

struct Norm {
  int64_t rows;
  int cols;
  const void* w;
  bool w_bf16;
  float eps;
};

// A weight's chunk, fp32 or bf16.
struct Weight {
  Raw<float> f;
  Raw<uint16_t> h;
};
template <bool kVec>
__device__ __forceinline__ void load_w(Weight& r, const Norm& n, int c) {
  if (n.w_bf16) load8<kVec>(r.h, rsrc(n.w, 2 * (uint64_t)n.cols), c, n.cols);
  else load8<kVec>(r.f, rsrc(n.w, 4 * (uint64_t)n.cols), c, n.cols);
}
template <bool kVec>
__device__ __forceinline__ void values_w(const Weight& r, const Norm& n, int c, float* v) {
  if (n.w_bf16) values8<kVec>(r.h, c, n.cols, v);
  else values8<kVec>(r.f, c, n.cols, v);
}

template <int kRow>
constexpr int threads() { return kRow < 256 ? 256 : kRow; }

// kRow threads a row (four rows a work group of 256 if 64), kC chunks a thread.  S may be X or R
// (no __restrict__; a thread has read what it overwrites, and of other threads' columns uses none).
template <typename T, int kRow, int kC, bool kVec>
__global__ __launch_bounds__(threads<kRow>()) void k_norm_fwd(const T* X, const T* R, Norm n, T* S,
                                                             uint16_t* __restrict__ Y, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  constexpr int kRows = threads<kRow>() / kRow;
  __shared__ f32x4 slot[2][kRow / 64];
  const int t = threadIdx.x % kRow, cols = n.cols;
  const double per = 1.0 / cols;
  Weight w[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) load_w<kVec>(w[i], n, 8 * (t + kRow * i));
  // a row (four) a work group while the launch can count them; m is uniform over a row's threads
  int turn = 0;
  const int64_t first = (int64_t)blockIdx.x * kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / kRow);
  for (int64_t m = first; m < n.rows; m += (int64_t)gridDim.x * kRows, turn ^= 1) {
    Raw<T> x[kC], u[kC];
    const __amdgpu_buffer_rsrc_t rx = rsrc(X + m * cols, sizeof(T) * (uint64_t)cols),
                                 rr = rsrc(R ? R + m * cols : X, R ? sizeof(T) * (uint64_t)cols : 0);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      load8<kVec>(x[i], rx, 8 * (t + kRow * i), cols);
      load8<kVec>(u[i], rr, 8 * (t + kRow * i), cols);     // zeros without R
    }
    float v[kC][8];
    float sum = 0.0f, none = 0.0f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      values8<kVec>(x[i], c, cols, v[i]);
      if (R) {
        float a[8];
        values8<kVec>(u[i], c, cols, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += a[j];
        round8(X, v[i]);                   // the norm is that of the sum as stored, which the backward reads
        if (c < cols) store8<kVec>(S + m * cols, c, cols, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    }
    row_sums<kRow>(sum, none, slot[turn]);
    const float inv = inverse_rms(sum, per, n.eps);
    const int pc = (int)mx8::padded(cols);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      if (c >= pc) break;
      float y[8];
      values_w<kVec>(w[i], n, c, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[i][j] * y[j] * inv;      // bf16 times bf16 is exact; zeros past the end
      if (Y && c < cols) store8<kVec>(Y + m * cols, c, cols, y);
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

// A work group takes rows blockIdx.x, + gridDim.x, .., the next one's in flight while it finishes
// one, and keeps its share of dw in registers; the shares, part[gridDim.x][cols], are added
// in order by k_norm_dw.  dX may be dS or S.
template <typename T, int kRow, int kC, bool kVec>
__global__ __launch_bounds__(threads<kRow>()) void k_norm_bwd(const uint16_t* __restrict__ dY, const T* S, const T* dS,
                                                             Norm n, T* dX, float* __restrict__ part) {
  constexpr int kRows = threads<kRow>() / kRow;
  __shared__ f32x4 slot[2][kRow / 64];
  const int t = threadIdx.x % kRow, cols = n.cols;
  const double per = 1.0 / cols;
  float dw[kC][8] = {};
  Weight w[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) load_w<kVec>(w[i], n, 8 * (t + kRow * i));
  struct Row {
    Raw<T> s[kC], g[kC];
    Raw<uint16_t> d[kC];
  };
  auto load = [&](int64_t m) {
    Row q;
    const bool in = m < n.rows;            // past the last row: descriptors of no bytes
    const uint64_t len = in ? (uint64_t)cols : 0;
    const __amdgpu_buffer_rsrc_t rs = rsrc(in ? S + m * cols : S, sizeof(T) * len), rd = rsrc(in ? dY + m * cols : dY, 2 * len),
                                 rg = rsrc(in && dS ? dS + m * cols : S, dS ? sizeof(T) * len : 0);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      load8<kVec>(q.s[i], rs, c, cols);
      load8<kVec>(q.d[i], rd, c, cols);
      load8<kVec>(q.g[i], rg, c, cols);    // zeros without dS
    }
    return q;
  };
  int turn = 0;
  int64_t m = (int64_t)blockIdx.x * kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / kRow);
  Row cur = load(m);
  for (; m < n.rows; m += (int64_t)gridDim.x * kRows, turn ^= 1) {
    const Row nxt = load(m + (int64_t)gridDim.x * kRows);
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      float s[8], d[8], k[8];
      values8<kVec>(cur.s[i], c, cols, s);
      values8<kVec>(cur.d[i], c, cols, d);
      values_w<kVec>(w[i], n, c, k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(s[j], s[j], sum);
        dot = fmaf(s[j] * k[j], d[j], dot);
      }
    }
    row_sums<kRow>(sum, dot, slot[turn]);
    const float inv = inverse_rms(sum, per, n.eps);
    const float mean = (float)((double)dot * inv * per);   // of n d
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = 8 * (t + kRow * i);
      float s[8], d[8], k[8], g[8];
      values8<kVec>(cur.s[i], c, cols, s);
      values8<kVec>(cur.d[i], c, cols, d);
      values_w<kVec>(w[i], n, c, k);
      values8<kVec>(cur.g[i], c, cols, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float nj = s[j] * inv;
        dw[i][j] = fmaf(nj, d[j], dw[i][j]);
        g[j] = fmaf(inv, k[j] * d[j] - nj * mean, g[j]);
      }
      if (dX && c < cols) store8<kVec>(dX + m * cols, c, cols, g);
    }
    cur = nxt;
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
      if (c < cols) store8<kVec>(part + (int64_t)blockIdx.x * cols, c, cols, dw[i]);
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
    for (; i + 8 <= end; i += 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = part[(int64_t)(i + k) * cols + c];
      u += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
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
  const int64_t per = cols <= 1024 ? 4 : 1;
  return std::min<int64_t>((rows + per - 1) / per, 512);
}

// Calls f with the threads of a row and the chunks of a thread: two chunks before more threads, so
// that more rows share a CU.  4096 rows of bf16 with the residual, us, so / with one chunk and twice
// the threads: 8192 columns forward 47 / 59, backward 54 / 56; 4096 columns 23 / 22, 29.0 / 29.3; 1024
// columns 12.6 / 12.5, 17.8 / 17.7.
template <typename F>
void by_columns(int64_t cols, F f) {
  if (cols <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (cols <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (cols <= 2048) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  else if (cols <= 4096) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else if (cols <= 8192) f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  else if (cols <= 16384) f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

template <typename T>
hipError_t fwd(const T* X, const T* R, const Norm& n, T* S, uint16_t* Y, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  by_columns(n.cols, [&](auto row, auto chunks) {
    constexpr int kRow = decltype(row)::value, kC = decltype(chunks)::value, kRows = threads<kRow>() / kRow;
    const dim3 grid((unsigned)std::min<int64_t>((n.rows + kRows - 1) / kRows, 1 << 20));
    if (n.cols % 8 == 0)
      hipLaunchKernelGGL((k_norm_fwd<T, kRow, kC, true>), grid, dim3(threads<kRow>()), 0, s, X, R, n, S, Y, codes, scales);
    else
      hipLaunchKernelGGL((k_norm_fwd<T, kRow, kC, false>), grid, dim3(threads<kRow>()), 0, s, X, R, n, S, Y, codes, scales);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t bwd(const uint16_t* dY, const T* S, const T* dS, const Norm& n, T* dX, float* dw, float* ws, hipStream_t s) {
  const int shares = (int)shares_of(n.rows, n.cols);
  float* part = dw ? ws : nullptr;
  by_columns(n.cols, [&](auto row, auto chunks) {
    constexpr int kRow = decltype(row)::value, kC = decltype(chunks)::value;
    const dim3 grid((unsigned)shares);
    if (n.cols % 8 == 0)
      hipLaunchKernelGGL((k_norm_bwd<T, kRow, kC, true>), grid, dim3(threads<kRow>()), 0, s, dY, S, dS, n, dX, part);
    else
      hipLaunchKernelGGL((k_norm_bwd<T, kRow, kC, false>), grid, dim3(threads<kRow>()), 0, s, dY, S, dS, n, dX, part);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dw) return e;
  hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)((n.cols + 63) / 64)), dim3(1024), 0, s, ws, shares, n.cols, dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const void* X, const void* R, bool bf16, int64_t rows, int64_t cols, const void* w, bool w_bf16,
                           float eps, void* S, uint16_t* Y, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const Norm n{rows, (int)cols, w, w_bf16, eps};
  if (bf16) return fwd((const uint16_t*)X, (const uint16_t*)R, n, (uint16_t*)S, Y, codes, scales, s);
  return fwd((const float*)X, (const float*)R, n, (float*)S, Y, codes, scales, s);
}

size_t norm_bwd_ws(int64_t rows, int64_t cols) { return (size_t)shares_of(rows, cols) * cols * sizeof(float); }

hipError_t launch_norm_bwd(const uint16_t* dY, const void* S, const void* dS, bool bf16, int64_t rows, int64_t cols,
                           const void* w, bool w_bf16, float eps, void* dX, float* dw, float* ws, hipStream_t s) {
  const Norm n{rows, (int)cols, w, w_bf16, eps};
  if (bf16) return bwd(dY, (const uint16_t*)S, (const uint16_t*)dS, n, (uint16_t*)dX, dw, ws, s);
  return bwd(dY, (const float*)S, (const float*)dS, n, (float*)dX, dw, ws, s);
}
