// Products of two microscaled 4-bit matrices (layout: mx4.h) on the scaled matrix
// instruction, with the adapter term in the same tile:
//   C[m][p] = bf16(sum_b 2^(ea + eb) sum_{32} a b + adapter[m][p]),  A [M, R], B [P, R]
//   forward   adapter = s (T L2)         T [M, r], L2 [r, P]
//   backward  adapter = D o (G L1^T)     G [M, r], L1 [P, r]
// fp32 accumulators throughout, one rounding at the end.
#include "mx4.h"

#include "kernels.h"

namespace {

using namespace mx4;

constexpr int kThreads = 256;
constexpr int kBM = 128, kBP = 128;
constexpr int kPL = 64 + 8;       // pitch of [row][c] adapter tiles
constexpr int kPD = kBP + 8;      // pitch of the [c][p] tile

__device__ __forceinline__ u32x4 load_row8(const uint16_t* __restrict__ row, int64_t col, int64_t ncols) {
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t h = (col + j < ncols) ? row[col + j] : 0;
    v[j >> 1] |= h << (16 * (j & 1));
  }
  return v;
}

// kMode: 0 no adapter, 1 forward, 2 backward, 3 backward with dropout.
template <int kMode>
__global__ __launch_bounds__(kThreads) void k_mx4_gemm(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                       int64_t M, const uint8_t* __restrict__ bc,
                                                       const uint8_t* __restrict__ bs, int64_t P, int64_t words,
                                                       Mx4Lora lo, uint16_t* __restrict__ C) {
  __shared__ __attribute__((aligned(16))) uint16_t la[kBM * kPL];
  __shared__ __attribute__((aligned(16))) uint16_t lb[kBP * kPL > 64 * kPD ? kBP * kPL : 64 * kPD];
  __shared__ __attribute__((aligned(16))) uint8_t mask[kMode == 3 ? kBM * drop::bit_pitch(kBP) : 16];
  const int t = threadIdx.x, w = t >> 6, l = t & 63;
  const int wm = w & 1, wp = w >> 1, h = l >> 5;
  const int64_t m0 = (int64_t)blockIdx.y * kBM, p0 = (int64_t)blockIdx.x * kBP;
  f32x16 acc[2][2] = {};
  if constexpr (kMode != 0) {
    const int r = lo.r;
    for (int i = t; i < kBM * 8; i += kThreads) {
      const int row = i >> 3, c = (i & 7) * 8;
      u32x4 v = {0, 0, 0, 0};
      if (m0 + row < M) v = load_row8(lo.A + (m0 + row) * r, c, r);
      *(LDS_AS u32x4*)((LDS_AS uint16_t*)la + row * kPL + c) = v;
    }
    if constexpr (kMode == 1) {
      for (int i = t; i < 64 * (kBP / 8); i += kThreads) {
        const int c = i / (kBP / 8), p = (i % (kBP / 8)) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (c < r) v = load_row8(lo.B + c * P, p0 + p, P);
        *(LDS_AS u32x4*)((LDS_AS uint16_t*)lb + c * kPD + p) = v;
      }
    } else {
      for (int i = t; i < kBP * 8; i += kThreads) {
        const int row = i >> 3, c = (i & 7) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (p0 + row < P) v = load_row8(lo.B + (p0 + row) * r, c, r);
        *(LDS_AS u32x4*)((LDS_AS uint16_t*)lb + row * kPL + c) = v;
      }
    }
    if constexpr (kMode == 3) drop::fill_bits<kBM, kBP>((LDS_AS uint8_t*)mask, lo.d, m0, p0, t, kThreads);
    __syncthreads();
    for (int s = 0; s < (r + 15) / 16; ++s) {
      bf16x8 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = qk::frag_rowmajor((const LDS_AS uint16_t*)la, kPL, 64 * wm + 32 * i, 16 * s);
        b[i] = kMode == 1 ? qk::frag_kmajor((const LDS_AS uint16_t*)lb, kPD, 16 * s, 64 * wp + 32 * i)
                          : qk::frag_rowmajor((const LDS_AS uint16_t*)lb, kPL, 64 * wp + 32 * i, 16 * s);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = qk::mfma32(a[i], b[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if constexpr (kMode == 1) acc[i][j][e] *= lo.scale;
          if constexpr (kMode == 3)
            acc[i][j][e] = drop::kept<kBP>((const LDS_AS uint8_t*)mask, 64 * wm + 32 * i + qk::acc_row(e),
                                           64 * wp + 32 * j + qk::acc_col())
                               ? lo.d.scale * acc[i][j][e]
                               : 0.0f;
        }
  }
  // rows past the end repeat the last one: their results are not stored
  int64_t ra[2], rb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ra[i] = min(m0 + 64 * wm + 32 * i + (l & 31), M - 1);
    rb[i] = min(p0 + 64 * wp + 32 * i + (l & 31), P - 1);
  }
  for (int64_t q = 0; q < words; ++q) {
    // step s of the word: lane half h takes block 2 h + s of both operands
    u32x4 a[2][2], b[2][2];
    uint32_t sa[2], sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sa[i] = *(const uint32_t*)(as + (q * M + ra[i]) * 4) >> (16 * h);
      sb[i] = *(const uint32_t*)(bs + (q * P + rb[i]) * 4) >> (16 * h);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        a[i][s] = *(const u32x4*)(ac + ((4 * q + 2 * h + s) * M + ra[i]) * 16);
        b[i][s] = *(const u32x4*)(bc + ((4 * q + 2 * h + s) * P + rb[i]) * 16);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[i][j] = mx4::mfma32<0, 0>(a[i][0], sa[i], b[j][0], sb[j], acc[i][j]);
        acc[i][j] = mx4::mfma32<1, 1>(a[i][1], sa[i], b[j][1], sb[j], acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t p = p0 + 64 * wp + 32 * j + qk::acc_col();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t m = m0 + 64 * wm + 32 * i + qk::acc_row(e);
        if (m < M && p < P) C[m * P + p] = qk::f32_to_bf16(acc[i][j][e]);
      }
    }
}

}  // namespace

hipError_t launch_mx4_gemm(const uint8_t* ac, const uint8_t* as, int64_t M, const uint8_t* bc, const uint8_t* bs,
                           int64_t P, int64_t R, const Mx4Lora& lora, uint16_t* C, hipStream_t s) {
  const dim3 grid((unsigned)((P + kBP - 1) / kBP), (unsigned)((M + kBM - 1) / kBM));
  const int64_t words = padded(R) / kPad;
#define QL_MX(MODE) \
  hipLaunchKernelGGL(k_mx4_gemm<MODE>, grid, dim3(kThreads), 0, s, ac, as, M, bc, bs, P, words, lora, C)
  if (!lora.A) QL_MX(0);
  else if (!lora.bwd) QL_MX(1);
  else if (lora.d.cut == 0) QL_MX(2);
  else QL_MX(3);
#undef QL_MX
  return hipGetLastError();
}
