// Elementwise dropout, Y = D o X with D the mask of philox.h: kept elements times
// 65536 / (65536 - cut), dropped ones 0 whatever they hold.  D o is its own
// transpose, so the same call is the backward.
//
// In place (Y = X): a thread stores only elements that it alone uses.  The piece at a
// row's end is read with elements of the piece before it, which are shifted out.
//
// One thread takes the eight elements of a row that share a draw.  Bound: HBM for
// large bf16 matrices; the draws' quarter-rate products cost about the same time
// as the traffic of a bf16 element (4 bytes), and overlap with it: a thread's next
// piece is on its way while one is drawn.  4096 x 11008 bf16 33 us (5.5 TB/s; 43 us
// with one piece at a time and a division for each), 4096 x 11007 36 us, 2048 x 8192
// fp32 28 us.
#include "philox.h"

#include "kernels.h"

namespace {

constexpr int kThreads = 256;

// kWhole: cols % 8 == 0, no piece crosses a row's end.
template <bool kBf16, bool kWhole, bool kPast>
__global__ __launch_bounds__(kThreads) void k_dropout(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                      int64_t ld, drop::Params d, void* __restrict__ Y) {
  const int64_t octs = (cols + 7) / 8, stride = (int64_t)gridDim.x * kThreads;
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  // row and octet of the thread's pieces, `stride` apart: one division, then steps
  const int64_t step_m = stride / octs, step_q = stride - step_m * octs;
  int64_t m = first / octs, q = first - m * octs;
  struct Piece {
    u32x4 v[kBf16 ? 1 : 2];
  };
  auto load = [&](int64_t m, int64_t q) {
    Piece x = {};
    if constexpr (kBf16) {
      const uint16_t* src = (const uint16_t*)X + m * ld;
      if (kWhole || 8 * q + 8 <= cols) x.v[0] = qk::load_past<kPast>((const u32x4_a2*)(src + 8 * q));
      else x.v[0] = qk::load8_row(src, 8 * q, cols);
    } else {
      const float* src = (const float*)X + m * ld + 8 * q;
      if (kWhole || 8 * q + 8 <= cols) {
        x.v[0] = __builtin_bit_cast(u32x4, qk::load_past<kPast>((const f32x4_a4*)src));
        x.v[1] = __builtin_bit_cast(u32x4, qk::load_past<kPast>((const f32x4_a4*)(src + 4)));
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j) x.v[j >> 2][j & 3] = 8 * q + j < cols ? __float_as_uint(src[j]) : 0u;
      }
    }
    return x;
  };
  if (m >= rows) return;
  Piece next = load(m, q);
  while (m < rows) {
    Piece x = next;
    int64_t m1 = m + step_m, q1 = q + step_q;
    if (q1 >= octs) {
      q1 -= octs;
      ++m1;
    }
    if (m1 < rows) next = load(m1, q1);              // on its way while this piece is drawn
    const int n = kWhole ? 8 : (int)min((int64_t)8, cols - 8 * q);
    if (d.cut) {
      const u32x4 u = drop::draw8(d, (uint32_t)m, (uint32_t)q);
      if constexpr (kBf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t y = x.v[0][j] & drop::keep2(u[j], d.cut);
          x.v[0][j] = qk::pack_bf16x2(__uint_as_float(y << 16) * d.scale, __uint_as_float(y & 0xFFFF0000u) * d.scale);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool keep = ((u[j >> 1] >> (16 * (j & 1))) & 0xFFFFu) >= d.cut;
          x.v[j >> 2][j & 3] = keep ? __float_as_uint(__uint_as_float(x.v[j >> 2][j & 3]) * d.scale) : 0u;
        }
      }
    }
    if constexpr (kBf16) {
      qk::store8_row<kPast>((uint16_t*)Y + m * cols + 8 * q, x.v[0], n);
    } else {
      float* dst = (float*)Y + m * cols + 8 * q;
      if (n == 8) {
        if constexpr (kPast) {
          __builtin_nontemporal_store(__builtin_bit_cast(f32x4, x.v[0]), (f32x4_a4*)dst);
          __builtin_nontemporal_store(__builtin_bit_cast(f32x4, x.v[1]), (f32x4_a4*)(dst + 4));
        } else {
          *(f32x4_a4*)dst = __builtin_bit_cast(f32x4, x.v[0]);
          *(f32x4_a4*)(dst + 4) = __builtin_bit_cast(f32x4, x.v[1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < n) dst[j] = __uint_as_float(x.v[j >> 2][j & 3]);
      }
    }
    m = m1;
    q = q1;
  }
}

}  // namespace

hipError_t launch_dropout(const void* X, bool bf16, int64_t rows, int64_t cols, int64_t ld, const drop::Params& d,
                          void* Y, hipStream_t s) {
  const int64_t octs = rows * ((cols + 7) / 8);
  int64_t grid = (octs + kThreads - 1) / kThreads;
  if (grid > 8192) grid = 8192;
  const bool whole = cols % 8 == 0;
  const bool past = rows * cols * (bf16 ? 2 : 4) > qk::kStreamBytes;
#define QL_DROP(B, W, P) \
  hipLaunchKernelGGL((k_dropout<B, W, P>), dim3((unsigned)grid), dim3(kThreads), 0, s, X, rows, cols, ld, d, Y)
#define QL_DROP_W(B, P)           \
  do {                            \
    if (whole) QL_DROP(B, true, P); \
    else QL_DROP(B, false, P);    \
  } while (0)
  if (bf16) {
    if (past) QL_DROP_W(true, true);
    else QL_DROP_W(true, false);
  } else {
    if (past) QL_DROP_W(false, true);
    else QL_DROP_W(false, false);
  }
#undef QL_DROP_W
#undef QL_DROP
  return hipGetLastError();
}
