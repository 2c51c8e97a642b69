// Quantisation to microscaled 4-bit (layout and rule: mx4.h) along the rows or the
// columns of a matrix, and back.  Memory-bound: 2 (bf16) or 4 (fp32) bytes read
// and 17/32 byte written per element.
#include "mx4.h"

#include "kernels.h"

namespace {

using namespace mx4;

constexpr int kThreads = 256;

// Largest of the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad_perm [1,0,3,2]
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true)); // quad_perm [2,3,0,1]
}

// Or over the 16 lanes of a DPP row of values that are equal within quads.
__device__ __forceinline__ uint32_t row_or(uint32_t v) {
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, true);   // row_ror:4
  return v | (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true);   // row_ror:8
}

// Along the rows: 16 lanes take 128 elements of a row (a quad one block, a lane
// eight elements), a wave four rows at a time and kRows / 4 such groups with all
// their loads in flight: 256 contiguous bytes read per row, 64 written per block
// position and group.  Rows past the end repeat the last one and are not written.
// 22016 x 8192 bf16 78 us (5.9 TB/s; a large copy moves 5.1), 4096 x 11007 21 us,
// 512 x 1000 2.5 us.
constexpr int kRows = 16;

// kShort: rows of fewer than eight elements.
template <bool kBf16, bool kShort, bool kPast>
__global__ __launch_bounds__(kThreads) void k_mx4_quant(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                        int64_t ld, int64_t words, uint32_t* __restrict__ codes,
                                                        uint32_t* __restrict__ scales) {
  const int l = threadIdx.x & 63, part = l & 15, rl = l >> 4;
  const int64_t tiles = (rows + kRows - 1) / kRows * words;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 64);
  for (int64_t tile = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); tile < tiles; tile += stride) {
    const int64_t rt = tile / words, w = tile - rt * words;      // row tile, 128-element piece
    const int64_t col = 128 * w + 8 * part;
    u32x4 v[kRows / 4];
    f32x4 f[kRows / 4][2];
    // every load on its way before the first is used: a piece that crosses the row's end is
    // read as the row's last eight and moved afterwards
    const int64_t at = min(col, cols - 8);
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      const int64_t row = min(kRows * rt + 4 * i + rl, rows - 1);
      if constexpr (kBf16) {
        const uint16_t* p = (const uint16_t*)X + row * ld;
        if constexpr (kShort) v[i] = qk::load8_row(p, col, cols);
        else v[i] = qk::load_past<kPast>((const u32x4_a2*)(p + at));
      } else {
        const float* p = (const float*)X + row * ld;
        if constexpr (kShort) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[i][j >> 2][j & 3] = col + j < cols ? p[col + j] : 0.0f;
        } else {
          f[i][0] = qk::load_past<kPast>((const f32x4_a4*)(p + at));
          f[i][1] = qk::load_past<kPast>((const f32x4_a4*)(p + at + 4));
        }
      }
    }
    if (!kShort && 128 * (w + 1) > cols) {                       // uniform
      const int s = (int)min((int64_t)8, col - at);
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        if constexpr (kBf16) v[i] = qk::drop_front8(v[i], s);
        else qk::drop_front8(f[i][0], f[i][1], s);
      }
    }
    // packed before any is stored: a load's wait would wait for the stores before it
    uint32_t c[kRows / 4], word[kRows / 4];
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      uint32_t top = 0;
      if constexpr (kBf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max((v[i][j] << 16) & 0x7FFFFFFFu, v[i][j] & 0x7FFF0000u));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[i][j >> 2][j & 3]) & 0x7FFFFFFFu);
      }
      const uint32_t sb = scale_byte(quad_max(top));
      if constexpr (kBf16) c[i] = encode8(v[i], scale_f32(sb));
      else {
        const float e[8] = {f[i][0][0], f[i][0][1], f[i][0][2], f[i][0][3], f[i][1][0], f[i][1][1], f[i][1][2], f[i][1][3]};
        c[i] = encode8(e, scale_f32(sb));
      }
      if (sb == 255u) c[i] = 0;
      word[i] = row_or(sb << (8 * (part >> 2)));
    }
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      const int64_t row = kRows * rt + 4 * i + rl;
      if (row < rows) {
        codes[((4 * w + (part >> 2)) * rows + row) * 4 + (part & 3)] = c[i];
        if (part == 0) scales[w * rows + row] = word[i];
      }
    }
  }
}

// Along the columns: the packed rows are the columns of X [len, cols].  A work
// group takes 128 columns and 128 rows, wave w its rows 32 w .. +31 (one block of
// each column), a lane two columns: no exchange between lanes, 256 contiguous
// bytes read per row (bf16), 32 written per lane.  The four waves' scale bytes
// meet in LDS.  22016 x 8192 bf16 77 us (5.9 TB/s), 4096 x 11007 26 us.
// kOne: cols == 1.
template <bool kBf16, bool kOne, bool kPast>
__global__ __launch_bounds__(kThreads) void k_mx4_quant_t(const void* __restrict__ X, int64_t len, int64_t cols,
                                                          int64_t ld, u32x4* __restrict__ codes,
                                                          uint32_t* __restrict__ scales) {
  __shared__ uint8_t sbytes[128][4];
  const int l = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t ctiles = (cols + 127) / 128, wg = blockIdx.x + (int64_t)gridDim.x * blockIdx.y;
  const int64_t ct = wg % ctiles, word = wg / ctiles;
  if (word >= (len + 127) / 128) return;
  const int64_t c0 = 128 * ct + 2 * l, r0 = 128 * word + 32 * wv;
  typedef uint32_t u32_a2 __attribute__((aligned(2)));
  typedef float f32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
  // rows past the end repeat the last one, columns past it the last pair; cleared below
  const int64_t at = cols > 1 ? min(c0, cols - 2) : 0;
  float x[2][32];
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const int64_t o = min(r0 + k, len - 1) * ld + at;
    if constexpr (kBf16) {
      const uint16_t* p = (const uint16_t*)X + o;
      const uint32_t d = kOne ? *p : qk::load_past<kPast>((const u32_a2*)p);
      x[0][k] = __uint_as_float(d << 16);
      x[1][k] = __uint_as_float(d & 0xFFFF0000u);
    } else {
      const float* p = (const float*)X + o;
      const f32x2_a4 y = kOne ? f32x2_a4{*p, 0.0f} : qk::load_past<kPast>((const f32x2_a4*)p);
      x[0][k] = y[0];
      x[1][k] = y[1];
    }
  }
  if (128 * (ct + 1) > cols || r0 + 32 > len) {                  // uniform
    const bool second = !kOne && c0 == cols - 1;                 // its pair was read one column early
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const bool in = r0 + k < len && c0 < cols;
      x[0][k] = in ? (second ? x[1][k] : x[0][k]) : 0.0f;
      x[1][k] = in && c0 + 1 < cols ? x[1][k] : 0.0f;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) top = max(top, __float_as_uint(x[c][k]) & 0x7FFFFFFFu);
    const uint32_t sb = scale_byte(top);
    const float s = scale_f32(sb);
    u32x4 o;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float e[8] = {x[c][8 * g], x[c][8 * g + 1], x[c][8 * g + 2], x[c][8 * g + 3],
                          x[c][8 * g + 4], x[c][8 * g + 5], x[c][8 * g + 6], x[c][8 * g + 7]};
      o[g] = sb == 255u ? 0u : encode8(e, s);
    }
    if (c0 + c < cols) codes[(4 * word + wv) * cols + c0 + c] = o;
    sbytes[2 * l + c][wv] = (uint8_t)sb;
  }
  __syncthreads();
  if (threadIdx.x < 128 && 128 * ct + threadIdx.x < cols)
    scales[word * cols + 128 * ct + threadIdx.x] = *(const uint32_t*)sbytes[threadIdx.x];
}

// Packed -> bf16 [rows, cols], the lanes as in k_mx4_quant.  22016 x 8192 70 to 87 us
// (5.2 to 6.5 TB/s), 4096 x 11007 32 us.
template <bool kPast>
__global__ __launch_bounds__(kThreads) void k_mx4_dequant(const uint32_t* __restrict__ codes,
                                                          const uint32_t* __restrict__ scales, int64_t rows,
                                                          int64_t cols, int64_t words, uint16_t* __restrict__ out) {
  const int l = threadIdx.x & 63, part = l & 15, rl = l >> 4;
  const int64_t tiles = (rows + kRows - 1) / kRows * words;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 64);
  for (int64_t tile = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); tile < tiles; tile += stride) {
    const int64_t rt = tile / words, w = tile - rt * words;
    const int64_t col = 128 * w + 8 * part;
    uint32_t c[kRows / 4], sw[kRows / 4];
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      const int64_t row = min(kRows * rt + 4 * i + rl, rows - 1);
      c[i] = codes[((4 * w + (part >> 2)) * rows + row) * 4 + (part & 3)];
      sw[i] = scales[w * rows + row];
    }
    u32x4 v[kRows / 4];
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      const uint32_t sb = (sw[i] >> (8 * (part >> 2))) & 255u;
      v[i] = decode8(c[i], scale_f32(sb));
      if (sb == 255u) v[i] = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    }
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      const int64_t row = kRows * rt + 4 * i + rl;
      if (row < rows && col < cols) qk::store8_row<kPast>(out + row * cols + col, v[i], (int)min((int64_t)8, cols - col));
    }
  }
}

unsigned tile_grid(int64_t rows, int64_t words) {
  const int64_t tiles = (rows + kRows - 1) / kRows * words;
  const int64_t g = (tiles + kThreads / 64 - 1) / (kThreads / 64);
  return (unsigned)(g > 65536 ? 65536 : g);
}

}  // namespace

hipError_t launch_mx4_quant(const void* X, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                            uint8_t* scales, hipStream_t s) {
  const int64_t words = padded(cols) / kPad;
  const bool past = rows * cols * (bf16 ? 2 : 4) > qk::kStreamBytes;
#define QL_MQ(B, S, P)                                                                                            \
  hipLaunchKernelGGL((k_mx4_quant<B, S, P>), dim3(tile_grid(rows, words)), dim3(kThreads), 0, s, X, rows, cols, ld, \
                     words, (uint32_t*)codes, (uint32_t*)scales)
  if (bf16) {
    if (cols < 8) QL_MQ(true, true, false);
    else if (past) QL_MQ(true, false, true);
    else QL_MQ(true, false, false);
  } else {
    if (cols < 8) QL_MQ(false, true, false);
    else if (past) QL_MQ(false, false, true);
    else QL_MQ(false, false, false);
  }
#undef QL_MQ
  return hipGetLastError();
}

hipError_t launch_mx4_quant_t(const void* X, bool bf16, int64_t len, int64_t cols, int64_t ld, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
  // a launch has fewer than 2^32 threads along x
  const int64_t groups = (cols + 127) / 128 * (padded(len) / kPad), gx = groups < (1 << 22) ? groups : 1 << 22;
  const dim3 grid((unsigned)gx, (unsigned)((groups + gx - 1) / gx));
  const bool past = len * cols * (bf16 ? 2 : 4) > qk::kStreamBytes;
#define QL_MQ(B, O, P)                                                                                           \
  hipLaunchKernelGGL((k_mx4_quant_t<B, O, P>), grid, dim3(kThreads), 0, s, X, len, cols, ld, (u32x4*)codes,      \
                     (uint32_t*)scales)
  if (bf16) {
    if (cols == 1) QL_MQ(true, true, false);
    else if (past) QL_MQ(true, false, true);
    else QL_MQ(true, false, false);
  } else {
    if (cols == 1) QL_MQ(false, true, false);
    else if (past) QL_MQ(false, false, true);
    else QL_MQ(false, false, false);
  }
#undef QL_MQ
  return hipGetLastError();
}

hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* out,
                              hipStream_t s) {
  const int64_t words = padded(cols) / kPad;
  const bool past = rows * cols * 2 > qk::kStreamBytes;
  hipLaunchKernelGGL((past ? k_mx4_dequant<true> : k_mx4_dequant<false>), dim3(tile_grid(rows, words)), dim3(kThreads), 0, s,
                     (const uint32_t*)codes, (const uint32_t*)scales, rows, cols, words, out);
  return hipGetLastError();
}
