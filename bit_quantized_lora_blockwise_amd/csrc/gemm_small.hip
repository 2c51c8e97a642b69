// The NF4 layer with dropout for few rows.  dX:
//   dX = bf16(dY W' + D o (G L1^T))       (transposed-weight path)
// Work group: 32 rows of dY, 64 columns of dX (one first-level block wide); eight waves
// split the reduction over W's stored rows, 32 rows at a time.  A wave rebuilds its 32 x 64
// piece of W' as bf16 in LDS of its own (no barrier in the loop) and reads it
// transposed as the matrix operand; the waves' sums meet in LDS in order.  32 rows of
// 512 x 512 with rank 8 take 6 us, nearly all of it latency.  The 256 x 256
// tiles of gemm_big.hip leave most CUs idle at such sizes and walk the whole reduction in
// one work group.
#include "dequant.h"
#include "glu.h"
#include "kernels.h"

namespace {

using namespace nf4;

constexpr int kW = 8;                  // waves
constexpr int kN = 32;                 // rows of W of a wave's step
constexpr int kP = 64;                 // columns of dX
constexpr int kPitch = kP + 8;         // LDS row of W' (elements)
constexpr uint32_t kOOB = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// Eight bf16 from byte offset `at`, element j present if j < n.
template <bool kVec>
__device__ __forceinline__ bf16x8 load8(__amdgpu_buffer_rsrc_t rs, uint32_t at, int n) {
  if (kVec) return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rs, n > 0 ? at : kOOB, 0, 0));
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_raw_buffer_load_b16(rs, j < n ? at + 2 * j : kOOB, 0, 0);
  return __builtin_bit_cast(bf16x8, u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16});
}

// Elements c .. c + 7 of row m of T or G from its S <= kSlices fp32 slices [M][r], `next` elements apart, added in order.
constexpr int kSlices = kSmallSlices;
__device__ __forceinline__ void sum8(__amdgpu_buffer_rsrc_t rp, int S, int M, int r, int m, int c, int next, float (&sum)[8]) {
  const uint32_t at = 4u * (uint32_t)(m * r + c);
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    u32x4 v[kSlices];                    // slices past the last read as zeros
#pragma unroll
    for (int n = 0; n < kSlices; ++n)
      v[n] = __builtin_amdgcn_raw_buffer_load_b128(rp, n < S && m < M && c < r ? at + 4u * k : kOOB, 4 * n * next, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float u = __uint_as_float(v[0][j]);
#pragma unroll
      for (int n = 1; n < kSlices; ++n) u += __uint_as_float(v[n][j]);
      sum[k + j] = c + k + j < r ? u : 0.0f;
    }
  }
}

// kVec: rows of dY in whole 16-byte pieces, zeros from N to ldy; kVecR: r % 8 == 0; kSum: G as slices.  kGlu: W's
// rows in two halves, each with a G (two planes [M][r]; slices [S][2][M][r], planes [2][3][M][..]) and an L1 [K][r] of
// its own, and no dropout; kTwo: rows of dY hold two matrices of ldy / 2 columns whose sum it is.  Both are the
// gated product's; decided at run time they cost the other layers' backwards 0.7 to 2 us of 14 to 60.
template <bool kVec, bool kVecR, bool kSum, bool kGlu, bool kTwo>
__global__ __launch_bounds__(64 * kW) void k_dx_small(const uint16_t* __restrict__ dY, int M, int K, int N,
                                                      const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ c2, const float* __restrict__ c1,
                                                      const uint16_t* __restrict__ G, const float* __restrict__ Gp, int S,
                                                      uint16_t* __restrict__ planes, const uint16_t* __restrict__ L1,
                                                      int r, uint16_t* __restrict__ dX, Nf4Params q, drop::Params d,
                                                      int ldy) {
  constexpr int halves = kGlu ? 2 : 1;
  if constexpr (!kGlu) ldy = N;
  __shared__ __attribute__((aligned(16))) uint16_t wt[kW][kN * kPitch];
  __shared__ f32x16 red[kW][2][64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, h = l >> 5, x = l & 31;
  const int p0 = kP * (int)blockIdx.x, m0 = 32 * (int)blockIdx.y, m = m0 + x;
  const int kb = K / 64;
  const __amdgpu_buffer_rsrc_t ry = rsrc(dY, (uint64_t)M * ldy * 2), rc = rsrc(codes, (uint64_t)N * (K / 2)),
                               r2 = rsrc(c2, (uint64_t)N * kb), r1 = rsrc(c1, 4 * (((uint64_t)N * kb + 255) / 256));
  const SplitConst kc = split_const();
  LDS_AS uint16_t* const tile = (LDS_AS uint16_t*)wt[w];

  // lane (x, h): row n0 + x of W, columns 32 h .. +31 of the block; rows past N read as zeros, and so does dY there
  struct Step {
    u32x4 c;
    uint32_t s2;
    float s1;
    bf16x8 y[2];
  };
  // the second term's steps follow the first's, from a whole round of the waves on
  const int next = (N + kN * kW - 1) / (kN * kW) * (kN * kW), end = kTwo ? next + N : N;
  auto load = [&](int n0) {
    Step s;
    int col0 = 0;
    if (kTwo && n0 >= next) {
      col0 = ldy / 2;
      n0 -= next;
    }
    const int n = n0 + x;
    const uint32_t b = (uint32_t)n * kb + blockIdx.x;
    s.c = __builtin_amdgcn_raw_buffer_load_b128(rc, n < N ? (uint32_t)n * (K / 2) + 32 * blockIdx.x + 16 * h : kOOB, 0, 0);
    s.s2 = __builtin_amdgcn_raw_buffer_load_b8(r2, n < N ? b : kOOB, 0, 0);
    s.s1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r1, n < N ? 4 * (b >> 8) : kOOB, 0, 0));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = n0 + 16 * u + 8 * h;
      s.y[u] = load8<kVec>(ry, (uint32_t)(m * ldy + col0 + k) * 2u, m < M ? N - k : 0);
    }
    return s;
  };
  f32x16 acc[2] = {};
  Step cur = load(kN * w);
  for (int n0 = kN * w; n0 < end; n0 += kN * kW) {
    const Step nxt = load(n0 + kN * kW);
    const BlockLut lut = make_lut(qk::e4m3fn_to_f32(cur.s2) * cur.s1, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) *(LDS_AS u32x4*)(tile + x * kPitch + 32 * h + 8 * i) = dequant8(lut, cur.c[i], kc);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[j] = qk::mfma32(qk::frag_kmajor(tile, kPitch, 16 * u, 32 * j), cur.y[u], acc[j]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    cur = nxt;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) red[w][j][l] = acc[j];
  // waves 0 and 1 finish 32 columns each
  f32x16 low = {};
  uint32_t keep = 0;
  const int p = p0 + 32 * w;
  if (w < 2) {
    // L1 from this wave's first column on: all of it may pass 2^31 bytes
    const int64_t first = __builtin_amdgcn_readfirstlane(p);
    const int pitch = (r + 7) / 8 * 8;
    const int64_t plane = (int64_t)M * pitch;
    for (int half = 0; half < halves; ++half) {
    const __amdgpu_buffer_rsrc_t rg = kSum ? rsrc(Gp + (int64_t)half * M * r, (uint64_t)M * r * 4 * (S * halves - half))
                                           : rsrc(G + (int64_t)half * halves * M * r, (uint64_t)M * r * 2 * halves),
                                 rl = rsrc(L1 + ((int64_t)half * K + first) * r, (uint64_t)32 * r * 2);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = 16 * s + 8 * h;
      if (16 * s >= r) break;                      // uniform
      const bf16x8 a = load8<kVecR>(rl, (uint32_t)(x * r + c) * 2u, r - c);
      bf16x8 b, rest;                              // two halves: 16 bits of G
      if constexpr (kSum) {
        float sum[8];
        sum8(rg, S, M, r, m, c, halves * M * r, sum);
        u32x4 v[3];                                // the planes: each what those before it rounded off
#pragma unroll
        for (int n = 0; n < 3; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[n][k] = qk::pack_bf16x2(sum[2 * k], sum[2 * k + 1]);
            sum[2 * k] -= __uint_as_float(v[n][k] << 16);
            sum[2 * k + 1] -= __uint_as_float(v[n][k] & 0xFFFF0000u);
          }
        b = __builtin_bit_cast(bf16x8, v[0]);
        rest = __builtin_bit_cast(bf16x8, v[1]);
        if (blockIdx.x == 0 && w == 0 && m < M && c < pitch)
#pragma unroll
          for (int n = 0; n < 3; ++n) *(u32x4*)(planes + (3 * half + n) * plane + (int64_t)m * pitch + c) = v[n];
      } else {
        b = load8<kVecR>(rg, (uint32_t)(m * r + c) * 2u, m < M ? r - c : 0);
        if constexpr (kGlu) rest = load8<kVecR>(rg, (uint32_t)((M + m) * r + c) * 2u, m < M ? r - c : 0);
      }
      low = qk::mfma32(a, b, low);
      if constexpr (kGlu) low = qk::mfma32(a, rest, low);
    }
    }
    if constexpr (!kGlu) {
    // half h draws octets 2 h and 2 h + 1 of its row; each lane takes its own columns 8 g + 4 h + e from both halves'
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) mine |= drop::bits8(d, (uint32_t)m, (uint32_t)(p >> 3) + 2 * h + i) << (16 * h + 8 * i);
    const u32x2 both = __builtin_amdgcn_permlane32_swap(mine, mine, false, false);
    keep = (both[0] | both[1]) >> (4 * h);
    }
  }
  __syncthreads();
  if (w >= 2 || m >= M) return;
  f32x16 sum = red[0][w][l];
#pragma unroll
  for (int i = 1; i < kW; ++i) sum += red[i][w][l];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = low[4 * g + e];
      o[e] = sum[4 * g + e] + (kGlu ? o[e] : (keep >> (8 * g + e)) & 1u ? d.scale * o[e] : 0.0f);
    }
    *(u32x2*)(dX + (int64_t)m * K + p + 8 * g + 4 * h) = u32x2{qk::pack_bf16x2(o[0], o[1]), qk::pack_bf16x2(o[2], o[3])};
  }
}

// Y of the NF4 layer for few rows: Y = bf16(X W'^T + s T L2).  Work group: 32 kI rows of X,
// 32 kJ rows of W; eight waves split the reduction, a block of 64 at a time.  The halves
// of a wave take the halves of a block, in both operands: the codes that a lane needs are
// 16 consecutive bytes, rebuilt in registers as the matrix operand, with no LDS but for
// the waves' sums, which meet there in order.  kSum: T as slices.
template <bool kVecR, int kI, int kJ, bool kSum>
__global__ __launch_bounds__(64 * kW) void k_fwd_small(const uint16_t* __restrict__ X, int M, int K, int N,
                                                       const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ c2, const float* __restrict__ c1,
                                                       const uint16_t* __restrict__ T, const float* __restrict__ Tp,
                                                       int S, uint16_t* __restrict__ T_out,
                                                       const uint16_t* __restrict__ L2, int r, float scale,
                                                       uint16_t* __restrict__ Y, Nf4Params q) {
  __shared__ f32x16 red[kW][kI * kJ][64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, h = l >> 5, x = l & 31;
  const int n0 = 32 * kJ * (int)blockIdx.x, m0 = 32 * kI * (int)blockIdx.y;
  const int kb = K / 64;
  const __amdgpu_buffer_rsrc_t rx = rsrc(X, (uint64_t)M * K * 2), rc = rsrc(codes, (uint64_t)N * (K / 2)),
                               r2 = rsrc(c2, (uint64_t)N * kb), r1 = rsrc(c1, 4 * (((uint64_t)N * kb + 255) / 256));
  const SplitConst kc = split_const();

  // block b: lane (x, h) holds columns 32 h .. +31 of it, of rows x, 32 + x, .. of X and W
  struct Step {
    u32x4 c[kJ];
    uint32_t s2[kJ];
    float s1[kJ];
    bf16x8 a[kI][4];
  };
  auto load = [&](int b) {
    Step s;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int n = n0 + 32 * j + x;
      const bool in = n < N && b < kb;
      const uint32_t at = (uint32_t)n * kb + b;
      s.c[j] = __builtin_amdgcn_raw_buffer_load_b128(rc, in ? (uint32_t)n * (K / 2) + 32 * b + 16 * h : kOOB, 0, 0);
      s.s2[j] = __builtin_amdgcn_raw_buffer_load_b8(r2, in ? at : kOOB, 0, 0);
      s.s1[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r1, in ? 4 * (at >> 8) : kOOB, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int m = m0 + 32 * i + x;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        s.a[i][u] = load8<true>(rx, ((uint32_t)m * K + 64 * b + 32 * h + 8 * u) * 2u, m < M && b < kb ? 8 : 0);
    }
    return s;
  };
  f32x16 acc[kI][kJ] = {};
  Step cur = load(w);
  for (int b = w; b < kb; b += kW) {
    const Step nxt = load(b + kW);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const BlockLut lut = make_lut(qk::e4m3fn_to_f32(cur.s2[j]) * cur.s1[j], q);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bf16x8 v = __builtin_bit_cast(bf16x8, dequant8(lut, cur.c[j][u], kc));
#pragma unroll
        for (int i = 0; i < kI; ++i) acc[i][j] = qk::mfma32(v, cur.a[i][u], acc[i][j]);
      }
    }
    cur = nxt;
  }
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int j = 0; j < kJ; ++j) red[w][kJ * i + j][l] = acc[i][j];
  // the first waves finish a tile of 32 x 32 each
  const int p = n0 + 32 * (w % kJ), m = m0 + 32 * (w / kJ) + x;
  f32x16 low = {};
  if (w < kI * kJ) {
    const __amdgpu_buffer_rsrc_t rt = rsrc(kSum ? (const void*)Tp : T, (uint64_t)M * r * (kSum ? 4 * S : 2)),
                                 rl = rsrc(L2, (uint64_t)N * r * 2);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = 16 * s + 8 * h;
      if (16 * s >= r) break;                      // uniform
      uint32_t e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        e[k] = __builtin_amdgcn_raw_buffer_load_b16(rl, c + k < r && p + x < N ? (uint32_t)((c + k) * N + p + x) * 2u : kOOB, 0, 0);
      const u32x4 a = {e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
      bf16x8 b;
      if constexpr (kSum) {
        float sum[8];
        sum8(rt, S, M, r, m, c, M * r, sum);
        u32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = qk::pack_bf16x2(sum[2 * k], sum[2 * k + 1]);
        b = __builtin_bit_cast(bf16x8, v);
        if (T_out && n0 == 0 && w % kJ == 0 && m < M && c < r) qk::store8_row(T_out + (int64_t)m * r + c, v, min(8, r - c));
      } else {
        b = load8<kVecR>(rt, (uint32_t)(m * r + c) * 2u, m < M ? r - c : 0);
      }
      low = qk::mfma32(__builtin_bit_cast(bf16x8, a), b, low);
    }
  }
  __syncthreads();
  if (w >= kI * kJ || m >= M) return;
  f32x16 sum = red[0][w][l];
#pragma unroll
  for (int i = 1; i < kW; ++i) sum += red[i][w][l];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int n = p + 8 * g + 4 * h;
    uint16_t* y = Y + (int64_t)m * N + n;
    const u32x2 o = {qk::pack_bf16x2(sum[4 * g] + scale * low[4 * g], sum[4 * g + 1] + scale * low[4 * g + 1]),
                     qk::pack_bf16x2(sum[4 * g + 2] + scale * low[4 * g + 2], sum[4 * g + 3] + scale * low[4 * g + 3])};
    if ((N & 3) == 0) {
      if (n < N) *(u32x2*)y = o;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) y[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// The gated product for few rows: H = bf16(silu(G) U), [G | U] = X W'^T + s T L2 for a stacked
// W [2 F, K].  As k_fwd_small, for 32 kI rows and the same 32 columns of both halves; 2 kI more
// waves form the adapter's term of one half of 32 rows each meanwhile, add the eight waves'
// sums in order and finish.  T enters as three bf16 planes (24 bits: G and U may be
// kept in 8): given [2 halves][3][M][pitch], or kSum: formed here from its slices [2][S][M][r].
// 17 rows 4096 -> 2 x 11008: 46 us, 47 MB at 1 TB/s; vector units busy for 14, the data return for 28
// (a lane's row is its own, so an instruction's 64 lanes read 64 lines), about 10 a launch's first
// loads and end.  Two blocks a step (a fifth fewer loads, half the tables) took 45 us, and 8192 -> 2
// x 22016 153 for 145; a wave's blocks side by side 47; two steps' registers in turn 48.  kI = 2 spills 17
// registers.
template <int kI, bool kSum>
__global__ __launch_bounds__(64 * (kW + 2 * kI)) void k_glu_small(const uint16_t* __restrict__ X, int M, int K, int F,
                                                       const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ c2, const float* __restrict__ c1,
                                                       const uint16_t* __restrict__ T, const float* __restrict__ Tp,
                                                       int S, uint16_t* __restrict__ T_out,
                                                       const uint16_t* __restrict__ L2, int r, float scale,
                                                       uint16_t* __restrict__ H, uint8_t* __restrict__ gu_codes,
                                                       uint8_t* __restrict__ gu_scales, Nf4Params q) {
  __shared__ f32x16 red[kW][kI * 2][64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, h = l >> 5, x = l & 31;
  const int n0 = 32 * (int)blockIdx.x, m0 = 32 * kI * (int)blockIdx.y;
  const int kb = K / 64;
  const int64_t N = 2 * (int64_t)F;
  const __amdgpu_buffer_rsrc_t rx = rsrc(X, (uint64_t)M * K * 2), rc = rsrc(codes, (uint64_t)N * (K / 2)),
                               r2 = rsrc(c2, (uint64_t)N * kb), r1 = rsrc(c1, 4 * (((uint64_t)N * kb + 255) / 256));
  const SplitConst kc = split_const();
  struct Step {
    u32x4 c[2];
    uint32_t s2[2];
    float s1[2];
    bf16x8 a[kI][4];
  };
  auto load = [&](int b) {
    Step s;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t n = (uint32_t)(j ? F : 0) + n0 + x;
      const bool in = n0 + x < F && b < kb;
      const uint32_t at = n * kb + b;
      s.c[j] = __builtin_amdgcn_raw_buffer_load_b128(rc, in ? n * (K / 2) + 32 * b + 16 * h : kOOB, 0, 0);
      s.s2[j] = __builtin_amdgcn_raw_buffer_load_b8(r2, in ? at : kOOB, 0, 0);
      s.s1[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r1, in ? 4 * (at >> 8) : kOOB, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int m = m0 + 32 * i + x;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        s.a[i][u] = load8<true>(rx, ((uint32_t)m * K + 64 * b + 32 * h + 8 * u) * 2u, m < M && b < kb ? 8 : 0);
    }
    return s;
  };
  if (w < kW) {
    f32x16 acc[kI][2] = {};
    Step cur = load(w);
    for (int b = w; b < kb; b += kW) {
      const Step nxt = load(b + kW);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const BlockLut lut = make_lut(qk::e4m3fn_to_f32(cur.s2[j]) * cur.s1[j], q);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bf16x8 v = __builtin_bit_cast(bf16x8, dequant8(lut, cur.c[j][u], kc));
#pragma unroll
          for (int i = 0; i < kI; ++i) acc[i][j] = qk::mfma32(v, cur.a[i][u], acc[i][j]);
        }
      }
      cur = nxt;
    }
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) red[w][2 * i + j][l] = acc[i][j];
  }
  const int wf = w - kW, j = wf & 1, i = wf >> 1, m = m0 + 32 * i + x;
  f32x16 sum = {};
  if (w >= kW) {
    const int pitch = (r + 7) / 8 * 8;
    const uint16_t* l2 = L2 + (int64_t)j * r * F;
    const uint16_t* t = T + (int64_t)j * 3 * M * pitch;      // its planes
    const __amdgpu_buffer_rsrc_t rt = kSum ? rsrc(Tp + (int64_t)j * S * M * r, (uint64_t)M * r * 4 * S)
                                           : rsrc(t, (uint64_t)M * pitch * 6);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = 16 * s + 8 * h;
      if (16 * s >= r) break;                      // uniform
      uint32_t e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = c + k < r && n0 + x < F ? l2[(int64_t)(c + k) * F + n0 + x] : 0;
      const bf16x8 a = __builtin_bit_cast(
          bf16x8, u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16});
      bf16x8 b[3];
      if constexpr (kSum) {
        float v[8];
        sum8(rt, S, M, r, m, c, M * r, v);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          const u32x4 p = glu::take_plane(v);
          b[n] = __builtin_bit_cast(bf16x8, p);
          if (n == 0 && T_out && n0 == 0 && m < M && c < r)
            qk::store8_row(T_out + ((int64_t)j * M + m) * r + c, p, min(8, r - c));
        }
      } else {
#pragma unroll
        for (int n = 0; n < 3; ++n)
          b[n] = load8<true>(rt, ((uint32_t)(n * M + m) * pitch + c) * 2u, m < M && c < pitch ? 8 : 0);
      }
#pragma unroll
      for (int n = 0; n < 3; ++n) sum = qk::mfma32(a, b[n], sum);
    }
    sum = scale * sum;
  }
  __syncthreads();
  if (w >= kW) {
    f32x16 base = red[0][wf][l];
#pragma unroll
    for (int k = 1; k < kW; ++k) base += red[k][wf][l];
    sum += base;
    if (gu_codes) {
      const int64_t fp = mx8::padded(F);
      glu::store_8(sum, gu_codes + j * M * fp, gu_scales + j * M * (fp / 32), m, M, n0, F);
    }
    if (j) red[0][wf][l] = sum;                    // this wave's alone until the barrier
  }
  __syncthreads();
  if (w >= kW && !j) glu::store_h(sum, red[0][wf + 1][l], H, m, M, n0, F);
}

}  // namespace

// Up to a work group of 64 rows x 32 columns of H a CU, and for 32 rows at any F (one work
// group's rows: no weight is rebuilt twice).  Whole forwards with the 8-bit copies, us, here / in
// large tiles: 4096 -> 2 x 11008 32 rows 59 / 83, 64 rows (344 work groups) 85 / 85, 128 rows (688)
// 132 / 87; 2048 -> 2 x 5504 64 rows (172) 37 / 58, 128 rows (344) 67 / 60; 512 -> 2 x 1376 256 rows
// (172) 37 / 39, 512 rows (344) 46 / 41; 8192 -> 2 x 22016 32 rows 151 / 204.
bool glu_small_ok(int64_t M, int64_t K, int64_t F) {
  return F < (int64_t(1) << 24) && (M <= 32 || (F + 31) / 32 * ((M + 63) / 64) <= 256);
}

hipError_t launch_glu_small(const uint16_t* X, int64_t M, int64_t K, int64_t F, const uint8_t* codes, const uint8_t* c2,
                            const float* c1, const uint16_t* T, const float* Tp, int S, uint16_t* T_out,
                            const uint16_t* L2, int r, float scale, uint16_t* H, uint8_t* gu_codes, uint8_t* gu_scales,
                            hipStream_t s) {
  const unsigned cols = (unsigned)((F + 31) / 32);
#define QL_GLU(I, A)                                                                                            \
  hipLaunchKernelGGL((k_glu_small<I, A>), dim3(cols, (unsigned)((M + 32 * I - 1) / (32 * I))),                  \
                     dim3(64 * (kW + 2 * I)), 0, s, X, (int)M, (int)K, (int)F, codes, c2, c1, T, Tp, S, T_out, L2, r, \
                     scale, H, gu_codes, gu_scales, nf4_params())
  // 32 rows a work group while those are at most one a CU: 4096 -> 2 x 1024 64 rows 26 us (64 rows a
  // group: 40), 1024 -> 2 x 1024 200 rows (224 groups) 14 (16); past that a CU would rebuild weights
  // twice: 2048 -> 2 x 5504 64 rows 45 us a call (37)
  const bool one = M <= 32 || cols * ((M + 31) / 32) <= 256;
  if (T) {
    if (one) QL_GLU(1, false);
    else QL_GLU(2, false);
  } else {
    if (one) QL_GLU(1, true);
    else QL_GLU(2, true);
  }
#undef QL_GLU
  return hipGetLastError();
}

// More rows than the decode kernels take at once (up to 48, three times as many, for any N
// that L2's 32-bit offsets reach), up to 2.5 work groups of 64 x 64 a CU: the large tiles walk
// the whole reduction in one work group, and leave CUs idle while they are few.  Whole forwards
// with dropout, us, decode kernels in passes of 16 rows or large tiles / here: 32 rows 512 -> 512 14 /
// 7.5, 4096 -> 11008 38 / 26, 11008 -> 4096 45 / 38, 8192 -> 22016 92 / 80; 128 rows 4096 -> 11008 95 / 67,
// 11008 -> 4096 222 / 57, 8576 -> 631 173 / 32; 512 rows 11008 -> 4096 229 / 146; 256 rows 4096 -> 11008
// (688 work groups) 98 / 97, 8192 -> 22016 (1376) 184 / 322.
bool fwd_small_ok(int64_t M, int64_t N) {
  return M > 16 && N < (int64_t(1) << 24) && (M <= 48 || (N + 63) / 64 * ((M + 63) / 64) <= 640);
}

// Bound: rebuilding the weights (3.6 vector instructions each) for every 32 kI rows, so
// tiles are as large as fills the chip: 64 rows 4096 -> 4096 25, 29 and 38 us with 32 x 32,
// 32 x 64 and 64 x 64 tiles, 128 rows 37, 30 and 39, 256 rows 62, 48 and 41.
hipError_t launch_fwd_small(const uint16_t* X, int64_t M, int64_t K, int64_t N, const uint8_t* codes, const uint8_t* c2,
                            const float* c1, const uint16_t* T, const float* Tp, int S, uint16_t* T_out,
                            const uint16_t* L2, int r, float scale, uint16_t* Y, hipStream_t s) {
  const int64_t rows = (M + 31) / 32;
#define QL_FW(V, I, J, A)                                                                                            \
  hipLaunchKernelGGL((k_fwd_small<V, I, J, A>),                                                                      \
                     dim3((unsigned)((N + 32 * J - 1) / (32 * J)), (unsigned)((M + 32 * I - 1) / (32 * I))),         \
                     dim3(64 * kW), 0, s, X, (int)M, (int)K, (int)N, codes, c2, c1, T, Tp, S, T_out, L2, r, scale, Y, \
                     nf4_params())
#define QL_FWT(I, J)                          \
  do {                                        \
    if (!T) QL_FW(false, I, J, true);         \
    else if (r % 8 == 0) QL_FW(true, I, J, false); \
    else QL_FW(false, I, J, false);           \
  } while (0)
  if ((N + 31) / 32 * rows <= 256) QL_FWT(1, 1);
  else if ((N + 63) / 64 * rows <= 256 || rows == 1) QL_FWT(1, 2);
  else QL_FWT(2, 2);
#undef QL_FWT
#undef QL_FW
  return hipGetLastError();
}

// Up to 64 rows, or up to three work groups (32 rows, 64 columns of dX) a CU.  Whole backwards
// with dropout, us, here / large tiles: 32 rows 4096 -> 11008 67 / 235, 11008 -> 4096 36 / 109,
// 8192 -> 22016 139 / 438, 512 -> 512 13 / 41; 128 rows 11008 -> 4096 85 / 112 (688 work groups),
// 8192 -> 22016 260 / 445 (512); 512 rows 4096 -> 4096 105 / 117 (1024); 256 rows 8192 -> 22016
// 489 / 446 (1024), 11008 -> 4096 159 / 116 (1376).
// From 2^29 columns on its launch would have 2^32 threads along x or more, which wrap.
bool dx_small_ok(int64_t M, int64_t K) {
  return (M <= 64 && K < (int64_t(1) << 29)) || (K / kP) * ((M + 31) / 32) <= 768;
}

hipError_t launch_dx_small(const uint16_t* dY, int64_t M, int64_t K, int64_t N, const uint8_t* codes, const uint8_t* c2,
                           const float* c1, const uint16_t* G, const float* Gp, int S, uint16_t* planes,
                           const uint16_t* L1, int r, uint16_t* dX, const drop::Params& d, hipStream_t s, int64_t ldy,
                           bool sum) {
  const dim3 grid((unsigned)(K / kP), (unsigned)((M + 31) / 32));
#define QL_DX(V, R, A, U, T)                                                                                               \
  hipLaunchKernelGGL((k_dx_small<V, R, A, U, T>), grid, dim3(64 * kW), 0, s, dY, (int)M, (int)K, (int)N, codes, c2, c1, \
                     G, Gp, S, planes, L1, r, dX, nf4_params(), d, (int)ldy)
#define QL_DXS(A)                                                       \
  do {                                                                  \
    if (glu && sum && vr) QL_DX(true, true, A, true, true);             \
    else if (glu && sum) QL_DX(true, false, A, true, true);             \
    else if (glu && vr) QL_DX(true, true, A, true, false);              \
    else if (glu) QL_DX(true, false, A, true, false);                   \
    else if (v && vr) QL_DX(true, true, A, false, false);               \
    else if (v) QL_DX(true, false, A, false, false);                    \
    else if (vr) QL_DX(false, true, A, false, false);                   \
    else QL_DX(false, false, A, false, false);                          \
  } while (0)
  const bool glu = ldy != 0, v = N % 8 == 0, vr = r % 8 == 0;
  if (G) QL_DXS(false);
  else QL_DXS(true);
#undef QL_DXS
#undef QL_DX
  return hipGetLastError();
}
