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

// Elements c .. c + 7 of row m of T or G from its S <= kSlices fp32 slices [M][r], added in order.
constexpr int kSlices = 8;
__device__ __forceinline__ void sum8(__amdgpu_buffer_rsrc_t rp, int S, int M, int r, int m, int c, float (&sum)[8]) {
  const uint32_t at = 4u * (uint32_t)(m * r + c);
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    u32x4 v[kSlices];                    // slices past the last read as zeros
#pragma unroll
    for (int n = 0; n < kSlices; ++n)
      v[n] = __builtin_amdgcn_raw_buffer_load_b128(rp, n < S && m < M && c < r ? at + 4u * k : kOOB, 4 * n * M * r, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float u = __uint_as_float(v[0][j]);
#pragma unroll
      for (int n = 1; n < kSlices; ++n) u += __uint_as_float(v[n][j]);
      sum[k + j] = c + k + j < r ? u : 0.0f;
    }
  }
}

// kVec: N % 8 == 0 (rows of dY in whole 16-byte pieces); kVecR: r % 8 == 0; kSum: G as slices.
template <bool kVec, bool kVecR, bool kSum>
__global__ __launch_bounds__(64 * kW) void k_dx_small(const uint16_t* __restrict__ dY, int M, int K, int N,
                                                      const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ c2, const float* __restrict__ c1,
                                                      const uint16_t* __restrict__ G, const float* __restrict__ Gp, int S,
                                                      uint16_t* __restrict__ planes, const uint16_t* __restrict__ L1,
                                                      int r, uint16_t* __restrict__ dX, Nf4Params q, drop::Params d) {
  __shared__ __attribute__((aligned(16))) uint16_t wt[kW][kN * kPitch];
  __shared__ f32x16 red[kW][2][64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, h = l >> 5, x = l & 31;
  const int p0 = kP * (int)blockIdx.x, m0 = 32 * (int)blockIdx.y, m = m0 + x;
  const int kb = K / 64;
  const __amdgpu_buffer_rsrc_t ry = rsrc(dY, (uint64_t)M * N * 2), rc = rsrc(codes, (uint64_t)N * (K / 2)),
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
  auto load = [&](int n0) {
    Step s;
    const int n = n0 + x;
    const uint32_t b = (uint32_t)n * kb + blockIdx.x;
    s.c = __builtin_amdgcn_raw_buffer_load_b128(rc, n < N ? (uint32_t)n * (K / 2) + 32 * blockIdx.x + 16 * h : kOOB, 0, 0);
    s.s2 = __builtin_amdgcn_raw_buffer_load_b8(r2, n < N ? b : kOOB, 0, 0);
    s.s1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r1, n < N ? 4 * (b >> 8) : kOOB, 0, 0));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = n0 + 16 * u + 8 * h;
      s.y[u] = load8<kVec>(ry, (uint32_t)(m * N + k) * 2u, m < M ? N - k : 0);
    }
    return s;
  };
  f32x16 acc[2] = {};
  Step cur = load(kN * w);
  for (int n0 = kN * w; n0 < N; n0 += kN * kW) {
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
    const __amdgpu_buffer_rsrc_t rg = rsrc(kSum ? (const void*)Gp : G, (uint64_t)M * r * (kSum ? 4 * S : 2)),
                                 rl = rsrc(L1 + first * r, (uint64_t)32 * r * 2);
    const int pitch = (r + 7) / 8 * 8;
    const int64_t plane = (int64_t)M * pitch;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = 16 * s + 8 * h;
      if (16 * s >= r) break;                      // uniform
      const bf16x8 a = load8<kVecR>(rl, (uint32_t)(x * r + c) * 2u, r - c);
      bf16x8 b;
      if constexpr (kSum) {
        float sum[8];
        sum8(rg, S, M, r, m, c, sum);
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
        if (blockIdx.x == 0 && w == 0 && m < M && c < pitch)
#pragma unroll
          for (int n = 0; n < 3; ++n) *(u32x4*)(planes + n * plane + (int64_t)m * pitch + c) = v[n];
      } else {
        b = load8<kVecR>(rg, (uint32_t)(m * r + c) * 2u, m < M ? r - c : 0);
      }
      low = qk::mfma32(a, b, low);
    }
    // half h draws octets 2 h and 2 h + 1 of its row; each lane takes its own columns 8 g + 4 h + e from both halves'
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) mine |= drop::bits8(d, (uint32_t)m, (uint32_t)(p >> 3) + 2 * h + i) << (16 * h + 8 * i);
    const u32x2 both = __builtin_amdgcn_permlane32_swap(mine, mine, false, false);
    keep = (both[0] | both[1]) >> (4 * h);
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
      o[e] = sum[4 * g + e] + ((keep >> (8 * g + e)) & 1u ? d.scale * o[e] : 0.0f);
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
        sum8(rt, S, M, r, m, c, sum);
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

}  // namespace

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
                           const uint16_t* L1, int r, uint16_t* dX, const drop::Params& d, hipStream_t s) {
  const dim3 grid((unsigned)(K / kP), (unsigned)((M + 31) / 32));
#define QL_DX(V, R, A)                                                                                                \
  hipLaunchKernelGGL((k_dx_small<V, R, A>), grid, dim3(64 * kW), 0, s, dY, (int)M, (int)K, (int)N, codes, c2, c1, \
                     G, Gp, S, planes, L1, r, dX, nf4_params(), d)
#define QL_DXS(A)                          \
  do {                                     \
    if (v && vr) QL_DX(true, true, A);     \
    else if (v) QL_DX(true, false, A);     \
    else if (vr) QL_DX(false, true, A);    \
    else QL_DX(false, false, A);           \
  } while (0)
  const bool v = N % 8 == 0, vr = r % 8 == 0;
  if (G) QL_DXS(false);
  else QL_DXS(true);
#undef QL_DXS
#undef QL_DX
  return hipGetLastError();
}
