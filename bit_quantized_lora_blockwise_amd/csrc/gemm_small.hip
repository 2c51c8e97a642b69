// dX of the NF4 layer for few rows:
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

// kVec: N % 8 == 0 (rows of dY in whole 16-byte pieces); kVecR: r % 8 == 0.
template <bool kVec, bool kVecR, bool kDrop>
__global__ __launch_bounds__(64 * kW) void k_dx_small(const uint16_t* __restrict__ dY, int M, int K, int N,
                                                      const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ c2, const float* __restrict__ c1,
                                                      const uint16_t* __restrict__ G, const uint16_t* __restrict__ L1,
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
    const __amdgpu_buffer_rsrc_t rg = rsrc(G, (uint64_t)M * r * 2), rl = rsrc(L1, (uint64_t)K * r * 2);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = 16 * s + 8 * h;
      const bf16x8 a = load8<kVecR>(rl, (uint32_t)((p + x) * r + c) * 2u, r - c);
      const bf16x8 b = load8<kVecR>(rg, (uint32_t)(m * r + c) * 2u, m < M ? r - c : 0);
      low = qk::mfma32(a, b, low);
    }
    if constexpr (kDrop) {
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
      if constexpr (kDrop) o[e] = (keep >> (8 * g + e)) & 1u ? d.scale * o[e] : 0.0f;
      o[e] += sum[4 * g + e];
    }
    *(u32x2*)(dX + (int64_t)m * K + p + 8 * g + 4 * h) = u32x2{qk::pack_bf16x2(o[0], o[1]), qk::pack_bf16x2(o[2], o[3])};
  }
}

}  // namespace

// Up to 64 rows, or more while the work groups (32 rows, 64 columns) are no more than
// CUs.  With 32 rows of them: 11008 -> 4096 23 us here, 87 us with the large tiles;
// 4096 -> 11008 53 and 213 us; 8192 -> 22016 117 and 406 us; 512 -> 512 5 and 22 us.
bool dx_small_ok(int64_t M, int64_t K) { return M <= 64 || (K / kP) * ((M + 31) / 32) <= 256; }

hipError_t launch_dx_small(const uint16_t* dY, int64_t M, int64_t K, int64_t N, const uint8_t* codes, const uint8_t* c2,
                           const float* c1, const uint16_t* G, const uint16_t* L1, int r, uint16_t* dX,
                           const drop::Params& d, hipStream_t s) {
  const dim3 grid((unsigned)(K / kP), (unsigned)((M + 31) / 32));
#define QL_DX(V, R, D)                                                                                                \
  hipLaunchKernelGGL((k_dx_small<V, R, D>), grid, dim3(64 * kW), 0, s, dY, (int)M, (int)K, (int)N, codes, c2, c1, G, L1, r, \
                     dX, nf4_params(), d)
  const bool v = N % 8 == 0, vr = r % 8 == 0, dr = d.cut != 0;
  if (v && vr) {
    if (dr) QL_DX(true, true, true);
    else QL_DX(true, true, false);
  } else if (v) {
    if (dr) QL_DX(true, false, true);
    else QL_DX(true, false, false);
  } else if (vr) {
    if (dr) QL_DX(false, true, true);
    else QL_DX(false, true, false);
  } else {
    if (dr) QL_DX(false, false, true);
    else QL_DX(false, false, false);
  }
#undef QL_DX
  return hipGetLastError();
}
