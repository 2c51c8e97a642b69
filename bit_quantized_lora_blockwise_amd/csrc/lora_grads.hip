// The adapter's gradients over many rows, both in one launch:
//   dL1 = (D o X)^T G  [K, r]   G as three bf16 planes (24 bits, see k_skinny_reduce3)
//   dL2 = s T^T dY     [r, N]
// Products that reduce over the long dimension M.  Bound: HBM, each activation read
// once; the draws of D (12 us of VALU for 4096 x 11008) and the products (7 us of MFMA
// with three planes) run beside it.
//
// Work group: 256 columns of the activation, all r columns of the other operand, a
// slice of M in steps of 64 rows; eight waves.  Wave w takes 64 of the columns
// (w % 4) and half of each step's rows (w / 4): 2 x 2 tiles of 32 x 32, so that one
// fragment read from LDS feeds two products.  (64 x 64 work groups of four waves,
// each 32 x 32, read twice as much LDS per product and kept a quarter of this in
// flight.)  A step's operands are loaded two steps ahead into registers, masked
// there (16 bytes are the eight elements of one draw) and stored to the other LDS
// buffer.  Slices are summed in order by k_tn_reduce_pair, so results repeat.
// 4096 rows of 11008 and 4096 columns, rank 64, dropout on the first: 38 us (4.4 TB/s counted).
#include <algorithm>

#include "kernels.h"

namespace {

constexpr int kT = 512;
constexpr int kP = 256;                    // activation columns of a work group
constexpr int kM = 64;                     // rows of a step
constexpr int kPitchB = 72;                // [m][c] tiles
constexpr int kABytes = kM * kP * 2;
constexpr int kBBytes = kM * kPitchB * 2;
constexpr uint32_t kOOB = 0x80000000u;

struct Job {
  const uint16_t* A;      // [M, P]
  const uint16_t* B;      // [M, r], kPlanes of them
  int P, tiles, slices;
  int rows;               // of a slice, a multiple of kM
  float* out;             // [slices][P][r]
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}

// A tile [m][256 columns], 512 bytes a row: 16-byte piece c of row m in slot
// c ^ 4 (m % 4), so that the rows a transposed read touches fall on different banks.
__device__ __forceinline__ bf16x8 frag_a(const LDS_AS uint8_t* a, int m0, int p0) {
  const int l = threadIdx.x & 63, G = l >> 4, i = l & 15;
  const int row = m0 + ((G >> 1) << 3) + (i >> 2), p = p0 + ((G & 1) << 4) + ((i & 3) << 2);
  const LDS_AS uint8_t* at = a + row * (kP * 2) + 16 * ((p >> 3) ^ (4 * (row & 3))) + 2 * (p & 7);
  const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)at);
  const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)(at + 4 * kP * 2));
  const u32x2 u = __builtin_bit_cast(u32x2, x), v = __builtin_bit_cast(u32x2, y);
  return __builtin_bit_cast(bf16x8, u32x4{u[0], u[1], v[0], v[1]});
}

template <int kPlanes, bool kDrop>
__device__ __forceinline__ void run(const Job& jb, int M, int r, int tile, int slice, const drop::Params& d,
                                    LDS_AS uint8_t* lds) {
  constexpr int kStage = kABytes + kPlanes * kBBytes;
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63;
  const int wp = w & 3, wk = w >> 2;
  const int p0 = tile * kP, m_beg = slice * jb.rows, m_end = min(M, m_beg + jb.rows);
  const int steps = (m_end - m_beg + kM - 1) / kM;
  const __amdgpu_buffer_rsrc_t ra = rsrc(jb.A, (uint64_t)M * jb.P * 2);
  // a descriptor for each plane: one stays below 2^31 bytes, all three together need not
  __amdgpu_buffer_rsrc_t rb[kPlanes];
#pragma unroll
  for (int j = 0; j < kPlanes; ++j) rb[j] = rsrc(jb.B + (int64_t)j * M * r, (uint64_t)M * r * 2);
  // thread t: rows t / 32 + 16 i, columns 8 (t % 32) of A; row t / 8, columns 8 (t % 8) of each plane
  const int arow = t >> 5, ac = t & 31, brow = t >> 3, bc = t & 7;
  struct Regs {
    u32x4 a[4], b[kPlanes];
  };
  auto load = [&](int st, Regs& g) {
    const int m = m_beg + st * kM;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m + arow + 16 * i, p = p0 + 8 * ac;
      g.a[i] = __builtin_amdgcn_raw_buffer_load_b128(
          ra, row < m_end && p < jb.P ? (uint32_t)(row * jb.P + p) * 2u : kOOB, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kPlanes; ++j)
      g.b[j] = __builtin_amdgcn_raw_buffer_load_b128(
          rb[j], m + brow < m_end && 8 * bc < r ? (uint32_t)((m + brow) * r + 8 * bc) * 2u : kOOB, 0, 0);
  };
  auto store = [&](int st, Regs& g) {
    LDS_AS uint8_t* a = lds + (st & 1) * kStage;
#pragma unroll
    for (int j = 0; j < kPlanes; ++j)
      *(LDS_AS u32x4*)(a + kABytes + j * kBBytes + brow * (kPitchB * 2) + 16 * bc) = g.b[j];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = arow + 16 * i;
      if constexpr (kDrop)
        g.a[i] = drop::mask8(g.a[i], d, (uint32_t)(m_beg + st * kM + row), (uint32_t)(p0 >> 3) + ac);
      *(LDS_AS u32x4*)(a + row * (kP * 2) + 16 * (ac ^ (4 * (row & 3)))) = g.a[i];
    }
  };
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  auto compute = [&](int st) {
    const LDS_AS uint8_t* a = lds + (st & 1) * kStage;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int m = 32 * wk + 16 * s;
      const bf16x8 x0 = frag_a(a, m, 64 * wp), x1 = frag_a(a, m, 64 * wp + 32);
#pragma unroll
      for (int j = 0; j < kPlanes; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const bf16x8 y = qk::frag_kmajor((const LDS_AS uint16_t*)(a + kABytes + j * kBBytes), kPitchB, m, 32 * c);
          acc[0][c] = qk::mfma32(x0, y, acc[0][c]);
          acc[1][c] = qk::mfma32(x1, y, acc[1][c]);
        }
    }
  };
  Regs g0, g1;
  load(0, g0);
  load(1, g1);
  store(0, g0);
  __syncthreads();
  // two steps a round (register sets alternate); past the slice's end everything reads as zeros
  for (int st = 0; st < steps; st += 2) {
    load(st + 2, g0);
    compute(st);
    store(st + 1, g1);
    __syncthreads();
    load(st + 3, g1);
    compute(st + 1);
    store(st + 2, g0);
    __syncthreads();
  }
  // the two halves of each step's rows
  LDS_AS float* red = (LDS_AS float*)lds + wp * 4096 + l;
  if (wk == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) red[((2 * i + j) * 16 + e) * 64] = acc[i][j][e];
  }
  __syncthreads();
  if (wk == 1) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = 32 * j + qk::acc_col();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int p = p0 + 64 * wp + 32 * i + qk::acc_row(e);
        if (p < jb.P && c < r) jb.out[((int64_t)slice * jb.P + p) * r + c] = acc[i][j][e] + red[((2 * i + j) * 16 + e) * 64];
      }
    }
}

template <bool kDrop>
__global__ __launch_bounds__(kT, 2) void k_lora_grads(Job j0, Job j1, int M, int r, drop::Params d) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * (kABytes + 3 * kBBytes)];
  const int n0 = j0.tiles * j0.slices, b = (int)blockIdx.x;
  if (b < n0) run<3, kDrop>(j0, M, r, b % j0.tiles, b / j0.tiles, d, (LDS_AS uint8_t*)lds);
  else run<1, false>(j1, M, r, (b - n0) % j1.tiles, (b - n0) / j1.tiles, d, (LDS_AS uint8_t*)lds);
}

// Slices of the two products: one work group a CU in all, the first product's work
// groups (three planes and the draws) with half as many rows as the second's.
struct Plan {
  int t0, t1, s0, s1, rows0, rows1;
};
Plan plan(int64_t M, int64_t K, int64_t N) {
  static const int cus = [] {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
      n = 256;
    return n;
  }();
  Plan p;
  p.t0 = (int)((K + kP - 1) / kP);
  p.t1 = (int)((N + kP - 1) / kP);
  const int steps = (int)((M + kM - 1) / kM);
  p.s1 = std::max(1, cus / (2 * p.t0 + p.t1));
  p.s0 = std::max(1, (cus - p.t1 * p.s1) / p.t0);
  auto rows = [&](int& s) {
    const int per = (steps + s - 1) / s;
    s = (steps + per - 1) / per;
    return per * kM;
  };
  p.rows0 = rows(p.s0);
  p.rows1 = rows(p.s1);
  return p;
}

}  // namespace

bool lora_grads_wide_ok(int64_t M, int64_t K, int64_t N, int r) {
  return M >= 512 && (K % 8) == 0 && (N % 8) == 0 && (r % 8) == 0;
}

size_t lora_grads_wide_ws(int64_t M, int64_t K, int64_t N, int r) {
  const Plan p = plan(M, K, N);
  return ((size_t)p.s0 * K * r * 4 + 255) / 256 * 256 + (size_t)p.s1 * N * r * 4;
}

hipError_t launch_lora_grads_wide(const uint16_t* X, int64_t K, const uint16_t* G, const drop::Params& d, float* dL1,
                                  const uint16_t* dY, int64_t N, const uint16_t* T, float scale, float* dL2, int64_t M,
                                  int r, float* ws, hipStream_t s) {
  const Plan p = plan(M, K, N);
  float* part1 = ws + ((size_t)p.s0 * K * r * 4 + 255) / 256 * 64;
  const Job j0{X, G, (int)K, p.t0, p.s0, p.rows0, ws}, j1{dY, T, (int)N, p.t1, p.s1, p.rows1, part1};
  const dim3 grid((unsigned)(p.t0 * p.s0 + p.t1 * p.s1));
  if (d.cut)
    hipLaunchKernelGGL(k_lora_grads<true>, grid, dim3(kT), 0, s, j0, j1, (int)M, r, d);
  else
    hipLaunchKernelGGL(k_lora_grads<false>, grid, dim3(kT), 0, s, j0, j1, (int)M, r, d);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_tn_reduce_pair(ws, p.s0, K, d.scale, dL1, part1, p.s1, N, scale, dL2, r, s);
}
