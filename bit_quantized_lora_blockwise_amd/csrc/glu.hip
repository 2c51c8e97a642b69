// The passes around the gated product of gemm_big.hip: T's planes, the gradients of G and U
// from dH, and the adapter's gradients from activations kept in 8 bits (mx8.h).
//
//   dG = dH U sig (1 + G (1 - sig)), dU = dH G sig, sig = 1 / (1 + e^-G)     (glu.h)
//   Gr = s dZ L2^T, dL1 = X^T Gr, dL2 = s T^T dZ       for dZ = dG and dU (or a linear's dY)
//
// dL1 and dL2 are fp32, so what enters them is kept to 24 bits: dZ and Gr as three bf16
// planes whose sum they are (each takes what the ones before it rounded off).  dZ's planes
// exist in registers alone: the pass that forms Gr (k_glu_back) writes the first one, which
// is what the dX product takes, and the pass that forms dL2 (k_grads8) computes dZ again from
// the 4 bytes an element that it came from.
#include <algorithm>

#include "glu.h"
#include "kernels.h"
#include "mx8.h"

namespace {

constexpr int kT = 256;

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight fp32 as bf16, which they keep the rest of.
__device__ __forceinline__ u32x4 take_plane(float (&v)[8]) {
  u32x4 p;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    p[k] = qk::pack_bf16x2(v[2 * k], v[2 * k + 1]);
    v[2 * k] -= __uint_as_float(p[k] << 16);
    v[2 * k + 1] -= __uint_as_float(p[k] & 0xFFFF0000u);
  }
  return p;
}

// ---- T's planes ------------------------------------------------------------------
__global__ __launch_bounds__(kT) void k_t_planes(const float* __restrict__ part, int64_t pitch, int slices, int64_t M,
                                                 int r, int rp, uint16_t* __restrict__ planes,
                                                 uint16_t* __restrict__ T_out) {
  const int h = blockIdx.y;
  part += h * pitch;
  planes += h * 2 * M * rp;
  for (int64_t i = (int64_t)blockIdx.x * kT + threadIdx.x; i < M * rp; i += (int64_t)gridDim.x * kT) {
    const int64_t m = i / rp;
    const int c = (int)(i - m * rp);
    float x = 0.0f;
    if (c < r) {
      const float* p = part + m * r + c;
      for (int k = 0; k < slices; ++k) x += p[k * M * r];
    }
    const uint16_t hi = qk::f32_to_bf16(x);
    planes[i] = hi;
    planes[M * rp + i] = qk::f32_to_bf16(x - qk::bf16_to_f32(hi));
    if (T_out && c < r) T_out[(h * M + m) * r + c] = hi;
  }
}

// ---- operands turned ----------------------------------------------------------------
// Work group: 32 rows m of one half of G (blockIdx.z = 0) or T (1).
__global__ __launch_bounds__(kT) void k_turn(Turn q, int halves, int64_t M, int r) {
  __shared__ float tile[64][33];
  const int h = blockIdx.y, rk = (r + 15) / 16 * 16;
  const bool is_t = blockIdx.z == 1;
  const int64_t m0 = 32 * (int64_t)blockIdx.x, mp = (M + 31) / 32 * 32;
  for (int e = threadIdx.x; e < 32 * r; e += kT) {
    const int y = e / r, c = e - y * r;
    const int64_t m = m0 + y, at = ((int64_t)h * M + m) * r + c;
    float x = 0.0f;
    if (m < M) {
      if (is_t) {
        x = qk::bf16_to_f32(q.T[at]);
      } else {
        for (int k = 0; k < q.slices; ++k) x += q.part[(int64_t)k * halves * M * r + at];
        x *= q.scale;
        q.G[at] = qk::f32_to_bf16(x);
      }
    }
    tile[c][y] = x;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * rk; e += kT) {
    const int c = e >> 5, y = e & 31;
    float x = c < r ? tile[c][y] : 0.0f;
    if (is_t) {
      q.Tt[((int64_t)h * rk + c) * mp + m0 + y] = qk::f32_to_bf16(x);
    } else {
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const uint16_t b = qk::f32_to_bf16(x);
        q.Gt[(((int64_t)h * 3 + n) * rk + c) * mp + m0 + y] = b;
        x -= qk::bf16_to_f32(b);
      }
    }
  }
}

// ---- dZ and the slices of dZ L2^T ----------------------------------------------------
// Work group: 64 rows, four waves of 16, and a slice of the columns in steps of 32: lane
// (x, q) holds row x, columns 8 q .. + 7 of a step, which is the matrix operand as it is.
__global__ __launch_bounds__(kT) void k_glu_back(const uint16_t* __restrict__ dH, int64_t M, int64_t F,
                                                 const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                 const uint16_t* __restrict__ L2, int r, int64_t chunk, int64_t ldz,
                                                 uint16_t* __restrict__ dZ, float* __restrict__ part) {
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, x = l & 15, q = l >> 4;
  const int64_t m = 64 * (int64_t)blockIdx.x + 16 * w + x;
  const int64_t f_beg = blockIdx.y * chunk, f_end = min(F, f_beg + chunk);
  const int64_t fp = mx8::padded(F);
  const bool ok = m < M;
  const int64_t mc = ok ? m : 0;
  const uint8_t *cg = codes + mc * fp, *cu = codes + (M + mc) * fp;
  const uint8_t *sg = scales + mc * (fp / 32), *su = scales + (M + mc) * (fp / 32);
  const uint16_t* dh = dH + mc * F;
  const int nt = (r + 15) / 16;
  f32x4 acc[2][4] = {};
  struct Step {
    u32x2 g, u;
    u32x4 d;
    uint32_t sg, su;
  };
  auto load = [&](int64_t f0) {
    Step s = {};
    const int64_t f = f0 + 8 * q;
    if (ok && f < f_end) {
      s.g = *(const u32x2*)(cg + f);
      s.u = *(const u32x2*)(cu + f);
      s.sg = sg[f >> 5];
      s.su = su[f >> 5];
      s.d = qk::load8_row(dh, f, F);
    }
    return s;
  };
  Step cur = load(f_beg);
  for (int64_t f0 = f_beg; f0 < f_end; f0 += 32) {
    const Step nxt = load(f0 + 32);
    const int64_t f = f0 + 8 * q;
    float g[8], u[8], dz[2][8];
    const float ks = mx8::scale_f32(cur.sg), ku = mx8::scale_f32(cur.su);
    mx8::decode4(cur.g[0], ks, g);
    mx8::decode4(cur.g[1], ks, g + 4);
    mx8::decode4(cur.u[0], ku, u);
    mx8::decode4(cur.u[1], ku, u + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      glu::back(g[j], u[j], __uint_as_float(j & 1 ? cur.d[j >> 1] & 0xFFFF0000u : cur.d[j >> 1] << 16), dz[0][j], dz[1][j]);
    u32x4 b[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 16 * j + x;
        b[h][j] = j < nt && c < r && f < F ? qk::load8_row(L2 + ((int64_t)h * r + c) * F, f, F) : u32x4{0, 0, 0, 0};
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const u32x4 a = take_plane(dz[h]);
        if (n == 0 && ok && f < F) qk::store8_row(dZ + m * ldz + h * F + f, a, (int)min((int64_t)8, F - f));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nt) acc[h][j] = mfma16(a, b[h][j], acc[h][j]);
      }
    cur = nxt;
  }
  if (f_end == F && ok && q == 0)
    for (int64_t f = 2 * F; f < ldz; ++f) dZ[m * ldz + f] = 0;
  // lane: column 16 j + x, rows 4 q + v
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t mm = 64 * (int64_t)blockIdx.x + 16 * w + 4 * q + v;
        const int c = 16 * j + x;
        if (mm < M && c < r) part[(((int64_t)blockIdx.y * 2 + h) * M + mm) * r + c] = acc[h][j][v];
      }
}

// ---- dL1 and dL2 ---------------------------------------------------------------------
// Products that reduce over the rows.  A wave takes 64 columns in steps of 32 rows: lane
// (x, q) loads columns 4 x .. + 3 of rows 8 q .. + 7 and so has, for each of its columns,
// eight consecutive rows, which is the matrix operand of a tile whose columns are 4 apart:
// tile t holds columns 4 x + t, and nothing is turned in LDS.  The other operand lies turned
// in memory (k_turn).  The four waves of a work group take its steps in turn and their sums
// meet in LDS in order; slices are added in order by k_grads8_sum.
enum Kind { kPacked, kDense, kGated };

struct Job8 {
  const uint8_t* codes;     // kPacked: X; kGated: G over U
  const uint8_t* scales;
  const uint16_t* d;        // kDense: dY; kGated: dH
  const uint16_t* B;        // [halves][planes][rk][mp]
  int64_t P;                // columns
  int64_t chunk;            // rows of a slice, a multiple of 32
  int tiles, slices;
  float* out;               // slices [..][halves * P * r] (dL1: [P][r] each half, dL2: [r][P])
  float scale;
};

// 4 columns of one row as bf16 pairs {0, 1}, {2, 3}
__device__ __forceinline__ u32x2 load4_row(const uint16_t* row, int64_t c, int64_t cols) {
  if (c + 4 <= cols) {
    typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
    return *(const u32x2_a2*)(row + c);
  }
  u32x2 v = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < cols) v[j >> 1] |= (uint32_t)row[c + j] << (16 * (j & 1));
  return v;
}

template <Kind kKind, int kHalves>
__device__ __forceinline__ void grads8(const Job8& jb, int64_t M, int r, int tile, int slice, f32x4* red) {
  constexpr int kPA = kKind == kGated ? 3 : 1, kPB = kKind == kPacked ? 3 : 1;
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, x = l & 15, q = l >> 4;
  const int nt = (r + 15) / 16, rk = 16 * nt;
  const int64_t mp = (M + 31) / 32 * 32;
  const int64_t p0 = 64 * (int64_t)tile, p = p0 + 4 * x;
  const int64_t m_beg = slice * jb.chunk, m_end = min(M, m_beg + jb.chunk);
  const int64_t cp = mx8::padded(jb.P);
  f32x4 acc[kHalves][4][4] = {};
  for (int64_t m0 = m_beg + 32 * w; m0 < m_end; m0 += 128) {
    const int64_t mq = m0 + 8 * q;
    // A: per half, column t, plane n
    float z[kHalves][4][8];                          // kGated: [half][column][row]
    u32x4 a1[4];                                     // the others: operands as they are
    if constexpr (kKind == kPacked) {
      u32x2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = mq + i < m_end && p < cp;
        const uint32_t c = ok ? *(const uint32_t*)(jb.codes + (mq + i) * cp + p) : 0u;
        const float s = mx8::scale_f32(ok ? jb.scales[(mq + i) * (cp / 32) + (p >> 5)] : 127u);
        float f[4];
        mx8::decode4(c, s, f);
        v[i] = u32x2{qk::pack_bf16x2(f[0], f[1]), qk::pack_bf16x2(f[2], f[3])};
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          a1[t][k] = __builtin_amdgcn_perm(v[2 * k + 1][t >> 1], v[2 * k][t >> 1], t & 1 ? 0x07060302u : 0x05040100u);
    } else if constexpr (kKind == kDense) {
      u32x2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = mq + i < m_end && p < jb.P ? load4_row(jb.d + (mq + i) * jb.P, p, jb.P) : u32x2{0, 0};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          a1[t][k] = __builtin_amdgcn_perm(v[2 * k + 1][t >> 1], v[2 * k][t >> 1], t & 1 ? 0x07060302u : 0x05040100u);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = mq + i < m_end && p < jb.P;
        const int64_t mg = ok ? mq + i : 0, pg = ok ? p : 0;
        const uint32_t cg = *(const uint32_t*)(jb.codes + mg * cp + pg), cu = *(const uint32_t*)(jb.codes + (M + mg) * cp + pg);
        const float sg = mx8::scale_f32(jb.scales[mg * (cp / 32) + (pg >> 5)]);
        const float su = mx8::scale_f32(jb.scales[(M + mg) * (cp / 32) + (pg >> 5)]);
        const u32x2 d = ok ? load4_row(jb.d + mg * jb.P, pg, jb.P) : u32x2{0, 0};
        float g[4], u[4];
        mx8::decode4(cg, sg, g);
        mx8::decode4(cu, su, u);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          glu::back(g[t], u[t], __uint_as_float(t & 1 ? d[t >> 1] & 0xFFFF0000u : d[t >> 1] << 16), z[0][t][i],
                    z[kHalves - 1][t][i]);
      }
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int nb = 0; nb < kPB; ++nb) {
        u32x4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[j] = j < nt ? *(const u32x4*)(jb.B + (((int64_t)h * kPB + nb) * rk + 16 * j + x) * mp + mq) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int na = 0; na < kPA; ++na) {
            const u32x4 a = kKind == kGated ? take_plane(z[h][t]) : a1[t];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < nt) {
                if constexpr (kKind == kPacked) acc[h][t][j] = mfma16(a, b[j], acc[h][t][j]);   // rows p, columns c
                else acc[h][t][j] = mfma16(b[j], a, acc[h][t][j]);                              // rows c, columns p
              }
          }
      }
  }
  // the waves' sums, added in order
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    if (h) __syncthreads();
    if (w) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[((w - 1) * 16 + 4 * t + j) * 64 + l] = acc[h][t][j];
    }
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int i = 0; i < 3; ++i) acc[h][t][j] += red[(i * 16 + 4 * t + j) * 64 + l];
          acc[h][t][j] *= jb.scale;
        }
      float* out = jb.out + ((int64_t)slice * kHalves + h) * jb.P * r;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if constexpr (kKind == kPacked) {        // lane: column c = 16 j + x, row 4 q + v of the tile
              const int64_t pp = p0 + 4 * (4 * q + v) + t;
              if (16 * j + x < r && pp < jb.P) out[pp * r + 16 * j + x] = acc[h][t][j][v];
            } else {                                 // lane: column x of the tile, row c = 16 j + 4 q + v
              const int c = 16 * j + 4 * q + v;
              if (c < r && p + t < jb.P) out[(int64_t)c * jb.P + p + t] = acc[h][t][j][v];
            }
          }
    }
  }
}

template <int kHalves>
__global__ __launch_bounds__(kT) void k_grads8(Job8 j0, Job8 j1, int64_t M, int r) {
  __shared__ f32x4 red[3 * 16 * 64];
  const int n0 = j0.tiles * j0.slices, b = (int)blockIdx.x;
  if (b < n0) grads8<kPacked, kHalves>(j0, M, r, b % j0.tiles, b / j0.tiles, red);
  else grads8<kHalves == 2 ? kGated : kDense, kHalves>(j1, M, r, (b - n0) % j1.tiles, (b - n0) / j1.tiles, red);
}

// Both outputs as their slices' sums, added in order.
__global__ __launch_bounds__(kT) void k_grads8_sum(const float* __restrict__ p0, int s0, int64_t n0, float* __restrict__ o0,
                                                   const float* __restrict__ p1, int s1, int64_t n1,
                                                   float* __restrict__ o1, int nb0) {
  const bool first = (int)blockIdx.x < nb0;
  const float* p = first ? p0 : p1;
  float* o = first ? o0 : o1;
  const int s = first ? s0 : s1;
  const int64_t n = first ? n0 : n1;
  const int blk = first ? blockIdx.x : blockIdx.x - nb0, nblk = first ? nb0 : gridDim.x - nb0;
  for (int64_t i = (int64_t)blk * kT + threadIdx.x; i < n; i += (int64_t)nblk * kT) {
    float u = p[i];
    for (int k = 1; k < s; ++k) u += p[k * n + i];
    o[i] = u;
  }
}

// Work groups of the backward's passes over the rows: a slice for every 512 / tiles, of 128 rows at least.
struct Plan8 {
  int tiles, slices;
  int64_t chunk;
};
Plan8 plan8(int64_t P, int64_t M) {
  Plan8 p;
  p.tiles = (int)((P + 63) / 64);
  int64_t s = std::max<int64_t>(1, std::min<int64_t>(512 / p.tiles, M / 128));
  p.chunk = ((M + s - 1) / s + 31) / 32 * 32;
  p.slices = (int)((M + p.chunk - 1) / p.chunk);
  return p;
}

Plan8 plan_back(int64_t M, int64_t F) {
  Plan8 p;
  p.tiles = (int)((M + 63) / 64);
  int64_t s = std::max<int64_t>(1, std::min<int64_t>(1024 / p.tiles, F / 128));
  p.chunk = ((F + s - 1) / s + 31) / 32 * 32;
  p.slices = (int)((F + p.chunk - 1) / p.chunk);
  return p;
}

unsigned blocks(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + kT - 1) / kT, 4096)); }

}  // namespace

hipError_t launch_t_planes(const float* part, int64_t pitch, int slices, int halves, int64_t M, int r, uint16_t* planes,
                           uint16_t* T_out, hipStream_t s) {
  const int rp = g_pitch(r);
  hipLaunchKernelGGL(k_t_planes, dim3(blocks(M * rp), (unsigned)halves), dim3(kT), 0, s, part, pitch, slices, M, r, rp,
                     planes, T_out);
  return hipGetLastError();
}

hipError_t launch_turn(const Turn& t, int halves, int64_t M, int r, hipStream_t s) {
  hipLaunchKernelGGL(k_turn, dim3((unsigned)((M + 31) / 32), (unsigned)halves, 2), dim3(kT), 0, s, t, halves, M, r);
  return hipGetLastError();
}

size_t glu_back_ws(int64_t M, int64_t F, int r) { return (size_t)plan_back(M, F).slices * 2 * M * r * sizeof(float); }

hipError_t launch_glu_back(const uint16_t* dH, int64_t M, int64_t F, const uint8_t* gu_codes, const uint8_t* gu_scales,
                           const uint16_t* L2, int r, uint16_t* dZ, float* part, int* slices, hipStream_t s) {
  const Plan8 p = plan_back(M, F);
  *slices = p.slices;
  hipLaunchKernelGGL(k_glu_back, dim3((unsigned)p.tiles, (unsigned)p.slices), dim3(kT), 0, s, dH, M, F, gu_codes, gu_scales,
                     L2, r, p.chunk, glu_ldz(F), dZ, part);
  return hipGetLastError();
}

size_t grads8_ws(int64_t M, int64_t K, int64_t N, int halves, int r) {
  return (size_t)halves * r * sizeof(float) * (plan8(K, M).slices * K + plan8(N, M).slices * N);
}

hipError_t launch_grads8(const Grads8& g, int64_t M, int64_t K, int64_t N, int halves, int r, float* ws, hipStream_t s) {
  const Plan8 a = plan8(K, M), b = plan8(N, M);
  const int64_t n0 = (int64_t)halves * K * r, n1 = (int64_t)halves * N * r;
  float* part1 = ws + a.slices * n0;
  const Job8 j0{g.x_codes, g.x_scales, nullptr, g.Gt, K, a.chunk, a.tiles, a.slices, a.slices > 1 ? ws : g.dL1, 1.0f};
  const Job8 j1{g.gu_codes, g.gu_scales, g.d, g.Tt, N, b.chunk, b.tiles, b.slices, b.slices > 1 ? part1 : g.dL2, g.scale};
  const dim3 grid((unsigned)(a.tiles * a.slices + b.tiles * b.slices));
  if (halves == 2) hipLaunchKernelGGL(k_grads8<2>, grid, dim3(kT), 0, s, j0, j1, M, r);
  else hipLaunchKernelGGL(k_grads8<1>, grid, dim3(kT), 0, s, j0, j1, M, r);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (a.slices == 1 && b.slices == 1)) return e;
  const int nb0 = a.slices > 1 ? (int)blocks(n0) : 0, nb1 = b.slices > 1 ? (int)blocks(n1) : 0;
  hipLaunchKernelGGL(k_grads8_sum, dim3((unsigned)(nb0 + nb1)), dim3(kT), 0, s, ws, a.slices, n0, g.dL1, part1, b.slices, n1,
                     g.dL2, nb0);
  return hipGetLastError();
}
