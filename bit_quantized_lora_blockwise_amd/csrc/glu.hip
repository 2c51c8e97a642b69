// The passes around the gated product of gemm_big.hip: T's planes, the gradients of G and U from
// dH (mx8.h), and what the adapter's gradients (grads8.hip) multiply.
//
//   dG = dH U sig (1 + G (1 - sig)), dU = dH G sig, sig = 1 / (1 + e^-G)     (glu.h)
//   Gr = s dZ L2^T, dL1 = X^T Gr, dL2 = s T^T dZ       for dZ = dG and dU (or a linear's dY)
//
// dL1 and dL2 are fp32, so what enters them is not rounded again: dZ and Gr, formed in fp32, go in as
// three bf16 planes whose sum they are to 24 bits (each takes what the ones before it rounded off).  dZ's planes
// exist on chip alone: the pass that forms Gr (k_glu_back) writes the first one, which is
// what the dX product takes, and the pass that forms dL2 (grads8.hip) computes dZ again from the
// 4 bytes an element that it came from.
#include <algorithm>

#include "glu.h"
#include "kernels.h"
#include "mx8.h"

namespace {

using glu::kOOB;
using glu::rsrc;

constexpr int kT = 256;
// ---- T's planes ------------------------------------------------------------------
__global__ __launch_bounds__(kT) void k_t_planes(const float* __restrict__ part, int64_t pitch, int slices, int64_t M,
                                                 int r, int rp, uint16_t* __restrict__ planes,
                                                 uint16_t* __restrict__ T_out) {
  const int h = blockIdx.y;
  part += h * pitch;
  planes += h * 3 * M * rp;
  for (int64_t i = (int64_t)blockIdx.x * kT + threadIdx.x; i < M * rp; i += (int64_t)gridDim.x * kT) {
    const int64_t m = i / rp;
    const int c = (int)(i - m * rp);
    float x = 0.0f;
    if (c < r) {
      const float* p = part + m * r + c;
      for (int k = 0; k < slices; ++k) x += p[k * M * r];
    }
    const uint16_t hi = qk::f32_to_bf16(x);
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const uint16_t b = qk::f32_to_bf16(x);
      planes[n * M * rp + i] = b;
      x -= qk::bf16_to_f32(b);
    }
    if (T_out && c < r) T_out[(h * M + m) * r + c] = hi;
  }
}

// ---- Gr's planes ---------------------------------------------------------------------
// The slices of Gr summed in order, scaled: bf16 [halves][M][r] and three planes [halves][3][M][rp].  kN columns a
// thread (16-byte loads if 4).
template <int kN>
__global__ __launch_bounds__(kT) void k_low(Low q, int halves, int64_t M, int r, int rp) {
  const int h = blockIdx.y;
  const int64_t pitch = (int64_t)halves * M * r, n = M * rp;
  for (int64_t i = kN * ((int64_t)blockIdx.x * kT + threadIdx.x); i < n; i += (int64_t)kN * gridDim.x * kT) {
    const int64_t m = i / rp;
    const int c = (int)(i - m * rp);
    const int64_t at = ((int64_t)h * M + m) * r + c;
    float x[kN] = {};
    if (c < r) {                           // kN = 4: r is a multiple of 4, and so all four or none
      const float* p = q.part + at;
      int k = 0;
      for (; k + 4 <= q.slices; k += 4) {  // four in flight
        float v[4][kN];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          if constexpr (kN == 4) {
            const f32x4 u = *(const f32x4*)(p + (k + a) * pitch);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[a][j] = u[j];
          } else {
            v[a][0] = p[(k + a) * pitch];
          }
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int j = 0; j < kN; ++j) x[j] += v[a][j];
      }
      for (; k < q.slices; ++k)
#pragma unroll
        for (int j = 0; j < kN; ++j) x[j] += p[k * pitch + j];
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) x[j] *= q.scale;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      uint16_t b[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        b[j] = qk::f32_to_bf16(x[j]);
        x[j] -= qk::bf16_to_f32(b[j]);
        if (a <= q.two && c < r) q.G[at + (int64_t)((q.two ? h : 0) + a) * M * r + j] = b[j];
      }
      uint16_t* to = q.planes + ((int64_t)h * 3 + a) * n + i;
      if constexpr (kN == 4) *(u32x2*)to = u32x2{b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16};
      else to[0] = b[0];
    }
  }
}

// ---- dZ and the slices of dZ L2^T ----------------------------------------------------
// Work group: 64 rows, a slice of the columns in steps of 64 (or 32 rows, steps of 128).  A
// step's dZ is formed in row-major pieces of eight columns a thread (so that a row's bytes are
// read and written in whole cache lines: with 16 rows a wave and lanes that held operands as
// they are, lines were read and written in quarters, 180 us at 4096 x 2 x 11008), stored, split
// into planes and put into LDS with L2's share of the step.  Wave w multiplies half w / 4, 32 ranks (w / 2 % 2),
// half of the step's columns (w % 2).  The next step's dH, G and U are loaded as soon as this
// one's have become dZ; one LDS buffer and two barriers a step, so that two work groups share a CU.
// 32 rows take L2 from memory straight to registers, a row a lane: 64 lines an instruction,
// which cost 45 of 127 us at 4096 rows, but a step less LDS and shorter: 64 rows 10 / 15 us (rows of
// 32 / of 64), 256 rows 13 / 16, 512 rows 20 / 19, 1024 rows 36 / 32, 4096 rows 123 / 101.
//
// 4096 x 2 x 11008: 363 MB, 70 us at a copy's rate; 36 vector instructions an element take 43 us
// of each SIMD, three planes' products 14, and what the two phases of a step do not overlap is the rest.
constexpr int kBT = 512;
constexpr int kBElems = 4096;              // of a step: 32 rows x 128 columns or 64 x 64

// kVec: F % 8 == 0.  plane: columns of a plane of dZ, of which a row holds ldz / plane.
template <int kBM, bool kVec>
__global__ __launch_bounds__(kBT, 4) void k_glu_back(const uint16_t* __restrict__ dH, int M, int F,
                                                     const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales,
                                                     const uint16_t* __restrict__ L2, int r, float scale, int chunk, int ldz,
                                                     int plane, uint16_t* __restrict__ dZ, float* __restrict__ part) {
  constexpr int kBC = kBElems / kBM;       // columns of a step
  constexpr int kBPitch = kBC + 8;         // LDS row (elements): 16 rows' pieces of 16 bytes on different banks
  constexpr int kRows = kBM / 32;          // row tiles of 32
  constexpr int kKs = kBC / 32;            // MFMA steps of a wave's half of the columns
  __shared__ __attribute__((aligned(16))) uint16_t lds[6 * kBM * kBPitch];      // [half][plane][row][column]
  // 64 rows: L2's share of a step, [half][rank][column]
  __shared__ __attribute__((aligned(16))) uint16_t lds_b[kBM == 64 ? 2 * 64 * kBPitch : 8];
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, hl = l >> 5;
  const int wh = w >> 2, wc = (w >> 1) & 1, wk = w & 1;
  const int f_beg = (int)blockIdx.y * chunk, f_end = min(F, f_beg + chunk);
  const int fp = (F + 31) / 32 * 32, nb = fp / 32;
  // all below 2^31 bytes; the up half's codes and scales follow the gate's
  const __amdgpu_buffer_rsrc_t rc = rsrc(codes, (uint64_t)2 * M * fp), rs = rsrc(scales, (uint64_t)2 * M * nb),
                               rd = rsrc(dH, (uint64_t)M * F * 2), rl = rsrc(L2, (uint64_t)2 * r * F * 2);
  const uint32_t up_c = (uint32_t)M * fp, up_s = (uint32_t)M * nb;
  // thread t: eight columns of a row of the step
  const int row = t / (kBC / 8), col = 8 * (t % (kBC / 8)), m = kBM * (int)blockIdx.x + row;
  // lane (x, hl) of a wave: rank 32 wc + x, a quarter of a step's columns, number 2 wk + hl
  const int c = 32 * wc + (l & 31), kcol = kBC / 4 * (2 * wk + hl);
  struct Step {
    u32x2 g, u;
    u32x4 d;
    uint8_t sg, su;
  };
  auto load = [&](int f0) {
    Step s;
    const int f = f0 + col;
    const bool in = m < M && f < f_end;    // rows of codes go on to a multiple of 32
    const uint32_t oc = in ? (uint32_t)m * fp + f : kOOB, os = in ? (uint32_t)m * nb + (f >> 5) : kOOB;
    s.g = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, oc, 0, 0));
    s.u = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, in ? oc + up_c : kOOB, 0, 0));
    s.sg = __builtin_amdgcn_raw_buffer_load_b8(rs, os, 0, 0);
    s.su = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? os + up_s : kOOB, 0, 0);
    s.d = glu::load8<kVec>(rd, (uint32_t)m * F * 2u, f, F, in);
    return s;
  };
  f32x16 acc[kRows] = {};
  Step cur = load(f_beg);
  for (int f0 = f_beg; f0 < f_end; f0 += kBC) {
    const int f = f0 + col;
    u32x4 b[kKs];
#pragma unroll
    for (int i = 0; i < kKs; ++i)
      if constexpr (kBM == 64)             // half i, rank `row`, columns `col`
        b[i] = glu::load8<kVec>(rl, (uint32_t)(i * r + row) * F * 2u, f, F, row < r && f < f_end);
      else
        b[i] = glu::load8<kVec>(rl, (uint32_t)(wh * r + c) * F * 2u, f0 + kcol + 8 * i, F, c < r && f0 + kcol + 8 * i < f_end);
    const float ks = mx8::scale_f32(cur.sg), ku = mx8::scale_f32(cur.su);
    const u32x4 d = glu::fit8<kVec>(cur.d, f, F);
    float dz[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float g[4], u[4];
      mx8::decode4(cur.g[k], ks, g);
      mx8::decode4(cur.u[k], ku, u);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        glu::back(g[j], u[j], __uint_as_float(j & 1 ? d[2 * k + (j >> 1)] & 0xFFFF0000u : d[2 * k + (j >> 1)] << 16),
                  dz[0][4 * k + j], dz[1][4 * k + j]);
    }
    cur = load(f0 + kBC);
    __syncthreads();                       // the last step has been read
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const u32x4 a = glu::take_plane(dz[h]);
        *(LDS_AS u32x4*)((LDS_AS uint16_t*)lds + ((3 * h + n) * kBM + row) * kBPitch + col) = a;
        if (n * plane < ldz && m < M && f < F) qk::store8_row(dZ + (int64_t)m * ldz + n * plane + h * F + f, a, min(8, F - f));
      }
    if constexpr (kBM == 64)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *(LDS_AS u32x4*)((LDS_AS uint16_t*)lds_b + (64 * i + row) * kBPitch + col) = glu::fit8<kVec>(b[i], f, F);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKs; ++i) {
      bf16x8 l2;
      if constexpr (kBM == 64)
        l2 = *(const LDS_AS bf16x8*)((const LDS_AS uint16_t*)lds_b + (64 * wh + c) * kBPitch + kcol + 8 * i);
      else
        l2 = __builtin_bit_cast(bf16x8, glu::fit8<kVec>(b[i], f0 + kcol + 8 * i, F));
#pragma unroll
      for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int q = 0; q < kRows; ++q)
          acc[q] = qk::mfma32(*(const LDS_AS bf16x8*)((const LDS_AS uint16_t*)lds +
                                                      ((3 * wh + n) * kBM + 32 * q + (l & 31)) * kBPitch + kcol + 8 * i),
                              l2, acc[q]);
    }
  }
  if (f_end == F && m < M)                 // up to 63 columns of a plane past 2 F
    for (int n = 0; n < ldz; n += plane)
      for (int f = 2 * F + col / 8; f < plane; f += kBC / 8) dZ[(int64_t)m * ldz + n + f] = 0;
  // the two halves of the steps' columns
  __syncthreads();
  LDS_AS float* red = (LDS_AS float*)lds + (w >> 1) * (kRows * 1024) + l;
  static_assert(4 * kRows * 1024 * sizeof(float) <= sizeof(lds), "the sums fit");
  if (wk)
#pragma unroll
    for (int q = 0; q < kRows; ++q)
#pragma unroll
      for (int e = 0; e < 16; ++e) red[64 * (16 * q + e)] = acc[q][e];
  __syncthreads();
  if (wk) return;
#pragma unroll
  for (int q = 0; q < kRows; ++q)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int mm = kBM * (int)blockIdx.x + 32 * q + qk::acc_row(e);
      if (mm < M && c < r)
        part[(((int64_t)blockIdx.y * 2 + wh) * M + mm) * r + c] = scale * (acc[q][e] + red[64 * (16 * q + e)]);
    }
}

// Slices of that pass: about 512 work groups (1024: 114 us for 111 at 4096 x 2 x 11008, 256: 121), but no
// more than 32 slices to add up for each row, and as many as the product for few rows adds up
// itself where the pass is short all the same (up to four steps).
struct PlanBack {
  int rows, tiles, slices;
  int64_t chunk;
};
PlanBack plan_back(int64_t M, int64_t F) {
  PlanBack p;
  p.rows = M >= 512 ? 64 : 32;             // both sides measured above
  p.tiles = (int)((M + p.rows - 1) / p.rows);
  const int cols = kBElems / p.rows;
  const int64_t steps = (F + cols - 1) / cols, most = steps <= 4 * kSmallSlices ? kSmallSlices : 32;
  const int64_t s = std::max<int64_t>(1, std::min<int64_t>({512 / p.tiles, steps, most}));
  p.chunk = (steps + s - 1) / s * cols;
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

hipError_t launch_low(const Low& q, int halves, int64_t M, int r, hipStream_t s) {
  const int rp = g_pitch(r);
  if (r % 4 == 0)
    hipLaunchKernelGGL(k_low<4>, dim3(blocks(M * rp / 4), (unsigned)halves), dim3(kT), 0, s, q, halves, M, r, rp);
  else
    hipLaunchKernelGGL(k_low<1>, dim3(blocks(M * rp), (unsigned)halves), dim3(kT), 0, s, q, halves, M, r, rp);
  return hipGetLastError();
}

size_t glu_back_ws(int64_t M, int64_t F, int r) { return (size_t)plan_back(M, F).slices * 2 * M * r * sizeof(float); }

hipError_t launch_glu_back(const uint16_t* dH, int64_t M, int64_t F, const uint8_t* gu_codes, const uint8_t* gu_scales,
                           const uint16_t* L2, int r, float scale, uint16_t* dZ, float* part, int* slices, hipStream_t s) {
  const PlanBack p = plan_back(M, F);
  *slices = p.slices;
  const dim3 grid((unsigned)p.tiles, (unsigned)p.slices);
#define QL_BACK(R, V)                                                                                                      \
  hipLaunchKernelGGL((k_glu_back<R, V>), grid, dim3(kBT), 0, s, dH, (int)M, (int)F, gu_codes, gu_scales, L2, r, scale,  \
                     (int)p.chunk, (int)glu_ldz(F), (int)glu_plane(F), dZ, part)
  if (p.rows == 64) {
    if (F % 8 == 0) QL_BACK(64, true);
    else QL_BACK(64, false);
  } else {
    if (F % 8 == 0) QL_BACK(32, true);
    else QL_BACK(32, false);
  }
#undef QL_BACK
  return hipGetLastError();
}
